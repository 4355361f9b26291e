"""GPU tests of calls on the 4-bit cache that lie at the edge of what its interface allows.

Where two calls compute the same numbers (a table at another address, a looser bound on the query
lengths, values that a row does not see, operands scaled by powers of two) their results are
compared bit for bit; bytes of the cache are compared with the numpy restatement of the format
(tests/q4_reference.py).
"""
import numpy as np
import pytest

from oracle import lazy_oracle as lo
from tests import q4_reference as q4
from tests.gpu_common import lib
from tests.test_gpu_q4 import POISON, _bf, _bits, _clean, _dev, _i32, _tensor, _ws
from workloads import alibi_slopes_input

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lk():
    return lib()


# ------------------------------------------------------------------ cos/sin tables
@pytest.mark.parametrize("offset", [1, 2, 3, 4])
@pytest.mark.parametrize("D,Hkv,T", [(128, 8, 37), (64, 3, 50), (128, 2, 40000)])
def test_a_table_may_start_at_any_float(lk, D, Hkv, T, offset):
    """A contiguous table inside a larger buffer, on 4-, 8- and 16-byte boundaries: the same bytes as from
    one of its own."""
    import torch
    rng = np.random.default_rng([D, T, offset])
    n = 2000
    cfg = lk.pos_cfg_from("rope", D, rope_theta=1e4)
    table = torch.empty((n, D), dtype=torch.float32, device="cuda")
    lk.build_rope_table(cfg, n, table)
    moved = torch.full((n * D + 8,), np.nan, dtype=torch.float32, device="cuda")[offset:offset + n * D].view(n, D)
    moved.copy_(table)
    assert moved.data_ptr() % 16 == 4 * offset % 16
    k, v = _tensor(_bf(rng, T, Hkv, D)), _tensor(_bf(rng, T, Hkv, D))
    slots, lp = _i32(rng.permutation(T + 9)[:T]), _i32(rng.integers(0, n + 50, T))  # some beyond the table
    caches = []
    for t in (table, moved):
        c = torch.full(lk.q4_cache_shape(T // 16 + 2, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
        lk.kv_write_q4(k, v, slots, lp, c, lk.pos_cfg_from("rope", D, rope_theta=1e4, cos_sin=t))
        caches.append(c)
    _clean(lk)
    assert torch.equal(*caches)


# ------------------------------------------------------------------ bounds on the query lengths
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (32, 1), (136, 1)])
@pytest.mark.parametrize("q_len", [[5, 0, 3], [70, 9, 1]])
def test_max_q_may_be_any_upper_bound(lk, Hq, Hkv, q_len):
    """A looser bound than the longest question, up to the largest int, changes nothing."""
    import torch
    D, B = 128, len(q_len)
    rng = np.random.default_rng([Hq, q_len[0]])
    T, n = max(q_len), -(-max(q_len) // 16)
    cache = torch.full(lk.q4_cache_shape(n, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
    cfg, t = lk.pos_cfg_from("rope", D), np.arange(T)
    lk.kv_write_q4(_tensor(_bf(rng, T, Hkv, D)), _tensor(_bf(rng, T, Hkv, D)), _i32(t), _i32(t), cache, cfg)
    _, meta, _, _, _ = lk.build_doc_meta([0, 0], [], [], [0], [], [T], [0, n], t[:n], n)
    meta, cu = _dev(meta.view(np.int64)).repeat(B, 1), np.r_[0, np.cumsum(q_len)]
    q = _tensor(_bf(rng, cu[-1], Hq, D))
    ws = _ws(lk, lk.PHASE_PREFILL_Q4, len(q), B, n, Hq, Hkv, D)
    outs = []
    for max_q in (max(q_len), max(q_len) + 1, len(q) + 1000, 2 ** 31 - 1):
        out, lse = torch.full_like(q, np.nan), torch.full((len(q), Hq), np.nan, device="cuda")
        lk.attn_prefill_q4(q, _i32(cu), _i32([0] * B), _i32([0] * B), meta, cache, cfg, out, max_q, lse=lse, ws=ws)
        _clean(lk)
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
        outs.append((out, lse))
    # the bound decides which warps share a row's keys: the same operands and scores, the weights rounded (2^-11)
    # against other maxima and summed in another order.  Both results lie within 2^-8 |x| + 2^-10 max |v| of the
    # exact one for those scores, so twice that apart.
    vmax = np.nanmax(np.abs(lo.bf16_bits_to_f64(q4.load(cache.cpu().numpy(), D)[1])))
    for out, lse in outs[1:]:
        a, b = out.float(), outs[0][0].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -9 * vmax).all()
        np.testing.assert_allclose(lse.cpu().numpy(), outs[0][1].cpu().numpy(), rtol=1e-5, atol=1e-4)
    for out, lse in outs[3:]:
        assert torch.equal(out, outs[2][0]) and torch.equal(lse, outs[2][1])


# ------------------------------------------------------------------ NaN in values that some rows do not see
@pytest.mark.parametrize("D,Hq,Hkv,L", [(128, 8, 2, 150), (64, 8, 2, 150), (128, 8, 2, 30), (64, 8, 8, 300), (128, 32, 1, 9),
                                        (64, 16, 1, 8), (128, 24, 1, 40), (128, 136, 1, 20)])
@pytest.mark.parametrize("kind", ["rope", "interleaved", "alibi"])
def test_a_nan_value_reaches_only_the_rows_that_see_it(lk, D, Hq, Hkv, L, kind):
    """Values with an infinity or a NaN at the document's end, inside the query segment and at its last token.
    A row's outputs are NaN in exactly the groups of 16 dimensions (and KV heads) where it sees one, even where
    the key's weight is 0 in f16; all else keeps its bits.  Prefill, then the decode of the same rows with few
    blocks and with many (key splits)."""
    import torch
    rng = np.random.default_rng([D, Hq, L])
    P, T = 41, 41 + L
    nd, nq = -(-P // 16), -(-L // 16)
    ids = rng.permutation(nd + nq + 2)[:nd + nq]
    t = np.arange(T)
    own = np.where(t < P, t, t - P)
    slot = np.where(t < P, ids[own // 16 % nd], ids[(nd + own // 16) % (nd + nq)]) * 16 + own % 16
    extra = dict(interleaved=True) if kind == "interleaved" else {}
    if kind == "alibi":
        extra = dict(alibi_slopes=_dev(np.asarray(alibi_slopes_input(Hq), np.float32)))
    cfg = lk.pos_cfg_from("alibi" if kind == "alibi" else "rope", D, rotary_dim=D, **extra)
    q, k, v = _tensor(_bf(rng, L, Hq, D)), _tensor(_bf(rng, T, Hkv, D)), _tensor(_bf(rng, T, Hkv, D))
    bad = [(P - 1, 0, D // 16 - 1, np.nan), (P + L // 3, 0, 1, -np.inf), (P + L // 3 + 2, Hkv - 1, 1, np.nan),
           (P + L // 2, Hkv - 1, 2, np.inf), (T - 1, 0, 0, np.nan)]  # position, KV head, group, value
    _, meta, _, q_start, doc_blocks = lk.build_doc_meta([0, 1], [0], [P], [0, nd], ids[:nd], [L], [0, nq], ids[nd:],
                                                       nd + nq)
    assert q_start[0] == P and doc_blocks[0] == nd
    caches = []
    for spoil in (False, True):
        x = v.clone()
        if spoil:
            for p, h, g, val in bad:
                x[p, h, 16 * g + p % 16] = val
        c = torch.full(lk.q4_cache_shape(nd + nq + 2, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
        lk.kv_write_q4(k, x, _i32(slot), _i32(own), c, cfg)
        caches.append(c)
    m = P + np.arange(L)
    want = np.zeros((L, Hq, D // 16), bool)
    for p, h, g, _ in bad:
        want[m >= p, h * (Hq // Hkv):(h + 1) * (Hq // Hkv), g] = True
    want = torch.from_numpy(want).cuda().repeat_interleave(16, 2)
    assert want.any() and not want.all()

    def check(what, outs):
        (a, la), (b, lb) = outs
        assert torch.isfinite(a.float()).all(), what
        assert torch.equal(torch.isnan(b), want), f"{what}: NaN in {int(torch.isnan(b).sum())}, not {int(want.sum())}"
        assert torch.equal(a[~want], b[~want]) and torch.equal(la, lb), what

    def both(call):
        res = []
        for c in caches:
            out, lse = torch.full_like(q, 7.0), torch.full((L, Hq), np.nan, device="cuda")
            call(c, out, lse)
            _clean(lk)
            res.append((out, lse))
        return res

    md = _dev(meta.view(np.int64))
    ws = _ws(lk, lk.PHASE_PREFILL_Q4, L, 1, nd + nq, Hq, Hkv, D)
    check("prefill", both(lambda c, out, lse: lk.attn_prefill_q4(
        q, _i32([0, L]), _i32([P]), _i32([nd]), md, c, cfg, out, L, lse=lse, ws=ws)))
    for blocks in (nd + nq, 3000):
        wide = torch.zeros((L, blocks), dtype=torch.int64, device="cuda")
        wide[:, :nd + nq] = md
        wd = _ws(lk, lk.PHASE_DECODE_Q4, L, L, blocks, Hq, Hkv, D)
        check(f"decode, {blocks} blocks", both(lambda c, out, lse: lk.attn_decode_q4(
            q, _i32(m + 1), _i32([P] * L), _i32([nd] * L), wide, c, cfg, out, lse=lse, ws=wd)))


@pytest.mark.parametrize("D,Hq,Hkv,L", [(128, 8, 2, 150), (64, 8, 8, 300), (128, 8, 2, 30), (64, 16, 1, 8), (128, 136, 1, 20)])
@pytest.mark.parametrize("kind", ["rope", "none"])
def test_a_nan_key_reaches_only_the_rows_that_see_it(lk, D, Hq, Hkv, L, kind):
    """A key with a NaN inside the query segment: its KV head's outputs and lse are NaN in the rows that see
    it, and keep their bits in the others."""
    import torch
    rng = np.random.default_rng([D, Hq, L])
    blocks, t, bad = -(-L // 16), np.arange(L), L // 2
    cfg = lk.pos_cfg_from(kind, D)
    q, k, v = _tensor(_bf(rng, L, Hq, D)), _tensor(_bf(rng, L, Hkv, D)), _tensor(_bf(rng, L, Hkv, D))
    _, meta, _, _, _ = lk.build_doc_meta([0, 0], [], [], [0], [], [L], [0, blocks], t[:blocks], blocks)
    md = _dev(meta.view(np.int64))
    res = []
    for spoil in (False, True):
        x = k.clone()
        if spoil:
            x[bad, Hkv - 1, 5] = np.nan
        c = torch.full(lk.q4_cache_shape(blocks, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
        lk.kv_write_q4(x, v, _i32(t), _i32(t), c, cfg)
        for call in ("prefill", "decode"):
            out, lse = torch.full_like(q, 7.0), torch.full((L, Hq), 7.0, device="cuda")
            if call == "prefill":
                lk.attn_prefill_q4(q, _i32([0, L]), _i32([0]), _i32([0]), md, c, cfg, out, L, lse=lse,
                                   ws=_ws(lk, lk.PHASE_PREFILL_Q4, L, 1, blocks, Hq, Hkv, D))
            else:
                lk.attn_decode_q4(q, _i32(t + 1), _i32([0] * L), _i32([0] * L), md.repeat(L, 1), c, cfg, out, lse=lse,
                                  ws=_ws(lk, lk.PHASE_DECODE_Q4, L, L, blocks, Hq, Hkv, D))
            _clean(lk)
            res.append((out, lse))
    want = torch.zeros((L, Hq), dtype=torch.bool, device="cuda")
    want[bad:, (Hkv - 1) * (Hq // Hkv):] = True
    for (a, la), (b, lb) in zip(res[:2], res[2:]):
        assert torch.isfinite(a.float()).all() and torch.isfinite(la).all()
        assert torch.equal(torch.isnan(b), want[..., None].expand_as(b)) and torch.equal(torch.isnan(lb), want)
        assert torch.equal(a[~want], b[~want]) and torch.equal(la[~want], lb[~want])


# ------------------------------------------------------------------ small queries under a large scale
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 16, 2), (64, 32, 1), (128, 136, 1)])
@pytest.mark.parametrize("shift", [40, 55, 62, 70])
def test_small_queries_under_a_large_scale(lk, D, Hq, Hkv, shift):
    """Queries times 2^-shift and the scale times 2^shift: every product is the same number, so are the
    results' bits.  (The scale stays below 2^60, the queries above bf16's smallest normal number.)"""
    import torch
    rng = np.random.default_rng([D, Hq, shift])
    T, blocks, cfg = 200, 13, lk.pos_cfg_from("rope", D)
    t = np.arange(T)
    cache = torch.full(lk.q4_cache_shape(blocks, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
    k = (_tensor(_bf(rng, T, Hkv, D)).float() * 256).to(torch.bfloat16)
    lk.kv_write_q4(k, _tensor(_bf(rng, T, Hkv, D)), _i32(t), _i32(t), cache, cfg)
    _, meta, _, _, _ = lk.build_doc_meta([0, 0], [], [], [0], [], [T], [0, blocks], t[:blocks], blocks)
    md = _dev(meta.view(np.int64))
    q = _tensor(_bf(rng, T, Hq, D))
    res = []
    for s in (0, shift):
        x = (q.float() * 2.0 ** -s).to(torch.bfloat16)
        scale = 2.0 ** (s - 11)
        out, lse = torch.empty_like(q), torch.empty((T, Hq), device="cuda")
        lk.attn_prefill_q4(x, _i32([0, T]), _i32([0]), _i32([0]), md, cache, cfg, out, T, lse=lse, scale=scale,
                           ws=_ws(lk, lk.PHASE_PREFILL_Q4, T, 1, blocks, Hq, Hkv, D))
        res.append([out, lse])
        for n, wide in ((6, md), (6, torch.cat([md, torch.zeros((1, 3000), dtype=torch.int64, device="cuda")], 1))):
            out, lse = torch.empty_like(q[:n]), torch.empty((n, Hq), device="cuda")
            lk.attn_decode_q4(x[-n:], _i32(t[-n:] + 1), _i32([0] * n), _i32([0] * n), wide.repeat(n, 1), cache, cfg, out,
                              lse=lse, scale=scale,
                              ws=_ws(lk, lk.PHASE_DECODE_Q4, n, n, wide.shape[1], Hq, Hkv, D))
            res[-1] += [out, lse]
    _clean(lk)
    assert (res[0][1] - torch.log(_dev(t + 1.0))[:, None]).abs().max() > 0.3  # the logits do not vanish
    for a, b in zip(*res):
        assert torch.equal(a, b)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 2), (32, 1)])
@pytest.mark.parametrize("scale", [2.0 ** -59, 2.0 ** -11, 2.0 ** 59])
def test_queries_next_to_zero(lk, Hq, Hkv, scale):
    """Rows of zeros, of subnormal numbers and of bf16's smallest normal ones: the logits vanish under every
    scale that is accepted, so each visible key weighs the same.  2^-8 for the output's rounding and 2^-10
    of the mean magnitude for the weights'."""
    import torch
    D, T, blocks, cfg = 128, 100, 7, lk.pos_cfg_from("rope", 128)
    rng = np.random.default_rng(Hq)
    t = np.arange(T)
    cache = torch.full(lk.q4_cache_shape(blocks, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
    lk.kv_write_q4(_tensor(_bf(rng, T, Hkv, D)), _tensor(_bf(rng, T, Hkv, D)), _i32(t), _i32(t), cache, cfg)
    vv = lo.bf16_bits_to_f64(q4.load(cache.cpu().numpy(), D)[1]).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:T]
    want = np.cumsum(vv, 0) / (t + 1.0)[:, None, None]
    mag = np.cumsum(np.abs(vv), 0) / (t + 1.0)[:, None, None]
    _, meta, _, _, _ = lk.build_doc_meta([0, 0], [], [], [0], [], [T], [0, blocks], t[:blocks], blocks)
    md = _dev(meta.view(np.int64))
    for top in (0.0, 2.0 ** -130, 2.0 ** -126):
        x = (_tensor(_bf(rng, T, Hq, D)).sign().double() * top).to(torch.bfloat16)
        assert float(x.abs().max()) == top
        out, lse = torch.empty_like(x), torch.empty((T, Hq), device="cuda")
        lk.attn_prefill_q4(x, _i32([0, T]), _i32([0]), _i32([0]), md, cache, cfg, out, T, lse=lse, scale=scale,
                           ws=_ws(lk, lk.PHASE_PREFILL_Q4, T, 1, blocks, Hq, Hkv, D))
        one, lone = torch.empty_like(x[-1:]), torch.empty((1, Hq), device="cuda")
        lk.attn_decode_q4(x[-1:], _i32([T]), _i32([0]), _i32([0]), md, cache, cfg, one, lse=lone, scale=scale,
                          ws=_ws(lk, lk.PHASE_DECODE_Q4, 1, 1, blocks, Hq, Hkv, D))
        _clean(lk)
        for got, l, rows in ((out, lse, slice(None)), (one, lone, slice(T - 1, T))):
            w, a = (np.repeat(z[rows], Hq // Hkv, 1) for z in (want, mag))
            err = np.abs(got.float().cpu().numpy() - w)
            assert (err <= 2.0 ** -8 * np.abs(w) + 2.0 ** -10 * a + 1e-30).all()
            np.testing.assert_allclose(l.cpu().numpy(), np.log(t[rows] + 1.0)[:, None].repeat(Hq, 1), atol=1e-5)


# ------------------------------------------------------------------ calls large enough for several heads per thread
def _store_all(cache, slots, k, v):
    """q4_reference.store for many tokens at once."""
    D = k.shape[-1]
    kc, ks, vc, vs = q4.offsets(D)
    p, r, h = (slots // 16)[:, None, None], slots % 16, np.arange(k.shape[1])[None, :, None]
    for x, co, so in ((k, kc, ks), (v, vc, vs)):
        code, scale = q4.quantise(x)
        cache[p, h, co[r][:, None, 0::2]] = code[..., 0::2] | (code[..., 1::2] << 4)
        cache[p, h, so[r][:, None, ::16]] = scale


def _tokens(Hkv, D, per_sm, dims):
    """Tokens that give each SM `per_sm` threads of `dims` dimensions and a head, and a few more."""
    import torch
    n = torch.cuda.get_device_properties(0).multi_processor_count * per_sm
    return -(-n // (Hkv * (D // dims))) + 13


@pytest.mark.parametrize("D,Hkv", [(128, 8), (128, 3), (64, 5), (64, 8), (128, 1), (64, 2)])
@pytest.mark.parametrize("rotate", [True, False])
def test_write_of_many_tokens_is_bit_exact(lk, D, Hkv, rotate):
    """Four heads per thread from 2048 threads per SM on, head counts that are no multiple of four, and
    some bad slots among them."""
    import torch
    T, n = _tokens(Hkv, D, 2048, 16), 1500
    rng = np.random.default_rng([D, Hkv, rotate])
    pages = T // 16 + 3
    slots, lp = rng.permutation(16 * pages)[:T], rng.integers(0, n, T)
    k, v = _bf(rng, T, Hkv, D), _bf(rng, T, Hkv, D)
    kf = lo.bf16_bits_to_f64(k)
    cfg = lk.pos_cfg_from("none", D)
    if rotate:
        table = torch.empty((n, D), dtype=torch.float32, device="cuda")
        lk.build_rope_table(lk.pos_cfg_from("rope", D), n, table)
        cfg = lk.pos_cfg_from("rope", D, cos_sin=table)
        kf = q4.rotate_f32(kf, lp, table.cpu().numpy(), False)
    bad = rng.choice(T, 9, replace=False)
    given = slots.copy()
    given[bad] = rng.choice([-1, 16 * pages, 2 ** 31 - 1], 9)
    cache = torch.full(lk.q4_cache_shape(pages, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
    lk.kv_write_q4(_tensor(k), _tensor(v), _i32(given), _i32(lp), cache, cfg)
    assert lk.device_status() == 2  # LAZY_STATUS_BAD_SLOT
    ref = np.full(cache.shape, POISON, np.uint8)
    ok = np.setdiff1d(np.arange(T), bad)
    _store_all(ref, slots[ok], kf[ok], lo.bf16_bits_to_f64(v[ok]))
    np.testing.assert_array_equal(cache.cpu().numpy(), ref)


@pytest.mark.parametrize("D,Hkv", [(128, 8), (128, 3), (64, 5), (64, 8), (128, 1)])
def test_read_of_many_tokens_is_exact(lk, D, Hkv):
    """Two heads per thread from 4096 threads per SM on, odd head counts, some bad slots (rows that stay)."""
    import torch
    T = _tokens(Hkv, D, 4096, 8)
    rng = np.random.default_rng([D, Hkv])
    pages = 300
    raw = rng.integers(0, 256, (pages, Hkv, 18 * D), dtype=np.uint8)
    for a, b in ((8 * D, 9 * D), (17 * D, 18 * D)):
        raw[..., a:b] = np.minimum(raw[..., a:b] & 0x7F, 0x7E)  # no NaN
    slots = rng.integers(0, 16 * pages, T)
    bad = rng.choice(T, 9, replace=False)
    given = slots.copy()
    given[bad] = rng.choice([-1, 16 * pages, 2 ** 31 - 1], 9)
    ko = torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    lk.kv_read_q4(_i32(given), _dev(raw), ko, vo, k_scale=0.25, v_scale=2.0)
    assert lk.device_status() == 2  # LAZY_STATUS_BAD_SLOT
    for got, want in zip((ko, vo), q4.load(raw, D, 0.25, 2.0)):
        w = lo.bf16_bits_to_f64(want)[slots // 16, :, slots % 16]
        w[bad] = 7.0
        np.testing.assert_array_equal(lo.bf16_bits_to_f64(_bits(got)), w)
