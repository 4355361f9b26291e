"""GPU tests of the 4-bit paged cache: writing, reading back, decode and prefill over it.

The write is compared byte for byte with a numpy restatement of the format
(tests/q4_reference.py), the read bit for bit, and the attention with the fp64 oracle on the
values that the cache holds.

Tolerances of the attention, from the arithmetic that the kernels document.  With A = sum_j p_j |v_j|:
  * the output is rounded to bf16: at most 2^-8 of it;
  * the weights p are rounded to f16, 2^-11 of each, and sums run in fp32: 2^-10 A covers both;
  * the tensor-core kernel (prefill; decode of head groups above 8) rounds queries to f16 (2^-11) and
    rotates keys in f16: cos, sin, a product and the sum each 2^-11, so a key is off by at most
    3 sqrt(2) 2^-11 |k|, a score by at most E = 6 * 2^-11 |q| |k| scale, a weight by 2 E of itself:
    2 E A more;
  * a weight is held as 2^(s - max + 7), max a score that was met, so the sum of the weights is at
    least 2^7; weights below 2^-14 are subnormal f16 numbers, off by at most 2^-25, which is 2^-32 of
    the sum: 2^-32 max |v| more per key.  Inputs are N(0, 1): |v| < 8.
These are worst cases; typically the roundings average out, so the relative Frobenius error is held
to 2^-8, the largest that the rounding of the output alone can reach.
"""
import numpy as np
import pytest

import oracle
from oracle import lazy_oracle as lo
from tests import q4_reference as q4
from tests.gpu_common import lib
from tests.oracle_setup import oracle_meta
from workloads import PosCfg, alibi_slopes_input, f32_to_bf16_bits, make_custom, make_workload

pytestmark = pytest.mark.gpu

POISON = 0x7F  # as a scale: NaN; as codes: +6, +6


@pytest.fixture(scope="module")
def lk():
    return lib()


def _bits(t):
    import torch
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _bf(rng, *shape):
    return f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def _dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _i32(x):
    return _dev(np.asarray(x, np.int32))


def _tensor(bits):
    from position_agnostic_kv_gb300.runner import bits_to_tensor
    return bits_to_tensor(bits, "cuda")


def _clean(lk):
    assert lk.device_status() == 0


# ------------------------------------------------------------------ writing
WRITES = [  # D, Hkv, kind, rotary_dim, interleaved, T, factors
    (128, 8, "rope", 128, False, 37, (1.0, 1.0)),
    (128, 2, "yarn", 128, False, 1, (1.0, 1.0)),
    (128, 1, "rope", 96, False, 100, (0.25, 4.0)),
    (128, 3, "rope", 16, False, 33, (1.0, 1.0)),
    (128, 2, "rope", 48, True, 65, (1.0, 0.5)),
    (64, 2, "rope", 64, False, 50, (1.0, 1.0)),
    (64, 5, "yarn", 48, False, 17, (2.0, 1.0)),
    (64, 1, "rope", 32, True, 129, (1.0, 1.0)),
    (128, 2, "none", 128, False, 31, (1.0, 1.0)),
    (64, 4, "none", 64, False, 15, (1.0, 8.0)),
]


def _write_case(lk, D, Hkv, kind, rd, inter, T, factors, table=True, seed=0):
    import torch
    rng = np.random.default_rng([D, Hkv, rd, T, seed])
    pages = T // 16 + 3
    slots = rng.permutation(16 * pages)[:T]
    lp = rng.integers(0, 2000, T)
    k, v = _bf(rng, T, Hkv, D), _bf(rng, T, Hkv, D)
    tab = None
    if kind != "none":
        cfg = lk.pos_cfg_from(kind, D, rope_theta=1e4, yarn_factor=8.0, yarn_orig_ctx=512, rotary_dim=rd,
                              interleaved=inter)
        tab = torch.empty((2000, rd), dtype=torch.float32, device="cuda")
        lk.build_rope_table(cfg, 2000, tab)
    cfg = lk.pos_cfg_from(kind, D, rope_theta=1e4, yarn_factor=8.0, yarn_orig_ctx=512, rotary_dim=rd,
                          interleaved=inter, cos_sin=tab if table else None)
    cache = torch.full(lk.q4_cache_shape(pages, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
    f = dict(k_scale=factors[0], v_scale=factors[1])
    lk.kv_write_q4(_tensor(k), _tensor(v), _i32(slots), _i32(lp), cache, cfg, **f)
    ref = np.full(cache.shape, POISON, np.uint8)
    kf = lo.bf16_bits_to_f64(k)
    rot = kf if tab is None else q4.rotate_f32(kf, lp, tab.cpu().numpy(), inter)
    q4.store(ref, slots, rot, lo.bf16_bits_to_f64(v), *factors)
    return cache, ref, slots, f


@pytest.mark.parametrize("D,Hkv,kind,rd,inter,T,factors", WRITES)
def test_write_is_bit_exact_with_a_table(lk, D, Hkv, kind, rd, inter, T, factors):
    """Codes, scales and every byte of the rows that were not written."""
    cache, ref, _, _ = _write_case(lk, D, Hkv, kind, rd, inter, T, factors)
    np.testing.assert_array_equal(cache.cpu().numpy(), ref)
    _clean(lk)


@pytest.mark.parametrize("D,Hkv,kind,rd,inter,T,factors", [w for w in WRITES if w[2] != "none"])
def test_write_with_angles_on_the_fly(lk, D, Hkv, kind, rd, inter, T, factors):
    """Angles computed in the kernel differ from the table's by ~5e-7, which moves a rounding to bf16
    (2^-8) in a few values of 10^4, and of those a code or scale in about one of 16."""
    cache, ref, slots, _ = _write_case(lk, D, Hkv, kind, rd, inter, T, factors, table=False)
    got, want = cache.cpu().numpy(), ref
    np.testing.assert_array_equal(got[..., 9 * D:], want[..., 9 * D:])  # values are not rotated
    n = (got != want).sum()
    assert n <= 8 + 1e-3 * 9 * D * Hkv * T / 16, n
    kg, _ = q4.load(got, D, *factors)
    kw, _ = q4.load(want, D, *factors)
    a = lo.bf16_bits_to_f64(kg)[slots // 16, :, slots % 16]
    b = lo.bf16_bits_to_f64(kw)[slots // 16, :, slots % 16]
    top = np.abs(b).reshape(*b.shape[:2], -1, 16).max(-1)
    # a moved code is one step (at most 2 of 6), a moved scale 2^-3 of everything
    assert (np.abs(a - b).reshape(*b.shape[:2], -1, 16) <= top[..., None] * (2 / 6 + 2.0 ** -3)).all()
    _clean(lk)


@pytest.mark.parametrize("D", [64, 128])
def test_write_of_extreme_values(lk, D):
    """Zeros, values whose scale underflows, saturating ones, ties, infinities and NaN, per group."""
    import torch
    groups = [np.zeros(16), np.full(16, 2.0 ** -11), np.full(16, -6 * 2.0 ** -10), np.full(16, 6 * 2.0 ** -9),
              np.linspace(-3e5, 3e5, 16), np.array([2688.0, 2624.0, 2752.0] + [1.0] * 13),
              np.array([np.inf] + [1.0] * 15), np.array([1.0] * 15 + [-np.inf]), np.array([np.nan] * 16),
              np.array([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5]),
              np.array([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5]) * 1.125,
              np.array([-0.0] * 8 + [1e-38, -1e-38, 1e-3, -1e-3, 3e38, 0, 0, 0])]
    flat = np.concatenate(groups)
    T = -(-flat.size // D)
    x = np.zeros(T * D, np.float32)
    x[:flat.size] = flat
    bits = f32_to_bf16_bits(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf))
    bits = np.where(np.isnan(x), np.uint16(0x7FC0), bits).reshape(T, 1, D)
    cache = torch.full(lk.q4_cache_shape(2, 1, D), POISON, dtype=torch.uint8, device="cuda")
    slots = np.arange(T) + 5
    lk.kv_write_q4(_tensor(bits), _tensor(bits), _i32(slots), _i32(slots), cache, lk.pos_cfg_from("none", D))
    ref = np.full(cache.shape, POISON, np.uint8)
    val = lo.bf16_bits_to_f64(bits)
    q4.store(ref, slots, val, val)
    got = cache.cpu().numpy()
    kg, vg = q4.load(got, D)
    kr, vr = q4.load(ref, D)
    # codes of a zero may carry either sign: compare values, and scales as bytes
    np.testing.assert_array_equal(lo.bf16_bits_to_f64(kg), lo.bf16_bits_to_f64(kr))
    np.testing.assert_array_equal(lo.bf16_bits_to_f64(vg), lo.bf16_bits_to_f64(vr))
    np.testing.assert_array_equal(got[..., 8 * D:9 * D], ref[..., 8 * D:9 * D])
    np.testing.assert_array_equal(got[..., 17 * D:], ref[..., 17 * D:])
    _clean(lk)


@pytest.mark.parametrize("factor", [2.0 ** -32, 1.0, 2.0 ** 32])
@pytest.mark.parametrize("D", [64, 128])
def test_write_of_values_far_beyond_the_scales(lk, D, factor):
    """Quotients by the largest scale that exceed fp32 saturate with their own sign."""
    T = 5 if D == 64 else 40000  # enough for several heads per thread too
    big = np.array([3e38, -3e38, 1e31, -1e31, 1e20, -1e20, 5e12, -5e12, 1.0, -1.0, 1e-7, -1e-7, 1e-38, -1e-38, 0, 7])
    bits = f32_to_bf16_bits(np.resize(np.concatenate([big, big * 1e-6, big * 1e-30]), (T, 1, D)).astype(np.float32))
    import torch
    cache = torch.full(lk.q4_cache_shape(T // 16 + 1, 1, D), POISON, dtype=torch.uint8, device="cuda")
    slots = np.arange(T) + 3
    lk.kv_write_q4(_tensor(bits), _tensor(bits), _i32(slots), _i32(slots), cache, lk.pos_cfg_from("none", D), factor,
                   factor)
    ref = np.full(cache.shape, POISON, np.uint8)
    val = lo.bf16_bits_to_f64(bits)
    q4.store(ref, slots, val, val, factor, factor)
    for g, r in zip(q4.load(cache.cpu().numpy(), D, factor, factor), q4.load(ref, D, factor, factor)):
        np.testing.assert_array_equal(lo.bf16_bits_to_f64(g), lo.bf16_bits_to_f64(r))
    _clean(lk)


def test_write_and_read_skip_bad_slots(lk):
    import torch
    D, Hkv, pages = 128, 2, 3
    rng = np.random.default_rng(1)
    k, v = _bf(rng, 5, Hkv, D), _bf(rng, 5, Hkv, D)
    slots = np.array([4, -1, 16 * pages, 7, 2 ** 31 - 1])
    cache = torch.full(lk.q4_cache_shape(pages, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
    lk.kv_write_q4(_tensor(k), _tensor(v), _i32(slots), _i32(np.arange(5)), cache, lk.pos_cfg_from("none", D))
    assert lk.device_status() == 2  # LAZY_STATUS_BAD_SLOT
    ref = np.full(cache.shape, POISON, np.uint8)
    q4.store(ref, slots[[0, 3]], lo.bf16_bits_to_f64(k[[0, 3]]), lo.bf16_bits_to_f64(v[[0, 3]]))
    np.testing.assert_array_equal(cache.cpu().numpy(), ref)
    ko = torch.full((5, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    lk.kv_read_q4(_i32(slots), cache, ko, vo)
    assert lk.device_status() == 2
    kr, _ = q4.load(ref, D)
    got = _bits(ko)
    np.testing.assert_array_equal(got[[0, 3]], kr[slots[[0, 3]] // 16, :, slots[[0, 3]] % 16])
    assert (ko[[1, 2, 4]] == 7.0).all() and (vo[[1, 2, 4]] == 7.0).all()


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("D,Hkv,T,factors", [(128, 8, 77, (1.0, 1.0)), (64, 2, 33, (0.25, 16.0)), (128, 1, 1, (1.0, 1.0)),
                                             (64, 3, 500, (1.0, 1.0)), (128, 5, 2000, (4.0, 0.5))])
def test_read_is_exact(lk, D, Hkv, T, factors):
    """Every code, every finite scale, rows in any order, some of them more than once."""
    import torch
    rng = np.random.default_rng([D, T])
    pages = T // 16 + 2
    raw = rng.integers(0, 256, (pages, Hkv, 18 * D), dtype=np.uint8)
    for lo_, hi in ((8 * D, 9 * D), (17 * D, 18 * D)):
        raw[..., lo_:hi] &= 0x7F
        raw[..., lo_:hi][raw[..., lo_:hi] == 0x7F] = 0x7E
    slots = rng.integers(0, 16 * pages, T)
    ko = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    lk.kv_read_q4(_i32(slots), _dev(raw), ko, vo, k_scale=factors[0], v_scale=factors[1])
    kr, vr = q4.load(raw, D, *factors)
    for got, want in ((ko, kr), (vo, vr)):
        np.testing.assert_array_equal(lo.bf16_bits_to_f64(_bits(got)),
                                      lo.bf16_bits_to_f64(want)[slots // 16, :, slots % 16])
    _clean(lk)


def test_what_was_written_reads_back(lk):
    import torch
    cache, ref, slots, f = _write_case(lk, 128, 4, "rope", 128, False, 90, (0.5, 2.0), seed=3)
    ko = torch.empty((90, 4, 128), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    lk.kv_read_q4(_i32(slots), cache, ko, vo, **f)
    kr, vr = q4.load(ref, 128, 0.5, 2.0)
    np.testing.assert_array_equal(_bits(ko) & 0x7FFF, kr[slots // 16, :, slots % 16] & 0x7FFF)
    np.testing.assert_array_equal(_bits(vo) & 0x7FFF, vr[slots // 16, :, slots % 16] & 0x7FFF)
    # NaN rows read back as NaN
    free = np.setdiff1d(np.arange(16 * cache.shape[0]), slots)[:4]
    lk.kv_read_q4(_i32(free), cache, ko[:4], vo[:4], **f)
    assert torch.isnan(ko[:4]).all() and torch.isnan(vo[:4]).all()
    _clean(lk)


# ------------------------------------------------------------------ attention
def _check_attention(got, want, absv, score_err, keys, what):
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2 * score_err) * absv + keys * 2.0 ** -32 * 8
    worst = (np.abs(g - want) / bound).max()
    rel = np.linalg.norm(g - want) / max(np.linalg.norm(want), 1e-30)
    assert worst <= 1.0 and rel <= 2.0 ** -8, f"{what}: {worst:.3f} of the bound, relative {rel:.3e}"


def _score_err(w, q, kb):
    """E of the module's docstring."""
    kv = lo.bf16_bits_to_f64(kb)
    kmax = np.sqrt((np.nan_to_num(kv) ** 2).sum(-1).max())
    qmax = np.sqrt((lo.bf16_bits_to_f64(q) ** 2).sum(-1).max()) if len(q) else 0.0
    return 6 * 2.0 ** -11 * qmax * kmax * lo.softmax_scale(w.pos.as_dict(), w.D)


def _load(raw, D, kf=1.0, vf=1.0):
    """Bits of the keys and values held, rows that were never written (NaN) as zeros: the oracle's
    textbook softmax multiplies hidden values by zero weights."""
    return [np.where((x & 0x7FFF) > 0x7F80, np.uint16(0), x) for x in q4.load(raw, D, kf, vf)]


def _values(v):
    return v & np.uint16(0x7FFF)  # |v|


def _run(lk, w, reqs, n_steps, check, use_table=False, factors=(1.0, 1.0), sharpen=1.0):
    """Fill, prefill and decode over a cache that starts as NaN; compare with the oracle on the
    values that the cache holds (the query tokens' own included)."""
    import torch
    from position_agnostic_kv_gb300.runner import PagedBatch
    pb = PagedBatch(w, device="cuda", use_table=use_table, kv_bits=4, k_scale=factors[0], v_scale=factors[1])
    pb.kv_cache.fill_(POISON)
    pb.ws.fill_(0xFF)
    pb.fill_documents()
    inp = pb.upload_prefill()
    if sharpen != 1.0:
        inp["q"] = (inp["q"].float() * sharpen).to(torch.bfloat16)
    lse_p = torch.full((max(pb.total_q, 1), w.Hq), np.nan, dtype=torch.float32, device="cuda")[:pb.total_q]
    out_p = pb.prefill(inp, lse=lse_p)
    got = {}
    for t in range(n_steps):
        l = torch.full((w.B, w.Hq), np.nan, dtype=torch.float32, device="cuda")
        o = pb.decode_step(pb.upload_decode(t), lse=l)
        if t in check:
            got[t] = (o.clone(), l)
    torch.cuda.synchronize()
    _clean(lk)
    _, meta, seq_len, q_start, doc_blocks = oracle_meta(w)
    used = sorted({int(word) >> 40 for b in reqs for word in meta[b]})
    raw = np.full(pb.kv_cache.shape, 0, np.uint8)
    raw[used] = pb.kv_cache[torch.tensor(used, device="cuda")].cpu().numpy()
    kb, vb = np.zeros((w.num_pages, w.Hkv, 16, w.D), np.uint16), np.zeros((w.num_pages, w.Hkv, 16, w.D), np.uint16)
    kb[used], vb[used] = _load(raw[used], w.D, *factors)
    pos = w.pos.as_dict()
    if w.q_len.sum():
        qb = _bits(inp["q"])
        args = (qb, w.cu_q, q_start, doc_blocks, meta, kb)
        ref, lse = lo.prefill(*args, vb, pos, requests=reqs)
        a, _ = lo.prefill(*args, _values(vb), pos, requests=reqs)
        rows = np.concatenate([np.arange(w.cu_q[b], w.cu_q[b + 1]) for b in reqs])
        e = _score_err(w, qb[rows], kb[used])
        _check_attention(out_p[rows], ref[rows], a[rows], e, int(seq_len.max()), f"{w.name} prefill")
        np.testing.assert_allclose(lse_p[rows].cpu().numpy(), lse[rows], rtol=1e-5, atol=e + 1e-4)
    for t in sorted(got):
        # later tokens are in the cache already; causality hides them from step t
        qd = w.decode_tokens(t)[0]
        args = (qd, seq_len + t + 1, q_start, doc_blocks, meta, kb)
        ref, lse = lo.decode(*args, vb, pos, requests=reqs)
        a, _ = lo.decode(*args, _values(vb), pos, requests=reqs)
        # wide head groups may run on the tensor-core kernel, which rounds queries and keys to f16
        e = _score_err(w, qd[reqs], kb[used]) if w.Hq // w.Hkv > 8 else 0.0
        _check_attention(got[t][0][reqs], ref[reqs], a[reqs], e, int(seq_len.max()) + t + 1, f"{w.name} decode step {t}")
        np.testing.assert_allclose(got[t][1][reqs].cpu().numpy(), lse[reqs], rtol=1e-5, atol=e + 1e-4)


SHAPES = [(64, 4, 4), (64, 8, 2), (128, 8, 1), (128, 16, 2), (64, 16, 2), (128, 4, 2), (128, 24, 1), (64, 48, 2),
          (128, 32, 1), (64, 16, 1), (128, 64, 1), (64, 128, 1), (128, 72, 1), (64, 120, 1), (128, 136, 1)]


@pytest.mark.parametrize("D,Hq,Hkv", SHAPES)
def test_attention_head_shapes(lk, D, Hq, Hkv):
    """Documents of 1, 15, 16, 17 and 33 tokens, requests without a query segment or with one token."""
    w = make_custom([1, 15, 16, 17, 33], [[4, 0, 2], [1, 3], [2, 4, 1, 0], [0]], Hq, Hkv, D, PosCfg("rope", 1e4, D),
                    [3, 0, 17, 1], 5, seed=D + Hq)
    _run(lk, w, [0, 1, 2, 3], 5, {0, 4})


@pytest.mark.parametrize("D,Hq,Hkv,rd,inter,kind,table", [
    (128, 8, 2, 64, False, "rope", False), (128, 8, 2, 128, True, "rope", True), (64, 4, 4, 32, True, "yarn", False),
    (64, 16, 2, 48, False, "rope", True), (128, 32, 1, 32, True, "rope", False), (128, 32, 4, 16, False, "yarn", True),
    (128, 24, 1, 96, False, "rope", True), (128, 8, 2, 128, False, "rope", True), (64, 8, 1, 64, False, "yarn", True),
    (128, 16, 2, 128, False, "alibi", False), (64, 4, 4, 64, False, "alibi", False), (64, 24, 1, 64, False, "alibi", False)])
def test_attention_positional_variants(lk, D, Hq, Hkv, rd, inter, kind, table):
    extra = dict(yarn_factor=8.0, yarn_orig_ctx=512) if kind == "yarn" else {}
    if kind == "alibi":
        extra = dict(alibi_slopes=alibi_slopes_input(Hq))
    w = make_custom([1, 15, 16, 17, 333], [[4, 0, 2], [1, 3], [2, 4, 1, 0]], Hq, Hkv, D,
                    PosCfg(kind, 1e4, rd, interleaved=inter, **extra), [3, 0, 17], 4, seed=D + Hq + rd)
    _run(lk, w, [0, 1, 2], 4, {0, 3}, use_table=table)


@pytest.mark.parametrize("name,batch,reqs,steps", [("tiny", None, [0], 8), ("rag8b", None, [0, 5, 15], 4),
                                                   ("yarn8b", None, [0, 31], 2), ("mqa_alibi", None, [0, 13], 2),
                                                   ("prefill70b", None, [0, 7], 0), ("decode32k", 24, [0, 23], 2)])
def test_attention_workloads(lk, name, batch, reqs, steps):
    w = make_workload(name, batch=batch)
    _run(lk, w, reqs, steps, set(range(steps)) if steps > 4 else {0, max(0, steps - 1)} if steps else set())


@pytest.mark.parametrize("Hq,Hkv,q_len", [(8, 2, [70, 33, 100, 1]), (8, 8, [300, 129, 1, 128]), (64, 8, [64, 16, 17, 40]),
                                          (32, 1, [9, 4, 1, 5]), (24, 1, [20, 7, 32, 1]), (24, 1, [5, 4, 1, 3]), (128, 1, [3, 2, 1, 5])])
@pytest.mark.parametrize("kind", ["rope", "alibi"])
def test_prefill_query_lengths(lk, Hq, Hkv, q_len, kind):
    """Query segments longer and shorter than a tile of query rows, over no document at all too."""
    pos = PosCfg("rope", 1e4, 128) if kind == "rope" else PosCfg("alibi", alibi_slopes=alibi_slopes_input(Hq), rotary_dim=128)
    w = make_custom([700, 16, 5, 130], [[0, 2], [3, 1, 0], [], [2]], Hq, Hkv, 128, pos, q_len, 0, seed=sum(q_len))
    _run(lk, w, [0, 1, 2, 3], 0, set())


def test_attention_long_context(lk):
    """136 072 tokens, the last page index of a document (2047), angles at 1.36e5."""
    w = make_custom([32768, 16384, 16384, 16384, 16384, 16384, 16384, 5000], [[3, 0, 7, 1, 6, 2, 5, 4]], 8, 2, 128,
                    PosCfg("rope", 5e5, 128), [16], 2, seed=1280)
    _run(lk, w, [0], 2, {0, 1})


@pytest.mark.parametrize("name", ["rag8b", "mqa_alibi"])
def test_attention_sharpened_queries(lk, name):
    """Queries x 4: the softmax rests on few keys."""
    _run(lk, make_workload(name, batch=2), [0, 1], 0, set(), sharpen=4.0)


@pytest.mark.parametrize("factors", [(0.25, 4.0), (8.0, 2.0 ** -6)])
def test_attention_with_cache_factors(lk, factors):
    w = make_custom([100, 40], [[0, 1], [1]], 8, 2, 128, PosCfg("rope", 1e4, 128), [5, 20], 2, seed=8)
    _run(lk, w, [0, 1], 2, {0, 1}, factors=factors)


def test_factors_scale_exactly(lk):
    """Keys 8 times as large in a cache of factor 8, queries' scale an eighth: the same bytes and outputs."""
    import torch
    rng = np.random.default_rng(5)
    D, Hq, Hkv, T = 128, 8, 2, 200
    k, v, q = _tensor(_bf(rng, T, Hkv, D)), _tensor(_bf(rng, T, Hkv, D)), _tensor(_bf(rng, 4, Hq, D))
    _, meta, _, q_start, doc_blocks = lk.build_doc_meta([0, 0], [], [], [0], [], [T], [0, 13], np.arange(13), 13)
    meta = _dev(meta.view(np.int64)).repeat(4, 1)
    cfg = lk.pos_cfg_from("rope", D)
    outs = []
    for f in (1.0, 8.0):
        cache = torch.full(lk.q4_cache_shape(13, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
        lk.kv_write_q4(k * f, v * f, _i32(np.arange(T)), _i32(np.arange(T)), cache, cfg, k_scale=f, v_scale=f)
        out, kb, vb = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        lk.attn_decode_q4(q, _i32([200, 1, 17, 150]), _i32([0] * 4), _i32([0] * 4), meta, cache, cfg, out,
                          ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), scale=0.1 / f, k_scale=f, v_scale=f)
        lk.kv_read_q4(_i32(np.arange(T)), cache, kb, vb, k_scale=f, v_scale=f)
        outs.append((cache, out, kb, vb))
    assert torch.equal(outs[0][0], outs[1][0])
    for a, b in zip(outs[0][1:], outs[1][1:]):
        assert torch.equal(a.float() * 8.0, b.float())
    _clean(lk)


# ------------------------------------------------------------------ edges
def _one_request(lk, D=128, Hq=8, Hkv=2, T=100, seed=2, pages=None):
    import torch
    rng = np.random.default_rng(seed)
    n = -(-T // 16)
    ids = np.arange(n) if pages is None else np.asarray(pages)[:n]
    cache = torch.full(lk.q4_cache_shape(int(ids.max()) + 1, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
    cfg = lk.pos_cfg_from("rope", D)
    t = np.arange(T)
    k, v = _bf(rng, T, Hkv, D), _bf(rng, T, Hkv, D)
    lk.kv_write_q4(_tensor(k), _tensor(v), _i32(ids[t // 16] * 16 + t % 16), _i32(t), cache, cfg)
    _, meta, _, _, _ = lk.build_doc_meta([0, 0], [], [], [0], [], [T], [0, n], ids, n)
    return dict(cache=cache, cfg=cfg, meta_h=meta, meta=_dev(meta.view(np.int64)), rng=rng, D=D, Hq=Hq, Hkv=Hkv, T=T)


def _ws(lk, phase, rows, B, mb, Hq, Hkv, D):
    import torch
    return torch.empty(max(lk.workspace_size(phase, rows, B, mb, Hq, Hkv, D), 256), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (8, 8), (32, 1), (24, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing(lk, D, Hq, Hkv):
    """A length of zero: out 0 and lse -inf; its neighbours of one and more tokens are unaffected."""
    import torch
    s = _one_request(lk, D, Hq, Hkv)
    q = _tensor(_bf(s["rng"], 4, Hq, D))
    lens = [0, 1, 100, 0]
    meta = s["meta"].repeat(4, 1)
    out = torch.full_like(q, np.nan)
    lse = torch.full((4, Hq), np.nan, device="cuda")
    ws = _ws(lk, lk.PHASE_DECODE_Q4, 4, 4, meta.shape[1], Hq, Hkv, D)
    ws.fill_(0xFF)
    lk.attn_decode_q4(q, _i32(lens), _i32([0] * 4), _i32([0] * 4), meta, s["cache"], s["cfg"], out, lse=lse, ws=ws)
    _clean(lk)
    kb, vb = _load(s["cache"].cpu().numpy(), D)
    pos = PosCfg("rope", 1e4, D).as_dict()
    args = (_bits(q), np.array(lens), [0] * 4, [0] * 4, s["meta_h"].repeat(4, 0), kb)
    ref, rl = lo.decode(*args, vb, pos, requests=[1, 2])
    a, _ = lo.decode(*args, _values(vb), pos, requests=[1, 2])
    for b in (0, 3):
        assert (out[b] == 0).all() and (lse[b] == -np.inf).all()
    e = 0.05 if Hq // Hkv > 8 else 0.0
    _check_attention(out[[1, 2]], ref[[1, 2]], a[[1, 2]], e, 100, "decode beside empty rows")
    np.testing.assert_allclose(lse[[1, 2]].cpu().numpy(), rl[[1, 2]], rtol=1e-5, atol=e + 1e-4)


def test_nothing_to_do(lk):
    """No tokens, no requests, no query rows: nothing is launched, nothing refused."""
    import torch
    s = _one_request(lk)
    e = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    before = s["cache"].clone()
    lk.kv_write_q4(e, e, z, z, s["cache"], s["cfg"])
    lk.kv_read_q4(z, s["cache"], e, e)
    q = torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    lk.attn_decode_q4(q, z, z, z, s["meta"][:0], s["cache"], s["cfg"], q)
    lk.attn_prefill_q4(q, _i32([0, 0]), _i32([0]), _i32([0]), s["meta"], s["cache"], s["cfg"], q, 0)
    _clean(lk)
    assert torch.equal(before, s["cache"])


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (32, 1), (24, 1)])
def test_bad_pages_are_skipped(lk, Hq, Hkv):
    """A block word that names a page outside the cache: the status bit, and the block's keys are
    left out; the other blocks count as before."""
    import torch
    D = 128
    s = _one_request(lk, D, Hq, Hkv)
    words = s["meta_h"].copy()
    words[0, 2] |= np.uint64(1000) << np.uint64(40)
    q = _tensor(_bf(s["rng"], 100, Hq, D))
    meta = _dev(words.view(np.int64))
    for what in ("decode", "prefill"):
        out = torch.full_like(q, np.nan)
        n = 100 if what == "prefill" else 1
        if what == "decode":
            ws = _ws(lk, lk.PHASE_DECODE_Q4, 1, 1, meta.shape[1], Hq, Hkv, D)
            lk.attn_decode_q4(q[:1], _i32([100]), _i32([0]), _i32([0]), meta, s["cache"], s["cfg"], out[:1], ws=ws)
        else:
            ws = _ws(lk, lk.PHASE_PREFILL_Q4, 100, 1, meta.shape[1], Hq, Hkv, D)
            lk.attn_prefill_q4(q, _i32([0, 100]), _i32([0]), _i32([0]), meta, s["cache"], s["cfg"], out, 100, ws=ws)
        assert lk.device_status() == 1  # LAZY_STATUS_BAD_PAGE
        kb, vb = (lo.bf16_bits_to_f64(x) for x in _load(s["cache"].cpu().numpy(), D))
        keep = np.r_[0:32, 48:100]
        kk = kb.transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[keep]
        vv = vb.transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[keep]
        m = np.array([99]) if what == "decode" else np.arange(100)
        inv = lo.rope_inv_freq(D, 1e4)
        qr = lo.rotate(lo.bf16_bits_to_f64(_bits(q[:n])), m[:, None], inv)
        ref, _ = lo.softmax_attention(qr, m, kk, vv, keep, 1 / np.sqrt(D))
        a, _ = lo.softmax_attention(qr, m, kk, np.abs(vv), keep, 1 / np.sqrt(D))
        e = 0.05 if what == "prefill" or Hq // Hkv > 8 else 0.0
        _check_attention(out[:n], ref, a, e, 100, what)


def test_prefill_rows_beyond_the_last_request_stay(lk):
    import torch
    s = _one_request(lk)
    q = _tensor(_bf(s["rng"], 9, 8, 128))
    out = torch.full_like(q, 5.0)
    ws = _ws(lk, lk.PHASE_PREFILL_Q4, 9, 1, s["meta"].shape[1], 8, 2, 128)
    lk.attn_prefill_q4(q[:4], _i32([0, 4]), _i32([0]), _i32([0]), s["meta"], s["cache"], s["cfg"], out[:4], 4, ws=ws)
    _clean(lk)
    assert (out[4:] == 5.0).all() and torch.isfinite(out[:4].float()).all()


@pytest.mark.parametrize("first,n,total", [(3, 30, 40), (0, 1, 2)])
@pytest.mark.parametrize("blocks", [7, 4000])  # 4000: key splits, those of (136, 1) merged through the workspace
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (32, 1), (24, 1), (136, 1), (272, 2)])
def test_a_batch_padded_to_a_fixed_number_of_rows(lk, Hq, Hkv, blocks, first, n, total):
    """Rows outside [cu_q[0], cu_q[B]) belong to no request: out and lse keep what they held.  The others
    may be split over keys otherwise than without the padding: both results lie within 2^-8 |x| +
    2^-10 max |v| of the exact one (_check_attention), so twice that apart."""
    import torch
    s = _one_request(lk, 128, Hq, Hkv)
    meta = torch.zeros((1, blocks), dtype=torch.int64, device="cuda")
    x = min(blocks, s["meta"].shape[1])
    meta[:, :x] = s["meta"][:, :x]
    q = _tensor(_bf(s["rng"], total, Hq, 128))
    last = first + n

    def run(q, cu):
        out, lse = torch.full_like(q, 5.0), torch.full((len(q), Hq), 5.0, device="cuda")
        ws = _ws(lk, lk.PHASE_PREFILL_Q4, len(q), 1, blocks, Hq, Hkv, 128)
        ws.fill_(0xFF)
        lk.attn_prefill_q4(q, _i32(cu), _i32([60]), _i32([0]), meta, s["cache"], s["cfg"], out, 30, lse=lse, ws=ws)
        _clean(lk)
        return out, lse

    out, lse = run(q, [first, last])
    want, wlse = run(q[first:last].contiguous(), [0, n])
    for x in (out, lse):
        assert (x[:first] == 5.0).all() and (x[last:] == 5.0).all()
    vmax = np.abs(lo.bf16_bits_to_f64(_load(s["cache"].cpu().numpy(), 128)[1])).max()
    a, b = out[first:last].float(), want.float()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -9 * vmax).all()
    np.testing.assert_allclose(lse[first:last].cpu().numpy(), wlse.cpu().numpy(), rtol=1e-5, atol=1e-4)


def test_offsets_beyond_32_bits(lk):
    """The request's pages lie past the first 4 GiB of the cache."""
    import torch
    Hkv, D, T = 8, 128, 50
    pages = (1 << 32) // (Hkv * 18 * D) + 100
    s = _one_request(lk, D, 32, Hkv, T, pages=[pages - 1, pages - 40, pages - 2, 3])
    q = _tensor(_bf(s["rng"], T, 32, D))
    out_d, out_p = torch.empty_like(q[:1]), torch.empty_like(q)
    ws = _ws(lk, lk.PHASE_DECODE_Q4, 2, 1, 4, 32, Hkv, D)
    lk.attn_decode_q4(q[-1:], _i32([T]), _i32([0]), _i32([0]), s["meta"], s["cache"], s["cfg"], out_d, ws=ws)
    lk.attn_prefill_q4(q, _i32([0, T]), _i32([0]), _i32([0]), s["meta"], s["cache"], s["cfg"], out_p, T,
                       ws=_ws(lk, lk.PHASE_PREFILL_Q4, T, 1, 4, 32, Hkv, D))
    ko = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    t = np.arange(T)
    ids = np.array([pages - 1, pages - 40, pages - 2, 3])
    lk.kv_read_q4(_i32(ids[t // 16] * 16 + t % 16), s["cache"], ko, vo)
    _clean(lk)
    k, v = lo.bf16_bits_to_f64(_bits(ko)), lo.bf16_bits_to_f64(_bits(vo))
    m = t
    qr = lo.rotate(lo.bf16_bits_to_f64(_bits(q)), m[:, None], lo.rope_inv_freq(D, 1e4))
    ref, _ = lo.softmax_attention(qr, m, k, v, t, 1 / np.sqrt(D))
    a, _ = lo.softmax_attention(qr, m, k, np.abs(v), t, 1 / np.sqrt(D))
    _check_attention(out_d, ref[-1:], a[-1:], 0.0, T, "decode")
    _check_attention(out_p, ref, a, 0.05, T, "prefill")


def test_one_large_key(lk):
    """A key whose logit lies hundreds of base-2 units above all others, met last."""
    import torch
    D, Hq, Hkv, T = 128, 8, 2, 300
    rng = np.random.default_rng(11)
    k, v, q = _bf(rng, T, Hkv, D), _bf(rng, T, Hkv, D), _bf(rng, T, Hq, D)
    k[T - 3] = 0
    k[T - 3, :, 63] = f32_to_bf16_bits(np.full(Hkv, 1024.0, np.float32))
    cfg = lk.pos_cfg_from("rope", D)
    cache = torch.full(lk.q4_cache_shape(19, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
    t = np.arange(T)
    lk.kv_write_q4(_tensor(k), _tensor(v), _i32(t), _i32(t), cache, cfg)
    _, meta, _, _, _ = lk.build_doc_meta([0, 0], [], [], [0], [], [T], [0, 19], t[:19], 19)
    out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    md = _dev(meta.view(np.int64))
    lk.attn_prefill_q4(_tensor(q), _i32([0, T]), _i32([0]), _i32([0]), md, cache, cfg, out, T,
                       ws=_ws(lk, lk.PHASE_PREFILL_Q4, T, 1, 19, Hq, Hkv, D))
    out_d = torch.empty((1, Hq, D), dtype=torch.bfloat16, device="cuda")
    lk.attn_decode_q4(_tensor(q[-1:]), _i32([T]), _i32([0]), _i32([0]), md, cache, cfg, out_d,
                      ws=_ws(lk, lk.PHASE_DECODE_Q4, 1, 1, 19, Hq, Hkv, D))
    _clean(lk)
    kb, vb = _load(cache.cpu().numpy(), D)
    pos = PosCfg("rope", 1e4, D).as_dict()
    ref, _ = lo.prefill(q, [0, T], [0], [0], meta, kb, vb, pos)
    a, _ = lo.prefill(q, [0, T], [0], [0], meta, kb, _values(vb), pos)
    # the large key's f16 roundings move its logit by at most 6 * 2^-11 of its two components' products,
    # which matters only where it is within reach of the others (below 16)
    _check_attention(out, ref, a, 6 * 2.0 ** -11 * 16, T, "prefill")
    _check_attention(out_d, ref[-1:], a[-1:], 0.0, T, "decode")


# ------------------------------------------------------------------ streams, graphs, workspaces
def test_streams_and_captured_graphs(lk):
    """Eager on another stream, and a captured write -> prefill -> decode replayed on new inputs,
    give the bytes that the eager default-stream run gives."""
    import torch
    from position_agnostic_kv_gb300.runner import PagedBatch
    w = make_workload("rag8b", batch=3)

    def run(pb, inp, dec):
        a = pb.prefill(inp)
        return a, pb.decode_step(dec)

    base = PagedBatch(w, kv_bits=4)
    base.fill_documents()
    inp, dec = base.upload_prefill(), base.upload_decode(0)
    want = run(base, inp, dec)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pb = PagedBatch(w, kv_bits=4)
        pb.fill_documents()
        got = run(pb, inp, dec)
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    # capture with other inputs in the buffers, then replay on the real ones
    pb = PagedBatch(w, kv_bits=4)
    pb.fill_documents()
    gi = {n: torch.zeros_like(x) if x.dtype == torch.bfloat16 else x for n, x in inp.items()}
    gd = {n: torch.zeros_like(x) if x.dtype == torch.bfloat16 else x for n, x in dec.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go = run(pb, gi, gd)
    for _ in range(2):
        for a, b in ((gi, inp), (gd, dec)):
            for n in a:
                a[n].copy_(b[n])
        for o in go:
            o.fill_(np.nan)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(go, want):
            assert torch.equal(x, y)
    _clean(lk)


def test_two_calls_at_once_with_their_own_workspaces(lk):
    """Two streams decode at the same time from one cache; results do not depend on it."""
    import torch
    from position_agnostic_kv_gb300.runner import PagedBatch
    w = make_workload("yarn8b", batch=4)
    pb = PagedBatch(w, kv_bits=4)
    pb.fill_documents()
    pb.prefill(pb.upload_prefill())
    d = pb.upload_decode(0)
    want = pb.decode_step(d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss, outs = [torch.empty_like(pb.ws) for _ in range(2)], [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            o = torch.empty_like(want)
            lk.attn_decode_q4(d["q"], d["seq_len"], pb.q_start, pb.doc_blocks, pb.meta, pb.kv_cache, pb.cfg, o, ws=wss[i],
                              stream=st)
            outs[i].append(o)
    torch.cuda.synchronize()
    _clean(lk)
    for o in outs[0] + outs[1]:
        assert torch.equal(o, want)


def test_a_short_workspace_is_refused(lk):
    import torch
    from position_agnostic_kv_gb300.runner import PagedBatch
    w = make_workload("yarn8b", batch=1)
    pb = PagedBatch(w, kv_bits=4)
    need = lk.workspace_size(lk.PHASE_DECODE_Q4, w.B, w.B, w.max_blocks, w.Hq, w.Hkv, w.D)
    assert need > 0  # one row over a long context: more key splits than a cluster holds
    d = pb.upload_decode(0)
    out = torch.full_like(d["q"], 3.0)
    call = lambda ws: lk.attn_decode_q4(d["q"], d["seq_len"], pb.q_start, pb.doc_blocks, pb.meta,  # noqa: E731
                                        pb.kv_cache, pb.cfg, out, ws=ws)
    big = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    for ws, text in ((None, "workspace"), (big[:need - 1], "workspace"), (big[16:need + 16], "256-byte")):
        with pytest.raises(lk.LazyError, match=text):
            call(ws)
    torch.cuda.synchronize()
    assert (out == 3.0).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("D,Hq,Hkv,L", [(128, 8, 2, 200), (64, 4, 4, 33), (128, 32, 1, 130)])
def test_encode_then_reuse_then_read_back(lk, D, Hq, Hkv, L):
    """A document encoded once over the 4-bit cache, reused by a later request at another offset with
    decode steps, and read back: a run of all four operators."""
    import torch
    from position_agnostic_kv_gb300.runner import encode_document
    rng = np.random.default_rng([L, D, Hq])
    q, k, v = _bf(rng, L, Hq, D), _bf(rng, L, Hkv, D), _bf(rng, L, Hkv, D)
    n = -(-L // 16)
    ids = rng.permutation(n + 6)
    pages, pre, qp = ids[:n], ids[n:n + 3], ids[n + 3:n + 4]
    cache = torch.full(lk.q4_cache_shape(n + 6, Hkv, D), POISON, dtype=torch.uint8, device="cuda")
    cfg = lk.pos_cfg_from("rope", D)
    out = encode_document(_tensor(q), _tensor(k), _tensor(v), pages, cache, None, cfg, k_scale=0.5, v_scale=1.0)
    _clean(lk)
    pos = PosCfg("rope", 1e4, D).as_dict()

    def held():
        return [lo.bf16_bits_to_f64(x) for x in _load(cache.cpu().numpy(), D, 0.5, 1.0)]

    t = np.arange(L)
    kk, vv = (x[pages[t // 16], :, t % 16] for x in held())
    inv, sc = lo.rope_inv_freq(D, 1e4), 1 / np.sqrt(D)
    qr = lo.rotate(lo.bf16_bits_to_f64(q), t[:, None], inv)
    ref, _ = lo.softmax_attention(qr, t, kk, vv, t, sc)
    a, _ = lo.softmax_attention(qr, t, kk, np.abs(vv), t, sc)
    _check_attention(out, ref, a, 0.05, L, "cold document")
    # reuse at offset 37 with a 5-token query, then one decode token
    P, ql = 37, 6
    kp, vp = _bf(rng, P, Hkv, D), _bf(rng, P, Hkv, D)
    qq, kq, vq = _bf(rng, ql, Hq, D), _bf(rng, ql, Hkv, D), _bf(rng, ql, Hkv, D)
    tp, tq = np.arange(P), np.arange(ql)
    f = dict(k_scale=0.5, v_scale=1.0)
    lk.kv_write_q4(_tensor(kp), _tensor(vp), _i32(pre[tp // 16] * 16 + tp % 16), _i32(tp), cache, cfg, **f)
    mb = 3 + n + 1
    _, meta, seq_len, q_start, doc_blocks = lk.build_doc_meta([0, 2], [0, 1], [P, L], [0, 3, 3 + n], np.r_[pre, pages],
                                                             [5], [0, 1], qp, mb)
    md = _dev(meta.view(np.int64))
    lk.kv_write_q4(_tensor(kq[:5]), _tensor(vq[:5]), _i32(qp[0] * 16 + tq[:5]), _i32(tq[:5]), cache, cfg, **f)
    out_p = torch.empty((5, Hq, D), dtype=torch.bfloat16, device="cuda")
    lk.attn_prefill_q4(_tensor(qq[:5]), _i32([0, 5]), _i32(q_start), _i32(doc_blocks), md, cache, cfg, out_p, 5,
                       ws=_ws(lk, lk.PHASE_PREFILL_Q4, 5, 1, mb, Hq, Hkv, D), **f)
    lk.kv_write_q4(_tensor(kq[5:]), _tensor(vq[5:]), _i32(qp[0] * 16 + tq[5:]), _i32(tq[5:]), cache, cfg, **f)
    out_d = torch.empty((1, Hq, D), dtype=torch.bfloat16, device="cuda")
    lk.attn_decode_q4(_tensor(qq[5:]), _i32(seq_len + 1), _i32(q_start), _i32(doc_blocks), md, cache, cfg, out_d,
                      ws=_ws(lk, lk.PHASE_DECODE_Q4, 1, 1, mb, Hq, Hkv, D), **f)
    _clean(lk)
    kc, vc = held()
    slots = np.r_[pre[tp // 16] * 16 + tp % 16, pages[t // 16] * 16 + t % 16, qp[0] * 16 + tq]
    off = np.r_[np.zeros(P), np.full(L, P), np.full(ql, P + L)].astype(int)
    p = np.r_[tp, P + t, P + L + tq]
    kk = lo.rotate(kc[slots // 16, :, slots % 16], off[:, None], inv)
    vv = vc[slots // 16, :, slots % 16]
    qr = lo.rotate(lo.bf16_bits_to_f64(qq), (P + L + tq)[:, None], inv)
    ref, _ = lo.softmax_attention(qr, P + L + tq, kk, vv, p, sc)
    a, _ = lo.softmax_attention(qr, P + L + tq, kk, np.abs(vv), p, sc)
    _check_attention(out_p, ref[:5], a[:5], 0.05, P + L + ql, "reuse, prefill")
    _check_attention(out_d, ref[5:], a[5:], 0.05 if Hq // Hkv > 8 else 0.0, P + L + ql, "reuse, decode")
    ko = torch.empty((len(slots), Hkv, D), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    lk.kv_read_q4(_i32(slots), cache, ko, vo, **f)
    _clean(lk)
    np.testing.assert_array_equal(lo.bf16_bits_to_f64(_bits(ko)), kc[slots // 16, :, slots % 16])
    np.testing.assert_array_equal(lo.bf16_bits_to_f64(_bits(vo)), vv)
