"""CPU tests of the calls over shared lists and of eviction: every refusal (arguments are checked before the
device is, with host addresses that are never read), workspace sizes, and the test-side reference against the
oracle's decode."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import lazy_oracle as lo
from tests import share_reference as ref

EINVAL, ERANGE = -1, -2


@pytest.fixture(scope="module")
def lk():
    import __graft_entry__
    __graft_entry__.build()
    import position_agnostic_kv_gb300 as m
    return m


class _Args:
    """Valid arguments of each call, at addresses that nothing reads."""

    def __init__(self, lk):
        self.lk = lk
        self.buf = ctypes.create_string_buffer(4096)
        self.p = (ctypes.addressof(self.buf) + 1023) & ~1023
        self.cfg = lk.PosCfg()
        self.cfg.kind, self.cfg.rotary_dim, self.cfg.rope_theta = 0, 64, 1e4

    def call(self, what, **kw):
        p, c = self.p, ctypes.byref(self.cfg)
        d = dict(q=p, lse=p, cu_q=p, seq_len=p, q_start=p, doc_blocks=p, meta=p, group_off=p, shared_blocks=p, n_groups=1,
                 max_group=2, max_shared=3, B=2, max_blocks=4, total_q=2, max_q=1, window=0, k=p, v=p, num_pages=8, Hq=4,
                 Hkv=2, D=64, scale=0.0, cfg=c, accumulate=0, weights=p, out=p, ws=p, ws_bytes=1 << 30, keep=p, first=0,
                 recent=0, dst_pages=p, max_dst=4, new_meta=p + 512, new_doc_blocks=p, src=p, dst=p, new_weights=p + 512,
                 T=3)
        d.update(kw)
        names = {
            "attn_decode_shared": "q seq_len q_start doc_blocks meta group_off shared_blocks n_groups max_group "
                                  "max_shared B max_blocks k v num_pages Hq Hkv D scale cfg out lse ws ws_bytes",
            "attn_key_weights": "q lse cu_q seq_len q_start doc_blocks meta B max_blocks total_q max_q window k "
                                "num_pages Hq Hkv D scale cfg accumulate weights ws ws_bytes",
            "evict_plan": "weights meta doc_blocks keep first recent dst_pages max_dst B max_blocks num_pages cfg "
                          "new_meta new_doc_blocks src dst new_weights",
            "kv_move": "src dst T Hkv D k v num_pages"}[what]
        return getattr(self.lk.lib, "lazy_" + what)(*(d[n] for n in names.split()), None)


ATTN = [
    (dict(B=-1), EINVAL, "bad sizes"), (dict(max_blocks=0), EINVAL, "bad sizes"), (dict(Hq=0), EINVAL, "bad sizes"),
    (dict(Hkv=0), EINVAL, "bad sizes"), (dict(num_pages=0), EINVAL, "bad sizes"), (dict(D=96), EINVAL, "head_dim"),
    (dict(Hq=5), EINVAL, "multiple"), (dict(num_pages=(1 << 24) + 1), ERANGE, "num_pages"),
    (dict(max_blocks=(1 << 26) + 1), ERANGE, "lists"), (dict(B=65536), ERANGE, "65536"),
    (dict(scale=-1.0), EINVAL, "scale"), (dict(scale=float("nan")), EINVAL, "scale"),
    (dict(scale=float("inf")), EINVAL, "scale"), (dict(scale=1e-30), EINVAL, "2^-60"), (dict(scale=1e30), EINVAL, "2^-60"),
    (dict(meta=None), EINVAL, "NULL"), (dict(k=None), EINVAL, "NULL"), (dict(q=None), EINVAL, "NULL"),
    (dict(seq_len=None), EINVAL, "NULL"), (dict(q_start=None), EINVAL, "NULL"), (dict(doc_blocks=None), EINVAL, "NULL"),
    (dict(cfg=None), EINVAL, "cfg"),
]
SHARED = ATTN + [
    (dict(n_groups=-1), EINVAL, "n_groups"), (dict(max_group=-1), EINVAL, "max_group"),
    (dict(max_shared=-1), EINVAL, "max_shared"), (dict(n_groups=65536), ERANGE, "65536"),
    (dict(group_off=None), EINVAL, "NULL"), (dict(shared_blocks=None), EINVAL, "NULL"), (dict(v=None), EINVAL, "NULL"),
    (dict(out=None), EINVAL, "NULL"), (dict(num_pages=1 << 24, Hkv=128, Hq=128), ERANGE, "2^31"),
]
WEIGHTS = ATTN + [
    (dict(total_q=-1), EINVAL, "total_q"), (dict(max_q=-1), EINVAL, "max_q"), (dict(window=-1), EINVAL, "window"),
    (dict(lse=None), EINVAL, "NULL"), (dict(cu_q=None), EINVAL, "NULL"), (dict(weights=None), EINVAL, "NULL"),
    (dict(ws=None), EINVAL, "workspace"), (dict(ws_bytes=1023), EINVAL, "workspace"),
]
PLAN = [
    (dict(B=-1), EINVAL, "bad sizes"), (dict(max_blocks=0), EINVAL, "bad sizes"), (dict(max_dst=0), EINVAL, "bad sizes"),
    (dict(num_pages=0), EINVAL, "bad sizes"), (dict(first=-1), EINVAL, "first"), (dict(recent=-1), EINVAL, "recent"),
    (dict(num_pages=(1 << 24) + 1), ERANGE, "num_pages"), (dict(max_dst=(1 << 26) + 1), ERANGE, "lists"),
    (dict(cfg=None), EINVAL, "cfg"), (dict(B=(1 << 24) + 1), ERANGE, "2^24"),
] + [(dict([(n, None)]), EINVAL, "NULL") for n in ("weights", "meta", "doc_blocks", "keep", "dst_pages", "new_meta",
                                                   "new_doc_blocks", "src", "dst", "new_weights")]
MOVE = [
    (dict(T=-1), EINVAL, "bad sizes"), (dict(Hkv=0), EINVAL, "bad sizes"), (dict(num_pages=0), EINVAL, "bad sizes"),
    (dict(D=32), EINVAL, "head_dim"), (dict(num_pages=(1 << 24) + 1), ERANGE, "num_pages"), (dict(src=None), EINVAL, "NULL"),
    (dict(dst=None), EINVAL, "NULL"), (dict(k=None), EINVAL, "NULL"), (dict(v=None), EINVAL, "NULL"),
]
ALL = [(w, *c) for w, cs in (("attn_decode_shared", SHARED), ("attn_key_weights", WEIGHTS), ("evict_plan", PLAN),
                             ("kv_move", MOVE)) for c in cs]


@pytest.mark.parametrize("what,kw,code,text", ALL, ids=lambda x: str(x)[:40])
def test_refusals(lk, what, kw, code, text):
    a = _Args(lk)
    assert a.call(what, **kw) == code
    assert text in lk.lib.lazy_last_error().decode()


@pytest.mark.parametrize("what,name", [(w, n) for w, ns in (
    ("attn_decode_shared", ("q", "k", "v", "out")), ("attn_key_weights", ("q", "k")), ("kv_move", ("k", "v"))) for n in ns])
def test_misaligned_tensors_are_refused(lk, what, name):
    a = _Args(lk)
    assert a.call(what, **{name: a.p + 8}) == EINVAL
    assert "aligned" in lk.lib.lazy_last_error().decode()


@pytest.mark.parametrize("what", ["attn_decode_shared", "attn_key_weights", "evict_plan"])
def test_misaligned_words_are_refused(lk, what):
    a = _Args(lk)
    assert a.call(what, meta=a.p + 4) == EINVAL
    assert "aligned" in lk.lib.lazy_last_error().decode()


def test_plan_refusals_of_its_own(lk):
    a = _Args(lk)
    assert a.call("evict_plan", new_meta=a.p) == EINVAL and "place" in lk.lib.lazy_last_error().decode()
    assert a.call("evict_plan", new_weights=a.p) == EINVAL and "place" in lk.lib.lazy_last_error().decode()
    a.cfg.kind = 2
    assert a.call("evict_plan") == EINVAL and "ALiBi" in lk.lib.lazy_last_error().decode()
    a.cfg.kind = 7
    assert a.call("evict_plan") == EINVAL and "kind" in lk.lib.lazy_last_error().decode()


def test_workspace_sizes(lk):
    size = lk.decode_shared_workspace_size
    assert size(0, 0, 0, 0, 4, 4, 2, 64) == 0 and size(2, 1, 2, 3, 4, 4, 3, 64) == 0 and size(2, 1, 2, 3, 0, 4, 2, 64) == 0
    assert size(4, 1, 4, 100, 104, 32, 8, 128) >= 4 * 32 * (128 + 2) * 4
    assert lk.workspace_size(lk.PHASE_KEY_WEIGHTS, 1, 3, 5, 8, 2, 64) >= 2 * 3 * 5 * 16 * 4


def test_python_calls_refuse_tensors(lk):
    import torch
    t = lambda *s, d=torch.int32: torch.zeros(s, dtype=d)  # noqa: E731
    bf = torch.bfloat16
    cfg = lk.pos_cfg_from("rope", 64)
    k = t(8, 2, 16, 64, d=bf)
    with pytest.raises(ValueError, match="CUDA device"):
        lk.attn_decode_shared(t(2, 4, 64, d=bf), t(2), t(2), t(2), t(2, 4, d=torch.int64), t(2), t(1), 2, 3, k, k, cfg,
                              t(2, 4, 64, d=bf))
    with pytest.raises(ValueError, match="group_off"):
        lk.attn_decode_shared(t(2, 4, 64, d=bf), t(2), t(2), t(2), t(2, 4, d=torch.int64), t(3), t(1), 2, 3, k, k, cfg,
                              t(2, 4, 64, d=bf))
    with pytest.raises(TypeError, match="seq_len"):
        lk.attn_decode_shared(t(2, 4, 64, d=bf), t(2, d=torch.int64), t(2), t(2), t(2, 4, d=torch.int64), t(2), t(1), 2, 3,
                              k, k, cfg, t(2, 4, 64, d=bf))
    with pytest.raises(ValueError, match="weights"):
        lk.attn_key_weights(t(2, 4, 64, d=bf), t(2, 4, d=torch.float32), t(3), t(2), t(2), t(2), t(2, 4, d=torch.int64), k,
                            cfg, t(2, 63, d=torch.float32), 1)
    with pytest.raises(TypeError, match="lse"):
        lk.attn_key_weights(t(2, 4, 64, d=bf), t(2, 4, d=bf), t(3), t(2), t(2), t(2), t(2, 4, d=torch.int64), k, cfg,
                            t(2, 64, d=torch.float32), 1)
    f = torch.float32
    with pytest.raises(ValueError, match="src_slot"):
        lk.evict_plan(t(2, 64, d=f), t(2, 4, d=torch.int64), t(2), t(2), t(2, 3), 8, cfg, t(2, 4, d=torch.int64), t(2),
                      t(2, 47), t(2, 48), t(2, 64, d=f))
    with pytest.raises(ValueError, match="dst_pages"):
        lk.evict_plan(t(2, 64, d=f), t(2, 4, d=torch.int64), t(2), t(2), t(6), 8, cfg, t(2, 4, d=torch.int64), t(2),
                      t(2, 48), t(2, 48), t(2, 64, d=f))
    with pytest.raises(ValueError, match="contiguous"):
        lk.kv_move(t(3, 2)[:, 0], t(3), k, k)
    with pytest.raises(ValueError, match="k_cache"):
        lk.kv_move(t(3), t(3), k[0], k[0])


@pytest.mark.parametrize("kind,inter,rd", [("rope", False, 64), ("rope", True, 32), ("alibi", False, 64)])
def test_reference_agrees_with_the_oracle(kind, inter, rd):
    """The reference's decode over lists with common documents is the oracle's decode of each list."""
    rng = np.random.default_rng(5)
    pos = dict(kind=kind, theta=1e4, rotary_dim=rd, interleaved=inter)
    x = ref.Lists(rng, [(2, [20, 7]), (1, [33])], [[5], [], [16], [40]], [3, 17, 1, 5], 4, 2, 64, pos)
    to_bits = lambda a: (np.nan_to_num(a).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)  # noqa: E731
    p = dict(kind=kind, rope_theta=1e4, rotary_dim=rd, interleaved=inter, alibi_slopes=x.slopes)
    out, lse = oracle.decode(to_bits(x.q), x.seq_len, x.q_start, x.doc_blocks, x.meta, to_bits(x.k), to_bits(x.v), p)
    mine, ls, _, _ = ref.decode(x)
    assert np.abs(mine - out).max() < 1e-9 and np.abs(ls - lse).max() < 1e-9
    assert np.array_equal(lo.bf16_bits_to_f64(to_bits(x.q)), x.q)


def test_reference_plan_keeps_attention(lk):
    """Decode over the packed copies of some keys is decode over those keys where they were."""
    rng = np.random.default_rng(6)
    pos = dict(kind="rope", theta=1e4, rotary_dim=64, interleaved=False)
    x = ref.Lists(rng, [], [[20, 7, 40], [33]], [3, 17], 4, 2, 64, pos, spare=12)
    w = rng.random((2, x.max_blocks * 16)).astype(np.float32)
    dst = x.spare.reshape(2, 6)
    nm, nd, src, to, nw = ref.plan(w, x.meta, x.doc_blocks, [30, 9], dst, x.num_pages, 2, 3)
    k, v = ref.move(src, to, x.k, x.v)
    out, _, _, _ = ref.decode(x, nm, nd, k, v)
    for b in range(2):
        stay = set(src[b][src[b] >= 0])
        s, ks = ref.scores(x, b, x.q[b:b + 1], [int(x.seq_len[b]) - 1])
        here = np.array([i >= x.doc_blocks[b] * 16 or page * 16 + row in stay for i, _, _, page, row in ks])
        wgt, _ = ref.softmax(np.where(here, s[0], -np.inf))
        vv = np.repeat(x.v[ks[:, 3], :, ks[:, 4]], 2, 1)
        assert np.abs(out[b] - np.einsum("ht,thd->hd", wgt, vv)).max() < 1e-12
        assert len(stay) == [30, 9][b]


def test_common_prefixes(lk):
    """Neighbouring requests whose lists begin alike."""
    from position_agnostic_kv_gb300.runner import common_prefixes
    meta = np.array([[1, 2, 3, 9], [1, 2, 4, 9], [1, 2, 3, 9], [5, 2, 3, 9], [5, 2, 3, 9], [7, 0, 0, 0]], np.uint64)
    nd = np.array([3, 3, 2, 3, 3, 0], np.int32)
    off, shared = common_prefixes(meta, nd)
    assert off.tolist() == [0, 3, 5, 6] and shared.tolist() == [2, 3, 0]
    off, shared = common_prefixes(meta, nd, min_blocks=3)
    assert off.tolist() == [0, 1, 2, 3, 5, 6] and shared.tolist() == [3, 3, 2, 3, 0]
    off, shared = common_prefixes(meta[:0], nd[:0])
    assert off.tolist() == [0] and shared.tolist() == []


def test_kv_move_of_more_rows_than_an_int_counts(lk):
    """Refused before anything is launched, by the call and by its Python form."""
    import torch
    a = _Args(lk)
    for T in (2 ** 31 - 7, 2 ** 31 - 1):
        assert a.call("kv_move", T=T) == ERANGE and "2^31" in lk.lib.lazy_last_error().decode()
    slots, k = (torch.empty(s, dtype=d, device="meta") for s, d in (((2 ** 32 + 5,), torch.int32), ((8, 2, 16, 64), torch.bfloat16)))
    with pytest.raises(ValueError, match="2\\^31"):
        lk.kv_move(slots, slots, k, k)


@pytest.mark.parametrize("B,groups,deep,Hq,Hkv,alone", [
    (64, 32, 260, 32, 8, True), (64, 32, 60, 64, 8, True), (64, 16, 30, 32, 8, True), (12, 6, 600, 64, 8, True),
    (64, 16, 260, 32, 8, False), (64, 8, 130, 32, 8, False), (64, 1, 2000, 32, 8, False), (12, 6, 600, 32, 32, False)])
def test_groups_too_small_to_gain_are_decoded_alone(lk, B, groups, deep, Hq, Hkv, alone):
    """Such a call needs the workspace of one without groups."""
    size = lk.decode_shared_workspace_size
    got = size(B, groups, B // groups, deep, deep + 3, Hq, Hkv, 128)
    assert (got == size(B, 0, 0, 0, deep + 3, Hq, Hkv, 128)) == alone
