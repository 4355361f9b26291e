"""CPU tests of the 4-bit cache: the test-side format against itself, and every refusal.

The entry points check their arguments before they look at the device, so what they refuse is
tested here, with host addresses that are never read.
"""
import ctypes

import numpy as np
import pytest

from oracle import lazy_oracle as lo
from tests import q4_reference as ref


@pytest.fixture(scope="module")
def lk():
    import __graft_entry__
    __graft_entry__.build()
    import position_agnostic_kv_gb300 as m
    return m


@pytest.mark.parametrize("D", [64, 128])
def test_block_offsets_cover_the_block_once(D):
    kc, ks, vc, vs = ref.offsets(D)
    bytes_ = np.concatenate([kc[:, ::2].ravel(), ks[:, ::16].ravel(), vc[:, ::2].ravel(), vs[:, ::16].ravel()])
    assert sorted(bytes_) == list(range(18 * D))
    for o in (ks, vs):  # one scale per 16 dimensions
        assert (o.reshape(16, -1, 16) == o.reshape(16, -1, 16)[..., :1]).all()


def test_quantiser_rules():
    # every e4m3 scale reproduces the levels exactly; halves go to the even code; 5 s and more is 6 s
    for s in (2.0 ** -9, 0.0625, 1.0, 1.125, 448.0):
        y = np.zeros(16)
        y[:8], y[8:] = ref.LEVELS * s, [0.25 * s, 0.75 * s, 1.25 * s, 1.75 * s, 2.5 * s, 3.5 * s, 5 * s, -6 * s]
        code, sb = ref.quantise(y)
        assert ref.E4M3[sb[0]] == s
        assert list(code) == [0, 1, 2, 3, 4, 5, 6, 7, 0, 2, 2, 4, 4, 6, 6, 15]
    code, sb = ref.quantise(np.full(16, 6 * 2.0 ** -10))  # max / 6 half way between 0 and the least scale
    assert sb[0] == 0 and not code.any()
    code, sb = ref.quantise(np.array([1e5] + [2688.0] + [0.0] * 14))  # beyond 448 * 6: saturates
    assert ref.E4M3[sb[0]] == 448.0 and code[0] == 7 and code[1] == 7
    for bad in (np.inf, -np.inf, np.nan):
        code, sb = ref.quantise(np.array([1.0, bad] + [0.0] * 14))
        assert sb[0] == 0x7F and not code.any()


@pytest.mark.parametrize("D", [64, 128])
def test_store_then_load_is_a_quantised_copy(D):
    rng = np.random.default_rng(D)
    k, v = rng.standard_normal((40, 2, D)), rng.standard_normal((40, 2, D)) * 3
    slots = rng.permutation(64)[:40]
    cache = np.full((4, 2, 18 * D), 0x7F, np.uint8)
    ref.store(cache, slots, k, v, 0.25, 2.0)
    kb, vb = ref.load(cache, D, 0.25, 2.0)
    for x, bits in ((k, kb), (v, vb)):
        got = lo.bf16_bits_to_f64(bits)[slots // 16, :, slots % 16]
        top = np.abs(x).reshape(40, 2, -1, 16).max(-1)[..., None]
        # a code is off by at most half its widest step (1 of 6), the scale by 2^-4 of itself
        assert (np.abs(got - x).reshape(40, 2, -1, 16) <= top / 6 * (1 + 2.0 ** -4) + 1e-12).all()
    free = np.setdiff1d(np.arange(64), slots)
    assert np.isnan(lo.bf16_bits_to_f64(kb)[free // 16, :, free % 16]).all()


# ------------------------------------------------------------------ refusals of the C entry points
class _Args:
    """Valid arguments of one call (host addresses, 256-byte aligned), some of them replaced."""

    def __init__(self, lk):
        self.lk = lk
        self.buf = ctypes.create_string_buffer(1 << 16)
        self.p = (ctypes.addressof(self.buf) + 255) & ~255
        self.cfg = lk.PosCfg(lk.POS_ROPE, 128, 1e4, 1.0, 0, 32.0, 1.0, None, None, 0, 0)

    def call(self, what, **kw):
        p, cfg, lib = self.p, self.cfg, self.lk.lib
        cfg = kw.pop("cfg", cfg)
        d = dict(B=2, max_blocks=4, total_q=3, max_q=2, cache=p, num_pages=8, Hq=8, Hkv=2, D=128, q=p, seq_len=p,
                 cu_q=p, q_start=p, doc_blocks=p, meta=p, out=p, k_scale=1.0, v_scale=1.0, ws=None, ws_bytes=0, T=3,
                 k=p, v=p, slot=p, local_pos=p, scale=0.0)
        unknown = set(kw) - set(d)
        assert not unknown, unknown
        d.update(kw)
        c = ctypes.byref(cfg) if cfg is not None else None
        g = lambda *names: [d[n] for n in names]  # noqa: E731
        if what == "write":
            return lib.lazy_kv_write_q4(*g("k", "v", "slot", "local_pos", "T", "Hkv", "D", "cache", "num_pages"), c,
                                        *g("k_scale", "v_scale"), None)
        if what == "read":
            return lib.lazy_kv_read_q4(*g("slot", "T", "Hkv", "D", "cache", "num_pages", "k_scale", "v_scale", "k", "v"),
                                       None)
        if what == "decode":
            return lib.lazy_attn_decode_q4(*g("q", "seq_len", "q_start", "doc_blocks", "meta", "B", "max_blocks",
                                              "cache", "num_pages", "Hq", "Hkv", "D", "scale"),
                                           *g("k_scale", "v_scale"), c, *g("out"), None, *g("ws", "ws_bytes"), None)
        return lib.lazy_attn_prefill_q4(*g("q", "cu_q", "q_start", "doc_blocks", "meta", "B", "max_blocks", "total_q",
                                           "max_q", "cache", "num_pages", "Hq", "Hkv", "D", "scale"),
                                        *g("k_scale", "v_scale"), c, *g("out"), None, *g("ws", "ws_bytes"), None)


EVERY = ("write", "read", "decode", "prefill")
REFUSED = [
    # calls, replaced arguments, code, part of the message
    (EVERY, dict(D=96), -1, "head_dim must be 64 or 128"),
    (EVERY, dict(Hkv=0), -1, "bad sizes"),
    (EVERY, dict(num_pages=0), -1, "bad sizes"),
    (EVERY, dict(num_pages=(1 << 24) + 1), -2, "num_pages above"),
    (EVERY, dict(cache=None), -1, "NULL pointer"),
    (EVERY, dict(k_scale=3.0), -1, "powers of two"),
    (EVERY, dict(v_scale=-1.0), -1, "powers of two"),
    (EVERY, dict(k_scale=float("inf")), -1, "powers of two"),
    (EVERY, dict(v_scale=2.0 ** 33), -1, "powers of two"),
    (EVERY, dict(k_scale=float("nan")), -1, "powers of two"),
    (("write", "read"), dict(T=-1), -1, "bad sizes"),
    (("write", "read"), dict(k=None), -1, "NULL pointer"),
    (("write", "read"), dict(v=None), -1, "NULL pointer"),
    (("write", "read"), dict(slot=None), -1, "NULL pointer"),
    (("write", "read"), dict(T=(1 << 31) - 1, Hkv=1024), -2, "too many tokens"),
    (("write",), dict(local_pos=None), -1, "local_pos"),
    (("write", "decode", "prefill"), dict(cfg=None), -1, "pos cfg"),
    (("decode", "prefill"), dict(B=-1), -1, "bad sizes"),
    (("decode", "prefill"), dict(max_blocks=0), -1, "bad sizes"),
    (("decode", "prefill"), dict(Hq=9), -1, "multiple of Hkv"),
    (("decode", "prefill"), dict(Hq=12), -1, "power of two below 8"),
    (("decode", "prefill"), dict(Hq=24), -1, "multiple of 8"),
    (("decode", "prefill"), dict(scale=-0.1), -1, "scale must be positive"),
    (("decode", "prefill"), dict(scale=float("nan")), -1, "scale must be positive"),
    (("decode", "prefill"), dict(scale=float("inf")), -1, "scale must be positive"),
    (("decode", "prefill"), dict(scale=1e-30, k_scale=2.0 ** -32), -1, "scale times k_scale"),
    (("decode", "prefill"), dict(scale=1e30), -1, "scale times k_scale"),
    (("decode", "prefill"), dict(q=None), -1, "NULL pointer"),
    (("decode", "prefill"), dict(out=None), -1, "NULL pointer"),
    (("decode", "prefill"), dict(meta=None), -1, "NULL pointer"),
    (("decode", "prefill"), dict(q_start=None), -1, "NULL pointer"),
    (("decode", "prefill"), dict(doc_blocks=None), -1, "NULL pointer"),
    (("decode",), dict(seq_len=None), -1, "seq_len"),
    (("prefill",), dict(cu_q=None), -1, "cu_q"),
    (("prefill",), dict(total_q=-1), -1, "total_q"),
    (("prefill",), dict(max_q=-1), -1, "max_q"),
]


@pytest.mark.parametrize("what,kw,code,text", [(w, kw, c, t) for ws, kw, c, t in REFUSED for w in ws])
def test_refusals(lk, what, kw, code, text):
    a = _Args(lk)
    assert a.call(what, **kw) == code
    assert text in lk.lib.lazy_last_error().decode()


@pytest.mark.parametrize("what,name", [(w, n) for w, ns in (("write", ("k", "v", "cache")), ("read", ("k", "v", "cache")),
                                                            ("decode", ("q", "cache", "out")),
                                                            ("prefill", ("q", "cache", "out"))) for n in ns])
def test_misaligned_tensors_are_refused(lk, what, name):
    a = _Args(lk)
    assert a.call(what, **{name: a.p + 8}) == -1
    assert "16-byte aligned" in lk.lib.lazy_last_error().decode()
    if what in ("decode", "prefill"):
        assert a.call(what, meta=a.p + 4) == -1
        assert "8-byte aligned" in lk.lib.lazy_last_error().decode()


@pytest.mark.parametrize("field,value,text", [("kind", 9, "positional kind"), ("rotary_dim", 24, "rotary_dim"),
                                              ("rotary_dim", 144, "rotary_dim"), ("rope_theta", 1.0, "rope_theta")])
def test_bad_positional_configurations_are_refused(lk, field, value, text):
    for what in ("write", "decode", "prefill"):
        a = _Args(lk)
        setattr(a.cfg, field, value)
        assert a.call(what) == -1
        assert text in lk.lib.lazy_last_error().decode()


def test_binding_refuses_tensors_it_cannot_pass_on(lk):
    import torch
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    idx = torch.zeros(3, dtype=torch.int32)
    cache = torch.zeros(lk.q4_cache_shape(4, 2, 64), dtype=torch.uint8)
    cfg = lk.pos_cfg_from("rope", 64)
    assert cache.shape == (4, 2, 1152)
    with pytest.raises(ValueError, match="head_dim"):
        lk.q4_cache_shape(4, 2, 96)
    with pytest.raises(ValueError, match="CUDA device"):
        lk.kv_write_q4(k, k, idx, idx, cache, cfg)
    with pytest.raises(ValueError, match="kv_cache must be"):
        lk.kv_write_q4(k, k, idx, idx, cache[:, :1], cfg)
    with pytest.raises(TypeError, match="torch.bfloat16"):
        lk.kv_write_q4(k.float(), k, idx, idx, cache, cfg)
    with pytest.raises(ValueError, match="shape"):
        lk.kv_write_q4(k, k[:2], idx, idx, cache, cfg)
    with pytest.raises(ValueError, match="contiguous"):
        lk.kv_read_q4(idx, cache, torch.zeros((2, 3, 64), dtype=torch.bfloat16).transpose(0, 1), k)
    with pytest.raises(TypeError, match="torch.int32"):
        lk.kv_read_q4(idx.long(), cache, k, k)
    with pytest.raises(TypeError, match="torch.uint8"):
        lk.kv_read_q4(idx, cache.to(torch.int8), k, k)


def test_binding_refuses_before_any_gpu_work(lk):
    import torch
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    a = _Args(lk)
    for what in EVERY:  # valid arguments, no usable GPU: an error code, no crash
        assert a.call(what) in (-3, -4)
