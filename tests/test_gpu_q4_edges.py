"""GPU tests of calls on the 4-bit cache that lie at the edge of what its interface allows.

Where two calls compute the same numbers (a table at another address, a looser bound on the query
lengths) their results are compared bit for bit.
"""
import numpy as np
import pytest

from oracle import lazy_oracle as lo
from tests import q4_reference as q4
from tests.gpu_common import lib
from tests.test_gpu_q4 import POISON, _bf, _clean, _dev, _i32, _tensor, _ws

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
