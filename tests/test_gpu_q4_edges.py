"""GPU tests of calls on the 4-bit cache that lie at the edge of what its interface allows.

Where two calls compute the same numbers (a table at another address) their results are
compared bit for bit.
"""
import numpy as np
import pytest

from tests.gpu_common import lib
from tests.test_gpu_q4 import POISON, _bf, _clean, _i32, _tensor

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
