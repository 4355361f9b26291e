"""CPU tests of the key weights' workspace: the size call against the sums that a call writes, counted from its launch's
definition (row blocks, groups of them, sums per group) over heads, rows, lists and positional kinds."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def lk():
    import __graft_entry__
    __graft_entry__.build()
    import position_agnostic_kv_gb300 as m
    return m


def planes_written(R, pages, sms, alibi):
    """Sums per key and KV head that a call writes whose longest request has R rows per KV head; ``pages``: list blocks of
    all requests and KV heads."""
    rows = min(max(16, -(-R // 16) * 16), 64 if alibi else 128)  # a block's
    blocks = -(-R // rows)
    per = max(1, blocks * pages // (32 * sms))  # row blocks in a group
    groups = min(8, max(1, -(-blocks // per)))
    return groups * (1 if rows <= 32 else 2)  # of many rows each warpgroup has half of the columns


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 20])
def test_workspace_holds_every_sum(lk, G, alibi):
    for total in np.unique(np.concatenate([np.arange(1, 300), np.geomspace(300, 40000, 60).astype(int)])):
        for B, Hkv, blocks in ((1, 1, 1), (1, 8, 100), (7, 2, 40), (64, 8, 2100)):
            size = lk.workspace_size(lk.PHASE_KEY_WEIGHTS, int(total), B, blocks, G * Hkv, Hkv, 128)
            plane = Hkv * B * blocks * 16 * 4
            assert size % plane == 0
            # requests that have all of the rows, and down to one
            for n in {int(total), -(-int(total) // B), 1}:
                assert planes_written(n * G, B * Hkv * blocks, 152, alibi) * plane <= size, (total, B, Hkv, blocks, n)


def test_workspace_grows_with_rows(lk):
    """A buffer for more rows serves a call with fewer."""
    sizes = [lk.workspace_size(lk.PHASE_KEY_WEIGHTS, n, 2, 10, 8, 2, 64) for n in range(1, 400)]
    assert sizes == sorted(sizes)
