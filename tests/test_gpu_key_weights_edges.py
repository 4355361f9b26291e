"""GPU tests of key weights: query rows with a NaN, windows and bounds around one another, and the runner's bound of a
request's rows.  Tolerances are those of the call's own tests (``Votes.check``)."""
import numpy as np
import pytest

from tests import share_reference as ref
from tests.gpu_common import lib
from tests.test_gpu_evict import Votes, dev
from tests.test_gpu_runner_shared import batch
from tests.test_gpu_shared import bf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lk():
    return lib()


# up to 32 query rows per KV head, more of them, and with a bias
@pytest.mark.parametrize("name,b,row", [("odd_heads", 0, 0), ("odd_heads", 1, 1), ("interleaved", 0, 3), ("all_rows", 2, 0),
                                        ("all_rows", 0, 17), ("alibi", 0, 0), ("alibi", 0, 19), ("prompt", 0, 100)])
def test_a_nan_row_takes_the_keys_that_it_sees(lk, name, b, row):
    v = Votes(lk, name)
    clean = v.run().copy()
    x, i = v.x, int(v.cu[b]) + row
    v.qh[i, 1, 3] = np.nan
    v.q.copy_(bf(v.qh))
    v.lse[i, 1] = float("nan")  # as attention leaves it
    got = v.run()
    m = int(x.seq_len[b]) - int(v.cu[b + 1]) + i
    seen = np.zeros(got.shape, bool)
    seen[b, [k[0] for k in ref.keys(x.meta[b], x.doc_blocks[b], x.q_start[b], x.seq_len[b]) if k[1] <= m]] = True
    assert seen.any() and np.array_equal(np.isnan(got), seen)
    assert np.array_equal(np.where(seen, 0, got), np.where(seen, 0, clean))


@pytest.mark.parametrize("name", ["all_rows", "odd_heads", "alibi"])
@pytest.mark.parametrize("window,max_q", [(1, None), (7, 7), (10 ** 6, None), (2 ** 31 - 1, 2 ** 31 - 1), (9, 2 ** 31 - 1)])
def test_windows_and_bounds(lk, name, window, max_q):
    """A window may be longer than any request, and max_q longer than both."""
    v = Votes(lk, name)
    rows = max(np.diff(v.cu))
    got = v.run(window=window, max_q=rows if max_q is None or max_q < min(window, rows) else max_q)
    v.window = window
    v.check(got)
    assert lk.device_status() == 0


def test_runner_bounds_the_rows_of_a_request(lk):
    """Four tokens of each request: the bits of the call with max_q = 4."""
    import torch
    w, pb = batch(lk)
    n, D = 4 * pb.B, pb.D
    rng = np.random.default_rng(2)
    q = bf(rng.standard_normal((n, pb.Hq, D)))
    lse = dev(rng.standard_normal((n, pb.Hq)).astype(np.float32) + 4)
    cu = torch.arange(0, n + 1, 4, dtype=torch.int32, device="cuda")
    got = pb.key_weights(q, lse, pb.seq_len0, cu_q=cu, max_q=4)
    want = torch.empty_like(got)
    lk.attn_key_weights(q, lse, cu, pb.seq_len0, pb.q_start, pb.doc_blocks, pb.meta, pb.k_cache, pb.cfg, want, 4, ws=pb.ws)
    assert torch.equal(got, want) and got.any()
    assert lk.device_status() == 0


@pytest.mark.parametrize("name", ["window", "odd_heads", "alibi"])
def test_a_list_longer_than_the_row_of_words(lk, name):
    """A position behind the last word of the list: the status says so, as it does for attention."""
    v = Votes(lk, name)
    x = v.x
    x.seq_len[0] += 16 * 40
    v.g.seq_len.copy_(dev(x.seq_len.astype(np.int32)))
    got = v.run()
    x.meta = np.pad(x.meta, ((0, 0), (0, 40)))  # words without keys
    want = ref.key_weights(x, v.qh, v.lse_h, v.cu, v.window)
    nan = np.isnan(want)  # the rest of the segment's last page, visible now, was never written
    assert nan[0].any() and np.array_equal(np.isnan(got), nan)
    x.k = np.nan_to_num(x.k)
    v.check(np.where(nan, ref.key_weights(x, v.qh, v.lse_h, v.cu, v.window), got))
    assert lk.device_status() == 8


def test_idle_requests_and_requests_without_rows_report_nothing(lk):
    v = Votes(lk, "no_rows")
    v.x.seq_len[0] = 10 ** 6  # no rows
    v.x.seq_len[1] = 0
    v.g.seq_len.copy_(dev(v.x.seq_len.astype(np.int32)))
    assert not v.run().any()
    assert lk.device_status() == 0
