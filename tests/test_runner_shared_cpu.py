"""CPU tests of the runner's host side over shared lists and of its eviction: buffers that captured steps name."""
import gc
import weakref

import numpy as np
import pytest

from tests import share_reference as ref
from workloads import PosCfg, make_custom


@pytest.fixture(scope="module")
def runner():
    import __graft_entry__
    __graft_entry__.build()
    from position_agnostic_kv_gb300 import runner as m
    return m


def batch(runner, **kw):
    docs = [[0, 1, 2], [0, 1], [0, 1, 3], [3, 2]] + [[4, 1, 0]] * 30
    w = make_custom([40, 200, 33, 17, 130], docs, 64, 32, 64, PosCfg("rope", rope_theta=1e4, rotary_dim=64),
                    [20, 17, 16, 5] + [3] * 30, 3)
    return w, runner.PagedBatch(w, device="cpu", **kw)


def fake_plan(weights, meta, doc_blocks, keep, dst, num_pages, cfg, new_meta, new_nd, src, to, new_w, first=0, recent=0):
    import torch
    got = ref.plan(weights.numpy(), meta.numpy().view(np.uint64), doc_blocks.numpy(), keep.numpy(), dst.numpy(), num_pages,
                   first, recent)
    for t, a in zip((new_meta, new_nd, src, to, new_w), got):
        t.copy_(torch.from_numpy(a.view(np.int64) if a.dtype == np.uint64 else a))


def test_outgrown_workspaces_stay(runner, monkeypatch):
    """A captured step goes on writing to the workspace that it was captured with."""
    import torch
    monkeypatch.setattr(runner, "attn_key_weights", lambda *a, **kw: None)
    _, pb = batch(runner)
    first, n = weakref.ref(pb.ws), pb.ws.numel()
    pb.share_prefixes(min_blocks=4)
    q, lse = torch.zeros((pb.B, pb.Hq, pb.D), dtype=torch.bfloat16), torch.zeros((pb.B, pb.Hq))
    pb.key_weights(q, lse, pb.seq_len0)
    gc.collect()
    assert pb.ws.numel() > n and first() is not None


def test_former_groups_stay(runner):
    _, pb = batch(runner)
    pb.share_prefixes(min_blocks=4)
    former = [weakref.ref(t) for t in pb.groups[:2]]
    pb.share_prefixes(min_blocks=1)
    gc.collect()
    assert all(r() is not None for r in former)


def test_eviction_changes_the_lists_in_place(runner, monkeypatch):
    """A step that was captured before an eviction reads the lists of after it, and takes nothing for common: requests
    that shared documents have copies of their own now."""
    import torch
    monkeypatch.setattr(runner, "evict_plan", fake_plan)
    monkeypatch.setattr(runner, "kv_move", lambda *a: None)
    w, pb = batch(runner, spare_pages=34 * 10)
    pb.share_prefixes(min_blocks=1)
    former = [pb.groups[1]]
    pb.share_prefixes(min_blocks=4)
    former.append(pb.groups[1])
    assert all(t.any() for t in former)
    meta, nd = pb.meta, pb.doc_blocks
    want_meta, want_nd = meta.clone(), nd.clone()
    rng = np.random.default_rng(0)
    weights = torch.from_numpy(rng.random((pb.B, 16 * pb.max_blocks)).astype(np.float32))
    pages = w.num_pages + np.arange(340).reshape(34, 10)
    want = ref.plan(weights.numpy(), meta.numpy().view(np.uint64).copy(), nd.numpy().copy(), np.full(34, 50), pages, w.num_pages + 340,
                    0, 0)
    pb.evict(weights, np.full(pb.B, 50), pages)
    assert not torch.equal(meta, want_meta) and not torch.equal(nd, want_nd)
    assert np.array_equal(meta.numpy().view(np.uint64), want[0]) and np.array_equal(nd.numpy(), want[1])
    assert pb.meta.data_ptr() == meta.data_ptr() and pb.doc_blocks.data_ptr() == nd.data_ptr()
    assert pb.groups is None and not any(t.any() for t in former)


def test_key_weights_copy_nothing_from_the_host(runner, monkeypatch):
    """A decode loop captures its weights with its step, and a capture takes no copies from pageable memory."""
    import torch
    seen = []
    monkeypatch.setattr(runner, "attn_key_weights", lambda q, lse, cu_q, *a, **kw: seen.append(cu_q))
    _, pb = batch(runner)
    monkeypatch.setattr(runner, "i32", lambda *a: pytest.fail("a copy from the host"))
    pb.key_weights(torch.zeros((pb.B, pb.Hq, pb.D), dtype=torch.bfloat16), torch.zeros((pb.B, pb.Hq)), pb.seq_len0)
    assert seen[0].dtype == torch.int32 and seen[0].tolist() == list(range(pb.B + 1))


def test_key_weights_pass_the_rows_of_a_request(runner, monkeypatch):
    """The bound of a request's rows decides with how many bits queries count: it is not the batch's number of rows."""
    import torch
    seen = []
    monkeypatch.setattr(runner, "attn_key_weights", lambda *a, **kw: seen.append(a[10]))
    _, pb = batch(runner)
    n = 4 * pb.B
    rows = lambda n: (torch.zeros((n, pb.Hq, pb.D), dtype=torch.bfloat16), torch.zeros((n, pb.Hq)), pb.seq_len0)  # noqa: E731
    cu = torch.arange(0, n + 1, 4, dtype=torch.int32)
    pb.key_weights(*rows(n), cu_q=cu, max_q=4)
    pb.key_weights(*rows(n), cu_q=cu)  # unknown: all rows could be one request's
    pb.key_weights(*rows(n), cu_q=cu, max_q=10 ** 6)
    pb.key_weights(*rows(pb.total_q), cu_q=pb.cu_q)  # the prefill's rows
    pb.key_weights(*rows(pb.B))
    assert seen == [4, n, n, 20, 1]
    with pytest.raises(ValueError, match="max_q"):
        pb.key_weights(*rows(n), cu_q=cu, max_q=-1)
