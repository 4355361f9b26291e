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
    pb.share_prefixes(min_blocks=1000)
    gc.collect()
    assert all(r() is not None for r in former)


def test_eviction_changes_the_lists_in_place(runner, monkeypatch):
    """A step that was captured before an eviction reads the lists of after it, and takes nothing for common: requests
    that shared documents have copies of their own now."""
    import torch
    monkeypatch.setattr(runner, "evict_plan", fake_plan)
    monkeypatch.setattr(runner, "kv_move", lambda *a: None)
    w, pb = batch(runner, spare_pages=34 * 10)
    pb.share_prefixes(min_blocks=1000)
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


def saved(meta, nd, off, shared, least):
    """What a grouping saves: a group's common words once instead of for every request, at the price of two readings, less
    the price of a group for every cut between requests that could be in one.  Checks that it is a grouping."""
    assert off[0] == 0 and off[-1] == len(nd) and (np.diff(off) > 0).all() and len(shared) == len(off) - 1
    total = 0
    for g, n in enumerate(shared):
        lo, hi = off[g], off[g + 1]
        assert all(nd[b] >= n and np.array_equal(meta[b, :n], meta[lo, :n]) for b in range(lo, hi))
        total += max(hi - lo - 2, 0) * int(n)
        if lo and min(nd[lo - 1], nd[lo]) >= least and np.array_equal(meta[lo, :least], meta[lo - 1, :least]):
            total -= 256
    return total


def lists(*prefixes, width=300):
    """Requests whose lists are these words, then words of their own."""
    meta = np.zeros((len(prefixes), width), np.uint64)
    nd = np.zeros(len(prefixes), np.int32)
    for b, p in enumerate(prefixes):
        nd[b] = len(p) + 3
        meta[b, :nd[b]] = list(p) + [10 ** 6 + 3 * b + i for i in range(3)]
    return meta, nd


SYSTEM = list(range(8))
LEFT, RIGHT = SYSTEM + list(range(100, 200)), SYSTEM + list(range(200, 300))


@pytest.mark.parametrize("name,requests,min_blocks,off,shared", [
    ("system_prompt", [LEFT] * 4 + [RIGHT] * 4, 8, [0, 4, 8], [108, 108]),
    ("outsider", [LEFT] * 13 + [SYSTEM] + [LEFT] * 14, 8, [0, 13, 14, 28], [108, 11, 108]),
    ("outsider_at_the_end", [LEFT] * 5 + [SYSTEM], 1, [0, 5, 6], [108, 11]),
    ("only_the_prompt", [SYSTEM + [1000 + b] * 50 for b in range(6)], 8, [0, 6], [8]),
    ("pairs", [SYSTEM + [1000 + b // 2] * 250 for b in range(6)], 8, [0, 6], [8]),  # (pairs gain nothing)
    ("shallow", [SYSTEM + [1000 + b // 8] * 30 for b in range(64)], 8, [0, 64], [8]),
    ("deep", [SYSTEM + [1000 + b // 8] * 120 for b in range(64)], 8, list(range(0, 72, 8)), [128] * 8),
    ("below_the_least", [LEFT] * 2 + [SYSTEM[:7]] * 2, 8, [0, 2, 3, 4], [108, 10, 10]),
])
def test_common_prefixes_keep_deep_sharing(runner, name, requests, min_blocks, off, shared):
    """What requests share beyond a prompt that all of them begin with is not given away for it."""
    meta, nd = lists(*requests)
    got = runner.common_prefixes(meta, nd, min_blocks)
    assert got[0].tolist() == off and got[1].tolist() == shared
    assert got[0].dtype == np.int32 and got[1].dtype == np.int32


@pytest.mark.parametrize("seed", range(40))
def test_common_prefixes_save_the_most(runner, seed):
    """Against every way to cut a batch of up to nine requests."""
    rng = np.random.default_rng(seed)
    n, least, width = int(rng.integers(1, 10)), int(rng.integers(1, 40)), 600
    deep = np.exp(rng.uniform(0, np.log(width), n)).astype(int)  # with the request before
    meta, nd = np.zeros((n, width), np.uint64), rng.integers(300, width, n).astype(np.int32)
    meta[0] = rng.integers(1, 1 << 40, width)
    for b in range(1, n):
        meta[b] = rng.integers(1, 1 << 40, width)
        meta[b, :deep[b]] = meta[b - 1, :deep[b]]
    off, shared = runner.common_prefixes(meta, nd, least)
    best = None
    for cuts in range(1 << (n - 1)):
        ends = [0] + [b for b in range(1, n) if cuts >> (b - 1) & 1] + [n]
        common = []
        for lo, hi in zip(ends, ends[1:]):
            same = (meta[lo:hi] == meta[lo]).all(0)
            k = int(min(nd[lo:hi].min(), width if same.all() else np.argmin(same)))
            common.append(int(nd[lo]) if hi - lo == 1 else k)
        if all(k >= least or hi - lo == 1 for k, lo, hi in zip(common, ends, ends[1:])):
            one = saved(meta, nd, np.array(ends), common, least)
            best = one if best is None else max(best, one)
    assert saved(meta, nd, off, shared, least) == best


def test_common_prefixes_of_a_large_batch(runner):
    """Thousands of requests: groups of unequal depth under one prompt."""
    meta, nd = lists(*[SYSTEM + [1000 + b // 37] * 60 for b in range(4000)], width=80)
    off, shared = runner.common_prefixes(meta, nd, 8)
    assert off.tolist() == list(range(0, 4000, 37)) + [4000] and (shared == 68).all()


def test_sharing_again_takes_no_more_memory(runner):
    """A loop that calls it before every step: groups that have not changed are the same tensors."""
    _, pb = batch(runner)
    n = pb.share_prefixes(min_blocks=4)
    groups = pb.groups
    for _ in range(3):
        assert pb.share_prefixes(min_blocks=4) == n
    assert pb.groups is groups and len(pb._all_groups) == 1
    pb.share_prefixes(min_blocks=1000)
    assert pb.groups is not groups and len(pb._all_groups) == 2
