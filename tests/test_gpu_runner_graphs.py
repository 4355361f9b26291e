"""GPU tests of the runner's steps in graphs that were captured before the batch's groups, workspace or lists changed."""
import numpy as np
import pytest

import oracle
from tests.gpu_common import assert_close, lib, oracle_caches_for
from tests.oracle_setup import oracle_meta
from tests.test_gpu_runner_shared import batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lk():
    return lib()


def captured(step):
    import torch
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    return graph


def test_captured_steps_outlive_groups_workspaces_and_lists(lk):
    import torch
    w, pb = batch(lk, many=True, spare_pages=34 * 8)
    inp = pb.upload_decode(0)
    outs = [torch.empty((pb.B, pb.Hq, pb.D), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    lse = torch.empty((pb.B, pb.Hq), device="cuda")
    graphs, sizes = [captured(lambda: pb.decode_step(inp, out=outs[0]))], [pb.ws.numel()]
    pb.share_prefixes(min_blocks=4)
    graphs.append(captured(lambda: pb.decode_step(inp, out=outs[1])))
    sizes.append(pb.ws.numel())
    pb.share_prefixes(min_blocks=1000)  # every request a group of its own
    graphs.append(captured(lambda: pb.decode_step(inp, out=outs[2], lse=lse)))
    sizes.append(pb.ws.numel())
    weights = pb.key_weights(torch.cat([inp["q"]] * 9), torch.cat([lse] * 9), inp["seq_len"],
                             cu_q=torch.arange(0, 9 * pb.B + 1, 9, dtype=torch.int32, device="cuda"))  # (a larger workspace)
    assert pb.ws.numel() > sizes[0]
    # what could take the place of freed buffers
    others = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes + [8 * pb.meta.numel()] for _ in range(3)]
    kc, vc = oracle_caches_for(w, decode_steps=1)
    _, meta, seq_len, q_start, doc_blocks = oracle_meta(w)
    want, _ = oracle.decode(w.decode_tokens(0)[0], seq_len + 1, q_start, doc_blocks, meta, kc, vc, w.pos.as_dict())

    def replay():
        for o, g in zip(outs, graphs):
            o.fill_(float("nan"))
            g.replay()
        torch.cuda.synchronize()
        assert all((t == 0x5A).all() for t in others)

    replay()
    for i, o in enumerate(outs):
        assert_close(o, want, f"step {i}")
    pages = w.num_pages + np.arange(34 * 8).reshape(34, 8)
    weights = pb.key_weights(inp["q"], lse, inp["seq_len"])
    pb.evict(weights, np.full(pb.B, 60), pages, first=2, recent=4)
    others += [torch.full((8 * pb.meta.numel(),), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(4)]
    replay()
    now = pb.decode_step(inp)
    assert pb.groups is None and torch.equal(outs[0], now)
    for o in outs[1:]:
        assert_close(o, now.float().cpu().numpy().astype(np.float64), "after the eviction")
    assert not torch.equal(now.float(), torch.from_numpy(want).cuda().float())
    assert lk.device_status() == 0


def test_captured_step_with_its_weights(lk):
    """A decode step and the weights that its rows give, summed over replays of one graph."""
    import torch
    _, pb = batch(lk)
    inp = pb.upload_decode(0)
    lse = torch.empty((pb.B, pb.Hq), device="cuda")
    total = torch.zeros((pb.B, 16 * pb.max_blocks), device="cuda")

    def step():
        pb.decode_step(inp, lse=lse)
        pb.key_weights(inp["q"], lse, inp["seq_len"], weights=total)

    graph = captured(step)
    once = total.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert once.any() and torch.equal(total, 2 * once)  # (a sum of two equal numbers is exact)
    assert lk.device_status() == 0
