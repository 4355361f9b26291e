"""GPU tests of the runner's path over shared lists and of its eviction."""
import numpy as np
import pytest

import oracle
from tests.gpu_common import assert_close, lib, oracle_caches_for
from tests.oracle_setup import oracle_meta
from workloads import PosCfg, make_custom

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lk():
    return lib()


def batch(lk, many=False, **kw):
    from position_agnostic_kv_gb300.runner import PagedBatch
    docs = [[0, 1, 2], [0, 1], [0, 1, 3], [3, 2]] + [[4, 1, 0]] * (30 * many)
    w = make_custom([40, 200, 33, 17, 130], docs, 64 if many else 8, 32 if many else 2, 64,
                    PosCfg("rope", rope_theta=1e4, rotary_dim=64), [20, 17, 16, 5] + [3] * (30 * many), 3)
    pb = PagedBatch(w, **kw)
    pb.fill_documents()
    pb.prefill(pb.upload_prefill())
    return w, pb


@pytest.mark.parametrize("many", [False, True])
def test_decode_steps_over_shared_prefixes(lk, many):
    w, pb = batch(lk, many)
    _, plain = batch(lk, many)
    assert pb.share_prefixes(min_blocks=4) == 3 + 30 * many
    kc, vc = oracle_caches_for(w, decode_steps=2)
    _, meta, seq_len, q_start, doc_blocks = oracle_meta(w)
    for t in range(2):
        out = pb.decode_step(pb.upload_decode(t))
        other = plain.decode_step(plain.upload_decode(t))
        q = w.decode_tokens(t)[0]
        ref, _ = oracle.decode(q, seq_len + t + 1, q_start, doc_blocks, meta, kc, vc, w.pos.as_dict())
        assert_close(out, ref, f"step {t}, shared")
        assert_close(other, ref, f"step {t}")
    assert lk.device_status() == 0


def test_eviction_between_decode_steps(lk):
    """Weights summed over two steps; everything kept: the same answers from the packed copies; then a cut."""
    import torch
    w, pb = batch(lk, spare_pages=100)
    _, plain = batch(lk)
    weights = None
    for t in range(2):
        inp = pb.upload_decode(t)
        lse = torch.empty((w.B, w.Hq), dtype=torch.float32, device="cuda")
        pb.decode_step(inp, lse=lse)
        plain.decode_step(plain.upload_decode(t))
        weights = pb.key_weights(inp["q"], lse, inp["seq_len"], weights=weights)
    total = weights.sum(1).cpu().numpy()
    assert np.abs(total - 2 * w.Hq).max() <= 1e-3 * w.Hq  # every row gives its weights away
    pages = w.num_pages + np.arange(100).reshape(w.B, 25)
    nd = pb.doc_blocks.clone()
    moved = pb.evict(weights, np.full(w.B, 10 ** 6), pages)
    assert torch.equal(pb.doc_blocks, nd) and torch.equal(moved, weights)
    # different pages, the same keys in the same places
    assert_close(pb.decode_step(pb.upload_decode(2)), plain.decode_step(plain.upload_decode(2)).float().cpu().numpy(), "moved",
                 1e-6, 1e-6, 1e-6)
    free = np.setdiff1d(np.arange(w.num_pages), np.unique(pb.meta.cpu().numpy().view(np.uint64) >> np.uint64(40)))
    small = pb.evict(moved, np.full(w.B, 32), free[:w.B * 5].reshape(w.B, 5), first=2, recent=4)
    assert (pb.doc_blocks <= 5).all()
    out = pb.decode_step(pb.upload_decode(2))
    assert torch.isfinite(out.float()).all() and (small.sum(1) <= moved.sum(1)).all()
    assert lk.device_status() == 0


def test_four_bit_batches_refuse(lk):
    _, pb = batch(lk, kv_bits=4)
    for call in (pb.share_prefixes, lambda: pb.key_weights(None, None, None), lambda: pb.evict(None, None, None)):
        with pytest.raises(ValueError, match="bf16"):
            call()
