"""GPU tests of the decode over lists that share their first documents.

Tolerances, from the arithmetic that the kernels document.  With A = sum_j p_j |v_j|, and E the largest error of a
score, which changes a weight by at most E of itself and the sum of the weights by as much, so an output by 2 E A:
  * the output is rounded to bf16: at most 2^-8 of it;
  * own keys: queries and weights are held in two bf16 numbers, off by at most 2^-17 of themselves:
    E = 2^-17 |q| |k| scale;
  * common keys: queries and rotated keys are f16 numbers, off by at most 2^-11 each: E = 2^-10 |q| |k| scale; the
    weights are rounded to bf16, off by at most 2^-8: 2^-8 A (their sum is taken before the rounding);
  * angles are good to 2^-20 |q| |k| scale of a score, sums run in fp32: 2^-12 A covers both.
These are worst cases.  Roundings average out, so the relative Frobenius error is held to 2^-7: the two roundings
to bf16, each at its largest.
"""
import numpy as np
import pytest

from tests import share_reference as ref
from tests.gpu_common import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lk():
    return lib()


def dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def bf(x):
    import torch
    return dev(np.asarray(x, np.float32), torch.bfloat16)


def cfg_of(lk, pos, D, slopes=None):
    return lk.pos_cfg_from(pos["kind"], D, rope_theta=pos["theta"], yarn_factor=4.0, yarn_orig_ctx=4096, alibi_slopes=slopes,
                           rotary_dim=pos["rotary_dim"], interleaved=pos["interleaved"])


class OnGpu:
    """The tensors of a ``Lists`` batch, and its shared decode."""

    def __init__(self, lk, x, max_group=None, max_shared=None):
        import torch
        self.lk, self.x = lk, x
        self.q, self.k, self.v = bf(x.q), bf(x.k), bf(x.v)
        self.seq_len, self.q_start, self.doc_blocks = (dev(a.astype(np.int32)) for a in (x.seq_len, x.q_start, x.doc_blocks))
        self.meta = dev(x.meta.view(np.int64))
        self.off, self.shared = dev(np.array(x.off, np.int32)), dev(np.array(x.shared, np.int32))
        self.max_group = int(np.diff(x.off).max()) if max_group is None and len(x.shared) else (max_group or 0)
        self.max_shared = max(x.shared) if max_shared is None and len(x.shared) else (max_shared or 0)
        self.slopes = dev(x.slopes) if x.slopes is not None else None
        self.cfg = cfg_of(lk, x.pos, x.D, self.slopes)
        n = lk.decode_shared_workspace_size(x.B, len(x.shared), self.max_group, self.max_shared, x.max_blocks, x.Hq, x.Hkv, x.D)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        self.out, self.lse = torch.full_like(self.q, float("nan")), torch.full(self.q.shape[:2], float("nan"), device="cuda")

    def decode(self, **kw):
        self.lk.attn_decode_shared(self.q, self.seq_len, self.q_start, self.doc_blocks, self.meta, self.off, self.shared,
                                   self.max_group, self.max_shared, self.k, self.v, self.cfg, self.out, lse=self.lse,
                                   ws=self.ws, **kw)
        return self.out, self.lse


def check(out, lse, want):
    o, ls, mass, reach = want
    got = out.float().cpu().numpy().astype(np.float64)
    E = 2.0 ** -10 * reach
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -12 + 2 * E) * mass * (1 + 2.0 ** -6)
    assert np.isfinite(got).all()
    bad = np.abs(got - o) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - o).max())
    rel = np.linalg.norm(got - o) / max(np.linalg.norm(o), 1e-300)
    assert rel <= 2.0 ** -7, rel
    got = lse.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(got), np.isneginf(ls))
    f = ~np.isneginf(ls)
    assert (np.abs(got[f] - ls[f]) <= E + 2.0 ** -20 * (1 + np.abs(ls[f]))).all(), np.abs(got[f] - ls[f]).max()


ROPE = dict(kind="rope", theta=1e4, rotary_dim=128, interleaved=False)


def pos_of(kind="rope", rd=128, inter=False):
    return dict(kind=kind, theta=1e4, rotary_dim=rd, interleaved=inter)


def own_and_common(n=(14, 16), outside=2):
    """Two groups, requests outside them, and documents of some requests' own."""
    B = sum(n) + outside
    own = [[[], [20], [50, 3], [], [16]][i % 5] for i in range(B)]
    return [(n[0], [33, 64]), (n[1], [128, 7])], own, [[1, 17, 2, 16, 40, 33][i % 6] for i in range(B)]


# Few and short lists are decoded one by one; from some thousand pages on a group's common keys are taken together
# (tests below look at which it is).
ALONE = {  # groups (requests, common documents), own documents, segments, Hq, Hkv, D, pos
    "one_group": ([(3, [40, 200, 16])], [[]] * 3, [5, 1, 33], 8, 2, 128, pos_of()),
    "own_documents": ([(2, [33]), (3, [128, 7])], [[20], [], [50, 3], [], [16]], [1, 17, 2, 16, 40], 8, 2, 128, pos_of()),
    "outside": ([(2, [130])], [[], [], [300], [1]], [3, 3, 20, 1], 4, 4, 128, pos_of()),
    "no_groups": ([], [[5, 18], []], [4, 9], 4, 2, 64, pos_of(rd=64)),
    "nothing_common": ([(2, []), (1, [])], [[30], [], [17]], [2, 3, 4], 4, 1, 64, pos_of(rd=64)),
    "group_of_one": ([(1, [500])], [[]], [1], 8, 1, 128, pos_of()),
    "many_rows": ([(40, [100, 64])], [[]] * 40, [1 + i % 20 for i in range(40)], 8, 1, 128, pos_of()),
    "two_tiles": ([(33, [150])], [[]] * 33, [2] * 33, 16, 2, 64, pos_of(rd=64)),
    "wide_heads": ([(3, [300, 20])], [[], [7], []], [4, 5, 6], 24, 1, 128, pos_of()),
    "very_wide": ([(2, [140])], [[], []], [1, 2], 160, 1, 64, pos_of(rd=64)),
    "odd_heads": ([(5, [90])], [[]] * 5, [3] * 5, 10, 2, 64, pos_of(rd=64)),
    "short_documents": ([(4, [1, 2, 3, 16, 17, 15, 1, 40, 5, 31, 9])], [[]] * 4, [2, 1, 1, 3], 8, 2, 128, pos_of()),
    "interleaved": ([(3, [70, 33])], [[9], [], []], [1, 20, 3], 8, 2, 128, pos_of(inter=True)),
    "partial": ([(3, [70, 33])], [[9], [], []], [1, 20, 3], 8, 2, 128, pos_of(rd=48)),
    "partial_interleaved": ([(3, [70, 33])], [[9], [], []], [1, 20, 3], 4, 2, 64, pos_of(rd=16, inter=True)),
    "yarn": ([(3, [70, 233])], [[9], [], []], [1, 20, 3], 8, 2, 128, pos_of("yarn")),
    "alibi": ([(3, [70, 233])], [[9], [], []], [1, 20, 3], 8, 2, 128, pos_of("alibi")),
    "alibi_mqa": ([(6, [400])], [[]] * 6, [1, 2, 3, 4, 5, 6], 32, 1, 64, pos_of("alibi", 64)),
    "none": ([(3, [70, 33])], [[9], [], []], [1, 20, 3], 8, 2, 64, pos_of("none", 64)),
    "long": ([(9, [1600, 900, 33])], [[]] * 9, [33] * 9, 8, 2, 128, pos_of()),
    "own_long": ([(2, [64])], [[1500, 700], [900]], [3, 3], 4, 1, 128, pos_of()),
}
KINDS = ([(20, [70, 233, 5])], [[9] if i % 3 == 0 else [] for i in range(20)], [1 + i for i in range(20)])
TOGETHER = {
    "t_one_q_tile": ([(20, [40, 200, 16])], [[]] * 20, [1 + i % 18 for i in range(20)], 64, 32, 64, pos_of(rd=64)),
    "t_two_q_tiles": ([(40, [150, 33, 7])], [[]] * 40, [2] * 40, 64, 16, 128, pos_of()),
    "t_two_pairs": ([(40, [130])], [[]] * 40, [2] * 40, 160, 16, 64, pos_of(rd=64)),
    "t_one_head": ([(24, [400, 64])], [[]] * 24, [3] * 24, 16, 16, 128, pos_of()),
    "t_ragged": ([(13, [300, 20]), (1, [50]), (9, []), (30, [16] * 9)], [[7] if i % 4 == 0 else [] for i in range(55)],
                 [1 + i % 9 for i in range(55)], 16, 16, 128, pos_of()),
    "t_wide": ([(12, [300, 20])], [[]] * 12, [4] * 12, 384, 16, 64, pos_of(rd=64)),
    "t_very_wide": ([(4, [140])], [[]] * 4, [1, 2, 3, 4], 1920, 12, 64, pos_of(rd=64)),
    "t_own": (*own_and_common(), 64, 32, 64, pos_of(rd=64)),
    "t_short_documents": ([(30, [1, 2, 3, 16, 17, 15, 1, 40, 5, 31, 9])], [[]] * 30, [2] * 30, 32, 32, 128, pos_of()),
    "t_long": ([(9, [1600, 900, 33])], [[]] * 9, [33] * 9, 32, 8, 128, pos_of()),
    "t_long_small_heads": ([(9, [1600, 900, 33])], [[]] * 9, [33] * 9, 32, 8, 64, pos_of(rd=64)),
    "t_interleaved": (*KINDS, 64, 32, 128, pos_of(inter=True)),
    "t_partial": (*KINDS, 32, 32, 128, pos_of(rd=48)),
    "t_partial_interleaved": (*KINDS, 64, 32, 64, pos_of(rd=16, inter=True)),
    "t_yarn": (*KINDS, 32, 32, 128, pos_of("yarn")),
    "t_alibi": (*KINDS, 64, 32, 128, pos_of("alibi")),
    "t_alibi_two_q_tiles": ([(40, [150, 33, 7])], [[]] * 40, [2] * 40, 64, 16, 64, pos_of("alibi", 64)),
    "t_none": (*KINDS, 32, 32, 64, pos_of("none", 64)),
}
CASES = ALONE | TOGETHER
BOTH = pytest.mark.parametrize("name", ["own_documents", "t_own"])


def lists(name, seed=0, **kw):
    groups, own, seg, Hq, Hkv, D, pos = CASES[name]
    return ref.Lists(np.random.default_rng(seed + 17), groups, own, seg, Hq, Hkv, D, pos, **kw)


@pytest.mark.parametrize("name", CASES)
def test_decode_shared(lk, name):
    x = lists(name)
    g = OnGpu(lk, x)
    alone = lk.decode_shared_workspace_size(x.B, 0, 0, 0, x.max_blocks, x.Hq, x.Hkv, x.D)
    assert (g.ws.numel() != alone) == (name in TOGETHER)  # partial results of the common keys
    out, lse = g.decode()
    check(out, lse, ref.decode(x))
    assert lk.device_status() == 0


@BOTH
def test_agrees_with_decode(lk, name):
    """attn_decode over the same lists."""
    import torch
    x = lists(name)
    g = OnGpu(lk, x)
    out, lse = g.decode()
    n = lk.workspace_size(lk.PHASE_DECODE, x.B, x.B, x.max_blocks, x.Hq, x.Hkv, x.D)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    other, ols = torch.empty_like(out), torch.empty_like(lse)
    lk.attn_decode(g.q, g.seq_len, g.q_start, g.doc_blocks, g.meta, g.k, g.v, g.cfg, other, lse=ols, ws=ws)
    want = ref.decode(x)
    check(out, lse, want)
    check(other, ols, want)


@BOTH
@pytest.mark.parametrize("scale", [0.02, 2.0])
def test_scale(lk, scale, name):
    x = lists(name)
    out, lse = OnGpu(lk, x).decode(scale=scale)
    check(out, lse, ref.decode(x, scale=scale))


@BOTH
def test_small_queries_under_a_large_scale(lk, name):
    x = lists(name)
    x.q = x.q * 2.0 ** -40
    scale = 2.0 ** 40 / np.sqrt(x.D)
    out, lse = OnGpu(lk, x).decode(scale=scale)
    check(out, lse, ref.decode(x, scale=scale))


@BOTH
def test_idle_requests(lk, name):
    """Requests of length 0 inside and outside groups: zeros, and -inf."""
    x = lists(name)
    x.seq_len[[0, 3, x.B - 1]] = 0
    out, lse = OnGpu(lk, x).decode()
    want = ref.decode(x)
    check(out, lse, want)
    assert not out[[0, 3, x.B - 1]].any() and np.isneginf(lse[[0, 3, x.B - 1]].cpu().numpy()).all()
    assert lk.device_status() == 0


@pytest.mark.parametrize("name", ["one_group", "t_one_q_tile", "t_two_q_tiles", "t_alibi"])
def test_requests_inside_their_documents(lk, name):
    """A position before the end of the documents sees the keys up to itself."""
    x = lists(name)
    x.seq_len[:] = np.resize([100, 1, 250, 37, 16, 17], x.B)
    x.seq_len = np.minimum(x.seq_len, x.q_start + np.array(x.seg))
    out, lse = OnGpu(lk, x).decode()
    check(out, lse, ref.decode(x))


@pytest.mark.parametrize("name,max_group,max_shared", [
    ("own_documents", 2, None), ("own_documents", None, 3), ("own_documents", 1, 1), ("own_documents", 0, 0),
    ("t_own", 11, None), ("t_own", None, 8), ("t_two_q_tiles", 38, 13)])
def test_bounds_that_are_too_small(lk, name, max_group, max_shared):
    """What the call's bounds cut off is decoded alone: the same result, and a status bit."""
    x = lists(name)
    g = OnGpu(lk, x, max_group if max_group is not None else max(np.diff(x.off)),
              max_shared if max_shared is not None else max(x.shared))
    out, lse = g.decode()
    check(out, lse, ref.decode(x))
    assert lk.device_status() == 8


@BOTH
@pytest.mark.parametrize("max_group,max_shared", [(100, 10 ** 6), (17, 12)])
def test_bounds_that_are_too_large(lk, name, max_group, max_shared):
    x = lists(name)
    out, lse = OnGpu(lk, x, max_group, max_shared).decode()
    check(out, lse, ref.decode(x))
    assert lk.device_status() == 0


@BOTH
def test_pages_outside_the_cache(lk, name):
    """Their keys are left out and the status says so; in common documents and in a request's own."""
    x = lists(name)
    bad = [(b, 1) for b in range(x.off[1])] + [(b, 3) for b in range(x.off[1], x.off[2])] + [(x.off[1], int(x.shared[1]))]
    want = x.meta.copy()
    for b, j in bad:
        x.meta[b, j] = int(x.meta[b, j]) & ((1 << 40) - 1) | (x.num_pages + 5) << 40
        want[b, j] = int(want[b, j]) & ~31
    out, lse = OnGpu(lk, x).decode()
    check(out, lse, ref.decode(x, meta=want))
    assert lk.device_status() == 1


@BOTH
def test_nan_stays_in_its_request(lk, name):
    """A NaN in a request's own value reaches only its columns; in a common value, that column of the whole group."""
    x = lists(name)
    clean = ref.decode(x)
    G, lo, hi = x.Hq // x.Hkv, x.off[1], x.off[2]
    own = ref.keys(x.meta[0], x.doc_blocks[0], x.q_start[0], x.seq_len[0])[-1]
    com = ref.keys(x.meta[lo], x.doc_blocks[lo], x.q_start[lo], x.seq_len[lo])[5]
    x.v[own[3], 1, own[4], 7] = np.nan
    x.v[com[3], 0, com[4], 9] = np.nan
    g = OnGpu(lk, x)
    got = g.decode()[0].float().cpu().numpy()
    hit = np.zeros(got.shape, bool)
    hit[0, G:2 * G, 7] = True
    hit[lo:hi, :G, 9] = True
    assert np.array_equal(np.isnan(got), hit)
    assert np.abs(np.where(hit, 0, got - clean[0])).max() < 0.05


@pytest.mark.parametrize("name", ["one_group", "t_one_q_tile", "t_two_q_tiles"])
def test_nan_keys_and_queries(lk, name):
    x = lists(name)
    G = x.Hq // x.Hkv
    com = ref.keys(x.meta[0], x.doc_blocks[0], x.q_start[0], x.seq_len[0])[44]
    x.k[com[3], 1, com[4], 3] = np.nan
    x.q[1, 0] = np.nan
    got = OnGpu(lk, x).decode()[0].float().cpu().numpy()
    nan = np.isnan(got).all(-1)
    assert nan[:, G:2 * G].all() and nan[1, 0] and nan.sum() == x.B * G + 1
    assert np.isnan(got).sum() == nan.sum() * x.D


@pytest.mark.parametrize("name", ["many_rows", "t_two_q_tiles", "t_ragged"])
def test_repeats_itself(lk, name):
    x = lists(name)
    g = OnGpu(lk, x)
    a = [t.clone() for t in g.decode()]
    g.ws.fill_(0x55)
    b = g.decode()
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all()


@BOTH
def test_stream_and_graph(lk, name):
    """On another stream, and captured once and replayed on other queries, lengths and groups."""
    import torch
    x, y = lists(name), lists(name, 5)
    g = OnGpu(lk, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.decode(stream=s)
    s.synchronize()
    check(g.out, g.lse, ref.decode(x))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.decode()
    h = OnGpu(lk, y)
    y.off = [0, y.off[1], y.off[2] - 1]  # the last request of the second group leaves it
    for name in ("q", "k", "v", "meta", "seq_len"):
        getattr(g, name).copy_(getattr(h, name))
    g.off.copy_(dev(np.array(y.off, np.int32)))
    for _ in range(3):
        g.out.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    check(g.out, g.lse, ref.decode(y))


def test_back_to_back_calls_share_a_workspace(lk):
    """Calls of different sizes one after another on one stream and one workspace."""
    import torch
    gs = [OnGpu(lk, lists(n)) for n in ("many_rows", "t_two_q_tiles", "one_group", "t_ragged", "t_alibi", "long", "no_groups")]
    ws = max((g.ws for g in gs), key=lambda t: t.numel())
    for g in gs:
        g.ws = ws
    for _ in range(3):
        for g in gs:
            g.decode()
    torch.cuda.synchronize()
    for g in gs:
        check(g.out, g.lse, ref.decode(g.x))
