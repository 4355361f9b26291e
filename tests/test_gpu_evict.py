"""GPU tests of eviction inside a context: the weights that keys receive, the plan, the rows' copies, and the
run of them with prefill and decode.

Tolerance of the weights, from the arithmetic that the kernel documents: queries are held in two bf16 numbers, off
by at most 2^-17 of themselves, and angles are good to 2^-20, so a score is off by at most E = 2^-16 |q| |k| scale; score
and log-sum-exp are fp32 numbers in base 2 and their difference is rounded, 2^-23 (|s| + |lse|) in all.  A weight is
off by both times itself, plus 2^-22 for the exponential; a sum of n weights by n 2^-24 of itself more.  Roundings
average out: the relative Frobenius error is held to 1e-5.
"""
import numpy as np
import pytest

from tests import share_reference as ref
from tests.gpu_common import lib
from tests.test_gpu_shared import OnGpu, bf, cfg_of, check, dev, pos_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lk():
    return lib()


# ------------------------------------------------------------------ weights
WEIGHTS = {  # documents per request, segments, rows of q per request, window, Hq, Hkv, D, pos
    "step": ([[40, 200], [7], []], [5, 1, 33], [1, 1, 1], 0, 8, 2, 128, pos_of()),
    "window": ([[40, 200], [7], [300]], [5, 1, 40], [5, 1, 40], 8, 8, 2, 128, pos_of()),
    "all_rows": ([[40], [], [130, 33]], [50, 20, 40], [50, 20, 40], 0, 4, 1, 128, pos_of()),
    "no_rows": ([[40], [20], [9]], [5, 6, 7], [0, 6, 0], 0, 4, 2, 64, pos_of(rd=64)),
    "some_rows": ([[60], [20, 20]], [30, 40], [3, 17], 0, 4, 2, 64, pos_of(rd=64)),
    "wide": ([[100], [20]], [9, 3], [9, 3], 0, 24, 1, 64, pos_of(rd=64)),
    "very_wide": ([[100]], [4], [4], 0, 160, 1, 128, pos_of()),
    "odd_heads": ([[100], [20]], [9, 3], [2, 3], 0, 10, 2, 64, pos_of(rd=64)),
    "short_documents": ([[1, 2, 3, 16, 17, 15, 1, 40, 5, 31, 9], [1]], [4, 2], [4, 2], 0, 8, 2, 128, pos_of()),
    "interleaved": ([[70, 33], [9]], [20, 3], [20, 3], 0, 8, 2, 128, pos_of(inter=True)),
    "partial": ([[70, 33], [9]], [20, 3], [20, 1], 0, 8, 2, 128, pos_of(rd=48)),
    "partial_interleaved": ([[70, 33], [9]], [20, 3], [20, 3], 5, 4, 2, 64, pos_of(rd=16, inter=True)),
    "yarn": ([[70, 233], [9]], [20, 3], [20, 3], 0, 8, 2, 128, pos_of("yarn")),
    "alibi": ([[70, 233], [9]], [20, 3], [20, 3], 0, 8, 2, 128, pos_of("alibi")),
    "none": ([[70, 33], [9]], [20, 3], [1, 3], 0, 8, 2, 64, pos_of("none", 64)),
    "many_heads": ([[333], [90]], [2, 2], [2, 2], 0, 32, 32, 64, pos_of(rd=64)),
    "long": ([[1600, 900, 33], [2000]], [40, 33], [40, 33], 32, 8, 2, 128, pos_of()),
    "prompt": ([[]], [700], [700], 0, 4, 2, 128, pos_of()),
}


class Votes:
    """Queries of the last rows of every request, their log-sum-exp, and the call."""

    def __init__(self, lk, name, seed=0, accumulate=False):
        import torch
        docs, seg, rows, window, Hq, Hkv, D, pos = WEIGHTS[name]
        rng = np.random.default_rng(seed + 23)
        self.lk, self.window, self.accumulate = lk, window, accumulate
        self.x = x = ref.Lists(rng, [], docs, seg, Hq, Hkv, D, pos, slack=2)
        self.g = OnGpu(lk, x)
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.qh = ref.bf16(rng.standard_normal((int(self.cu[-1]), Hq, D)))
        self.lse_h = np.zeros(self.qh.shape[:2], np.float32)
        for b in range(x.B):
            lo, hi = self.cu[b], self.cu[b + 1]
            if hi > lo:
                self.lse_h[lo:hi] = ref.softmax(ref.scores(x, b, self.qh[lo:hi], x.seq_len[b] - hi + np.arange(lo, hi))[0])[1]
        self.q, self.lse, self.cu_q = bf(self.qh), dev(self.lse_h), dev(self.cu)
        self.max_q = max(rows)
        self.base = rng.random((x.B, x.max_blocks * 16)).astype(np.float32)
        self.weights = dev(self.base)
        n = lk.workspace_size(lk.PHASE_KEY_WEIGHTS, len(self.qh), x.B, x.max_blocks, Hq, Hkv, D)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, **kw):
        g = self.g
        kw = dict(window=self.window, accumulate=self.accumulate, max_q=self.max_q) | kw
        self.lk.attn_key_weights(self.q, self.lse, self.cu_q, g.seq_len, g.q_start, g.doc_blocks, g.meta, g.k, g.cfg,
                                 self.weights, ws=self.ws, **kw)
        return self.weights.cpu().numpy().astype(np.float64)

    def check(self, got, scale=None):
        x = self.x
        want = ref.key_weights(x, self.qh, self.lse_h, self.cu, self.window)
        base = self.base.astype(np.float64) if self.accumulate else 0.0
        real = np.nan_to_num(x.k)
        s = np.linalg.norm(self.qh, axis=-1).max(initial=0) * np.linalg.norm(real, axis=-1).max() * ref.scale_of(x.pos, x.D)
        s2 = 1.4427 * (s + np.abs(np.where(np.isneginf(self.lse_h), 0, self.lse_h)).max(initial=0))
        if x.pos["kind"] == "alibi":
            s2 += 1.4427 * x.seq_len.max()  # slopes are below 1
        n = self.max_q * x.Hq
        tol = (2.0 ** -16 * s + 2.0 ** -23 * s2 + 2.0 ** -22 + n * 2.0 ** -24) * want + 2.0 ** -24 * np.abs(want + base) + 1e-30
        off = np.abs(got - want - base)
        assert (off <= tol).all(), (np.argwhere(off > tol)[:5], off.max())
        if want.any() and not self.accumulate:
            assert np.linalg.norm(off) <= 1e-5 * np.linalg.norm(want), np.linalg.norm(off) / np.linalg.norm(want)
        if not self.accumulate:
            assert not got[want == 0].any()
        return want


@pytest.mark.parametrize("name", WEIGHTS)
def test_key_weights(lk, name):
    v = Votes(lk, name)
    v.check(v.run())
    assert lk.device_status() == 0


@pytest.mark.parametrize("name", ["step", "all_rows", "alibi"])
def test_key_weights_accumulate(lk, name):
    v = Votes(lk, name, accumulate=True)
    v.check(v.run())


def test_weights_of_all_rows_sum_to_their_number(lk):
    v = Votes(lk, "all_rows")
    got = v.run()
    n = np.diff(v.cu) * v.x.Hq
    assert np.abs(got.sum(1) - n).max() <= 1e-4 * n.max()


def test_key_weights_of_rows_without_a_key(lk):
    """lse = -inf marks a row that saw nothing: it counts nothing."""
    v = Votes(lk, "window")
    v.lse_h[1] = -np.inf
    v.lse_h[7, 3] = -np.inf
    v.lse.copy_(dev(v.lse_h))
    v.check(v.run())


def test_key_weights_bounds(lk):
    """max_q may be any upper bound, also of more rows than there are."""
    v = Votes(lk, "window")
    v.check(v.run(max_q=10 ** 6))
    v.weights.copy_(dev(v.base))
    v.check(v.run(window=0) if v.window == 0 else v.run())


def test_key_weights_of_idle_requests(lk):
    v = Votes(lk, "step")
    v.x.seq_len[1] = 0
    v.g.seq_len.copy_(dev(v.x.seq_len.astype(np.int32)))
    got = v.run()
    assert not got[1].any()
    v.check(got)


def test_key_weights_of_more_rows_than_tokens(lk):
    """Rows before the sequence's first token see nothing; the others' positions count from the end."""
    v = Votes(lk, "window")
    v.x.seq_len[0] = 3
    v.g.seq_len.copy_(dev(v.x.seq_len.astype(np.int32)))
    v.check(v.run())
    assert lk.device_status() == 0


def test_key_weights_beyond_max_q(lk):
    """Of more rows than max_q the last max_q count, and the status says so."""
    v = Votes(lk, "all_rows")
    got = v.run(max_q=17)
    v.window = 17
    v.check(got)
    assert lk.device_status() == 8


def test_key_weights_bad_page(lk):
    v = Votes(lk, "window")
    x = v.x
    want_meta = x.meta.copy()
    j = 1
    x.meta[0, j] = int(x.meta[0, j]) & ((1 << 40) - 1) | (x.num_pages + 3) << 40
    v.g.meta.copy_(dev(x.meta.view(np.int64)))
    got = v.run()
    want_meta[0, j] = int(want_meta[0, j]) & ~31
    x.meta = want_meta
    v.check(got)
    assert lk.device_status() == 1


def test_key_weights_nan(lk):
    """A NaN key takes its own weight; a NaN row takes the weights of every key that it sees."""
    v = Votes(lk, "all_rows")
    clean = v.run()
    x = v.x
    key = ref.keys(x.meta[0], x.doc_blocks[0], x.q_start[0], x.seq_len[0])[10]
    x.k[key[3], 0, key[4], 5] = np.nan
    v.g.k.copy_(bf(x.k))
    got = v.run()
    assert np.isnan(got[0, key[0]]) and np.isnan(got).sum() == 1
    got[0, key[0]] = clean[0, key[0]]
    assert np.array_equal(got, clean)


def test_key_weights_repeat_themselves(lk):
    v = Votes(lk, "long")
    a = v.run()
    v.ws.fill_(0x55)
    assert np.array_equal(a, v.run())


def test_key_weights_of_many_requests(lk):
    """More requests than a warp has lanes, of very different sizes, some without rows and some without keys."""
    n = 75
    WEIGHTS["many"] = ([[(37 * b) % 290] if b % 5 else [] for b in range(n)], [1 + b * b % 41 for b in range(n)],
                       [min(1 + b * b % 41, b % 4 * 3) for b in range(n)], 0, 8, 2, 128, pos_of())
    try:
        v = Votes(lk, "many")
    finally:
        del WEIGHTS["many"]
    for b in (0, 33, 63, 64, 74):
        v.x.seq_len[b] = 0
    v.g.seq_len.copy_(dev(v.x.seq_len.astype(np.int32)))
    got = v.run()
    assert not got[[0, 33, 63, 64, 74]].any()
    v.check(got)
    assert lk.device_status() == 0


@pytest.mark.parametrize("accumulate", [False, True])
def test_key_weights_without_rows(lk, accumulate):
    v = Votes(lk, "window", accumulate=accumulate)
    v.q, v.lse = v.q[:0], v.lse[:0]
    v.cu_q.zero_()
    assert np.array_equal(v.run(max_q=0), v.base if accumulate else 0 * v.base)
    assert lk.device_status() == 0


def test_key_weights_stream_and_graph(lk):
    import torch
    v, u = Votes(lk, "window"), Votes(lk, "window", 9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    v.run(stream=s)
    s.synchronize()
    v.check(v.weights.cpu().numpy().astype(np.float64))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v.lk.attn_key_weights(v.q, v.lse, v.cu_q, v.g.seq_len, v.g.q_start, v.g.doc_blocks, v.g.meta, v.g.k, v.g.cfg, v.weights,
                              v.max_q, window=v.window, ws=v.ws)
    for a, b in ((v.q, u.q), (v.lse, u.lse), (v.g.k, u.g.k), (v.g.meta, u.g.meta)):
        a.copy_(b)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    u.check(v.weights.cpu().numpy().astype(np.float64))


# ------------------------------------------------------------------ plan and move
class Cut:
    def __init__(self, lk, docs, seg, keep, first=0, recent=0, seed=0, room=None, D=64, Hkv=2):
        import torch
        rng = np.random.default_rng(seed + 31)
        n = room or max(1, max(max(k, 0) // 16 + len(d) for k, d in zip(keep, docs)))
        self.lk, self.first, self.recent = lk, first, recent
        self.x = x = ref.Lists(rng, [], docs, seg, 2 * Hkv, Hkv, D, pos_of(rd=D), spare=n * len(docs))
        self.w = np.exp(2 * rng.standard_normal((x.B, x.max_blocks * 16))).astype(np.float32)
        self.w[rng.random(self.w.shape) < 0.3] = 0.0
        self.keep, self.dst = np.array(keep, np.int32), x.spare.reshape(x.B, n)
        self.num_pages = x.num_pages
        self.new = [torch.full((x.B, x.max_blocks), -7, dtype=torch.int64, device="cuda"),
                    torch.full((x.B,), -7, dtype=torch.int32, device="cuda")]
        self.new += [torch.full((x.B, 16 * n), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.new += [torch.full((x.B, 16 * x.max_blocks), float("nan"), device="cuda")]

    def run(self):
        x, (nm, nd, src, dst, nw) = self.x, self.new
        self.args = (dev(self.w), dev(x.meta.view(np.int64)), dev(x.doc_blocks), dev(self.keep), dev(self.dst), self.num_pages,
                     cfg_of(self.lk, x.pos, x.D))
        self.lk.evict_plan(*self.args, nm, nd, src, dst, nw, first=self.first, recent=self.recent)
        return [t.cpu().numpy() for t in self.new]

    def check(self, got):
        x = self.x
        want = ref.plan(self.w, x.meta, x.doc_blocks, self.keep, self.dst, self.num_pages, self.first, self.recent)
        for a, b, n in zip(got, want, ("new_meta", "new_doc_blocks", "src_slot", "dst_slot", "new_weights")):
            a = a.view(np.uint64) if n == "new_meta" else a
            assert np.array_equal(a, b, equal_nan=n == "new_weights"), (n, np.argwhere(a != b)[:5])
        return want


PLANS = {
    "plain": dict(docs=[[40, 200], [7], [300, 16, 16]], seg=[5, 1, 33], keep=[50, 3, 100]),
    "protected": dict(docs=[[40, 200], [7], [300, 16, 16]], seg=[5, 1, 33], keep=[50, 3, 100], first=4, recent=20),
    "more_protected_than_kept": dict(docs=[[40, 200], [30]], seg=[5, 1], keep=[10, 12], first=8, recent=9),
    "everything_protected": dict(docs=[[40], [30]], seg=[5, 1], keep=[17, 5], first=100, recent=100),
    "keep_all": dict(docs=[[40, 200], [7]], seg=[5, 1], keep=[1000, 7]),
    "keep_none": dict(docs=[[40, 200], [7]], seg=[5, 1], keep=[0, 1]),
    "leave": dict(docs=[[40, 200], [7], [20]], seg=[5, 1, 2], keep=[-1, 3, -5]),
    "no_documents": dict(docs=[[], [7], []], seg=[20, 1, 0], keep=[5, 3, 1]),
    "single_keys": dict(docs=[[1] * 30, [1]], seg=[1, 1], keep=[11, 1]),
    "long": dict(docs=[[1600] * 6 + [33], [17000], [100] * 90], seg=[40, 3, 1], keep=[2000, 5000, 777], first=4, recent=64),
    "two_parts": dict(docs=[[1600] * 4, [33] * 130], seg=[40, 3], keep=[2000, 1500], first=4, recent=64),
    "longer": dict(docs=[[20000, 33, 20000], [300]], seg=[40, 3], keep=[12345, 300], first=4, recent=64),
    "longest": dict(docs=[[30000, 33, 30000, 30000, 30000, 12345], [300]], seg=[40, 3], keep=[33333, 20], first=4, recent=64),
    "many": dict(docs=[[1 + 7 * i % 50, 20] for i in range(200)], seg=[1 + i % 20 for i in range(200)],
                 keep=[i % 60 for i in range(200)], recent=5),
    "many_longer": dict(docs=[[4500, 20] if i % 40 == 0 else [20 + i] for i in range(160)], seg=[1] * 160,
                        keep=[5 * i for i in range(160)], first=3),
}


@pytest.mark.parametrize("name", PLANS)
def test_evict_plan(lk, name):
    c = Cut(lk, **PLANS[name])
    c.check(c.run())
    assert lk.device_status() == 0


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("weights", ["equal", "zero", "nan", "inf", "negative", "tiny"])
def test_evict_plan_orders_any_weights(lk, weights, long):
    c = Cut(lk, [[40, 200], [70], [300, 16, 16] + [3000] * 4 * long], [5, 1, 33], [51, 33, 100 + 5000 * long], first=1, recent=1)
    rng = np.random.default_rng(3)
    some = rng.random(c.w.shape) < 0.4
    if weights == "equal":
        c.w[:] = 0.25
    elif weights == "zero":
        c.w[:] = np.where(some, 0.0, -0.0)
    elif weights == "nan":
        c.w[some] = np.nan
        c.w[1] = -np.nan
    elif weights == "inf":
        c.w[some] = np.inf
        c.w[rng.random(c.w.shape) < 0.3] = -np.inf
    elif weights == "negative":
        c.w[some] *= -1
    else:
        c.w = (c.w * 1e-42).astype(np.float32)  # subnormal
    c.check(c.run())


def test_evict_plan_with_too_few_pages(lk):
    c = Cut(lk, [[40, 200], [70]], [5, 1], [100, 30], room=3)
    c.check(c.run())
    assert lk.device_status() == 1
    c = Cut(lk, [[40, 200], [70]], [5, 1], [100, 30])
    c.dst = c.dst.copy()
    c.dst[0, 2], c.dst[1, 0] = -1, c.num_pages
    c.check(c.run())
    assert lk.device_status() == 1


def test_evict_twice(lk):
    """The plan of a list that an eviction made."""
    c = Cut(lk, [[40, 200, 90], [70]], [5, 1], [100, 30])
    c.check(c.run())
    x = c.x
    x.meta, x.doc_blocks, c.w = (t.cpu().numpy() for t in (c.new[0], c.new[1], c.new[4]))
    x.meta = x.meta.view(np.uint64)
    rng = np.random.default_rng(4)
    c.keep, c.dst = np.array([33, 16], np.int32), rng.permutation(x.num_pages)[:c.dst.size].reshape(c.dst.shape).astype(np.int32)
    c.check(c.run())


@pytest.mark.parametrize("D,Hkv,T", [(128, 8, 100), (128, 1, 1), (64, 3, 33), (64, 2, 7), (128, 5, 64)])
def test_kv_move(lk, D, Hkv, T):
    import torch
    rng = np.random.default_rng(T)
    P = 2 * T // 16 + 3
    bits = [rng.integers(0, 1 << 16, (P, Hkv, 16, D)).astype(np.uint16) for _ in range(2)]
    slots = rng.permutation(16 * P)[:2 * T].astype(np.int32)
    src, dst = slots[:T].copy(), slots[T:].copy()
    src[rng.random(T) < 0.1] = -1
    dst[rng.random(T) < 0.1] = -1
    k, v = (dev(b.view(np.int16)).view(torch.bfloat16) for b in bits)
    lk.kv_move(dev(src), dev(dst), k, v)
    for got, want in zip((k, v), ref.move(src, dst, *bits)):
        assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), want)
    assert lk.device_status() == 0


def test_kv_move_outside_the_cache(lk):
    import torch
    k, v = (torch.randn((4, 2, 16, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    a, b = k.clone(), v.clone()
    lk.kv_move(dev(np.array([3, 64, 70, 2 ** 31 - 1], np.int32)), dev(np.array([64, 9, 10, 11], np.int32)), k, v)
    assert lk.device_status() == 2
    assert (k == a).all() and (v == b).all()
    lk.kv_move(dev(np.zeros(0, np.int32)), dev(np.zeros(0, np.int32)), k, v)
    assert lk.device_status() == 0


# ------------------------------------------------------------------ together
def test_prefill_vote_cut_and_decode(lk):
    """A question over documents, its last tokens' votes, the cut, and answers sampled over what stays: prefill,
    key weights, plan, move, then a decode step of several requests that share the packed documents."""
    import torch
    rng = np.random.default_rng(8)
    pos, Hq, Hkv, D, n = pos_of(rd=64), 8, 2, 64, 4
    docs, seg, keep = [150, 37, 220], 32, 120  # the question fills whole pages
    room = keep // 16 + len(docs)
    x = ref.Lists(rng, [], [docs], [seg], Hq, Hkv, D, pos, spare=room + n)
    g = OnGpu(lk, x)
    qh = ref.bf16(rng.standard_normal((seg, Hq, D)))
    q, cu = bf(qh), dev(np.array([0, seg], np.int32))
    out, lse = torch.empty_like(q), torch.empty((seg, Hq), device="cuda")
    lk.attn_prefill(q, cu, g.q_start, g.doc_blocks, g.meta, g.k, g.v, g.cfg, out, seg, lse=lse)
    w = torch.empty((1, 16 * x.max_blocks), device="cuda")
    ws = torch.empty(lk.workspace_size(lk.PHASE_KEY_WEIGHTS, seg, 1, x.max_blocks, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    lk.attn_key_weights(q, lse, cu, g.seq_len, g.q_start, g.doc_blocks, g.meta, g.k, g.cfg, w, seg, window=8, ws=ws)
    s = ref.scores(x, 0, qh, x.q_start[0] + np.arange(seg))[0]
    want = ref.key_weights(x, qh, ref.softmax(s)[1].astype(np.float32), [0, seg], 8)
    got = w.cpu().numpy()
    assert np.linalg.norm(got - want) <= 2.0 ** -9 * np.linalg.norm(want)  # the prefill's lse: f16 scores
    dst = x.spare[:room].reshape(1, room)
    nm, nw = torch.empty_like(g.meta), torch.empty_like(w)
    nd, src, to = torch.empty_like(g.doc_blocks), *(torch.empty((1, 16 * room), dtype=torch.int32, device="cuda") for _ in range(2))
    lk.evict_plan(w, g.meta, g.doc_blocks, dev(np.array([keep], np.int32)), dev(dst), x.num_pages, g.cfg, nm, nd, src, to, nw,
                  first=4, recent=8)
    lk.kv_move(src, to, g.k, g.v)
    pm, pd, ps, pt, pw = ref.plan(got, x.meta, x.doc_blocks, [keep], dst, x.num_pages, 4, 8)
    assert np.array_equal(nm.cpu().numpy().view(np.uint64), pm) and np.array_equal(nw.cpu().numpy(), pw)
    # n answers: each continues on a page of its own behind the packed documents and the question
    x.k, x.v = ref.move(ps, pt, x.k, x.v)
    tail = int(pd[0]) + seg // 16
    x.B, x.max_blocks = n, tail + 1
    x.meta = np.repeat(pm[:, :tail + 1], n, 0)
    tokens = [3, 1, 16, 7]
    for b in range(n):
        page = int(x.spare[room + b])
        x.meta[b, tail] = 16 | seg // 16 << 5 | int(x.q_start[0]) << 16 | page << 40
        x.k[page, :, :tokens[b]] = ref.bf16(rng.standard_normal((Hkv, tokens[b], D)))
        x.v[page, :, :tokens[b]] = ref.bf16(rng.standard_normal((Hkv, tokens[b], D)))
    x.seq_len = np.array([int(x.seq_len[0]) + t for t in tokens], np.int32)
    x.q_start, x.doc_blocks = np.repeat(x.q_start, n), np.repeat(pd, n)
    x.off, x.shared = [0, n], [int(pd[0])]
    x.q = ref.bf16(rng.standard_normal((n, Hq, D)))
    h = OnGpu(lk, x)
    for mine, theirs in ((g.k, h.k), (g.v, h.v)):
        for page in dst[0]:  # the moved rows are the reference's
            assert torch.equal(mine[int(page)].isnan(), theirs[int(page)].isnan())
            assert torch.equal(mine[int(page)].nan_to_num(), theirs[int(page)].nan_to_num())
    out, lse = h.decode()
    check(out, lse, ref.decode(x))
    assert lk.device_status() == 0
