"""Decoding a batch that shares documents, and evicting keys by the attention they receive.

Each case is one call that a serving program makes over a bf16 paged, position-free cache:
``attn_decode_shared`` (one decode step in which groups of requests list the same first documents),
``attn_key_weights`` (the attention weight that every cached key received from a set of query rows),
``evict_plan`` (which document keys of each request stay, and where they go) and ``kv_move`` (the rows'
copies).  ``run`` computes them with elementary torch operations in 32 bits, or, with ``own`` set, makes
the library's calls.  ``exact`` restates the definitions in 64 bits.

Caches are [pages][Hkv][16][D]; a request's list has one 64-bit word per page: bits [4:0] valid rows,
[15:5] page index in the document, [39:16] the document's offset Delta, [63:40] physical page.  Keys are
stored rotated by their position in the document; attention turns them by Delta and queries by their
position m.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    d = dict(name=name, op=op, Hq=32, Hkv=8, D=128, kind="rope", theta=5e5, rotary_dim=128, interleaved=False, ragged=False,
             layout=0)
    d.update(kw)
    return d


def listed():
    return [
        # two short requests over one small document, small heads: what a call costs by itself
        _case("shared_tiny", "shared", B=2, Hq=4, Hkv=2, D=64, rotary_dim=64, theta=1e4, groups=1, docs=1, doc_len=80,
              own_docs=0, seg=17),
        # sixteen answers sampled for one question over ten retrieved documents
        _case("shared_samples", "shared", B=16, groups=1, docs=10, doc_len=200, own_docs=0, seg=33),
        # a large batch of questions about the same 32 000 tokens
        _case("shared_long", "shared", B=64, groups=1, docs=20, doc_len=1600, own_docs=0, seg=33),
        # several groups of unequal size, each with documents of its own behind the common ones
        _case("shared_groups", "shared", B=64, Hq=64, groups=8, docs=20, doc_len=512, own_docs=2, seg=40, ragged=True),
        # one KV head for 32 query heads, linear biases
        _case("shared_mqa_alibi", "shared", B=32, Hkv=1, kind="alibi", groups=1, docs=12, doc_len=1000, own_docs=0, seg=33),
        # one decode step's weights added to the running sums of long contexts
        _case("weights_step", "weights", B=16, docs=20, doc_len=1600, seg=33, rows=1, window=0, add=True),
        # the last 32 tokens of 64-token questions vote on long contexts
        _case("weights_window", "weights", B=8, Hq=64, docs=20, doc_len=512, seg=64, rows=64, window=32, add=False),
        # every token of one question, and of the answer so far, over one document
        _case("weights_prompt", "weights", B=1, docs=1, doc_len=1600, seg=800, rows=800, window=0, add=False),
        # one request of ten retrieved documents cut to a quarter
        _case("plan_short", "plan", B=1, docs=10, doc_len=200, seg=64, keep=500, first=4, recent=32),
        # long contexts cut to an eighth
        _case("plan_long", "plan", B=16, docs=20, doc_len=1600, seg=64, keep=4000, first=4, recent=64),
        # the filled rows of the last page of a prompt, copied once for each of eight answers
        _case("move_fork", "move", B=8, docs=1, doc_len=9, seg=0, keep=9),
        # the rows that a cut of sixteen 8000-token contexts to a quarter keeps
        _case("move_kept", "move", B=16, docs=5, doc_len=1600, seg=0, keep=2000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    D = rng.choice([64, 128, 128])
    kind = rng.choice(["rope", "rope", "yarn", "alibi"])
    rd = D if kind == "alibi" or rng.random() < 0.6 else 16 * rng.randint(1, D // 16)
    Hq, Hkv = rng.choice([(4, 2), (8, 8), (16, 2), (32, 8), (32, 8), (32, 1), (64, 8), (24, 1)])
    op = rng.choice(["shared", "shared", "weights", "weights", "plan", "move"])
    c = dict(op=op, D=D, Hq=Hq, Hkv=Hkv, kind=kind, rotary_dim=rd, interleaved=kind != "alibi" and rng.random() < 0.25,
             theta=rng.choice([1e4, 5e5]), ragged=True, layout=rng.randint(1, 1 << 20), docs=rng.randint(1, 20),
             doc_len=_log(rng, 1, 1600))
    if op == "shared":
        c["B"], c["seg"], c["own_docs"] = _log(rng, 1, 64), rng.randint(1, 64), rng.choice([0, 0, 1, 2])
        c["groups"] = rng.randint(1, min(8, c["B"]))
    elif op == "weights":
        c["B"], c["seg"], c["add"] = _log(rng, 1, 16), _log(rng, 1, 64), rng.random() < 0.5
        if rng.random() < 0.2:
            c["B"], c["seg"], c["docs"] = 1, _log(rng, 64, 800), rng.randint(0, 2)
        c["rows"] = 1 if rng.random() < 0.4 else c["seg"]
        c["window"] = rng.choice([0, 8, 32]) if c["rows"] > 1 else 0
        # below the largest listed weights' work
        while c["B"] * min(c["rows"], c["window"] or c["rows"]) * (c["docs"] * c["doc_len"] + c["seg"]) * Hq > 1.6e8:
            c["doc_len"] = max(1, c["doc_len"] // 2)
            c["seg"] = max(1, c["seg"] - c["seg"] // 4)
            c["rows"] = min(c["rows"], c["seg"])
    else:
        c["B"], c["seg"] = _log(rng, 1, 16), rng.randint(1, 64)
        c["kind"] = "rope"  # neither depends on it
        if op == "move":
            c["docs"] = min(c["docs"], 5)
        c["keep"] = _log(rng, 1, max(1, c["docs"] * c["doc_len"] // 4))
        if op == "plan":
            c["first"], c["recent"] = rng.choice([0, 4]), rng.choice([0, 16, 64])
    return {k: c[k] for k in sorted(c)}


def _layout(case):
    """Lengths of every request's documents and of its query segment, and the groups that list the same first
    documents: (lens [B] of int arrays, seg [B], group_off [groups + 1], common [groups] of document counts)."""
    r = np.random.default_rng([int(case["layout"]), int(case["docs"]), int(case["doc_len"])])
    B, n, L = case["B"], case["docs"], case["doc_len"]
    one = lambda k: r.integers(1, L + 1, k) if case["ragged"] else np.full(k, L, np.int64)  # noqa: E731
    seg = np.full(B, case["seg"], np.int64)
    if case["op"] != "shared":
        if case["ragged"] and B > 1 and case["seg"] > 0:
            seg = r.integers(1, case["seg"] + 1, B)
            seg[r.integers(0, B)] = case["seg"]
        return [one(n) for _ in range(B)], seg, None, None
    if case["ragged"]:
        cuts = np.sort(r.choice(np.arange(1, B), case["groups"] - 1, replace=False)) if B > 1 else np.zeros(0, np.int64)
        seg = r.integers(1, case["seg"] + 1, B)
    else:
        cuts = np.arange(1, case["groups"]) * B // case["groups"]
    off = np.concatenate([[0], cuts, [B]]).astype(np.int64)
    lens = []
    for g in range(case["groups"]):
        common = one(n)
        lens += [np.concatenate([common, one(case["own_docs"])]) for _ in range(off[g + 1] - off[g])]
    return lens, seg, off, np.full(case["groups"], n)


def _blocks(lens):
    return -(-np.asarray(lens, np.int64) // PAGE)


def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    lens, seg, off, _ = _layout(case)
    docs = np.array([x.sum() for x in lens])
    blocks = np.array([_blocks(x).sum() for x in lens]) + _blocks(seg)
    keys = docs + seg
    if case["op"] == "shared":  # each common key once for its group
        once = keys.sum() - sum((off[g + 1] - off[g] - 1) * lens[off[g]][:case["docs"]].sum() for g in range(case["groups"]))
        return {"bytes": float(once * Hkv * D * 4 + 8 * blocks.sum() + case["B"] * Hq * D * 4),
                "flops": float(4 * D * Hq * keys.sum())}
    if case["op"] == "weights":
        n = np.minimum(seg, case["rows"])
        n = np.minimum(n, case["window"]) if case["window"] else n
        pairs = n * keys - n * (n - 1) // 2
        return {"bytes": float(keys.sum() * (Hkv * D * 2 + (8 if case["add"] else 4)) + 8 * blocks.sum()
                               + n.sum() * Hq * (2 * D + 4)), "flops": float(2 * D * Hq * pairs.sum())}
    kept = np.minimum(docs, case["keep"]).sum()
    if case["op"] == "plan":  # weights and words in; words, slots and the kept weights out
        return {"bytes": float(4 * keys.sum() + 8 * blocks.sum() + 8 * (kept / PAGE + _blocks(seg).sum()) + 12 * kept),
                "flops": 0}
    return {"bytes": float(kept * (8 * D * Hkv + 8)), "flops": 0}


# ------------------------------------------------------------------ inputs
def _freqs(case):
    """Angle per position of each rotated pair, float64."""
    rd = case["rotary_dim"]
    th = case["theta"] ** (-2.0 * np.arange(rd // 2) / rd)
    if case["kind"] == "yarn":
        r = 8192 * th / (2 * math.pi)
        g = np.clip((r - 1.0) / 31.0, 0.0, 1.0)
        th = (1 - g) * th / 8.0 + g * th
    return th


def _softmax_scale(case):
    s = 1.0 / math.sqrt(case["D"])
    return s * (0.1 * math.log(8.0) + 1.0) ** 2 if case["kind"] == "yarn" else s


def _words(case, lens, seg, off, rng):
    """Block words [B][max blocks] (numpy uint64), document blocks [B] and the number of pages.  The requests of a
    group name the same pages for their common documents."""
    B = case["B"]
    nb = [int(_blocks(x).sum()) for x in lens]
    meta = np.zeros((B, max(1, max(n + int(_blocks(s)) for n, s in zip(nb, seg)))), np.uint64)
    first = np.arange(B) if off is None else off[:-1].repeat(np.diff(off))
    at, pages = 0, []
    for b in range(B):
        ids, delta, j = [], 0, 0
        for d, x in enumerate(lens[b]):
            n = int(_blocks(x))
            if off is not None and first[b] != b and d < case["docs"]:
                ids.append(pages[first[b]][j:j + n])
            else:
                ids.append(np.arange(at, at + n))
                at += n
            pg = np.arange(n)
            meta[b, j:j + n] = (np.minimum(PAGE, x - PAGE * pg) | pg << 5 | delta << 16).astype(np.uint64)
            j, delta = j + n, delta + int(x)
        n = int(_blocks(seg[b]))
        ids.append(np.arange(at, at + n))
        at += n
        meta[b, j:j + n] = (PAGE | np.arange(n) << 5 | delta << 16).astype(np.uint64)
        pages.append(np.concatenate(ids))
    where = rng.permutation(at)
    for b in range(B):
        meta[b, :len(pages[b])] |= where[pages[b]].astype(np.uint64) << np.uint64(40)
    return meta, np.array(nb), at


def _fields(meta):
    return meta & 31, (meta >> 5) & 2047, (meta >> 16) & 0xFFFFFF, (meta >> 40) & 0xFFFFFF


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)  # noqa: E731
    s = {"case": dict(case)}
    B, Hq, H, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    lens, seg, off, common = _layout(case)
    meta, nb, pages = _words(case, lens, seg, off, rng)
    docs = np.array([x.sum() for x in lens])
    MB = meta.shape[1]
    s["meta"] = torch.from_numpy(meta.view(np.int64)).to(dev)
    s["doc_blocks"], s["q_start"], s["seq_len"] = i32(nb), i32(docs), i32(docs + seg)
    spread = torch.exp(0.5 * torch.randn((H, 1, D), generator=gen, device=dev))  # some channels of keys are larger

    def cache(n, c):
        t = torch.empty((n, H, PAGE, D), dtype=torch.bfloat16, device=dev)
        for p in range(0, n, 16384):
            x = torch.randn((min(16384, n - p), H, PAGE, D), generator=gen, device=dev)
            t[p:p + 16384] = x * c if c is not None else x
        return t

    if case["op"] == "plan":
        # most keys get little, a few much; far keys of sharp heads nothing at all
        w = torch.exp(2.0 * torch.randn((B, MB * PAGE), generator=gen, device=dev)) * 1e-3
        s["weights"] = torch.where(torch.rand(w.shape, generator=gen, device=dev) < 0.1, torch.zeros_like(w), w)
        s["keep"] = i32(np.full(B, case["keep"]))
        room = max(1, int(max((min(int(k), case["keep"]) // PAGE + len(x)) for k, x in zip(docs, lens))))
        s["num_pages"] = pages + B * room
        s["dst_pages"] = i32(pages + rng.permutation(B * room).reshape(B, room))
        s["new_meta"], s["new_weights"] = torch.zeros_like(s["meta"]), torch.zeros_like(s["weights"])
        s["new_doc_blocks"] = torch.zeros_like(s["doc_blocks"])
        s["src"] = torch.zeros((B, room * PAGE), dtype=torch.int32, device=dev)
        s["dst"] = torch.zeros_like(s["src"])
    elif case["op"] == "move":
        slots, to = [], []
        at = pages
        for b in range(B):
            nv, ids = (meta[b, :nb[b]] & np.uint64(31)).astype(np.int64), (meta[b, :nb[b]] >> np.uint64(40)).astype(np.int64)
            rows = (ids[:, None] * PAGE + np.arange(PAGE))[np.arange(PAGE) < nv[:, None]]
            keep = np.sort(rng.permutation(len(rows))[:case["keep"]])
            slots.append(rows[keep])
            to.append(at * PAGE + np.arange(len(keep)))
            at += int(_blocks(len(keep)))
        s["src"], s["dst"] = i32(np.concatenate(slots)), i32(np.concatenate(to))
        s["k"], s["v"] = cache(at, spread), cache(at, None)
    else:
        s["k"] = cache(pages, spread)
        if case["kind"] == "alibi":
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq).float()
    if case["op"] == "shared":
        s["v"] = cache(pages, None)
        s["q"] = torch.randn((B, Hq, D), generator=gen, device=dev).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["group_off"] = i32(off)
        shared = np.array([_blocks(lens[off[g]][:common[g]]).sum() for g in range(case["groups"])])
        s["shared_blocks"] = i32(shared)
        s["max_group"], s["max_shared"] = int(np.diff(off).max()), int(shared.max())
    if case["op"] == "weights":
        n = np.minimum(seg, case["rows"])
        s["cu_q"], s["max_q"] = i32(np.concatenate([[0], np.cumsum(n)])), int(n.max())
        s["q"] = torch.randn((int(n.sum()), Hq, D), generator=gen, device=dev).to(torch.bfloat16)
        s["weights"] = torch.zeros((B, MB * PAGE), device=dev)
        if case["add"]:
            s["weights"] += torch.rand(s["weights"].shape, generator=gen, device=dev)
        # the attention call's log-sum-exp
        lse = torch.empty((int(n.sum()), Hq), device=dev)
        cu = np.concatenate([[0], np.cumsum(n)])
        for b in range(B):
            one = dict(s, meta=s["meta"][b:b + 1], q=s["q"][cu[b]:cu[b + 1]], m=docs[b] + seg[b] - n[b] + np.arange(n[b]))
            lse[cu[b]:cu[b + 1]] = _lse(one, case)
        s["lse"] = lse
    torch.cuda.synchronize()
    return s


def _lse(s, case):
    """Log-sum-exp [n][Hq] of the rows q of one request at positions m."""
    dev, (n, Hq, D), H = s["q"].device, s["q"].shape, case["Hkv"]
    m = torch.from_numpy(np.asarray(s["m"])).to(dev)
    x = _scores(dict(s, q=s["q"].float()[None]), case, m[None])[0]  # [H, G, n, N]
    return torch.logsumexp(x, -1).permute(2, 0, 1).reshape(n, Hq)


# ------------------------------------------------------------------ the plain form
def _rotate(x, c, s, rd, interleaved):
    """Pairs of the first rd of x's last dimension turned by the angles whose cos and sin are given."""
    a, rest = x[..., :rd], x[..., rd:]
    if interleaved:
        x1, x2 = a[..., 0::2], a[..., 1::2]
        y = torch.stack([x1 * c - x2 * s, x1 * s + x2 * c], -1).flatten(-2)
    else:
        x1, x2 = a[..., :rd // 2], a[..., rd // 2:]
        y = torch.cat([x1 * c - x2 * s, x1 * s + x2 * c], -1)
    return torch.cat([y, rest], -1) if rd < x.shape[-1] else y


def _cos_sin(pos, case):
    a = pos.double().unsqueeze(-1) * torch.from_numpy(_freqs(case)).to(pos.device)
    return a.cos().float(), a.sin().float()


def _scores(s, case, m):
    """Scores [B, Hkv, G, n, keys] of q [B, n, Hq, D] (32 bits) at positions m [B, n]; -inf where a key is not seen."""
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    meta, q, G = s["meta"], s["q"], Hq // Hkv
    B, n = m.shape
    nv, pg, delta, page = _fields(meta)
    k = s["k"][page].float()  # [B, MB, H, 16, D]
    t = torch.arange(PAGE, device=meta.device)
    p = ((delta + PAGE * pg).unsqueeze(-1) + t).flatten(1)  # [B, N]
    valid = (t < nv.unsqueeze(-1)).flatten(1)
    if case["kind"] != "alibi":
        rd, il = case["rotary_dim"], case["interleaved"]
        c, sn = _cos_sin(delta, case)
        k = _rotate(k, c[:, :, None, None], sn[:, :, None, None], rd, il)
        c, sn = _cos_sin(m, case)
        q = _rotate(q, c[:, :, None], sn[:, :, None], rd, il)
    k = k.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    q = q.reshape(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, G, n, -1) * _softmax_scale(case)
    if case["kind"] == "alibi":
        x = x - s["slopes"].view(1, Hkv, G, 1, 1) * (m.unsqueeze(-1) - p.unsqueeze(1)).float()[:, None, None]
    see = valid.unsqueeze(1) & (p.unsqueeze(1) <= m.unsqueeze(-1))  # [B, n, N]
    return torch.where(see[:, None, None], x, -math.inf)


def _plain_shared(s, case):
    B, Hq, D, H = case["B"], case["Hq"], case["D"], case["Hkv"]
    x = _scores(dict(s, q=s["q"].float()[:, None]), case, s["seq_len"].long().view(B, 1) - 1)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    w = (e / e.sum(-1, keepdim=True)).view(B, H, Hq // H, -1)
    _, _, _, page = _fields(s["meta"])
    v = s["v"][page].float().permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    return torch.matmul(w, v).reshape(B, Hq, D).to(torch.bfloat16)


def _plain_weights(s, case):
    cu, n, H = s["cu_q"].long(), s["max_q"], case["Hkv"]
    length = (cu[1:] - cu[:-1]).unsqueeze(1)
    if case["window"]:
        n = min(n, case["window"])
    i = torch.arange(n, device=cu.device)  # counted back from each request's last row
    live = i < length
    at = torch.where(live, cu[1:].unsqueeze(1) - 1 - i, 0)
    m = s["seq_len"].long().unsqueeze(1) - 1 - i
    x = _scores(dict(s, q=s["q"].float()[at]), case, m)
    lse = s["lse"][at].view(*at.shape, H, -1).permute(0, 2, 3, 1).unsqueeze(-1)
    w = torch.where(live[:, None, None, :, None], torch.exp(x - lse), 0.0).sum((1, 2, 3))
    if case["add"]:
        s["weights"] += w
    else:
        s["weights"].copy_(w)
    return s["weights"]


def _plain_plan(s, case):
    meta, w, dev = s["meta"], s["weights"], s["meta"].device
    B, MB = meta.shape
    N = MB * PAGE
    nv, _, delta, page = _fields(meta)
    block = torch.arange(MB, device=dev)
    doc = block < s["doc_blocks"].unsqueeze(1)  # [B, MB]
    t = torch.arange(PAGE, device=dev)
    key = (doc.unsqueeze(-1) & (t < nv.unsqueeze(-1))).flatten(1)  # [B, N] document keys
    rank = key.long().cumsum(1) - 1
    total = key.sum(1, keepdim=True)
    safe = key & ((rank < case["first"]) | (rank >= total - case["recent"]))
    order = torch.where(safe, math.inf, torch.where(key, w, -math.inf))
    order = torch.where(key, order, -math.inf)
    at = torch.sort(order, dim=1, descending=True, stable=True).indices
    keep = torch.zeros_like(key).scatter(1, at, torch.arange(N, device=dev).expand(B, N) < s["keep"].unsqueeze(1)) & key
    # kept keys packed per document: a document is a run of blocks with one Delta
    start = doc & torch.cat([torch.ones_like(doc[:, :1]), delta[:, 1:] != delta[:, :-1]], 1)
    run = torch.where(doc, start.long().cumsum(1) - 1, MB)  # [B, MB]
    run_key = run.repeat_interleave(PAGE, 1)
    kept = torch.zeros((B, MB + 1), dtype=torch.long, device=dev).scatter_add(1, run_key, keep.long())
    blocks = -(-kept // PAGE)
    base = blocks.cumsum(1) - blocks  # first new block of each run
    before = kept.cumsum(1) - kept
    inside = keep.long().cumsum(1) - 1 - before.gather(1, run_key)
    new_block = base.gather(1, run_key) + inside // PAGE
    slot = new_block * PAGE + inside % PAGE  # position in the new list
    new_docs = blocks.sum(1)
    R = s["dst_pages"].shape[1]
    put = lambda out, val: out.scatter(1, torch.where(keep, slot, out.shape[1] - 1), torch.where(keep, val, 0))  # noqa: E731
    wide = lambda fill, n: torch.full((B, n + 1), fill, dtype=torch.long, device=dev)  # noqa: E731
    src = page.repeat_interleave(PAGE, 1) * PAGE + t.repeat(MB)
    to = s["dst_pages"].long()
    there = to.gather(1, new_block.clamp(0, R - 1)) * PAGE + inside % PAGE
    s["src"].copy_(put(wide(-1, R * PAGE), src)[:, :-1])
    s["dst"].copy_(put(wide(-1, R * PAGE), there)[:, :-1])
    new_w = torch.zeros((B, N + 1), device=dev).scatter(1, torch.where(keep, slot, N), torch.where(keep, w, 0.0))[:, :-1]
    # words: the last kept key of a page gives its number of rows
    word = (inside % PAGE + 1) | (inside // PAGE) << 5 | delta.repeat_interleave(PAGE, 1) << 16
    word = word | to.gather(1, new_block.clamp(0, R - 1)) << 40
    last = keep & ((inside % PAGE == PAGE - 1) | (inside == kept.gather(1, run_key) - 1))
    new = torch.zeros((B, MB + 1), dtype=torch.long, device=dev)
    new = new.scatter(1, torch.where(last, new_block, MB), torch.where(last, word, 0))[:, :-1]
    # the query segment's blocks and weights follow
    back = block - new_docs.unsqueeze(1) + s["doc_blocks"].unsqueeze(1)
    here = (block >= new_docs.unsqueeze(1)) & (back < MB)
    back = back.clamp(0, MB - 1)
    s["new_meta"].copy_(torch.where(here, meta.gather(1, back), new))
    seg_w = w.view(B, MB, PAGE).gather(1, back.unsqueeze(-1).expand(-1, -1, PAGE))
    s["new_weights"].copy_(torch.where(here.unsqueeze(-1), seg_w, new_w.view(B, MB, PAGE)).flatten(1))
    s["new_doc_blocks"].copy_(new_docs)
    return _plan_outputs(s)


def _plan_outputs(s):
    return [s["new_meta"], s["new_doc_blocks"], s["src"], s["dst"], s["new_weights"]]


def _plain_move(s):
    src, dst = s["src"].long(), s["dst"].long()
    for c in (s["k"], s["v"]):
        c[dst // PAGE, :, dst % PAGE] = c[src // PAGE, :, src % PAGE]
    return [s["k"], s["v"]]


# ------------------------------------------------------------------ the library's calls
def _plan(s):
    """What a program keeps: the positional configuration and the workspace."""
    import position_agnostic_kv_gb300 as lk
    case, ws = s["case"], None
    Hq, Hkv, D, B, MB = case["Hq"], case["Hkv"], case["D"], case["B"], s["meta"].shape[1]
    cfg = lk.pos_cfg_from(case["kind"], D, rope_theta=case["theta"], yarn_factor=8.0, yarn_orig_ctx=8192,
                          alibi_slopes=s.get("slopes"), rotary_dim=case["rotary_dim"], interleaved=case["interleaved"])
    if case["op"] == "shared":
        n = lk.decode_shared_workspace_size(B, s["group_off"].numel() - 1, s["max_group"], s["max_shared"], MB, Hq, Hkv, D)
        ws = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
    elif case["op"] == "weights":
        n = lk.workspace_size(lk.PHASE_KEY_WEIGHTS, s["q"].shape[0], B, MB, Hq, Hkv, D)
        ws = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
    s["plan"] = (lk, cfg, ws)
    return s["plan"]


def _own(s):
    lk, cfg, ws = s.get("plan") or _plan(s)
    case = s["case"]
    if case["op"] == "shared":
        lk.attn_decode_shared(s["q"], s["seq_len"], s["q_start"], s["doc_blocks"], s["meta"], s["group_off"],
                              s["shared_blocks"], s["max_group"], s["max_shared"], s["k"], s["v"], cfg, s["out"], ws=ws)
        return s["out"]
    if case["op"] == "weights":
        lk.attn_key_weights(s["q"], s["lse"], s["cu_q"], s["seq_len"], s["q_start"], s["doc_blocks"], s["meta"], s["k"],
                            cfg, s["weights"], s["max_q"], window=case["window"], accumulate=case["add"], ws=ws)
        return s["weights"]
    if case["op"] == "plan":
        lk.evict_plan(s["weights"], s["meta"], s["doc_blocks"], s["keep"], s["dst_pages"], s["num_pages"], cfg,
                      s["new_meta"], s["new_doc_blocks"], s["src"], s["dst"], s["new_weights"], first=case["first"],
                      recent=case["recent"])
        return _plan_outputs(s)
    lk.kv_move(s["src"], s["dst"], s["k"], s["v"])
    return [s["k"], s["v"]]


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "shared":
        return _plain_shared(state, case)
    if case["op"] == "weights":
        return _plain_weights(state, case)
    return _plain_plan(state, case) if case["op"] == "plan" else _plain_move(state)


# ------------------------------------------------------------------ the definition in 64 bits
def _turn64(x, pos, case):
    """x [..., D] float64 turned by its positions pos [...]."""
    f = torch.from_numpy(_freqs(case)).to(x.device)
    rd = case["rotary_dim"]
    z = x[..., :rd]
    z = torch.complex(z[..., 0::2], z[..., 1::2]) if case["interleaved"] else torch.complex(z[..., :rd // 2], z[..., rd // 2:])
    z = z * torch.polar(torch.ones_like(f), pos.double().unsqueeze(-1) * f)
    y = x.clone()
    if case["interleaved"]:
        y[..., 0:rd:2], y[..., 1:rd:2] = z.real, z.imag
    else:
        y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
    return y


def _request64(s, case, b, lens, seg):
    """One request's keys in list order: their places in the list, positions, and rows of the cache."""
    w = s["meta"][b].cpu().numpy().view(np.uint64)
    place, pos, off, rows, j, delta = [], [], [], [], 0, 0
    for x in list(lens[b]) + [seg[b]]:
        for i in range(int(x)):
            at = j + i // PAGE
            place.append(at * PAGE + i % PAGE)
            pos.append(delta + i)
            off.append(delta)
            rows.append(int(w[at] >> np.uint64(40)) * PAGE + i % PAGE)
        j += -(-int(x) // PAGE)
        delta += int(x)
    to = lambda a: torch.tensor(a, dtype=torch.long, device=s["meta"].device)  # noqa: E731
    return to(place), to(pos), to(off), to(rows)


def _exact_attention(s, case):
    B, Hq, H, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // H
    lens, seg, _, _ = _layout(case)
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=s["q"].device) if case["op"] == "shared" else s["weights"].double()
    if case["op"] == "weights" and not case["add"]:
        out.zero_()
    for b in range(B):
        place, p, off, rows = _request64(s, case, b, lens, seg)
        k = s["k"][rows // PAGE, :, rows % PAGE].double()
        last = int(lens[b].sum() + seg[b]) - 1
        if case["op"] == "shared":
            q, m, lse = s["q"][b:b + 1].double(), torch.tensor([last], device=p.device), None
        else:
            lo, hi = int(s["cu_q"][b]), int(s["cu_q"][b + 1])
            lo = max(lo, hi - case["window"]) if case["window"] else lo
            q, lse = s["q"][lo:hi].double(), s["lse"][lo:hi].double()
            m = last - torch.arange(hi - lo - 1, -1, -1, device=p.device)
        if case["kind"] != "alibi":
            k = _turn64(k, off.view(-1, 1).expand(-1, H), case)
            q = _turn64(q, m.view(-1, 1).expand(-1, Hq), case)
        for h in range(H):
            z = torch.einsum("ngd,td->ngt", q[:, h * G:(h + 1) * G], k[:, h]) * _softmax_scale(case)
            if case["kind"] == "alibi":
                z = z - s["slopes"][h * G:(h + 1) * G].double()[:, None] * (m.view(-1, 1, 1) - p)
            z = z.masked_fill((p > m.view(-1, 1)).unsqueeze(1), -math.inf)
            if case["op"] == "shared":
                v = s["v"][rows // PAGE, h, rows % PAGE].double()
                out[b, h * G:(h + 1) * G] = torch.einsum("gt,td->gd", torch.softmax(z[0], -1), v)
            else:
                out[b, place] += torch.exp(z - lse[:, h * G:(h + 1) * G].unsqueeze(-1)).sum((0, 1))
    return out


def _exact_plan(s, case):
    lens, seg, _, _ = _layout(case)
    words = s["meta"].cpu().numpy().view(np.uint64)
    weights = s["weights"].cpu().numpy().astype(np.float64)
    to = s["dst_pages"].cpu().numpy()
    B, MB = words.shape
    meta, docs = np.zeros((B, MB), np.int64), np.zeros(B, np.int32)
    src, dst = np.full((B, to.shape[1] * PAGE), -1, np.int32), np.full((B, to.shape[1] * PAGE), -1, np.int32)
    new_w = np.zeros((B, MB * PAGE))
    for b in range(B):
        keys, j = [], 0  # (document, block, row) in list order
        for d, x in enumerate(lens[b]):
            keys += [(d, j + i // PAGE, i % PAGE) for i in range(int(x))]
            j += -(-int(x) // PAGE)
        n = len(keys)
        rank = sorted(range(n), key=lambda i: (not (i < case["first"] or i >= n - case["recent"]),
                                               0.0 if i < case["first"] or i >= n - case["recent"]
                                               else -weights[b, keys[i][1] * PAGE + keys[i][2]], i))
        at, offset = 0, 0
        stay = sorted(rank[:case["keep"]])
        for d, x in enumerate(lens[b]):
            lo, hi = np.searchsorted(stay, [lens[b][:d].sum(), lens[b][:d + 1].sum()])
            mine = [keys[i] for i in stay[lo:hi]]
            for i, (_, blk, row) in enumerate(mine):
                page = int(to[b, at + i // PAGE])
                src[b, (at + i // PAGE) * PAGE + i % PAGE] = int(words[b, blk] >> np.uint64(40)) * PAGE + row
                dst[b, (at + i // PAGE) * PAGE + i % PAGE] = page * PAGE + i % PAGE
                new_w[b, (at + i // PAGE) * PAGE + i % PAGE] = weights[b, blk * PAGE + row]
                meta[b, at + i // PAGE] = i % PAGE + 1 | i // PAGE << 5 | offset << 16 | page << 40
            at += -(-len(mine) // PAGE)
            offset += int(x)
        docs[b] = at
        rest = min(MB - at, MB - j)
        meta[b, at:at + rest] = words[b, j:j + rest].view(np.int64)
        new_w[b, at * PAGE:(at + rest) * PAGE] = weights[b, j * PAGE:(j + rest) * PAGE]
    return [torch.from_numpy(x) for x in (meta, docs, src, dst, new_w)]


def exact(case, seed):
    if case["op"] == "move":
        return None  # values are copied, none is computed
    s = prepare(case, seed)
    return _exact_plan(s, case) if case["op"] == "plan" else _exact_attention(s, case)
