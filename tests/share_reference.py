"""Test-side restatement in 64 bits of the calls over shared lists and of eviction (numpy; no product code)."""
from __future__ import annotations

import math

import numpy as np

PAGE = 16


def bf16(x):
    """float64 values rounded to bf16 (nearest, ties to even)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def freqs(pos):
    rd = pos["rotary_dim"]
    th = pos["theta"] ** (-2.0 * np.arange(rd // 2) / rd)
    if pos["kind"] == "yarn":
        g = np.clip((4096 * th / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
        th = (1 - g) * th / 4.0 + g * th
    return th


def rotate(x, p, pos):
    """x [..., D] turned by positions p (broadcast over x's leading dimensions)."""
    if pos["kind"] not in ("rope", "yarn"):
        return x
    rd = pos["rotary_dim"]
    a = np.asarray(p, np.float64)[..., None] * freqs(pos)
    c, s = np.cos(a), np.sin(a)
    y = x.copy()
    if pos["interleaved"]:
        x1, x2 = x[..., 0:rd:2], x[..., 1:rd:2]
        y[..., 0:rd:2], y[..., 1:rd:2] = x1 * c - x2 * s, x1 * s + x2 * c
    else:
        h = rd // 2
        x1, x2 = x[..., :h], x[..., h:rd]
        y[..., :h], y[..., h:rd] = x1 * c - x2 * s, x1 * s + x2 * c
    return y


def scale_of(pos, D):
    s = 1.0 / math.sqrt(D)
    return s * (0.1 * math.log(4.0) + 1.0) ** 2 if pos["kind"] == "yarn" else s


class Lists:
    """Block lists, caches and queries of a small batch.  ``groups``: (requests, common document lengths) each;
    ``own``: per request the lengths of its further documents; ``seg``: per request the tokens of its query
    segment.  Rows and pages that hold no key hold NaN."""

    def __init__(self, rng, groups, own, seg, Hq, Hkv, D, pos, slack=1, spare=0):
        self.Hq, self.Hkv, self.D, self.pos = Hq, Hkv, D, pos
        self.seg = list(seg)
        self.lens, self.off, self.shared = [], [0], []
        b = 0
        for n, common in groups:
            self.shared.append(sum(-(-x // PAGE) for x in common))
            for _ in range(n):
                self.lens.append(list(common) + list(own[b]))
                b += 1
            self.off.append(b)
        while b < len(self.seg):  # outside every group
            self.lens.append(list(own[b]))
            b += 1
        self.B = b
        self.doc_blocks = np.array([sum(-(-x // PAGE) for x in le) for le in self.lens], np.int32)
        self.q_start = np.array([sum(le) for le in self.lens], np.int32)
        self.seq_len = self.q_start + np.array(self.seg, np.int32)
        self.max_blocks = max(1, max(int(d) + -(-s // PAGE) for d, s in zip(self.doc_blocks, self.seg)) + slack)
        pages, ids = 0, []
        for b in range(self.B):
            g = next((g for g in range(len(groups)) if self.off[g] <= b < self.off[g + 1]), None)
            n = int(self.doc_blocks[b]) + -(-self.seg[b] // PAGE)
            first = 0 if g is None or b == self.off[g] else self.shared[g]
            mine = list(ids[self.off[g]][:first]) if first else []
            mine += range(pages, pages + n - first)
            pages += n - first
            ids.append(mine)
        self.num_pages = pages + spare + 1
        where = rng.permutation(self.num_pages)
        self.spare = where[pages:pages + spare].astype(np.int32)
        self.meta = np.zeros((self.B, self.max_blocks), np.uint64)
        self.k = np.full((self.num_pages, Hkv, PAGE, D), np.nan)
        self.v = np.full((self.num_pages, Hkv, PAGE, D), np.nan)
        for b in range(self.B):
            j, delta = 0, 0
            for d, x in enumerate(self.lens[b] + [self.seg[b]]):
                for i in range(-(-x // PAGE)):
                    rows = min(PAGE, x - PAGE * i)
                    nv = PAGE if d == len(self.lens[b]) else rows
                    page = int(where[ids[b][j]])
                    self.meta[b, j] = nv | i << 5 | delta << 16 | page << 40
                    if np.isnan(self.k[page, 0, 0, 0]):
                        self.k[page, :, :rows] = bf16(rng.standard_normal((Hkv, rows, D)))
                        self.v[page, :, :rows] = bf16(rng.standard_normal((Hkv, rows, D)))
                    j += 1
                delta += x
        self.q = bf16(rng.standard_normal((self.B, Hq, D)))
        self.slopes = np.exp2(-8.0 * np.arange(1, Hq + 1) / Hq).astype(np.float32) if pos["kind"] == "alibi" else None


def keys(meta, doc_blocks, q_start, seq_len):
    """(place, position, Delta, page, row) of every key of one list, in order."""
    out = []
    nb = int(doc_blocks) + -(-max(0, int(seq_len) - int(q_start)) // PAGE)
    for j in range(nb):
        w = int(meta[j])
        nv, pg, delta, page = w & 31, w >> 5 & 2047, w >> 16 & 0xFFFFFF, w >> 40
        for t in range(nv):
            p = delta + PAGE * pg + t
            if p < seq_len:
                out.append((j * PAGE + t, p, delta, page, t))
    return np.array(out, np.int64).reshape(-1, 5)


def scores(x, b, q, m, meta=None, doc_blocks=None, k=None, scale=None):
    """(scores [n, Hq, keys], keys) of queries q [n, Hq, D] at positions m [n]; -inf where a key is not seen."""
    ks = keys((x.meta if meta is None else meta)[b], (x.doc_blocks if doc_blocks is None else doc_blocks)[b],
              x.q_start[b], x.seq_len[b])
    kc = x.k if k is None else k
    place, p, delta, page, row = ks.T
    kk = rotate(kc[page, :, row], delta[:, None], x.pos)  # [N, Hkv, D]
    qq = rotate(q, np.asarray(m)[:, None], x.pos)
    s = np.einsum("nhd,thd->nht", qq, np.repeat(kk, x.Hq // x.Hkv, 1))
    s = s * (scale_of(x.pos, x.D) if scale is None else scale)
    if x.pos["kind"] == "alibi":
        s = s - x.slopes.astype(np.float64)[:, None] * (np.asarray(m)[:, None, None] - p)
    return np.where(p <= np.asarray(m)[:, None, None], s, -np.inf), ks


def softmax(s):
    top = s.max(-1, keepdims=True) if s.shape[-1] else np.full(s.shape[:-1] + (1,), -np.inf)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    e = np.where(np.isneginf(s), 0.0, e)
    tot = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        return e / np.where(tot > 0, tot, 1.0), np.where(tot > 0, top + np.log(np.where(tot > 0, tot, 1.0)), -np.inf)[..., 0]


def decode(x, meta=None, doc_blocks=None, k=None, v=None, scale=None):
    """(out [B, Hq, D], lse [B, Hq], sum of p |v|, largest |q| |k| scale) of one decode step."""
    out, mass = np.zeros((x.B, x.Hq, x.D)), np.zeros((x.B, x.Hq, x.D))
    lse, reach = np.full((x.B, x.Hq), -np.inf), 0.0
    vc = x.v if v is None else v
    for b in range(x.B):
        if x.seq_len[b] <= 0:
            continue
        s, ks = scores(x, b, x.q[b:b + 1], [int(x.seq_len[b]) - 1], meta, doc_blocks, k, scale)
        if not len(ks):
            continue
        w, ls = softmax(s[0])
        vv = np.repeat(vc[ks[:, 3], :, ks[:, 4]], x.Hq // x.Hkv, 1)
        out[b], mass[b], lse[b] = np.einsum("ht,thd->hd", w, vv), np.einsum("ht,thd->hd", w, np.abs(vv)), ls
        kc = (x.k if k is None else k)[ks[:, 3], :, ks[:, 4]]
        reach = max(reach, np.linalg.norm(x.q[b], axis=-1).max() * np.linalg.norm(kc, axis=-1).max()
                    * (scale_of(x.pos, x.D) if scale is None else scale))
    return out, lse, mass, reach


def key_weights(x, q, lse, cu, window=0):
    """weights [B, 16 max_blocks] that the rows q of each request give."""
    w = np.zeros((x.B, x.max_blocks * PAGE))
    for b in range(x.B):
        lo, hi = int(cu[b]), int(cu[b + 1])
        lo = max(lo, hi - window) if window else lo
        if lo == hi:
            continue
        m = int(x.seq_len[b]) - hi + np.arange(lo, hi)
        s, ks = scores(x, b, q[lo:hi], m)
        ls = lse[lo:hi].astype(np.float64)[..., None]
        e = np.exp(s - np.where(np.isneginf(ls), 0.0, ls))
        w[b, ks[:, 0]] += np.where(np.isneginf(s) | np.isneginf(ls), 0.0, e).sum((0, 1))
    return w


def plan(weights, meta, doc_blocks, keep, dst, num_pages, first, recent):
    """What evict_plan writes: (new meta, new document blocks, source and destination slots, new weights)."""
    B, MB = meta.shape
    R = dst.shape[1]
    nm, nd = np.zeros_like(meta), np.zeros(B, np.int32)
    src, to = np.full((B, R * PAGE), -1, np.int32), np.full((B, R * PAGE), -1, np.int32)
    nw = np.zeros((B, MB * PAGE), np.float32)
    for b in range(B):
        if keep[b] < 0:
            nm[b], nd[b], nw[b] = meta[b], doc_blocks[b], weights[b]
            continue
        docs, last = [], None  # runs of blocks with one Delta
        for j in range(int(doc_blocks[b])):
            w = int(meta[b, j])
            if last != w >> 16 & 0xFFFFFF:
                last = w >> 16 & 0xFFFFFF
                docs.append([])
            docs[-1] += [(j, t) for t in range(min(w & 31, PAGE))]
        flat = [(d, j, t) for d, ks in enumerate(docs) for j, t in ks]
        n = len(flat)

        def rank(i):
            safe = i < first or i >= n - recent
            w = float(weights[b, flat[i][1] * PAGE + flat[i][2]])
            return (not safe, 0.0 if safe else (math.inf if math.isnan(w) else -w), not safe and math.isnan(w), i)

        stay = sorted(sorted(range(n), key=rank)[:int(keep[b])])
        at = 0
        for d in range(len(docs)):
            mine = [flat[i] for i in stay if flat[i][0] == d]
            for i, (_, j, t) in enumerate(mine):
                blk, row = at + i // PAGE, i % PAGE
                w = int(meta[b, j])
                page = int(dst[b, blk]) if blk < R else -1
                good = 0 <= page < num_pages
                nm[b, blk] = (row + 1 if good else 0) | i // PAGE << 5 | (w >> 16 & 0xFFFFFF) << 16 | (page if good else 0) << 40
                if good:
                    src[b, blk * PAGE + row] = (w >> 40) * PAGE + t
                    to[b, blk * PAGE + row] = page * PAGE + row
                    nw[b, blk * PAGE + row] = weights[b, j * PAGE + t]
            at += -(-len(mine) // PAGE)
        nd[b] = at
        rest = min(MB - at, MB - int(doc_blocks[b]))
        nm[b, at:at + rest] = meta[b, doc_blocks[b]:doc_blocks[b] + rest]
        nw[b, at * PAGE:(at + rest) * PAGE] = weights[b, doc_blocks[b] * PAGE:(doc_blocks[b] + rest) * PAGE]
    return nm, nd, src, to, nw


def move(src, dst, k, v):
    k, v = k.copy(), v.copy()
    for s, d in zip(np.asarray(src).ravel(), np.asarray(dst).ravel()):
        if s >= 0 and d >= 0:
            for c in (k, v):
                c[d // PAGE, :, d % PAGE] = c[s // PAGE, :, s % PAGE]
    return k, v
