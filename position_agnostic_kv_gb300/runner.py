"""Device-resident driver for one batch of requests over a paged, position-free KV cache.

This is the call sequence a serving engine makes, expressed through the public binding only:
build the block words on the host (``lazy_build_doc_meta``), write each cached document's
keys and values once (``lazy_kv_write`` at local positions), then per batch write the query
tokens, run the causal prefill, and for every decode step write the new token and attend.

The batch description is duck-typed (any object with the attributes used below, e.g. a
``workloads.Workload``); values arrive as bf16 bit patterns (numpy uint16).
"""
from __future__ import annotations

import numpy as np
import torch

from . import (PHASE_DECODE, PHASE_DECODE_Q4, PHASE_KEY_WEIGHTS, PHASE_PREFILL, PHASE_PREFILL_Q4, attn_decode,
               attn_decode_q4, attn_decode_shared, attn_key_weights, attn_prefill, attn_prefill_q4, build_doc_meta,
               build_rope_table, decode_shared_workspace_size, evict_plan, kv_move, kv_write, kv_write_q4,
               pos_cfg_from, q4_cache_shape, workspace_size)

PAGE = 16


def bits_to_tensor(bits: np.ndarray, device) -> torch.Tensor:
    """bf16 bit patterns (numpy uint16) -> bf16 tensor on ``device`` (exact)."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.view(torch.bfloat16).to(device)


def i32(x, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).to(device)


# What one group more costs, in page reads (of a request's 8 heads).  Reading a page for a group takes about as long as reading
# it twice alone, whatever the number of requests, and every group has a start, its results and their join: decode steps of
# 64 requests, 32 / 8 heads, that begin with 8 common pages, as one group / as groups of 8 that share 30, 60, 120, 250 pages
# more: 27.3 / 32.4, 35.5 / 34.5, 51.9 / 40.6, 88.7 / 54.9 us; of 4 with 60, 120, 250: 37.5 / 42.7, 53.9 / 54.9, 90.9 / 81.6.
# (Groups of 2, and of 4 with 30, the call decodes alone either way.)
_GROUP_COST = 256


def common_prefixes(meta: np.ndarray, doc_blocks, min_blocks: int = 1):
    """Groups of neighbouring requests whose lists begin with the same document blocks, as ``attn_decode_shared``
    takes them: (group_off [n + 1], shared_blocks [n], int32).  Neighbours with fewer than ``min_blocks`` common words are
    in different groups; others too where requests go deeper together than all share, and reading those pages once is
    worth more than another group costs (the order of the requests is the caller's)."""
    meta, nd = np.asarray(meta), np.asarray(doc_blocks).astype(np.int64)
    n = len(nd)
    if n == 0:
        return np.zeros(1, np.int32), np.zeros(0, np.int32)
    same = meta[1:] == meta[:-1]
    deep = np.where(same.all(1), meta.shape[1], np.argmin(same, 1))  # words that a request shares with the one before
    deep = np.minimum(deep, np.minimum(nd[1:], nd[:-1]))
    # What a group shares is the least over its neighbours.  best[j]: most that the first j requests save, with a last
    # group that begins at last[j]; low[i]: what requests i .. j - 1 share, from the first that can be in one group with j - 1.
    best, last, low, begin = np.zeros(n + 1, np.int64), np.zeros(n + 1, np.int64), np.zeros(n, np.int64), 0
    for j in range(1, n + 1):
        if j > 1:
            if deep[j - 2] < max(min_blocks, 1):
                begin = j - 1
            low[j - 2] = deep[j - 2]
            np.minimum(low[begin:j - 1], deep[j - 2], out=low[begin:j - 1])
        more = np.arange(j - 2 - begin, -2, -1)  # requests beyond two; -1 for one alone, where low is still 0
        save = best[begin:j] + low[begin:j] * more
        save[1:] -= _GROUP_COST  # a cut between requests that could be in one group
        last[j] = begin + int(np.argmax(save))
        best[j] = save[last[j] - begin]
    off = [n]
    while off[-1]:
        off.append(int(last[off[-1]]))
    off.reverse()
    shared = [int(nd[lo]) if hi - lo == 1 else int(deep[lo:hi - 1].min()) for lo, hi in zip(off, off[1:])]
    return np.array(off, np.int32), np.array(shared, np.int32)


class PagedBatch:
    """Caches, block words and per-request metadata of one batch, resident on one GPU.

    ``kv_bits=4`` keeps keys and values in one 4-bit cache (``kv_cache``, with the power-of-two
    factors ``k_scale`` / ``v_scale``) instead of the bf16 ``k_cache`` and ``v_cache``.  ``spare_pages`` adds
    free pages behind those of the workload (for ``evict``)."""

    def __init__(self, w, device="cuda", use_table: bool = False, pos_kind: str | None = None,
                 kv_bits: int = 16, k_scale: float = 1.0, v_scale: float = 1.0, spare_pages: int = 0):
        if kv_bits not in (4, 16):
            raise ValueError(f"kv_bits must be 16 or 4, got {kv_bits}")
        self.kv_bits, self.factors = kv_bits, dict(k_scale=k_scale, v_scale=v_scale)
        self.w = w
        self.device = torch.device(device)
        self.B, self.Hq, self.Hkv, self.D = w.B, w.Hq, w.Hkv, w.D
        (self.block_table, self.meta_h, self.seq_len0_h, self.q_start_h,
         self.doc_blocks_h) = build_doc_meta(w.req_inst_off, w.req_inst, w.inst_len,
                                             w.inst_page_off, w.inst_pages, w.q_len,
                                             w.q_page_off, w.q_pages, w.max_blocks)
        dev = self.device
        self.meta = torch.from_numpy(self.meta_h.view(np.int64)).to(dev)
        self.q_start = i32(self.q_start_h, dev)
        self.doc_blocks = i32(self.doc_blocks_h, dev)
        self.seq_len0 = i32(self.seq_len0_h, dev)
        self.cu_q = i32(w.cu_q, dev)
        self.max_q = int(np.max(w.q_len)) if len(w.q_len) else 0
        self.total_q = int(np.sum(w.q_len))
        shape = (w.num_pages + spare_pages, w.Hkv, PAGE, w.D)
        self.k_cache = self.v_cache = self.kv_cache = None
        if kv_bits == 4:
            self.kv_cache = torch.zeros(q4_cache_shape(w.num_pages + spare_pages, w.Hkv, w.D), dtype=torch.uint8, device=dev)
        else:
            self.k_cache = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
            self.v_cache = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        p = w.pos
        kind = pos_kind or p.kind
        self.slopes = None
        if p.alibi_slopes is not None:
            self.slopes = torch.from_numpy(np.asarray(p.alibi_slopes, np.float32)).to(dev)
        self.table = None
        rd = getattr(p, "rotary_dim", w.D) if kind in ("rope", "yarn") else w.D
        inter = bool(getattr(p, "interleaved", False))
        self.cfg = pos_cfg_from(kind, w.D, rope_theta=p.rope_theta, yarn_factor=p.yarn_factor,
                                yarn_orig_ctx=p.yarn_orig_ctx, yarn_beta_fast=p.yarn_beta_fast,
                                yarn_beta_slow=p.yarn_beta_slow, alibi_slopes=self.slopes,
                                rotary_dim=rd, interleaved=inter)
        if use_table and kind in ("rope", "yarn"):
            max_pos = int(self.q_start_h.max()) + int(np.max(w.q_len)) + w.n_decode + 1
            self.table = torch.empty((max_pos, rd), dtype=torch.float32, device=dev)
            build_rope_table(self.cfg, max_pos, self.table)
            self.cfg = pos_cfg_from(kind, w.D, rope_theta=p.rope_theta,
                                    yarn_factor=p.yarn_factor, yarn_orig_ctx=p.yarn_orig_ctx,
                                    yarn_beta_fast=p.yarn_beta_fast,
                                    yarn_beta_slow=p.yarn_beta_slow, alibi_slopes=self.slopes,
                                    cos_sin=self.table, rotary_dim=rd, interleaved=inter)
        self.max_blocks = w.max_blocks
        ph_dec, ph_pre = (PHASE_DECODE, PHASE_PREFILL) if kv_bits == 16 else (PHASE_DECODE_Q4, PHASE_PREFILL_Q4)
        ws_dec = workspace_size(ph_dec, self.B, self.B, self.max_blocks, self.Hq, self.Hkv,
                                self.D)
        ws_pre = workspace_size(ph_pre, max(self.total_q, 1), self.B, self.max_blocks,
                                self.Hq, self.Hkv, self.D)
        self.ws = torch.empty(max(ws_dec, ws_pre, 256), dtype=torch.uint8, device=dev)
        self.groups = None  # see share_prefixes
        # What calls took before it was replaced.  Steps that were captured into graphs name it by address, so it stays.
        self._former_ws, self._all_groups = [], []

    def _workspace(self, n: int):
        """From now on at least n bytes of workspace."""
        if n > self.ws.numel():
            self._former_ws.append(self.ws)
            self.ws = torch.empty(n, dtype=torch.uint8, device=self.device)

    def _write(self, k, v, slot, lp):
        if self.kv_bits == 4:
            kv_write_q4(k, v, slot, lp, self.kv_cache, self.cfg, **self.factors)
        else:
            kv_write(k, v, slot, lp, self.k_cache, self.v_cache, self.cfg)

    # ---------------------------------------------------------------- cache fill
    def fill_documents(self):
        """Write every document copy into the cache once (keys rotated by local position)."""
        w = self.w
        by_doc: dict[int, list[int]] = {}
        for i, d in enumerate(w.inst_doc):
            by_doc.setdefault(int(d), []).append(i)
        for d, insts in by_doc.items():
            k, v = w.doc_kv(d)
            kt, vt = bits_to_tensor(k, self.device), bits_to_tensor(v, self.device)
            for i in insts:
                slot, lp = w.inst_slots(i)
                self._write(kt, vt, i32(slot, self.device), i32(lp, self.device))

    # ---------------------------------------------------------------- prefill
    def upload_prefill(self):
        q, k, v, slot, lp = self.w.prefill_tokens()
        dev = self.device
        return dict(q=bits_to_tensor(q, dev), k=bits_to_tensor(k, dev), v=bits_to_tensor(v, dev),
                    slot=i32(slot, dev), lp=i32(lp, dev))

    def prefill(self, inp, out=None, lse=None):
        """Write the query tokens' keys/values, then the causal prefill of every query row."""
        if out is None:
            out = torch.empty((self.total_q, self.Hq, self.D), dtype=torch.bfloat16,
                              device=self.device)
        if self.total_q == 0:
            return out
        self._write(inp["k"], inp["v"], inp["slot"], inp["lp"])
        if self.kv_bits == 4:
            attn_prefill_q4(inp["q"], self.cu_q, self.q_start, self.doc_blocks, self.meta, self.kv_cache, self.cfg,
                            out, self.max_q, lse=lse, ws=self.ws, **self.factors)
        else:
            attn_prefill(inp["q"], self.cu_q, self.q_start, self.doc_blocks, self.meta, self.k_cache,
                         self.v_cache, self.cfg, out, self.max_q, lse=lse, ws=self.ws)
        return out

    # ---------------------------------------------------------------- decode
    def upload_decode(self, t: int):
        q, k, v, slot, lp = self.w.decode_tokens(t)
        dev = self.device
        seq = self.seq_len0_h + t + 1
        return dict(q=bits_to_tensor(q, dev), k=bits_to_tensor(k, dev), v=bits_to_tensor(v, dev),
                    slot=i32(slot, dev), lp=i32(lp, dev), seq_len=i32(seq, dev))

    def decode_step(self, inp, out=None, lse=None):
        """Write step t's token (at p = m) then attend from it."""
        if out is None:
            out = torch.empty((self.B, self.Hq, self.D), dtype=torch.bfloat16, device=self.device)
        self._write(inp["k"], inp["v"], inp["slot"], inp["lp"])
        if self.kv_bits == 4:
            attn_decode_q4(inp["q"], inp["seq_len"], self.q_start, self.doc_blocks, self.meta, self.kv_cache,
                           self.cfg, out, lse=lse, ws=self.ws, **self.factors)
        elif self.groups is not None:
            attn_decode_shared(inp["q"], inp["seq_len"], self.q_start, self.doc_blocks, self.meta, *self.groups,
                               self.k_cache, self.v_cache, self.cfg, out, lse=lse, ws=self.ws)
        else:
            attn_decode(inp["q"], inp["seq_len"], self.q_start, self.doc_blocks, self.meta,
                        self.k_cache, self.v_cache, self.cfg, out, lse=lse, ws=self.ws)
        return out

    def share_prefixes(self, min_blocks: int = 8):
        """From now on decode steps read the documents that neighbouring requests list first, in the same
        order, once per group (bf16 caches).  Returns the number of requests that share.  Keys that a group shares meet
        its queries in f16 and their weights are rounded to bf16, where a request's own keys and ``attn_decode`` keep more:
        relative to 64 bits 0.0024 instead of 0.0017, which is the result's rounding to bf16."""
        if self.kv_bits != 16:
            raise ValueError("share_prefixes: the calls over shared lists need a bf16 cache")
        off, shared = common_prefixes(self.meta.cpu().numpy(), self.doc_blocks.cpu().numpy(), min_blocks)
        size = np.diff(off)
        biggest, longest = int(size.max(initial=0)), int(shared.max(initial=0))
        self._workspace(decode_shared_workspace_size(self.B, len(shared), biggest, longest, self.max_blocks, self.Hq,
                                                     self.Hkv, self.D))
        if self.groups is None or not all(map(np.array_equal, self._grouping, (off, shared))):
            self.groups, self._grouping = (i32(off, self.device), i32(shared, self.device), biggest, longest), (off, shared)
            self._all_groups.append(self.groups)
        return int(size[size > 1].sum())

    # ---------------------------------------------------------------- eviction inside a context (bf16 caches)
    def key_weights(self, q, lse, seq_len, cu_q=None, window: int = 0, weights=None, max_q: int | None = None):
        """The attention weight that every key of the lists receives from the rows ``q`` (with the log-sum-exps of
        their attention call; requests' last tokens, split by ``cu_q``, by default one row per request), in a new
        tensor [B, 16 max_blocks], or added to ``weights``.  ``max_q`` bounds the rows of a request (by default the
        prefill's longest segment for its own ``cu_q``, all rows for another): give it, for where it and ``window`` leave
        up to 32 rows per KV head, queries count with 24 bits instead of 16 and the call is faster."""
        if self.kv_bits != 16:
            raise ValueError("key_weights: needs a bf16 cache")
        if max_q is None:
            max_q = 1 if cu_q is None else self.max_q if cu_q is self.cu_q else q.shape[0]
        if max_q < 0:
            raise ValueError(f"key_weights: max_q must not be negative, got {max_q}")
        if cu_q is None:
            cu_q = torch.arange(self.B + 1, dtype=torch.int32, device=self.device)  # made on the device: captures take it
        self._workspace(workspace_size(PHASE_KEY_WEIGHTS, q.shape[0], self.B, self.max_blocks, self.Hq, self.Hkv, self.D))
        add = weights is not None
        if not add:
            weights = torch.empty((self.B, PAGE * self.max_blocks), dtype=torch.float32, device=self.device)
        attn_key_weights(q, lse, cu_q, seq_len, self.q_start, self.doc_blocks, self.meta, self.k_cache, self.cfg, weights,
                         min(max_q, q.shape[0]), window=window, accumulate=add, ws=self.ws)
        return weights

    def evict(self, weights, keep, pages, first: int = 0, recent: int = 0):
        """Cut every request's documents to the ``keep`` keys of the largest ``weights`` (the ``first`` and
        ``recent`` ones before all others): the rows move to the free ``pages`` [B, n], the lists change, and the
        weights come back in the new order.  The old pages are the caller's to free.  The lists change in place: a
        step that was captured into a graph before reads the new ones, and takes nothing for common."""
        if self.kv_bits != 16:
            raise ValueError("evict: needs a bf16 cache")
        pages = i32(pages, self.device)
        meta, nd, new_w = torch.empty_like(self.meta), torch.empty_like(self.doc_blocks), torch.empty_like(weights)
        src = torch.empty((self.B, PAGE * pages.shape[1]), dtype=torch.int32, device=self.device)
        dst = torch.empty_like(src)
        evict_plan(weights, self.meta, self.doc_blocks, i32(keep, self.device), pages, self.k_cache.shape[0], self.cfg, meta,
                   nd, src, dst, new_w, first=first, recent=recent)
        kv_move(src, dst, self.k_cache, self.v_cache)
        self.meta.copy_(meta)
        self.doc_blocks.copy_(nd)
        for _, shared, _, _ in self._all_groups:  # nothing is common any more
            shared.zero_()
        self.groups = None
        return new_w


# -------------------------------------------------------------------- cold documents
def encode_document(q, k, v, pages, k_cache, v_cache, cfg, ws=None, out=None, **factors):
    """Cold-document processing: the first time a document is seen it is encoded alone, from
    local position 0 ([NOTE] 整体框架: each document's cache is built independently, indexed
    from 0).  Its keys (rotated by their local positions) and values are written into
    ``pages`` of the position-free cache, then the document's own causal attention runs as a
    request with no cached documents whose query segment is the document (Delta = 0).

    q, k, v: bf16 [L, Hq | Hkv, D] raw projections of the document's tokens; pages: int list
    of ceil(L / 16) physical page ids.  Returns the attention output [L, Hq, D] (bf16); the
    cached pages can then be reused by any later request at any document offset.

    With ``v_cache=None``, ``k_cache`` is a 4-bit cache that holds both (``factors``: its
    ``k_scale`` and ``v_scale``); the document then attends to its keys and values as stored."""
    L, Hq, D = q.shape
    dev = q.device
    pages = np.asarray(pages, dtype=np.int32)
    if len(pages) * PAGE < L:
        raise ValueError("encode_document: fewer pages than the document needs")
    t = np.arange(L, dtype=np.int32)
    slot, lp = i32(pages[t // PAGE] * PAGE + t % PAGE, dev), i32(t, dev)
    if v_cache is None:
        kv_write_q4(k, v, slot, lp, k_cache, cfg, **factors)
    else:
        kv_write(k, v, slot, lp, k_cache, v_cache, cfg, **factors)
    max_blocks = len(pages)
    _, meta_h, _, q_start_h, doc_blocks_h = build_doc_meta(
        [0, 0], [], [], [0], [], [L], [0, len(pages)], pages, max_blocks)
    meta = torch.from_numpy(meta_h.view(np.int64)).to(dev)
    if out is None:
        out = torch.empty((L, Hq, D), dtype=torch.bfloat16, device=dev)
    Hkv = k_cache.shape[1]
    if ws is None:
        n = workspace_size(PHASE_PREFILL_Q4 if v_cache is None else PHASE_PREFILL, L, 1, max_blocks, Hq, Hkv, D)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    if v_cache is None:
        attn_prefill_q4(q, i32([0, L], dev), i32(q_start_h, dev), i32(doc_blocks_h, dev), meta, k_cache, cfg, out, L,
                        ws=ws, **factors)
        return out
    attn_prefill(q, i32([0, L], dev), i32(q_start_h, dev), i32(doc_blocks_h, dev), meta, k_cache,
                 v_cache, cfg, out, L, ws=ws)
    return out
