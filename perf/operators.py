"""The operators of the 4-bit paged K/V cache, as cases to time and to compare.

Each case is one call that a serving program makes: writing tokens into the cache and reading
them back (``kv_write_q4``, ``kv_read_q4``), one decode step (``attn_decode_q4``) or one causal
prefill (``attn_prefill_q4``) over the cache.  ``run`` computes them with elementary torch
operations in 32 bits, or, with ``own`` set, makes the library's calls.  ``exact`` restates the
definitions in 64 bits.

The cache format (one uint8 block of 18 D bytes per page and KV head; D is the head dimension, a
page has 16 token rows): every 16 consecutive dimensions of a row form a group with one e4m3
scale, every value is an e2m1 code (sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6) times its group's scale
times the cache's power-of-two factor.  Byte offsets in a block, for row r and dimension d:
  K code   r D/2 + d/2, low half of the byte for even d
  K scale  8 D + ((r % 8) 4 + d / (D/4)) D/32 + (r / 8) D/64 + (d % (D/4)) / 16
  V code   9 D + (r / 8) A + (d / (D/8) 4 + (r % 8) / 2) 16 + (r % 2) D/16 + (d % (D/8)) / 2, where
           A = 512 for D = 128 and 8 for D = 64; low half of the byte for even d
  V scale  17 D + (d / 16) 16 + ((r % 8) / 2) 4 + (r / 8) 2 + r % 2
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # e2m1 magnitudes


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    d = dict(name=name, op=op, Hkv=8, D=128, kind="rope", theta=5e5, rotary_dim=128, interleaved=False,
             k_scale=1.0, v_scale=1.0, layout=0)
    d.update(kw)
    return d


def listed():
    return [
        # the new token of each of 64 requests, written between two decode steps
        _case("append_step", "write", T=64, doc_len=1),
        # twenty documents of 1600 tokens entering the cache
        _case("ingest_documents", "write", T=32000, doc_len=1600),
        # one 200-token document read back, e.g. to move it to another pool
        _case("read_document", "read", T=200, doc_len=200),
        # a long context read back whole
        _case("read_context", "read", T=128000, doc_len=1600),
        # a decode step of one short request, small heads
        _case("decode_tiny", "decode", B=1, Hq=4, Hkv=2, D=64, rotary_dim=64, theta=1e4, docs=2, doc_len=80,
              ragged=True, seg=17),
        # a decode step of a small batch over ten retrieved documents each
        _case("decode_rag", "decode", B=16, Hq=32, docs=10, doc_len=200, ragged=False, seg=33),
        # a decode step of a large batch over 32 000-token contexts
        _case("decode_long", "decode", B=64, Hq=32, docs=20, doc_len=1600, ragged=False, seg=1),
        # a decode step with one KV head for 32 query heads, and linear biases
        _case("decode_mqa_alibi", "decode", B=32, Hq=32, Hkv=1, kind="alibi", docs=12, doc_len=1000, ragged=False,
              seg=33),
        # the 32-token questions of a small batch over ten retrieved documents each
        _case("prefill_rag", "prefill", B=16, Hq=32, docs=10, doc_len=200, ragged=False, q_len=32),
        # 64-token questions of a model with 64 heads over long contexts
        _case("prefill_wide", "prefill", B=8, Hq=64, docs=20, doc_len=512, ragged=False, q_len=64),
        # one KV head for 32 query heads, linear biases, every question over twelve documents
        _case("prefill_mqa_alibi", "prefill", B=32, Hq=32, Hkv=1, kind="alibi", docs=12, doc_len=1000, ragged=False,
              q_len=32),
        # one 1600-token document seen for the first time: its own causal attention
        _case("encode_document", "prefill", B=1, Hq=32, docs=0, doc_len=0, ragged=False, q_len=1600),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    D = rng.choice([64, 128, 128])
    kind = rng.choice(["rope", "rope", "yarn", "alibi"])
    rd = D if kind == "alibi" or rng.random() < 0.6 else 16 * rng.randint(1, D // 16)
    common = dict(D=D, kind=kind, rotary_dim=rd, interleaved=kind != "alibi" and rng.random() < 0.25,
                  theta=rng.choice([1e4, 5e5]), k_scale=rng.choice([1.0, 1.0, 0.25, 4.0]),
                  v_scale=rng.choice([1.0, 1.0, 0.5]), layout=rng.randint(1, 1 << 20))
    op = rng.choice(["write", "read", "decode", "prefill"])
    if op in ("write", "read"):
        c = dict(op=op, Hkv=rng.choice([1, 2, 4, 8]), doc_len=_log(rng, 1, 1600), **common)
        c["T"] = _log(rng, 1, 32000 if op == "write" else 128000)
    else:
        Hq, Hkv = rng.choice([(4, 2), (8, 8), (16, 2), (32, 8), (32, 8), (32, 1), (64, 8), (24, 1)])
        docs, doc_len = rng.randint(1, 20), _log(rng, 1, 1600)
        if op == "decode":
            c = dict(op=op, B=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, docs=docs, doc_len=doc_len, ragged=True,
                     seg=rng.randint(1, 48), **common)
        else:
            B, q_len = _log(rng, 1, 16), _log(rng, 1, 100)
            if rng.random() < 0.25:
                B, q_len, docs = 1, _log(rng, 100, 1600), rng.randint(0, 2)
            while B * q_len * (docs * doc_len + q_len) * Hq > 2.5e8:  # below the largest listed prefill
                doc_len = max(1, doc_len // 2)
                q_len = max(1, q_len - q_len // 4)
            c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, docs=docs, doc_len=doc_len, ragged=True, q_len=q_len, **common)
    return {k: c[k] for k in sorted(c)}


def _lengths(case):
    """Document lengths [B][docs] of an attention case, and every request's query tokens."""
    r = np.random.default_rng([int(case["layout"]), int(case["docs"]), int(case["doc_len"])])
    B, n, L = case["B"], case["docs"], case["doc_len"]
    lens = r.integers(1, L + 1, (B, n)) if case["ragged"] and n else np.full((B, n), L, np.int64)
    q = np.full(B, case.get("q_len", case.get("seg", 0)), np.int64)
    if case["ragged"] and case["op"] == "prefill" and B > 1:
        q = r.integers(1, case["q_len"] + 1, B)
        q[r.integers(0, B)] = case["q_len"]
    return lens.astype(np.int64), q


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    cached = Hkv * 18 * D / 16  # bytes of one token's keys and values in the cache
    plain = Hkv * D * 4  # bytes of the same in bf16
    if case["op"] == "write":  # read in bf16, written in 4 bits, read in 4 bits, written in bf16
        return {"bytes": case["T"] * (2 * plain + 2 * cached + 12), "flops": 0}
    if case["op"] == "read":
        return {"bytes": case["T"] * (plain + cached + 4), "flops": 0}
    lens, q = _lengths(case)
    keys = lens.sum(1) + q  # cached keys of each request
    blocks = (-(-lens // PAGE)).sum(1) + -(-q // PAGE)
    rows = np.ones_like(q) if case["op"] == "decode" else q
    pairs = keys if case["op"] == "decode" else q * lens.sum(1) + q * (q + 1) // 2
    return {"bytes": float((keys * cached + blocks * 8 + rows * case["Hq"] * D * 4).sum()),
            "flops": float(4 * D * case["Hq"] * pairs.sum())}


# ------------------------------------------------------------------ inputs
def _spread(x, gen):
    """Some channels of keys are much larger than the others."""
    c = torch.exp(0.5 * torch.randn(x.shape[-2:], generator=gen, device=x.device))
    return x * c


def _quantise(x, factor):
    """Codes (uint8, one per value) and e4m3 scales of float32 x [..., D], groups of 16."""
    y = x.unflatten(-1, (-1, 16)) / factor
    s = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float().unsqueeze(-1)
    m = torch.where(sf > 0, y.abs() / sf, torch.zeros_like(y))
    # nearest level; a value half way between two goes to the one with the even code
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code + 8 * ((y < 0) & (sf > 0)).to(torch.uint8)
    return code.flatten(-2), s


def _pack(kc, ks, vc, vs):
    """Cache blocks [P, H, 18 D] from codes [P, H, 16, D] and scales [P, H, 16, D/16]."""
    P, H, _, D = kc.shape
    pairs = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)  # noqa: E731
    kb = pairs(kc).reshape(P, H, 8 * D)
    ksb = ks.view(torch.uint8).view(P, H, 2, 8, 4, D // 64).permute(0, 1, 3, 4, 2, 5).reshape(P, H, D)
    vb = pairs(vc).view(P, H, 2, 4, 2, 8, D // 16)  # half, t, odd, lane group, bytes
    order = (0, 1, 2, 5, 3, 4, 6) if D == 128 else (0, 1, 5, 3, 2, 4, 6)
    vb = vb.permute(*order).reshape(P, H, 8 * D)
    vsb = vs.view(torch.uint8).view(P, H, 2, 4, 2, D // 16).permute(0, 1, 5, 3, 2, 4).reshape(P, H, D)
    return torch.cat([kb, ksb, vb, vsb], -1)


def _random_cache(pages, case, gen, dev):
    H, D = case["Hkv"], case["D"]
    cache = torch.empty((pages, H, 18 * D), dtype=torch.uint8, device=dev)
    step = 16384
    for p in range(0, pages, step):
        n = min(step, pages - p)
        k = torch.randn((n, 16, H, D), generator=gen, device=dev)
        k = _spread(k, gen).transpose(1, 2).to(torch.bfloat16).float()
        v = torch.randn((n, H, 16, D), generator=gen, device=dev).to(torch.bfloat16).float()
        cache[p:p + n] = _pack(*_quantise(k, case["k_scale"]), *_quantise(v, case["v_scale"]))
    return cache


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


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)  # noqa: E731
    s = {"case": dict(case)}
    H, D = case["Hkv"], case["D"]
    if case["op"] in ("write", "read"):
        T, L = case["T"], case["doc_len"]
        local = np.arange(T) % L
        start = 0
        if L == 1:  # single tokens, each somewhere in a page of its own
            start = rng.integers(0, 2000, T)
        per = -(-L // PAGE)
        page = np.arange(T) // L * per + local // PAGE
        pages = int(page[-1]) + 1
        row = (local + start) % PAGE
        s["slot"] = i32(rng.permutation(pages)[page] * PAGE + row)
        s["local_pos"] = i32(local + start)
        for n in ("k", "v") if case["op"] == "write" else ():
            x = torch.randn((T, H, D), generator=gen, device=dev)
            s[n] = (_spread(x, gen) if n == "k" else x).to(torch.bfloat16)
        if case["op"] == "write":
            s["cache"] = torch.zeros((pages, H, 18 * D), dtype=torch.uint8, device=dev)
            if case["kind"] != "alibi":  # the program's cos/sin table
                a = torch.arange(int((local + start).max()) + 1, device=dev, dtype=torch.float64)[:, None]
                a = a * torch.from_numpy(_freqs(case)).to(dev)
                s["table"] = torch.cat([a.cos(), a.sin()], 1).float().contiguous()
        else:
            s["cache"] = _random_cache(pages, case, gen, dev)
        s["k_out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
    else:
        lens, q = _lengths(case)
        B = case["B"]
        dblocks = -(-lens // PAGE)
        qblocks = -(-q // PAGE)
        nb = dblocks.sum(1) + qblocks
        pages = int(nb.sum())
        ids = rng.permutation(pages)
        meta = np.zeros((B, max(1, int(nb.max()))), np.uint64)
        at = 0
        for b in range(B):
            segs = [(int(x), int(n)) for x, n in zip(lens[b], dblocks[b])] + [(PAGE * int(qblocks[b]), int(qblocks[b]))]
            j, delta = 0, 0
            for x, n in segs:
                pg = np.arange(n, dtype=np.uint64)
                nv = np.minimum(PAGE, x - PAGE * np.arange(n)).astype(np.uint64)
                w = nv | pg << np.uint64(5) | np.uint64(delta) << np.uint64(16)
                meta[b, j:j + n] = w | ids[at:at + n].astype(np.uint64) << np.uint64(40)
                j, at, delta = j + n, at + n, delta + x
        s["meta"] = torch.from_numpy(meta.view(np.int64)).to(dev)
        s["q_start"], s["doc_blocks"] = i32(lens.sum(1)), i32(dblocks.sum(1))
        s["seq_len"] = i32(lens.sum(1) + q)
        s["max_q"] = int(q.max())
        rows = B if case["op"] == "decode" else int(q.sum())
        s["cu_q"] = i32(np.concatenate([[0], np.cumsum(q)]))
        s["q"] = torch.randn((rows, case["Hq"], D), generator=gen, device=dev).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        if case["kind"] == "alibi":
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["Hq"] + 1, device=dev) / case["Hq"]).float()
        s["cache"] = _random_cache(pages, case, gen, dev)
    torch.cuda.synchronize()
    return s


# ------------------------------------------------------------------ the plain form
def _unpack(blocks, case):
    """Float32 keys and values [..., 16, D] (without the cache's factors) of blocks [..., 18 D]."""
    D, lead = case["D"], blocks.shape[:-1]
    dev = blocks.device
    mag = torch.tensor(LEVELS, device=dev)
    level = torch.cat([mag, -mag])
    byte = torch.arange(256, device=dev)
    two = torch.stack([level[byte & 15], level[byte >> 4]], 1)  # both values of a byte
    split = lambda c: two.index_select(0, c.reshape(-1).int())  # noqa: E731
    kb, ks, vb, vs = blocks.split([8 * D, D, 8 * D, D], -1)
    k = split(kb).view(*lead, 16, D // 16, 16)
    n = len(lead)
    at = list(range(n))
    ks = ks.reshape(*lead, 8, 4, 2, D // 64).permute(*at, n + 2, n, n + 1, n + 3).reshape(*lead, 16, D // 16)
    if D == 128:  # half, lane group, t, odd, values
        v = split(vb).view(*lead, 2, 8, 4, 2, D // 8).permute(*at, n, n + 2, n + 3, n + 1, n + 4)
    else:  # lane group, t, half, odd, values
        v = split(vb).view(*lead, 8, 4, 2, 2, D // 8).permute(*at, n + 2, n + 1, n + 3, n, n + 4)
    v = v.reshape(*lead, 16, D // 16, 16)
    vs = vs.reshape(*lead, D // 16, 4, 2, 2).permute(*at, n + 2, n + 1, n + 3, n).reshape(*lead, 16, D // 16)
    k = k * ks.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)
    v = v * vs.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return k.flatten(-2), v.flatten(-2)


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


def _plain_write(s):
    case = s["case"]
    k = s["k"].float()
    if "table" in s:
        cs = s["table"].index_select(0, s["local_pos"])[:, None, :]
        h = case["rotary_dim"] // 2
        k = _rotate(k, cs[..., :h], cs[..., h:], 2 * h, case["interleaved"]).to(torch.bfloat16).float()
    level = torch.tensor(LEVELS, device=k.device)
    level = torch.cat([level, -level])
    out = []
    for x, f in ((k, case["k_scale"]), (s["v"].float(), case["v_scale"])):
        code, scale = _quantise(x, f)
        y = level.index_select(0, code.reshape(-1).int()).view(*x.shape[:-1], -1, 16) * (scale.float() * f).unsqueeze(-1)
        out.append(y.flatten(-2).to(torch.bfloat16))
    return out


def _plain_read(s):
    case = s["case"]
    rows = s["slot"].long()
    k, v = _unpack(s["cache"].index_select(0, rows // PAGE), case)  # [T, H, 16, D]
    at = (rows % PAGE).view(-1, 1, 1, 1).expand(-1, k.shape[1], 1, k.shape[3])
    k, v = k.gather(2, at).squeeze(2), v.gather(2, at).squeeze(2)
    return [(k * case["k_scale"]).to(torch.bfloat16), (v * case["v_scale"]).to(torch.bfloat16)]


def _cos_sin(pos, case):
    a = pos.double().unsqueeze(-1) * torch.from_numpy(_freqs(case)).to(pos.device)
    return a.cos().float(), a.sin().float()


def _plain_attention(s):
    case = s["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    meta, dev = s["meta"], s["meta"].device
    MB = meta.shape[1]
    nv, pg, delta, page = meta & 31, (meta >> 5) & 2047, (meta >> 16) & 0xFFFFFF, (meta >> 40) & 0xFFFFFF
    k, v = _unpack(s["cache"][page], case)  # [B, MB, H, 16, D]
    t = torch.arange(PAGE, device=dev)
    p = (delta + PAGE * pg).unsqueeze(-1) + t  # [B, MB, 16]
    valid = (t < nv.unsqueeze(-1)).flatten(1)
    p = p.flatten(1)  # [B, N]
    if case["op"] == "decode":
        m = (s["seq_len"].long() - 1).view(B, 1)
        q = s["q"].float().view(B, 1, Hq, D)
    else:
        cu, n = s["cu_q"].long(), s["max_q"]
        i = torch.arange(n, device=dev)
        live = i < (cu[1:] - cu[:-1]).unsqueeze(1)  # [B, n]
        m = s["q_start"].long().view(B, 1) + i
        q = s["q"].float()[torch.where(live, cu[:-1].unsqueeze(1) + i, 0)]  # [B, n, Hq, D]
    if case["kind"] != "alibi":
        rd, il = case["rotary_dim"], case["interleaved"]
        c, sn = _cos_sin(delta, case)
        k = _rotate(k, c[:, :, None, None], sn[:, :, None, None], rd, il)
        c, sn = _cos_sin(m, case)
        q = _rotate(q, c[:, :, None], sn[:, :, None], rd, il)
    k = k.permute(0, 2, 1, 3, 4).reshape(B, Hkv, MB * PAGE, D)
    v = v.permute(0, 2, 1, 3, 4).reshape(B, Hkv, MB * PAGE, D)
    n = q.shape[1]
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * (_softmax_scale(case) * case["k_scale"])
    x = x.view(B, Hkv, G, n, -1)
    if case["kind"] == "alibi":
        x = x - s["slopes"].view(1, Hkv, G, 1, 1) * (m.unsqueeze(-1) - p.unsqueeze(1)).float()[:, None, None]
    see = valid.unsqueeze(1) & (p.unsqueeze(1) <= m.unsqueeze(-1))  # [B, n, N]
    x = torch.where(see[:, None, None], x, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    w = e / e.sum(-1, keepdim=True)
    o = torch.matmul(w.view(B, Hkv, G * n, -1), v) * case["v_scale"]
    o = o.view(B, Hkv, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(torch.bfloat16)
    return o[:, 0] if case["op"] == "decode" else o[live]


# ------------------------------------------------------------------ the library's calls
def _plan(s):
    """What a program keeps: the positional configuration and the workspace."""
    import position_agnostic_kv_gb300 as lk
    case = s["case"]
    D, Hkv = case["D"], case["Hkv"]
    cfg = lk.pos_cfg_from(case["kind"], D, rope_theta=case["theta"], yarn_factor=8.0, yarn_orig_ctx=8192,
                          alibi_slopes=s.get("slopes", s["cache"].new_zeros(1, dtype=torch.float32)),
                          cos_sin=s.get("table"), rotary_dim=case["rotary_dim"], interleaved=case["interleaved"])
    ws = None
    if case["op"] in ("decode", "prefill"):
        phase = lk.PHASE_DECODE_Q4 if case["op"] == "decode" else lk.PHASE_PREFILL_Q4
        n = lk.workspace_size(phase, s["q"].shape[0], case["B"], s["meta"].shape[1], case["Hq"], Hkv, D)
        ws = torch.empty(n, dtype=torch.uint8, device=s["q"].device) if n else None
    s["plan"] = (lk, cfg, ws)
    return s["plan"]


def _own(s):
    lk, cfg, ws = s.get("plan") or _plan(s)
    case = s["case"]
    f = dict(k_scale=case["k_scale"], v_scale=case["v_scale"])
    if case["op"] in ("write", "read"):
        if case["op"] == "write":
            lk.kv_write_q4(s["k"], s["v"], s["slot"], s["local_pos"], s["cache"], cfg, **f)
        lk.kv_read_q4(s["slot"], s["cache"], s["k_out"], s["v_out"], **f)
        return [s["k_out"], s["v_out"]]
    if case["op"] == "decode":
        lk.attn_decode_q4(s["q"], s["seq_len"], s["q_start"], s["doc_blocks"], s["meta"], s["cache"], cfg, s["out"],
                          ws=ws, **f)
    else:
        lk.attn_prefill_q4(s["q"], s["cu_q"], s["q_start"], s["doc_blocks"], s["meta"], s["cache"], cfg, s["out"],
                           s["max_q"], ws=ws, **f)
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "write":
        return _plain_write(state)
    if op == "read":
        return _plain_read(state)
    return _plain_attention(state)


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3(b):
    """float64 values of e4m3 bytes."""
    b = b.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where(b >= 128, -x, x)


def _values(blocks, D, which):
    """float64 values [..., 16, D] of the keys (0) or values (1) in blocks, offset by offset."""
    r = np.arange(16)[:, None]
    d = np.arange(D)[None, :]
    if which == 0:
        code = r * (D // 2) + d // 2
        scale = 8 * D + ((r % 8) * 4 + d // (D // 4)) * (D // 32) + r // 8 * (D // 64) + d % (D // 4) // 16
    else:
        code = (9 * D + r // 8 * (512 if D == 128 else 8) + (d // (D // 8) * 4 + r % 8 // 2) * 16 + r % 2 * (D // 16)
                + d % (D // 8) // 2)
        scale = 17 * D + d // 16 * 16 + r % 8 // 2 * 4 + r // 8 * 2 + r % 2 + 0 * d
    dev = blocks.device
    code, scale = torch.from_numpy(code).to(dev), torch.from_numpy(scale).to(dev)
    c = blocks[..., code].int() >> torch.from_numpy(4 * (d % 2)).to(dev).int()
    n = c & 7
    # e2m1: two exponent bits (bias 1), one fraction bit
    x = torch.where(n < 2, n / 2, (1 + (n & 1) / 2) * torch.exp2((n >> 1) - 1.0)).double()
    return torch.where((c & 8) != 0, -x, x) * _e4m3(blocks[..., scale])


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


def _exact_write(s, case):
    res = []
    for n, f in (("k", case["k_scale"]), ("v", case["v_scale"])):
        x = s[n].double()
        if n == "k" and case["kind"] != "alibi":
            x = _turn64(x, s["local_pos"].view(-1, 1).expand(-1, x.shape[1]), case).to(torch.bfloat16).double()
        y = x.unflatten(-1, (-1, 16)) / f
        a = (y.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0)
        # nearest e4m3: steps of 2^(e-3), no finer than 2^-9, ties to even
        step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
        sc = torch.round(a / step) * step
        m = y.abs() / torch.where(sc > 0, sc, 1.0)
        # nearest e2m1: steps of 0.5 below 2, 1 below 4, 2 above, ties to even, at most 6
        st = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
        lev = (torch.round(m / st) * st).clamp(max=6.0)
        z = torch.where(sc > 0, torch.sign(y) * lev * sc * f, 0.0)
        res.append(z.flatten(-2))
    return res


def _exact_attention(s, case):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    lens, q = _lengths(case)
    words = s["meta"].cpu().numpy().view(np.uint64)
    outs = []
    for b in range(B):
        nblk = int((-(-lens[b] // PAGE)).sum() + -(-q[b] // PAGE))
        w = words[b, :nblk]
        start = (w >> np.uint64(16) & np.uint64(0xFFFFFF)).astype(np.int64)
        first = start + PAGE * (w >> np.uint64(5) & np.uint64(2047)).astype(np.int64)
        rows = (w & np.uint64(31)).astype(np.int64)
        rows[int((-(-lens[b] // PAGE)).sum()):] = np.minimum(PAGE, lens[b].sum() + q[b] - first[int((-(-lens[b] // PAGE)).sum()):])
        keep = torch.from_numpy(np.flatnonzero((np.arange(PAGE) < rows[:, None]).reshape(-1))).to(s["q"].device)
        p = torch.from_numpy((first[:, None] + np.arange(PAGE)).reshape(-1)).to(keep.device)[keep]
        off = torch.from_numpy(np.repeat(start, PAGE)).to(keep.device)[keep]
        blocks = s["cache"][torch.from_numpy((w >> np.uint64(40)).astype(np.int64)).to(keep.device)]
        k, v = (_values(blocks, D, i).transpose(1, 2).reshape(-1, Hkv, D)[keep].transpose(0, 1) for i in (0, 1))
        if case["kind"] != "alibi":
            k = _turn64(k, off.expand(Hkv, -1), case)
        if case["op"] == "decode":
            qr, m = s["q"][b:b + 1].double(), torch.tensor([int(lens[b].sum() + q[b]) - 1], device=keep.device)
        else:
            at = int(q[:b].sum())
            qr = s["q"][at:at + int(q[b])].double()
            m = int(lens[b].sum()) + torch.arange(int(q[b]), device=keep.device)
        if case["kind"] != "alibi":
            qr = _turn64(qr, m.view(-1, 1).expand(-1, Hq), case)
        res = torch.empty_like(qr)
        for h in range(Hkv):
            z = torch.einsum("ngd,td->ngt", qr[:, h * G:(h + 1) * G], k[h]) * (_softmax_scale(case) * case["k_scale"])
            if case["kind"] == "alibi":
                z = z - s["slopes"][h * G:(h + 1) * G].double()[:, None] * (m.view(-1, 1, 1) - p)
            z = z.masked_fill((p > m.view(-1, 1)).unsqueeze(1), -math.inf)
            res[:, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", torch.softmax(z, -1), v[h]) * case["v_scale"]
        outs.append(res)
    return torch.cat(outs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(s, case)
    if case["op"] == "read":
        step, k, v = 8192, [], []
        for i in range(0, case["T"], step):
            rows = s["slot"][i:i + step].long()
            blocks = s["cache"][rows // PAGE]
            for which, f, to in ((0, case["k_scale"], k), (1, case["v_scale"], v)):
                x = _values(blocks, case["D"], which)
                to.append((x[torch.arange(len(rows), device=rows.device), :, rows % PAGE] * f).to(torch.bfloat16))
        return [torch.cat(k).double(), torch.cat(v).double()]  # 4-bit values times scales are bf16 values
    return _exact_attention(s, case)
