"""The 4-bit cache restated in numpy (test infrastructure): block offsets, quantiser, reader.

Shares nothing with the library: offsets are written out from the format's description, the
quantiser rounds in float64 on exact quotients, and the reader returns bf16 bit patterns (a code
times an e4m3 scale times a power of two has at most 6 significant bits), which the attention
oracle takes as they are.
"""
from __future__ import annotations

import numpy as np

from oracle import lazy_oracle as lo

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_table():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    x = np.where(e == 0, m / 512.0, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    x = np.where((b & 127) == 127, np.nan, x)
    return np.where(b >= 128, -x, x)


E4M3 = _e4m3_table()


def offsets(D):
    """Byte offsets [16, D] of the K codes, K scales, V codes and V scales in a block."""
    kc, ks, vc, vs = (np.zeros((16, D), int) for _ in range(4))
    for r in range(16):
        for d in range(D):
            kc[r, d] = r * (D // 2) + d // 2
            ks[r, d] = 8 * D + ((r % 8) * 4 + d // (D // 4)) * (D // 32) + (r // 8) * (D // 64) + (d % (D // 4)) // 16
            a = 512 if D == 128 else 8
            vc[r, d] = (9 * D + (r // 8) * a + ((d // (D // 8)) * 4 + (r % 8) // 2) * 16 + (r % 2) * (D // 16)
                        + (d % (D // 8)) // 2)
            vs[r, d] = 17 * D + (d // 16) * 16 + ((r % 8) // 2) * 4 + (r // 8) * 2 + r % 2
    return kc, ks, vc, vs


def quantise(y, factor=1.0):
    """Codes [..., D] and e4m3 scale bytes [..., D/16] of float64 y, straight from the definition."""
    g = np.asarray(y, np.float64).reshape(*y.shape[:-1], -1, 16) / factor
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    a = np.minimum(np.abs(g).max(-1) / 6, 448.0)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    s = np.round(a / step) * step  # numpy rounds half to even
    m = np.abs(g) / np.where(s > 0, s, 1)[..., None]
    st = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    level = np.minimum(np.round(m / st) * st, 6.0)
    code = np.searchsorted(LEVELS, level).astype(np.uint8) | (np.signbit(g) * 8).astype(np.uint8)
    code = np.where(((s == 0) | bad)[..., None], 0, code).astype(np.uint8)
    sb = np.searchsorted(E4M3[:127], s).astype(np.uint8)  # the positive e4m3 values ascend
    sb = np.where(bad, 0x7F, sb).astype(np.uint8)
    return code.reshape(y.shape), sb


def store(cache, slots, k, v, kf=1.0, vf=1.0):
    """Write tokens' keys and values [T, H, D] (float64, as quantised) into cache blocks [P, H, 18 D]."""
    T, H, D = k.shape
    kc, ks, vc, vs = offsets(D)
    ck, sk = quantise(k, kf)
    cv, sv = quantise(v, vf)
    for t in range(T):
        p, r = divmod(int(slots[t]), 16)
        for code, scale, co, so in ((ck[t], sk[t], kc[r], ks[r]), (cv[t], sv[t], vc[r], vs[r])):
            cache[p][:, co[0::2]] = code[:, 0::2] | (code[:, 1::2] << 4)
            cache[p][:, so[::16]] = scale


def load(cache, D, kf=1.0, vf=1.0):
    """Keys and values held in blocks [P, H, 18 D] as bf16 bits [P, H, 16, D] (NaN scales: NaN)."""
    kc, ks, vc, vs = offsets(D)
    out = []
    for co, so, f in ((kc, ks, kf), (vc, vs, vf)):
        code = (cache[..., co] >> (4 * (np.arange(D) % 2)).astype(np.uint8)) & 15
        x = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0) * E4M3[cache[..., so]] * f
        bits = lo.f64_to_bf16_bits(np.nan_to_num(x, nan=0.0))
        out.append(np.where(np.isnan(x), np.uint16(0x7FC0), bits).astype(np.uint16))
    return out


def rotate_f32(k, local_pos, table, interleaved):
    """bf16_RNE of the fp32 rotation that the write documents, from a cos/sin table [P, rd] (fp32)."""
    x = np.asarray(k, np.float32)
    rd, h = table.shape[1], table.shape[1] // 2
    c, s = table[local_pos][:, None, :h], table[local_pos][:, None, h:]
    y = x.copy()
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if interleaved else (x[..., :h], x[..., h:rd])
    y1, y2 = a * c - b * s, a * s + b * c  # one rounding per operation
    if interleaved:
        y[..., 0:rd:2], y[..., 1:rd:2] = y1, y2
    else:
        y[..., :h], y[..., h:rd] = y1, y2
    from workloads import f32_to_bf16_bits
    return lo.bf16_bits_to_f64(f32_to_bf16_bits(y))
