// Writing tokens into the 4-bit paged cache, and reading them back.
//
// A stored key is what the bf16 cache would hold, bf16_RNE(R_j k), quantised; a stored value is
// the bf16 input quantised.  Per row, every 16 consecutive dimensions y_0 .. y_15 form a group:
//   s = e4m3_RNE(min(max |y_i| / (6 f), 448)),   code_i = e2m1_RNE((y_i / f) / s)
// with f the cache's power-of-two factor (an exact division), e2m1 saturating at +-6 and every
// code 0 where s rounds to 0.  A group with an infinity or a NaN gets the scale NaN, so all of it
// reads back as NaN.  Read back, a value is code * s * f: at most 6 significant bits, exact in bf16.
#include <type_traits>

#include "q4.cuh"

namespace lazykv {

// Largest |y| of 8 bf16 numbers as an integer (infinities and NaN above every number).
__device__ __forceinline__ uint32_t top8(const uint4& y) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t t = __vmaxu2(__vmaxu2(y.x & m, y.y & m), __vmaxu2(y.z & m, y.w & m));
  return max(t & 0xFFFFu, t >> 16);
}

// e4m3 scale of a group whose largest |y| has the bf16 bits `top` (inv6 = 1 / (6 factor), rounded).  The product
// is off by at most 2^-22 of itself; max |y| has 8 bits and six times a point half way between two scales 7,
// so a quotient that is not half way is at least 2^-8 away from it, and rounding it to 12 bits (ties away)
// puts one that is exactly there.
__device__ __forceinline__ uint32_t group_scale(uint32_t top, float inv6) {
  const uint32_t a = (__float_as_uint(__uint_as_float(top << 16) * inv6) + 0x800u) & 0xFFFFF000u;
  uint16_t s;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s) : "f"(0.0f), "f"(__uint_as_float(a)));
  return top >= 0x7F80u ? 0x7Fu : s & 0xFFu;
}

// Codes of 8 bf16 numbers (a word, low half of a byte = even dimension).  A quotient by the scale (times the
// factor, a power of two) is a product with the approximate reciprocal, corrected once by its remainder
// (Markstein's correction), which one fused multiply-add gives exactly: so a value half way between two codes
// stays half way, and others stay on their side.  (Divisions cost ten instructions a value.)  With a
// factor below 2^-8 a quotient by the largest scale can exceed fp32: CUT cuts values at eight scales, more than
// any code.  Without a scale, or with a NaN one, every code is 0.
template <bool CUT>
__device__ __forceinline__ uint32_t codes8(const uint4& y, uint32_t scale, float factor) {
  const float s = e4m3_to_f(scale) * factor;
  const bool some = s > 0.0f;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(some ? s : 1.0f));
  const float2 r2 = make_float2(r, r), ns2 = make_float2(-s, -s);
  uint32_t w[4] = {y.x, y.y, y.z, y.w};
  if (CUT && scale == 0x7Eu) {
    const uint32_t lim = __float_as_uint(8.f * s) >> 16;  // a power of two times 3.5: exact in bf16
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __vminu2(w[i] & 0x7FFF7FFFu, lim * 0x10001u) | (w[i] & 0x80008000u);
  }
  float2 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = bf2_to_f2(w[i]);
    const float2 p = __fmul2_rn(x, r2);
    q[i] = __ffma2_rn(__ffma2_rn(p, ns2, x), r2, p);
  }
  uint32_t c;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(c)
      : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
  return some ? c : 0u;
}

// 8 bf16 values of a 16-byte chunk.
__device__ __forceinline__ void load8(const uint4& u, float* x) {
  x[0] = bf_lo(u.x); x[1] = bf_hi(u.x); x[2] = bf_lo(u.y); x[3] = bf_hi(u.y);
  x[4] = bf_lo(u.z); x[5] = bf_hi(u.z); x[6] = bf_lo(u.w); x[7] = bf_hi(u.w);
}

// The block of a slot's page and head 0, or null (and the status bit, from one thread) for a bad slot.
__device__ __forceinline__ uint8_t* page_of(uint8_t* cache, int sl, int num_pages, size_t page_bytes, bool report,
                                            uint32_t* status) {
  if (sl < 0 || sl >= num_pages * kPage) {
    if (report) set_status(status, LAZY_STATUS_BAD_SLOT);
    return nullptr;
  }
  return cache + (size_t)(sl / kPage) * page_bytes;
}

// Partial or interleaved rotations, or a cos/sin table off a 16-byte boundary: one thread per (token, head,
// group), which reads its partners' inputs too.
template <int D>
__global__ void __launch_bounds__(256) kv_write_q4_any_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                                                              const int32_t* __restrict__ slot,
                                                              const int32_t* __restrict__ local_pos, int T, int Hkv,
                                                              uint8_t* __restrict__ cache, int num_pages, float kf,
                                                              float vf, PosParams pos, uint32_t* status) {
  using Q = Q4<D>;
  pdl_wait();
  pdl_trigger();
  const long long gid = blockIdx.x * (long long)blockDim.x + threadIdx.x;
  const int q = int(gid % Q::GROUPS);
  const long long u = gid / Q::GROUPS;
  const int t = int(u % T), h = int(u / T);
  if (h >= Hkv) return;
  const int sl = slot[t], r = sl % kPage;
  uint8_t* blk = page_of(cache, sl, num_pages, (size_t)Hkv * Q::BYTES, q == 0 && h == 0, status);
  if (!blk) return;
  blk += (size_t)h * Q::BYTES;
  const uint4* krow = k + ((size_t)t * Hkv + h) * (D / 8);
  const uint4* vrow = v + ((size_t)t * Hkv + h) * (D / 8);
  const uint32_t j = uint32_t(local_pos[t]);
  const bool tab = pos.table != nullptr && j < uint32_t(pos.max_pos);
  const int rd = pos.rotary_dim, hr = rd / 2;
  auto cs = [&](int i, float& s, float& c) {
    if (tab) {
      c = pos.table[(size_t)j * rd + i];
      s = pos.table[(size_t)j * rd + hr + i];
    } else {
      turn_sincos(j, pos.turns[i], s, c);
    }
  };
  uint4 y[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int ch = 2 * q + half, d0 = 8 * ch;  // this chunk of 8 dimensions
    float x[8];
    load8(krow[ch], x);
    if (d0 < rd) {
      if (pos.interleaved) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float s, c;
          cs(d0 / 2 + w, s, c);
          const float a = x[2 * w], b = x[2 * w + 1];
          x[2 * w] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
          x[2 * w + 1] = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
        }
      } else {
        const bool first = d0 < hr;
        float p[8];
        load8(krow[first ? ch + hr / 8 : ch - hr / 8], p);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float s, c;
          cs(first ? d0 + e : d0 + e - hr, s, c);
          x[e] = first ? __fsub_rn(__fmul_rn(x[e], c), __fmul_rn(p[e], s))
                       : __fadd_rn(__fmul_rn(p[e], s), __fmul_rn(x[e], c));
        }
      }
    }
    y[half] = make_uint4(f2_to_bf2(x[0], x[1]), f2_to_bf2(x[2], x[3]), f2_to_bf2(x[4], x[5]), f2_to_bf2(x[6], x[7]));
  }
  const uint32_t ks = group_scale(max(top8(y[0]), top8(y[1])), 1.0f / (6.0f * kf));
  *reinterpret_cast<uint2*>(blk + Q::k_code(r, q)) = make_uint2(codes8<true>(y[0], ks, kf), codes8<true>(y[1], ks, kf));
  blk[Q::k_scale(r, q)] = uint8_t(ks);
  const uint4 a = vrow[2 * q], b = vrow[2 * q + 1];
  const uint32_t vs = group_scale(max(top8(a), top8(b)), 1.0f / (6.0f * vf));
  *reinterpret_cast<uint32_t*>(blk + Q::v_code(r, 16 * q)) = codes8<true>(a, vs, vf);
  *reinterpret_cast<uint32_t*>(blk + Q::v_code(r, 16 * q + 8)) = codes8<true>(b, vs, vf);
  blk[Q::v_scale(r, q)] = uint8_t(vs);
}

// Full half-split rotation, or none.  A thread takes chunk c (8 dimensions) and its partner chunk c + D/16 of
// one token for HEADS heads: it reads every input once, keeps its 8 cos/sin over the heads, and shares a
// group's maximum with the lane beside it.  Lanes run over the row's chunks, then over tokens, so loads take
// whole 128-byte lines and a warp's stores fill whole sectors of a block.
template <int D, bool ROTATE, int HEADS>
__global__ void __launch_bounds__(256, 4) kv_write_q4_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                                                          const int32_t* __restrict__ slot,
                                                          const int32_t* __restrict__ local_pos, int T, int Hkv,
                                                          uint8_t* __restrict__ cache, int num_pages, float kf,
                                                          float vf, PosParams pos, uint32_t* status) {
  using Q = Q4<D>;
  constexpr int NC = D / 16;  // chunk pairs of a row
  pdl_wait();
  pdl_trigger();
  const long long gid = blockIdx.x * (long long)blockDim.x + threadIdx.x;
  const int c = int(gid % NC);
  const long long u = gid / NC;
  const int t = int(u % T), h0 = int(u / T) * HEADS;
  // threads without a token, or with a bad slot, stay for the exchange between lanes and store nothing
  const bool live = h0 < Hkv;
  const int sl = live ? slot[t] : 0, r = sl % kPage;
  uint8_t* page = page_of(cache, sl, num_pages, (size_t)Hkv * Q::BYTES, live && c == 0 && h0 == 0, status);
  if (!live) page = nullptr;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 nk1 = zero, nk2 = zero, nv1 = zero, nv2 = zero;
  auto fetch = [&](int h) {  // the next head's inputs, loaded while this one is computed
    if (!page || h >= Hkv) return;
    const size_t at = ((size_t)t * Hkv + h) * (D / 8) + c;
    nk1 = k[at];
    nk2 = k[at + NC];
    nv1 = v[at];
    nv2 = v[at + NC];
  };
  fetch(h0);
  float2 co[4], sn[4];
  if constexpr (ROTATE) {
    const uint32_t j = live ? uint32_t(local_pos[t]) : 0u;
    if (pos.table != nullptr && j < uint32_t(pos.max_pos)) {
      const float4* row = reinterpret_cast<const float4*>(pos.table + (size_t)j * D + 8 * c);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 x = row[e], y = row[D / 8 + e];
        co[2 * e] = make_float2(x.x, x.y);
        co[2 * e + 1] = make_float2(x.z, x.w);
        sn[2 * e] = make_float2(y.x, y.y);
        sn[2 * e + 1] = make_float2(y.z, y.w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        turn_sincos(j, pos.turns[8 * c + 2 * e], sn[e].x, co[e].x);
        turn_sincos(j, pos.turns[8 * c + 2 * e + 1], sn[e].y, co[e].y);
      }
    }
  }
  const bool odd = c & 1;
  const float inv6 = 1.0f / (6.0f * (odd ? vf : kf));
#pragma unroll 1
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i;
    uint4 a = nk1, b = nk2;
    const uint4 va = nv1, vb = nv2;
    if (i + 1 < HEADS) fetch(h + 1);
    if constexpr (ROTATE) {
      uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
      uint32_t* pb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // each product and each sum rounded to fp32, then once to bf16
        const float2 x1 = bf2_to_f2(pa[e]), x2 = bf2_to_f2(pb[e]);
        const float2 u1 = __fmul2_rn(x1, co[e]), u2 = __fmul2_rn(x2, sn[e]);
        const float2 w1 = __fmul2_rn(x1, sn[e]), w2 = __fmul2_rn(x2, co[e]);
        pa[e] = f2_to_bf2(__fsub_rn(u1.x, u2.x), __fsub_rn(u1.y, u2.y));
        pb[e] = f2_to_bf2(__fadd_rn(w1.x, w2.x), __fadd_rn(w1.y, w2.y));
      }
    }
    // Maxima of this lane's four half groups, two to a word; of the lanes that share the groups the even
    // one takes the keys' maxima and computes their scales, the odd one the values'.
    const uint32_t tk = top8(a) | top8(b) << 16, tv = top8(va) | top8(vb) << 16;
    const uint32_t t2 = __vmaxu2(odd ? tv : tk, __shfl_xor_sync(0xffffffffu, odd ? tk : tv, 1));
    const uint32_t mine = group_scale(t2 & 0xFFFFu, inv6) | group_scale(t2 >> 16, inv6) << 8;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
    const uint32_t sk = odd ? other : mine, sv = odd ? mine : other;
    if (!page || h >= Hkv) continue;
    uint8_t* blk = page + (size_t)h * Q::BYTES;
    const int qa = c >> 1, qb = qa + NC / 2;  // the groups
    *reinterpret_cast<uint32_t*>(blk + Q::k_code(r, 0) + 4 * c) = codes8<HEADS == 1>(a, sk & 0xFFu, kf);
    *reinterpret_cast<uint32_t*>(blk + Q::k_code(r, 0) + 4 * (c + NC)) = codes8<HEADS == 1>(b, sk >> 8, kf);
    *reinterpret_cast<uint32_t*>(blk + Q::v_code(r, 8 * c)) = codes8<HEADS == 1>(va, sv & 0xFFu, vf);
    *reinterpret_cast<uint32_t*>(blk + Q::v_code(r, 8 * (c + NC))) = codes8<HEADS == 1>(vb, sv >> 8, vf);
    blk[odd ? Q::v_scale(r, qa) : Q::k_scale(r, qa)] = uint8_t(mine);
    blk[odd ? Q::v_scale(r, qb) : Q::k_scale(r, qb)] = uint8_t(mine >> 8);
  }
}

// 8 values (a word of codes, their scale, the factor) as bf16: exact.
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, uint32_t scale, float factor) {
  const float s = e4m3_to_f(scale) * factor;
  uint32_t h[4], o[4];
  e2m1x8_to_h2(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = h2_to_f2(h[i]);
    o[i] = f2_to_bf2(x.x * s, x.y * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// One thread per 8 dimensions of HEADS heads of a token: lanes run over the row, then over tokens, so a block
// of threads reads a page's block once and writes whole rows.
template <int D, int HEADS>
__global__ void __launch_bounds__(256) kv_read_q4_kernel(const int32_t* __restrict__ slot, int T, int Hkv,
                                                         const uint8_t* __restrict__ cache, int num_pages,
                                                         float k_factor, float v_factor, uint4* __restrict__ k,
                                                         uint4* __restrict__ v, uint32_t* status) {
  using Q = Q4<D>;
  pdl_wait();
  pdl_trigger();
  const long long gid = blockIdx.x * (long long)blockDim.x + threadIdx.x;
  const int c = int(gid % (D / 8));
  const long long u = gid / (D / 8);
  const int t = int(u % T), h0 = int(u / T) * HEADS;
  if (h0 >= Hkv) return;
  const int sl = slot[t], r = sl % kPage;
  const uint8_t* blk = page_of(const_cast<uint8_t*>(cache), sl, num_pages, (size_t)Hkv * Q::BYTES, c == 0 && h0 == 0,
                               status);
  if (!blk) return;
  blk += (size_t)h0 * Q::BYTES;
  uint32_t kc[HEADS], ks[HEADS], vc[HEADS], vs[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    if (h0 + i >= Hkv) break;
    const uint8_t* x = blk + (size_t)i * Q::BYTES;
    kc[i] = *reinterpret_cast<const uint32_t*>(x + Q::k_code(r, 0) + 4 * c);
    ks[i] = x[Q::k_scale(r, c / 2)];
    vc[i] = *reinterpret_cast<const uint32_t*>(x + Q::v_code(r, 8 * c));
    vs[i] = x[Q::v_scale(r, c / 2)];
  }
  const size_t at = ((size_t)t * Hkv + h0) * (D / 8) + c;
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    if (h0 + i >= Hkv) break;
    k[at + i * (D / 8)] = dequantise8(kc[i], ks[i], k_factor);
    v[at + i * (D / 8)] = dequantise8(vc[i], vs[i], v_factor);
  }
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// What both entry points refuse; nothing here needs a GPU.
static int check_cache_args(const char* what, int T, int Hkv, int D, int num_pages, const void* k, const void* v,
                            const int32_t* slot, const void* cache, float ks, float vs, float* kf, float* vf) {
  if (T < 0 || Hkv <= 0 || num_pages <= 0)
    return fail(LAZY_EINVAL, "%s: bad sizes (T=%d Hkv=%d num_pages=%d)", what, T, Hkv, num_pages);
  if (D != 64 && D != 128) return fail(LAZY_EINVAL, "%s: head_dim must be 64 or 128, got %d", what, D);
  if (num_pages > (1 << 24)) return fail(LAZY_ERANGE, "%s: num_pages above 2^24", what);
  if (!q4_factor(ks, kf) || !q4_factor(vs, vf))
    return fail(LAZY_EINVAL, "%s: k_scale and v_scale must be powers of two in [2^-32, 2^32] (or 0 for 1)", what);
  if (T == 0) return LAZY_OK;
  if (!k || !v || !slot || !cache) return fail(LAZY_EINVAL, "%s: NULL pointer", what);
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache))
    return fail(LAZY_EINVAL, "%s: tensors must be 16-byte aligned", what);
  if ((long long)T * Hkv * (D / 8) > (1ll << 31) * 128)
    return fail(LAZY_ERANGE, "%s: too many tokens in one call (T=%d Hkv=%d)", what, T, Hkv);
  return LAZY_OK;
}

}  // namespace lazykv

using namespace lazykv;

extern "C" int lazy_kv_write_q4(const void* k, const void* v, const int32_t* slot, const int32_t* local_pos, int T,
                                int Hkv, int D, void* kv_cache, int num_pages, const lazy_pos_cfg* cfg,
                                float k_scale, float v_scale, void* stream) {
  float kf, vf;
  int rc = check_cache_args("lazy_kv_write_q4", T, Hkv, D, num_pages, k, v, slot, kv_cache, k_scale, v_scale, &kf, &vf);
  if (rc) return rc;
  PosParams pos;
  rc = prepare_pos(cfg, 1, D, 0.f, &pos);
  if (!rc) rc = q4_check_table("lazy_kv_write_q4", pos);
  if (rc) return rc;
  const bool rotate = pos.kind == kRope || pos.kind == kYarn;
  if (rotate && T > 0 && !local_pos) return fail(LAZY_EINVAL, "lazy_kv_write_q4: local_pos is NULL");
  rc = check_device();
  if (rc || T == 0) return rc;
  // the full rotation's kernel reads the caller's cos/sin table 16 bytes at a time, the other one by floats (the
  // same arithmetic): a table that starts off a 16-byte boundary, inside a larger buffer, goes there
  const bool any = rotate && (pos.rotary_dim != D || pos.interleaved || !aligned16(pos.table));
  // Four heads per thread share its cos/sin and overlap loads with arithmetic, once single heads would fill
  // the GPU (4 CTAs of 256 per SM) twice.  Measured, 32 000 tokens of 8 heads: 39 us with a table and 41 without,
  // against 46 and 67 with one head per thread; below 4096 tokens both take their launch's time.
  // Only single heads cut values (codes8), which factors below 2^-8 need; four heads with it take 45 us.
  const long long rows = (long long)T * Hkv;
  const bool many = rows * (D / 16) >= (long long)sm_count() * 2048 && min(kf, vf) >= 0x1p-8f;
  const int threads = 256;
  const long long n = any ? rows * (D / 16) : (many ? (long long)T * ((Hkv + 3) / 4) : rows) * (D / 16);
  auto pick = [&](auto d) {
    constexpr int DD = decltype(d)::value;
    if (any) return kv_write_q4_any_kernel<DD>;
    if (rotate) return many ? kv_write_q4_kernel<DD, true, 4> : kv_write_q4_kernel<DD, true, 1>;
    return many ? kv_write_q4_kernel<DD, false, 4> : kv_write_q4_kernel<DD, false, 1>;
  };
  auto kern = D == 128 ? pick(std::integral_constant<int, 128>()) : pick(std::integral_constant<int, 64>());
  LAZY_CUDA_TRY(launch_pdl(kern, dim3(unsigned((n + threads - 1) / threads)), dim3(threads), 0,
                           static_cast<cudaStream_t>(stream), static_cast<const uint4*>(k),
                           static_cast<const uint4*>(v), slot, local_pos, T, Hkv, static_cast<uint8_t*>(kv_cache),
                           num_pages, kf, vf, pos, status_word()));
  return LAZY_OK;
}

extern "C" int lazy_kv_read_q4(const int32_t* slot, int T, int Hkv, int D, const void* kv_cache, int num_pages,
                               float k_scale, float v_scale, void* k, void* v, void* stream) {
  float kf, vf;
  int rc = check_cache_args("lazy_kv_read_q4", T, Hkv, D, num_pages, k, v, slot, kv_cache, k_scale, v_scale, &kf, &vf);
  if (rc) return rc;
  rc = check_device();
  if (rc || T == 0) return rc;
  // Two heads per thread keep more loads in flight once single heads would fill the GPU twice: 32 000 tokens of
  // 8 heads 28.6 us (5.9 TB/s) against 32.6.
  const bool many = (long long)T * Hkv * (D / 8) >= (long long)sm_count() * 2048 * 2;
  const long long n = (long long)T * (many ? (Hkv + 1) / 2 : Hkv) * (D / 8);
  const int threads = 256;
  auto kern = D == 128 ? (many ? kv_read_q4_kernel<128, 2> : kv_read_q4_kernel<128, 1>)
                       : (many ? kv_read_q4_kernel<64, 2> : kv_read_q4_kernel<64, 1>);
  LAZY_CUDA_TRY(launch_pdl(kern, dim3(unsigned((n + threads - 1) / threads)), dim3(threads), 0,
                           static_cast<cudaStream_t>(stream), slot, T, Hkv, static_cast<const uint8_t*>(kv_cache),
                           num_pages, kf, vf, static_cast<uint4*>(k), static_cast<uint4*>(v), status_word()));
  return LAZY_OK;
}
