// Writing tokens into the 4-bit paged cache, and reading them back.
//
// A stored key is what the bf16 cache would hold, bf16_RNE(R_j k), quantised; a stored value is
// the bf16 input quantised.  Per row, every 16 consecutive dimensions y_0 .. y_15 form a group:
//   s = e4m3_RNE(min(max |y_i| / (6 f), 448)),   code_i = e2m1_RNE((y_i / f) / s)
// with f the cache's power-of-two factor (an exact division), e2m1 saturating at +-6 and every
// code 0 where s rounds to 0.  A group with an infinity or a NaN gets the scale NaN, so all of it
// reads back as NaN.  Read back, a value is code * s * f: at most 6 significant bits, exact in bf16.
#include "q4.cuh"

namespace lazykv {

// Codes (8 bytes, low half of a byte = even dimension) and e4m3 scale of 16 values.
__device__ __forceinline__ void quantise16(const float (&y)[16], float inv_factor, uint2& codes, uint32_t& scale) {
  uint32_t top = 0;  // |y| ordered as integers: infinities and NaN compare above every number
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(y[e]) & 0x7FFFFFFFu);
  codes = make_uint2(0, 0);
  if (top >= 0x7F800000u) {
    scale = 0x7Fu;
    return;
  }
  const float a = __fdiv_rn(__uint_as_float(top) * inv_factor, 6.0f);
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.0f), "f"(a));
  scale = s2 & 0xFFu;
  if (scale == 0) return;
  const float s = e4m3_to_f(scale);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    // correctly rounded quotients: a value half way between two codes stays half way
    const float lo = __fdiv_rn(y[e] * inv_factor, s), hi = __fdiv_rn(y[e + 1] * inv_factor, s);
    uint32_t b;
    asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n cvt.u32.u8 %0, t;\n}\n" : "=r"(b) : "f"(lo), "f"(hi));
    w[e >> 3] |= b << (4 * (e & 7));
  }
  codes = make_uint2(w[0], w[1]);
}

// One thread per (token, head, group).
template <int D, bool ROTATE>
__global__ void __launch_bounds__(256) kv_write_q4_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                                                          const int32_t* __restrict__ slot,
                                                          const int32_t* __restrict__ local_pos, int T, int Hkv,
                                                          uint8_t* __restrict__ cache, int num_pages, float k_inv,
                                                          float v_inv, PosParams pos, uint32_t* status) {
  using Q = Q4<D>;
  pdl_wait();
  pdl_trigger();
  const long long gid = blockIdx.x * (long long)blockDim.x + threadIdx.x;
  const long long row = gid / Q::GROUPS;  // (token, head)
  const int q = int(gid % Q::GROUPS);
  if (row >= (long long)T * Hkv) return;
  const int t = int(row / Hkv), h = int(row % Hkv);
  const int sl = slot[t];
  if (sl < 0 || sl >= num_pages * kPage) {
    if (q == 0) set_status(status, LAZY_STATUS_BAD_SLOT);
    return;
  }
  const int r = sl % kPage;
  uint8_t* blk = cache + ((size_t)(sl / kPage) * Hkv + h) * Q::BYTES;
  auto load8 = [](const uint4* p, float* x) {
    const uint4 u = *p;
    x[0] = bf_lo(u.x); x[1] = bf_hi(u.x); x[2] = bf_lo(u.y); x[3] = bf_hi(u.y);
    x[4] = bf_lo(u.z); x[5] = bf_hi(u.z); x[6] = bf_lo(u.w); x[7] = bf_hi(u.w);
  };
  const uint4* krow = k + row * (D / 8);
  const uint4* vrow = v + row * (D / 8);
  float y[16];
  if constexpr (ROTATE) {
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
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int ch = 2 * q + half, d0 = 8 * ch;  // this chunk of 8 dimensions
      float x[8];
      load8(krow + ch, x);
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
          load8(krow + (first ? ch + hr / 8 : ch - hr / 8), p);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float s, c;
            cs(first ? d0 + e : d0 + e - hr, s, c);
            x[e] = first ? __fsub_rn(__fmul_rn(x[e], c), __fmul_rn(p[e], s))
                         : __fadd_rn(__fmul_rn(p[e], s), __fmul_rn(x[e], c));
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) y[8 * half + e] = __bfloat162float(__float2bfloat16_rn(x[e]));
    }
  } else {
    load8(krow + 2 * q, y);
    load8(krow + 2 * q + 1, y + 8);
  }
  uint2 c;
  uint32_t s;
  quantise16(y, k_inv, c, s);
  *reinterpret_cast<uint2*>(blk + Q::k_code(r, q)) = c;
  blk[Q::k_scale(r, q)] = uint8_t(s);
  load8(vrow + 2 * q, y);
  load8(vrow + 2 * q + 1, y + 8);
  quantise16(y, v_inv, c, s);
  if constexpr (D == 128) {
    *reinterpret_cast<uint2*>(blk + Q::v_code(r, 16 * q)) = c;
  } else {
    *reinterpret_cast<uint32_t*>(blk + Q::v_code(r, 16 * q)) = c.x;
    *reinterpret_cast<uint32_t*>(blk + Q::v_code(r, 16 * q + 8)) = c.y;
  }
  blk[Q::v_scale(r, q)] = uint8_t(s);
}

// 16 values of a group (codes, scale, factor) as bf16.
__device__ __forceinline__ void dequantise16(uint2 codes, uint32_t scale, float factor, uint4 (&out)[2]) {
  const float s = e4m3_to_f(scale) * factor;
  uint32_t h[8];
  e2m1x8_to_h2(codes.x, *reinterpret_cast<uint32_t(*)[4]>(h));
  e2m1x8_to_h2(codes.y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = h2_to_f2(h[i]);
    o[i] = f2_to_bf2(x.x * s, x.y * s);
  }
  out[0] = make_uint4(o[0], o[1], o[2], o[3]);
  out[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int D>
__global__ void __launch_bounds__(256) kv_read_q4_kernel(const int32_t* __restrict__ slot, int T, int Hkv,
                                                         const uint8_t* __restrict__ cache, int num_pages,
                                                         float k_factor, float v_factor, uint4* __restrict__ k,
                                                         uint4* __restrict__ v, uint32_t* status) {
  using Q = Q4<D>;
  pdl_wait();
  pdl_trigger();
  const long long gid = blockIdx.x * (long long)blockDim.x + threadIdx.x;
  const long long row = gid / Q::GROUPS;
  const int q = int(gid % Q::GROUPS);
  if (row >= (long long)T * Hkv) return;
  const int t = int(row / Hkv), h = int(row % Hkv);
  const int sl = slot[t];
  if (sl < 0 || sl >= num_pages * kPage) {
    if (q == 0) set_status(status, LAZY_STATUS_BAD_SLOT);
    return;
  }
  const int r = sl % kPage;
  const uint8_t* blk = cache + ((size_t)(sl / kPage) * Hkv + h) * Q::BYTES;
  uint4 o[2];
  dequantise16(*reinterpret_cast<const uint2*>(blk + Q::k_code(r, q)), blk[Q::k_scale(r, q)], k_factor, o);
  uint4* kd = k + row * (D / 8) + 2 * q;
  kd[0] = o[0];
  kd[1] = o[1];
  uint2 c;
  if constexpr (D == 128) {
    c = *reinterpret_cast<const uint2*>(blk + Q::v_code(r, 16 * q));
  } else {
    c.x = *reinterpret_cast<const uint32_t*>(blk + Q::v_code(r, 16 * q));
    c.y = *reinterpret_cast<const uint32_t*>(blk + Q::v_code(r, 16 * q + 8));
  }
  dequantise16(c, blk[Q::v_scale(r, q)], v_factor, o);
  uint4* vd = v + row * (D / 8) + 2 * q;
  vd[0] = o[0];
  vd[1] = o[1];
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
  if ((long long)T * Hkv * (D / 16) > (1ll << 31) * 128)
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
  if (rc) return rc;
  const bool rotate = pos.kind == kRope || pos.kind == kYarn;
  if (rotate && T > 0 && !local_pos) return fail(LAZY_EINVAL, "lazy_kv_write_q4: local_pos is NULL");
  rc = check_device();
  if (rc || T == 0) return rc;
  const long long n = (long long)T * Hkv * (D / 16);
  const int threads = 256;
  auto kern = D == 128 ? (rotate ? kv_write_q4_kernel<128, true> : kv_write_q4_kernel<128, false>)
                       : (rotate ? kv_write_q4_kernel<64, true> : kv_write_q4_kernel<64, false>);
  LAZY_CUDA_TRY(launch_pdl(kern, dim3(unsigned((n + threads - 1) / threads)), dim3(threads), 0,
                           static_cast<cudaStream_t>(stream), static_cast<const uint4*>(k),
                           static_cast<const uint4*>(v), slot, local_pos, T, Hkv, static_cast<uint8_t*>(kv_cache),
                           num_pages, 1.0f / kf, 1.0f / vf, pos, status_word()));
  return LAZY_OK;
}

extern "C" int lazy_kv_read_q4(const int32_t* slot, int T, int Hkv, int D, const void* kv_cache, int num_pages,
                               float k_scale, float v_scale, void* k, void* v, void* stream) {
  float kf, vf;
  int rc = check_cache_args("lazy_kv_read_q4", T, Hkv, D, num_pages, k, v, slot, kv_cache, k_scale, v_scale, &kf, &vf);
  if (rc) return rc;
  rc = check_device();
  if (rc || T == 0) return rc;
  const long long n = (long long)T * Hkv * (D / 16);
  const int threads = 256;
  auto kern = D == 128 ? kv_read_q4_kernel<128> : kv_read_q4_kernel<64>;
  LAZY_CUDA_TRY(launch_pdl(kern, dim3(unsigned((n + threads - 1) / threads)), dim3(threads), 0,
                           static_cast<cudaStream_t>(stream), slot, T, Hkv, static_cast<const uint8_t*>(kv_cache),
                           num_pages, kf, vf, static_cast<uint4*>(k), static_cast<uint4*>(v), status_word()));
  return LAZY_OK;
}
