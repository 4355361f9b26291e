// The 4-bit K/V cache block and its conversions (see lazykv.h, "4-bit caches", for the format).
//
// One block holds the 16 token rows of one page and KV head, keys and values together, in 18 D
// bytes (D = 128: 2304, D = 64: 1152; bf16 needs 8192 / 4096): K codes (8 D), K scales (D), V
// codes (8 D), V scales (D).  The order of the bytes follows the fragments of the 16x8x16 matrix
// instruction that the decode kernel feeds from registers (lane = 4 g + t):
//   K codes   row-major.  Lane (g, t) takes D/4 consecutive dimensions of rows g and g + 8, so
//             a page's keys are two fully coalesced warp-wide loads.
//   K scales  one word of D/32 bytes per lane: the scales of those dimensions, row g then g + 8.
//   V codes   lane (g, t) takes D/8 consecutive dimensions of rows 2t, 2t + 1, 2t + 8 and 2t + 9.
//             D = 128: [2 row halves][32 lanes][2 rows][8 bytes]; D = 64: [32 lanes][2][2][4].
//   V scales  one word per (group of 16 dimensions, t): rows 2t, 2t + 1, 2t + 8, 2t + 9.
#pragma once

#include "common.cuh"

namespace lazykv {

template <int D>
struct Q4 {
  static_assert(D == 64 || D == 128, "head dimensions of the 4-bit cache");
  static constexpr int BYTES = 18 * D;     // one block
  static constexpr int KS = 8 * D;         // K scales
  static constexpr int VC = 9 * D;         // V codes
  static constexpr int VS = 17 * D;        // V scales
  static constexpr int GROUPS = D / 16;    // groups of 16 dimensions in a row
  // byte offsets inside a block, for row r and group q (dimensions 16 q .. 16 q + 15)
  static __host__ __device__ constexpr int k_code(int r, int q) { return r * (D / 2) + q * 8; }
  static __host__ __device__ constexpr int k_scale(int r, int q) {
    constexpr int PER = D / 64;            // groups of a lane
    return KS + ((r & 7) * 4 + q / PER) * (2 * PER) + (r >> 3) * PER + q % PER;
  }
  // codes of dimensions d .. (8-byte runs of a group for D = 128, two 4-byte runs for D = 64)
  static __host__ __device__ constexpr int v_code(int r, int d) {
    constexpr int DL = D / 8;              // dimensions of a lane
    const int lane = (d / DL) * 4 + ((r & 7) >> 1);
    return VC + (r >> 3) * (D == 128 ? 512 : 8) + lane * 16 + (r & 1) * (DL / 2) + (d % DL) / 2;
  }
  static __host__ __device__ constexpr int v_scale(int r, int q) {
    return VS + q * 16 + ((r & 7) >> 1) * 4 + (r >> 3) * 2 + (r & 1);
  }
};

// The eight e2m1 codes of a word (low half of a byte first) as four f16 pairs; exact.
__device__ __forceinline__ void e2m1x8_to_h2(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Two e4m3 bytes (low byte first) as two f16; exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 a;\n cvt.u16.u32 a, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(r) : "r"(two));
  return r;
}

__device__ __forceinline__ float2 h2_to_f2(uint32_t h) {
  const __half2 x = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(x);
}

__device__ __forceinline__ float e4m3_to_f(uint32_t byte) { return h2_to_f2(e4m3x2_to_h2(byte & 0xFFu)).x; }

// Host side: the power-of-two factor of a cache (0 selects 1).
inline bool q4_factor(float f, float* out) {
  if (f == 0.0f) f = 1.0f;
  uint32_t u;
  static_assert(sizeof(u) == sizeof(f), "");
  __builtin_memcpy(&u, &f, 4);
  // a positive normal power of two between 2^-32 and 2^32
  if ((u >> 31) || (u & 0x7FFFFFu) || (u >> 23) < 127 - 32 || (u >> 23) > 127 + 32) return false;
  *out = f;
  return true;
}

// The kernels compare positions with max_pos as unsigned numbers: a negative one would cover every position.
inline int q4_check_table(const char* what, const PosParams& pos) {
  if (pos.max_pos >= 0) return LAZY_OK;
  return fail(LAZY_EINVAL, "%s: max_pos (%d) must not be negative", what, pos.max_pos);
}

}  // namespace lazykv
