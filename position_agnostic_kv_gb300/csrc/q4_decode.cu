// Attention of single query rows over the 4-bit cache: the decode step, and prefill rows.
//
// One CTA per (query row, KV head, up to 8 query heads of its group), tiles of 128 keys, one key
// per thread: the thread dequantises its key row, rotates it by its document's Delta and takes the
// dot products with the query heads (rotated by the absolute position m); an online softmax in
// base 2 over the tile; then one dimension per thread accumulates P V.
#include <cfloat>

#include "q4_attn.cuh"

namespace lazykv {

constexpr int kHeads = 8;  // query heads per CTA at most

template <int D>
__device__ __forceinline__ float q4_v_value(const uint8_t* blk, int r, int d) {
  using Q = Q4<D>;
  const uint32_t c = blk[Q::v_code(r, d)] >> (4 * (d & 1));
  return h2_to_f2(e2m1x2_to_h2(c & 15u)).x * e4m3_to_f(blk[Q::v_scale(r, d / 16)]);
}

template <int D, bool ROWS>
__global__ void __launch_bounds__(128) q4_rows_kernel(const Q4Args a, int heads, int ngrp) {
  using Q = Q4<D>;
  constexpr int NK = 128;          // keys per tile
  constexpr int KH = 128 / D;      // threads per dimension in the PV step
  __shared__ float qs[kHeads][D], ps[kHeads][NK], red[kHeads][4], mrun[kHeads], lrun[kHeads], alpha[kHeads];
  __shared__ float osum[KH > 1 ? kHeads : 1][D];
  __shared__ const uint8_t* vblk[NK / kPage];
  __shared__ int vrows[NK / kPage];
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = int(blockIdx.x % ngrp), g = int(blockIdx.x / ngrp) % a.Hkv, r = int(blockIdx.x / ngrp) / a.Hkv;
  const Q4Row w = q4_row<ROWS>(a, r);
  const int b = w.b, m = w.m;
  int nb = w.nb;
  if (nb > a.max_blocks) {
    if (tid == 0) set_status(a.status, LAZY_STATUS_BAD_ROW);
    nb = a.max_blocks;
  }
  const int h0 = g * (a.Hq / a.Hkv) + grp * heads;
  const bool rotary = a.pos.kind == kRope || a.pos.kind == kYarn;
  const int rd = rotary ? a.pos.rotary_dim : 0, hr = rd / 2;
  // queries, rotated by m
  for (int i = tid; i < heads * D; i += 128) {
    const int h = i / D, d = i % D;
    const __nv_bfloat16* qr = a.q + ((size_t)r * a.Hq + h0 + h) * D;
    float x = __bfloat162float(qr[d]);
    if (d < rd) {
      const int f = a.pos.interleaved ? d / 2 : d % hr;
      const bool first = a.pos.interleaved ? (d & 1) == 0 : d < hr;
      const float p = __bfloat162float(qr[a.pos.interleaved ? d ^ 1 : (first ? d + hr : d - hr)]);
      float s, c;
      turn_sincos(uint32_t(max(m, 0)), a.pos.turns[f], s, c);
      x = first ? x * c - p * s : p * s + x * c;
    }
    qs[h][d] = x * a.qk_log2;
  }
  if (tid < kHeads) {
    mrun[tid] = -INFINITY;
    lrun[tid] = 0.f;
  }
  float o[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) o[h] = 0.f;
  const uint64_t* mrow = a.meta + (size_t)b * a.max_blocks;
  for (int j0 = 0; j0 < nb; j0 += NK / kPage) {
    __syncthreads();
    const int jb = j0 + tid / kPage, t = tid % kPage;
    int rows = 0, start = 0;
    uint32_t delta = 0;
    const uint8_t* blk = nullptr;
    if (jb < nb) {
      const uint64_t mw = ldg_u64(mrow + jb);
      rows = q4_rows(mw, m);
      delta = word_delta(mw);
      start = int(delta + kPage * word_pg(mw));
      if (word_page(mw) >= uint32_t(a.num_pages)) {
        if (t == 0) set_status(a.status, LAZY_STATUS_BAD_PAGE);
        rows = 0;
      } else {
        blk = a.cache + ((size_t)word_page(mw) * a.Hkv + g) * Q::BYTES;
      }
    }
    if (t == 0) {
      vblk[tid / kPage] = blk;
      vrows[tid / kPage] = rows;
    }
    float s[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) s[h] = -INFINITY;
    if (t < rows) {
      float x[D];
#pragma unroll
      for (int q = 0; q < Q::GROUPS; ++q) {
        const uint2 c = *reinterpret_cast<const uint2*>(blk + Q::k_code(t, q));
        const float sc = e4m3_to_f(blk[Q::k_scale(t, q)]);
        uint32_t hh[8];
        e2m1x8_to_h2(c.x, *reinterpret_cast<uint32_t(*)[4]>(hh));
        e2m1x8_to_h2(c.y, *reinterpret_cast<uint32_t(*)[4]>(hh + 4));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = h2_to_f2(hh[e]);
          x[16 * q + 2 * e] = f.x * sc;
          x[16 * q + 2 * e + 1] = f.y * sc;
        }
      }
      for (int f = 0; f < hr; ++f) {
        const int d1 = a.pos.interleaved ? 2 * f : f, d2 = a.pos.interleaved ? 2 * f + 1 : f + hr;
        float sn, co;
        turn_sincos(delta, a.pos.turns[f], sn, co);
        const float x1 = x[d1], x2 = x[d2];
        x[d1] = x1 * co - x2 * sn;
        x[d2] = x1 * sn + x2 * co;
      }
      for (int h = 0; h < heads; ++h) {
        float acc = 0.f;
        for (int d = 0; d < D; ++d) acc = fmaf(qs[h][d], x[d], acc);
        if (a.pos.kind == kAlibi) acc -= a.pos.slopes[h0 + h] * 1.4426950408889634f * float(m - start - t);
        s[h] = acc;
      }
    }
    // tile maxima, then the weights
    for (int h = 0; h < heads; ++h) {
      float x = s[h];
      for (int off = 16; off; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
      // fmaxf drops a NaN score: carry it to the weights instead
      if (lane == 0) red[h][warp] = x;
    }
    __syncthreads();
    for (int h = 0; h < heads; ++h) {
      const float mx = fmaxf(fmaxf(red[h][0], red[h][1]), fmaxf(red[h][2], red[h][3]));
      const float mn = fmaxf(mrun[h], mx);
      ps[h][tid] = mn == -INFINITY ? (s[h] != s[h] ? s[h] : 0.f) : exp2f(s[h] - mn);
      if (tid == 0) alpha[h] = mn == -INFINITY ? 1.f : exp2f(mrun[h] - mn);
    }
    __syncthreads();
    if (tid < heads) {
      const float mx = fmaxf(fmaxf(red[tid][0], red[tid][1]), fmaxf(red[tid][2], red[tid][3]));
      mrun[tid] = fmaxf(mrun[tid], mx);
      float l = lrun[tid] * alpha[tid];
      for (int i = 0; i < NK; ++i) l += ps[tid][i];
      lrun[tid] = l;
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h < heads) o[h] *= alpha[h];
    const int d = tid % D, part = tid / D;
    for (int pg = part; pg < NK / kPage; pg += KH)
      for (int rr = 0; rr < vrows[pg]; ++rr) {
        const float v = q4_v_value<D>(vblk[pg], rr, d);
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
          if (h < heads) o[h] = fmaf(ps[h][pg * kPage + rr], v, o[h]);
      }
  }
  __syncthreads();
  pdl_trigger();
  if constexpr (KH > 1) {
    if (tid >= D)
      for (int h = 0; h < heads; ++h) osum[h][tid - D] = o[h];
    __syncthreads();
    if (tid >= D) return;
    for (int h = 0; h < heads; ++h) o[h] += osum[h][tid];
  }
  for (int h = 0; h < heads; ++h) {
    const float l = lrun[h];
    const float inv = l != 0.f ? a.v_factor / l : 0.f;
    const size_t row = (size_t)r * a.Hq + h0 + h;
    a.out[row * D + tid] = __float2bfloat16_rn(o[h] * inv);
    if (a.lse && tid == 0) a.lse[row] = (mrun[h] + log2f(l)) * 0.6931471805599453f;
  }
}

size_t q4_ws_bytes(int rows, int Hq, int Hkv, int D, int max_blocks, bool rows_mode) {
  (void)rows; (void)Hq; (void)Hkv; (void)D; (void)max_blocks; (void)rows_mode;
  return 0;
}

int run_q4_rows(Q4Args& a, int D, bool rows_mode, void* ws, size_t ws_bytes, cudaStream_t st) {
  (void)ws;
  (void)ws_bytes;
  const int G = a.Hq / a.Hkv, heads = G < kHeads ? G : kHeads, ngrp = G / heads;
  const long long ctas = (long long)a.rows * a.Hkv * ngrp;
  if (ctas > 0x7FFFFFFFll) return fail(LAZY_ERANGE, "too many query rows (%d rows, %d heads)", a.rows, a.Hq);
  auto kern = D == 128 ? (rows_mode ? q4_rows_kernel<128, true> : q4_rows_kernel<128, false>)
                       : (rows_mode ? q4_rows_kernel<64, true> : q4_rows_kernel<64, false>);
  LAZY_CUDA_TRY(launch_pdl(kern, dim3(unsigned(ctas)), dim3(128), 0, st, a, heads, ngrp));
  return LAZY_OK;
}

}  // namespace lazykv
