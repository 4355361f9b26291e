// Attention of single query rows over the 4-bit cache: the decode step, and prefill rows of head
// groups that do not fit the tensor-core prefill.
//
// Mathematics.  For one KV head and the (up to 8) query heads that share it, per page of 16 keys:
//   S^T [16 keys x 8] = K [16 x D] (R_{m - Delta} q)^T,   O^T [D x 8] += V^T [D x 16] P^T [16 x 8]
// with an online softmax in base 2 between them.  Both products run on 16x8x16 f16 matrix
// instructions whose 16-row operand (K rows, V columns) is dequantised into registers: a tile of a
// decode step has up to 8 rows of queries here, so the 128-row tcgen05 tiles would be nearly empty, and their
// operands would cross shared memory once more (2 x 2 bytes per value against 0.56 loaded).
//  * The cache block is laid out in fragment order (q4.cuh), so a page is four 16-byte shared loads
//    per lane plus two scale words, all without bank conflicts.
//  * A code times its e4m3 scale is exact in f16.  q is normalised per head by a power of two and
//    split in two f16 (hi + lo), 22 bits of the row's largest value; without a cos/sin table the angles'
//    sine and cosine are good to about 2^-20 (turn_sincos_fast).  Groups of at most 4 heads put hi in columns 0-3
//    and lo in columns 4-7 of one instruction; groups of 8 use two instructions.
//  * With at most 4 heads the two pages of a step share one softmax: the hi and lo parts are added so that
//    lanes t < 2 hold the even page's scores and lanes t >= 2 the odd page's, and the columns 0-3 and 4-7 of
//    O^T accumulate even and odd pages (P's other columns are zeroed), merged in the epilogue.
//  * q is rotated by R_{m - Delta} only when a page's Delta differs from the one before: the warp
//    computes the D/2 angles together (two per lane), then each lane its fragment.
//  * P is f16 (2^-11 relative), held as 2^(s - max + 7): the lazy maximum (moved only when a score
//    beats it by more than 8) keeps it below 2^15, and small weights stay normal numbers longer.
//  * P^T comes out of the S^T fragment by one 8x8 transpose per 8 keys.
//
// What bounds it: HBM and instruction issue together.  At the measured HBM rate an SM gets one page-head
// (18 D bytes) per 99 cycles = 396 issue slots; a page costs about 300 warp instructions (D = 128, 4 heads),
// issued by 16 warps per SM at 0.6 per cycle and scheduler.  64 requests over 32 000 keys, 32 heads of 8 KV
// heads: 434 us, 5440 GB/s, 80 % of the copy rate (the loads alone take 327 us); 16 requests over 2000 keys:
// 21 us, most of it latency.  Measured and left out (first shape): 5 CTAs per SM at 96 registers 485 us
// (spills), one page per step 474, three stages 469 (a CTA per SM less), one bulk copy per block 444 (84
// cycles of issue each, lane by lane).
//
// Work: a CTA = (query row, KV head, head group, key split), 4 warps, each with its own run of pages
// and a ring of stages of two page blocks, filled by its lanes' asynchronous 16-byte copies.  Block words are
// unpacked 32 at a time, one per lane.  The warps' partial (O, max, sum) are merged in shared
// memory; up to 8 splits form a thread-block cluster and are merged through distributed shared memory,
// more of them (few long rows) through the workspace and a second kernel.
#include <cfloat>

#include "q4_attn.cuh"

namespace lazykv {

namespace {

constexpr float kTau = 8.0f;   // the running maximum moves when a score beats it by more (base 2)
constexpr float kPOff = 7.0f;  // weights are held times 2^7
constexpr int kWarps = 4;
constexpr int kStages = 2;
constexpr int kPair = 2;       // pages per stage
constexpr int kMaxCluster = 8; // key splits merged inside a cluster

template <int D, bool H8>
struct DecL {
  static constexpr int DL = D / 4;                    // dimensions of a lane's K fragment
  static constexpr int QROW = 4 * (DL + 4);           // padded: 4 t-chunks fall on different banks
  static constexpr int STAGE = kPair * Q4<D>::BYTES;
  static constexpr int QS = kWarps * kStages * STAGE;          // float [8][QROW]
  static constexpr int CS = QS + (H8 ? 8 : 4) * QROW * 4;      // float2 [warp][D/2]
  static constexpr int SC = CS + kWarps * (D / 2) * 8;         // float [8] score factor of each head
  static constexpr int SLOT = SC + 32;                         // int2 {Delta | rows << 24, first position} [warp][64]
  static constexpr int SRC = SLOT + kWarps * 64 * 8;           // block addresses [warp][64] (0: nothing to read)
  static constexpr int SMEM = SRC + kWarps * 64 * 8;
  // the stages are reused to merge: the warps' partials, then (clusters) this CTA's
  static constexpr int ML = kWarps * 8 * D * 4;
  static constexpr int CO = ML + kWarps * 8 * 8;
  static constexpr int CML = CO + 8 * D * 4;
  static_assert(CML + 64 <= QS, "the merge buffers reuse the stages");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank) {  // a float of CTA `rank`'s shared memory
  float v;
  asm volatile("{\n .reg .b32 x;\n mapa.shared::cluster.u32 x, %1, %2;\n ld.shared::cluster.f32 %0, [x];\n}\n"
               : "=f"(v)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}

// H8: eight heads (columns = heads, hi and lo by two instructions); else up to four.
template <int D, bool H8, int POS>
__global__ void __launch_bounds__(kWarps * 32, H8 ? 3 : 4) q4_decode_kernel(const Q4Args a, int heads, int ngrp) {
  using L = DecL<D, H8>;
  using Q = Q4<D>;
  constexpr int NKS = D / 16;   // k-steps of S, and m-tiles of O^T
  constexpr int NW_ = D / 32;   // words of a K row per lane
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int split = int(blockIdx.x) % a.S;
  int u = int(blockIdx.x) / a.S;
  const int grp = u % ngrp;
  u /= ngrp;
  const int kvh = u % a.Hkv, r = u / a.Hkv;
  const int h0 = kvh * (a.Hq / a.Hkv) + grp * heads;
  pdl_wait();
  if (!q4_in_request(a.cu_q, a.B, r)) return;  // the whole cluster: its CTAs share the row
  const Q4Row row = a.cu_q ? q4_row<true>(a, r) : q4_row<false>(a, r);
  const int m = row.m;
  int nb = row.nb;
  if (nb > a.max_blocks) {
    if (threadIdx.x == 0) set_status(a.status, LAZY_STATUS_BAD_ROW);
    nb = a.max_blocks;
  }
  const int chunk = (nb + a.S - 1) / a.S;
  const int beg = min(nb, split * chunk), len = min(nb, beg + chunk) - beg;
  const int wb = beg + warp * len / kWarps;
  const int n = beg + (warp + 1) * len / kWarps - wb;
  const int ns = (n + kPair - 1) / kPair;

  float* qs = reinterpret_cast<float*>(smem + L::QS);
  float* scs = reinterpret_cast<float*>(smem + L::SC);
  float2* cs = reinterpret_cast<float2*>(smem + L::CS) + warp * (D / 2);
  int2* slots = reinterpret_cast<int2*>(smem + L::SLOT) + warp * 64;
  unsigned long long* srcs = reinterpret_cast<unsigned long long*>(smem + L::SRC) + warp * 64;
  const uint32_t stage0 = smem_u32(smem + warp * kStages * L::STAGE);

  // Block words, 32 pages at a time, one per lane: the lane unpacks its word and publishes its page's slot
  // (what the compute needs of it) and address, in two batches.
  const uint64_t* mrow = a.meta + (size_t)row.b * a.max_blocks + wb;
  uint64_t mnxt = lane < n ? ldg_u64(mrow + lane) : 0;
  int mbase = -32;
  auto next_batch = [&]() {
    const uint64_t w = mnxt;
    mbase += 32;
    mnxt = mbase + 32 + lane < n ? ldg_u64(mrow + mbase + 32 + lane) : 0;
    int rows = 0;
    if (mbase + lane < n) {
      rows = q4_rows(w, m);
      if (word_page(w) >= uint32_t(a.num_pages)) {
        set_status(a.status, LAZY_STATUS_BAD_PAGE);
        rows = 0;
      }
    }
    const int x = (mbase + lane) & 63;
    slots[x] = make_int2(int(word_delta(w) | uint32_t(rows) << 24), int(word_delta(w) + kPage * word_pg(w)));
    srcs[x] = rows > 0 ? reinterpret_cast<unsigned long long>(a.cache + ((size_t)word_page(w) * a.Hkv + kvh) * Q::BYTES)
                       : 0ull;
    __syncwarp();
  };

  auto issue = [&](int i) {  // stage i: pages 2i and 2i + 1; a group for every stage, empty ones past the end
    if (i < ns) {
      if (kPair * i >= mbase + 32) next_batch();
      const ulonglong2 src = *reinterpret_cast<const ulonglong2*>(srcs + ((kPair * i) & 63));
      const uint32_t dst = stage0 + uint32_t((i % kStages) * L::STAGE + lane * 16);
#pragma unroll
      for (int pp = 0; pp < kPair; ++pp) {
        const unsigned long long x = pp ? src.y : src.x;
        if (x == 0) continue;
#pragma unroll
        for (int c = 0; c < Q::BYTES; c += 512)
          if (c + 512 <= Q::BYTES || lane * 16 < Q::BYTES - c)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + uint32_t(pp * Q::BYTES + c)),
                         "l"(x + lane * 16 + c)
                         : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kStages; ++i) issue(i);

  // ---- queries: one warp per head, normalised by a power of two, in fp32
  for (int h = warp; h < (H8 ? 8 : 4); h += kWarps) {
    float x[D / 32];
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      x[e] = h < heads ? __bfloat162float(a.q[((size_t)r * a.Hq + h0 + h) * D + e * 32 + lane]) : 0.f;
      top = fmaxf(top, fabsf(x[e]));  // a NaN does not raise it, and passes through
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const int ex = q4_exponent(top, a.lowest_ex);
    const float inv = __uint_as_float(uint32_t(127 - ex) << 23);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const int d = e * 32 + lane;
      qs[h * L::QROW + (d / L::DL) * (L::DL + 4) + d % L::DL] = x[e] * inv;
    }
    if (lane == 0) scs[h] = a.qk_log2 * __uint_as_float(uint32_t(127 + ex) << 23);
  }
  __syncthreads();

  // columns 2t and 2t + 1 of the score fragment: their heads, factors and slopes
  const int c0 = H8 ? 2 * t : (2 * t) & 3, c1 = c0 + 1;
  const float sc0 = scs[c0], sc1 = scs[c1];
  float sl0 = 0.f, sl1 = 0.f;
  if constexpr (POS == kAlibi) {
    if (a.pos.slopes) {
      sl0 = c0 < heads ? a.pos.slopes[h0 + c0] * 1.4426950408889634f : 0.f;
      sl1 = c1 < heads ? a.pos.slopes[h0 + c1] * 1.4426950408889634f : 0.f;
    }
  }

  // ---- this lane's query fragment: column gr, dimensions DL t .. DL t + DL - 1
  uint32_t qhi[NKS][2], qlo[H8 ? NKS : 1][2];
  const float* qh = qs + (H8 ? gr : (gr & 3)) * L::QROW;
  const bool low_half = !H8 && gr >= 4;  // this lane holds the lo parts
  auto put = [&](int e, float y0, float y1) {  // dimensions e, e + 1 of the lane's run
    const uint32_t hi = pack_h2(y0, y1);
    const float2 f = h2_to_f2(hi);
    const uint32_t lo = pack_h2(y0 - f.x, y1 - f.y);
    if constexpr (H8) {
      qhi[e / 4][(e / 2) & 1] = hi;
      qlo[e / 4][(e / 2) & 1] = lo;
    } else {
      qhi[e / 4][(e / 2) & 1] = low_half ? lo : hi;
    }
  };
  if constexpr (POS == kAlibi) {
#pragma unroll
    for (int e = 0; e < L::DL; e += 2) put(e, qh[t * (L::DL + 4) + e], qh[t * (L::DL + 4) + e + 1]);
  }
  auto rotate_q = [&](uint32_t delta) {
    const uint32_t dp = uint32_t(m) - delta;
    const int rd = POS == kRope ? D : a.pos.rotary_dim, hr = rd / 2;
    const bool tab = a.pos.table != nullptr && dp < uint32_t(a.pos.max_pos);
    __syncwarp();
    for (int f = lane; f < hr; f += 32) {
      float s, c;
      if (tab) {
        c = a.pos.table[(size_t)dp * rd + f];
        s = a.pos.table[(size_t)dp * rd + hr + f];
      } else {
        turn_sincos_fast(dp, a.pos.turns[f], s, c);
      }
      cs[f] = make_float2(c, s);
    }
    __syncwarp();
    if constexpr (POS == kRope) {
      const bool first = t < 2;  // this run lies in the first half; its partner two chunks on
      const float* x1 = qh + (t & 1) * (L::DL + 4);
      const float* x2 = x1 + 2 * (L::DL + 4);
      const float4* cp = reinterpret_cast<const float4*>(cs + (t & 1) * L::DL);
#pragma unroll
      for (int e = 0; e < L::DL; e += 2) {
        const float4 w = cp[e / 2];  // cos, sin of two frequencies
        const float2 p1 = *reinterpret_cast<const float2*>(x1 + e), p2 = *reinterpret_cast<const float2*>(x2 + e);
        put(e, first ? p1.x * w.x - p2.x * w.y : p1.x * w.y + p2.x * w.x,
            first ? p1.y * w.z - p2.y * w.w : p1.y * w.w + p2.y * w.z);
      }
    } else {
      const bool inter = a.pos.interleaved != 0;
#pragma unroll
      for (int e = 0; e < L::DL; e += 2) {
        const int d = t * L::DL + e;
        auto at = [&](int i) { return qh[(i / L::DL) * (L::DL + 4) + i % L::DL]; };
        float y0 = at(d), y1 = at(d + 1);
        if (d < rd) {
          if (inter) {
            const float2 w = cs[d / 2];
            const float x0 = y0, x1 = y1;
            y0 = x0 * w.x - x1 * w.y;
            y1 = x0 * w.y + x1 * w.x;
          } else {  // hr is a multiple of 8: both dimensions lie in the same half
            const bool first = d < hr;
            const int f = first ? d : d - hr, o = first ? d + hr : d - hr;
            const float2 w0 = cs[f], w1 = cs[f + 1];
            const float p0 = at(o), p1 = at(o + 1);
            y0 = first ? y0 * w0.x - p0 * w0.y : p0 * w0.y + y0 * w0.x;
            y1 = first ? y1 * w1.x - p1 * w1.y : p1 * w1.y + y1 * w1.x;
          }
        }
        put(e, y0, y1);
      }
    }
  };

  float o[NKS][4];
#pragma unroll
  for (int i = 0; i < NKS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float m0 = -FLT_MAX, m1 = -FLT_MAX, l0 = 0.f, l1 = 0.f;
  uint32_t cur_delta = 0xFFFFFFFFu;
  bool first = true;
  constexpr int NS = H8 ? kPair : 1;  // score sets of a lane: both pages', or its own page's
  const bool mine1 = !H8 && t >= 2;   // this lane's page is the odd one

  for (int i = 0; i < ns; ++i) {
    const int st = i % kStages;
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint8_t* blk0 = smem + warp * kStages * L::STAGE + st * L::STAGE;
    const int4 w = *reinterpret_cast<const int4*>(slots + ((kPair * i) & 63));  // both pages' slots
    const int delta0 = w.x & 0xFFFFFF, delta1 = w.z & 0xFFFFFF, rows0 = w.x >> 24;
    const int rows1 = kPair * i + 1 < n ? w.z >> 24 : 0;
    // Both pages in one straight run of instructions, absent ones masked like absent rows.  Where the
    // document changes between the two, they take a pass each.
    const bool split_pair = POS != kAlibi && rows0 > 0 && rows1 > 0 && delta0 != delta1;
#pragma unroll 1
    for (int pass = 0; pass <= int(split_pair); ++pass) {
      const int rows[kPair] = {split_pair && pass == 1 ? 0 : rows0, split_pair && pass == 0 ? 0 : rows1};
      if constexpr (POS != kAlibi) {
        const uint32_t delta = uint32_t(rows[0] > 0 ? delta0 : delta1);
        if (delta != cur_delta && rows[0] + rows[1] > 0) {
          cur_delta = delta;
          rotate_q(delta);
        }
      }
      // ---- S^T = K q^T
      float acc[kPair][4];
      uint32_t kw[kPair][2][NW_], ksc[kPair][2][NW_ / 2];
#pragma unroll
      for (int pp = 0; pp < kPair; ++pp) {
        const uint8_t* blk = blk0 + pp * Q::BYTES;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[pp][e] = 0.f;
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(blk + lane * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(blk + 512 + lane * 16);
          kw[pp][0][0] = x.x; kw[pp][0][1] = x.y; kw[pp][0][2] = x.z; kw[pp][0][3] = x.w;
          kw[pp][1][0] = y.x; kw[pp][1][1] = y.y; kw[pp][1][2] = y.z; kw[pp][1][3] = y.w;
          const uint32_t sw = *reinterpret_cast<const uint32_t*>(blk + Q::KS + lane * 4);
          const uint32_t sa = e4m3x2_to_h2(sw & 0xFFFFu), sb = e4m3x2_to_h2(sw >> 16);
          ksc[pp][0][0] = __byte_perm(sa, 0, 0x1010);
          ksc[pp][0][1] = __byte_perm(sa, 0, 0x3232);
          ksc[pp][1][0] = __byte_perm(sb, 0, 0x1010);
          ksc[pp][1][1] = __byte_perm(sb, 0, 0x3232);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(blk + lane * 8);
          const uint2 y = *reinterpret_cast<const uint2*>(blk + 256 + lane * 8);
          kw[pp][0][0] = x.x; kw[pp][0][1] = x.y;
          kw[pp][1][0] = y.x; kw[pp][1][1] = y.y;
          const uint32_t sa = e4m3x2_to_h2(*reinterpret_cast<const uint16_t*>(blk + Q::KS + lane * 2));
          ksc[pp][0][0] = __byte_perm(sa, 0, 0x1010);
          ksc[pp][1][0] = __byte_perm(sa, 0, 0x3232);
        }
      }
#pragma unroll
      for (int x = 0; x < NW_; ++x)
#pragma unroll
        for (int pp = 0; pp < kPair; ++pp) {
          uint32_t ra[4], rb[4];
          e2m1x8_to_h2(kw[pp][0][x], ra);
          e2m1x8_to_h2(kw[pp][1][x], rb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ra[e] = hmul2(ra[e], ksc[pp][0][x / 2]);
            rb[e] = hmul2(rb[e], ksc[pp][1][x / 2]);
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            mma16816(acc[pp], ra[2 * v], rb[2 * v], ra[2 * v + 1], rb[2 * v + 1], qhi[2 * x + v][0], qhi[2 * x + v][1]);
            if constexpr (H8)
              mma16816(acc[pp], ra[2 * v], rb[2 * v], ra[2 * v + 1], rb[2 * v + 1], qlo[2 * x + v][0],
                       qlo[2 * x + v][1]);
          }
        }
      // ---- scores: [set][row gr | gr + 8][column 2t | 2t + 1], still without the factor sc (ALiBi: logits)
      float s[NS][4];
      if constexpr (H8) {
#pragma unroll
        for (int pp = 0; pp < kPair; ++pp)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[pp][e] = acc[pp][e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)  // hi + lo: each lane gives away its part of the other page
          s[0][e] = (mine1 ? acc[1][e] : acc[0][e]) + __shfl_xor_sync(0xffffffffu, mine1 ? acc[0][e] : acc[1][e], 2);
      }
      if constexpr (POS == kAlibi) {
#pragma unroll
        for (int x = 0; x < NS; ++x) {
          const float dist = float(((H8 ? x == 1 : mine1) ? w.w : w.y) + gr - m);
          s[x][0] = fmaf(s[x][0], sc0, sl0 * dist);
          s[x][1] = fmaf(s[x][1], sc1, sl1 * dist);
          s[x][2] = fmaf(s[x][2], sc0, sl0 * (dist + 8.f));
          s[x][3] = fmaf(s[x][3], sc1, sl1 * (dist + 8.f));
        }
      }
      if (min(rows[0], rows[1]) < kPage) {
#pragma unroll
        for (int x = 0; x < NS; ++x) {
          const int rr = (H8 ? x == 1 : mine1) ? rows[1] : rows[0];
          if (gr >= rr) s[x][0] = s[x][1] = -INFINITY;
          if (gr + 8 >= rr) s[x][2] = s[x][3] = -INFINITY;
        }
      }
      // ---- lazy running maximum of each column
      float x0 = fmaxf(s[0][0], s[0][2]), x1 = fmaxf(s[0][1], s[0][3]);
      if constexpr (H8) {
        x0 = fmaxf(x0, fmaxf(s[NS - 1][0], s[NS - 1][2]));
        x1 = fmaxf(x1, fmaxf(s[NS - 1][1], s[NS - 1][3]));
      }
      if constexpr (POS != kAlibi) {
        x0 *= sc0;
        x1 *= sc1;
      }
      if (__any_sync(0xffffffffu, first || x0 > m0 + kTau || x1 > m1 + kTau)) {
        first = false;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
        }
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float a0 = exp2f(m0 - n0), a1 = exp2f(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int x = 0; x < NKS; ++x) {
          o[x][0] *= a0;
          o[x][1] *= a1;
          o[x][2] *= a0;
          o[x][3] *= a1;
        }
      }
      const float f0 = kPOff - m0, f1 = kPOff - m1;
      uint32_t pb[NS][2];  // P^T fragments: keys 0-7 and 8-15
#pragma unroll
      for (int x = 0; x < NS; ++x) {
        const float k0 = POS == kAlibi ? 1.f : sc0, k1 = POS == kAlibi ? 1.f : sc1;
        const float p0 = ex2_approx(fmaf(s[x][0], k0, f0)), p1 = ex2_approx(fmaf(s[x][1], k1, f1));
        const float p2 = ex2_approx(fmaf(s[x][2], k0, f0)), p3 = ex2_approx(fmaf(s[x][3], k1, f1));
        l0 += p0 + p2;
        l1 += p1 + p3;
        pb[x][0] = transpose8(pack_h2(p0, p1));
        pb[x][1] = transpose8(pack_h2(p2, p3));
      }
#pragma unroll
      for (int pp = 0; pp < kPair; ++pp) {
        // columns of the other page take no part in this page's product
        const bool use = H8 || (gr >= 4) == (pp == 1);
        const uint32_t b0 = use ? pb[H8 ? pp : 0][0] : 0u, b1 = use ? pb[H8 ? pp : 0][1] : 0u;
        // ---- O^T += V^T P^T
        const uint8_t* blk = blk0 + pp * Q::BYTES;
        const int vg = D == 128 ? lane : (gr >> 1) * 4 + t;
        uint32_t sw = *reinterpret_cast<const uint32_t*>(blk + Q::VS + vg * 4);
        if (rows[pp] < kPage) {  // rows without a key: scale 0, so that what they hold cannot matter
          const int rr = rows[pp] - 2 * t;  // bytes: rows 2t, 2t + 1, 2t + 8, 2t + 9
          const uint32_t keep = (rr > 0 ? 0xFFu : 0u) | (rr > 1 ? 0xFF00u : 0u) | (rr > 8 ? 0xFF0000u : 0u) |
                                (rr > 9 ? 0xFF000000u : 0u);
          sw &= keep;
        }
        const uint32_t vs0 = e4m3x2_to_h2(sw & 0xFFFFu), vs1 = e4m3x2_to_h2(sw >> 16);
        uint32_t va[2][D / 64], vb[2][D / 64];  // [row half][word]: codes of the even and the odd row
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(blk + Q::VC + lane * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(blk + Q::VC + 512 + lane * 16);
          va[0][0] = x.x; va[0][1] = x.y; vb[0][0] = x.z; vb[0][1] = x.w;
          va[1][0] = y.x; va[1][1] = y.y; vb[1][0] = y.z; vb[1][1] = y.w;
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(blk + Q::VC + lane * 16);
          va[0][0] = x.x; vb[0][0] = x.y; va[1][0] = x.z; vb[1][0] = x.w;
        }
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint32_t e0[4], o0[4], e1[4], o1[4];  // even and odd dimensions of the word, both row halves
          const uint32_t A0 = va[0][w], B0 = vb[0][w], A1 = va[1][w], B1 = vb[1][w];
          // two rows' codes of one dimension side by side in a byte
          e2m1x8_to_h2((A0 & 0x0F0F0F0Fu) | ((B0 << 4) & 0xF0F0F0F0u), e0);
          e2m1x8_to_h2(((A0 >> 4) & 0x0F0F0F0Fu) | (B0 & 0xF0F0F0F0u), o0);
          e2m1x8_to_h2((A1 & 0x0F0F0F0Fu) | ((B1 << 4) & 0xF0F0F0F0u), e1);
          e2m1x8_to_h2(((A1 >> 4) & 0x0F0F0F0Fu) | (B1 & 0xF0F0F0F0u), o1);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mma16816(o[4 * w + x], hmul2(e0[x], vs0), hmul2(o0[x], vs0), hmul2(e1[x], vs1), hmul2(o1[x], vs1), b0, b1);
        }
      }
    }
    __syncwarp();
    issue(i + kStages);
  }
  pdl_trigger();

  // ---- merge the warps: O^T fragments hold dimensions D/8 gr + 2x (+1), columns 2t, 2t + 1.  With at most
  // four heads the columns h and h + 4 are two partials of head h.
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, off);
    l1 += __shfl_xor_sync(0xffffffffu, l1, off);
  }
  __syncthreads();  // every stage is consumed
  float* mo = reinterpret_cast<float*>(smem);                  // [warp][column][D]
  float2* mml = reinterpret_cast<float2*>(smem + L::ML);       // [warp][column]
#pragma unroll
  for (int x = 0; x < NKS; ++x) {
    const int d = (D / 8) * gr + 2 * x;
    *reinterpret_cast<float2*>(mo + (warp * 8 + 2 * t) * D + d) = make_float2(o[x][0], o[x][2]);
    *reinterpret_cast<float2*>(mo + (warp * 8 + 2 * t + 1) * D + d) = make_float2(o[x][1], o[x][3]);
  }
  if (gr == 0) {
    mml[warp * 8 + 2 * t] = make_float2(l0 != 0.f ? m0 : -INFINITY, l0);
    mml[warp * 8 + 2 * t + 1] = make_float2(l1 != 0.f ? m1 : -INFINITY, l1);
  }
  __syncthreads();
  constexpr int PARTS = H8 ? kWarps : 2 * kWarps;
  float* co = reinterpret_cast<float*>(smem + L::CO);          // [head][D] (clusters)
  float2* cml = reinterpret_cast<float2*>(smem + L::CML);      // [head]
  for (int x = threadIdx.x; x < heads * D; x += kWarps * 32) {
    const int h = x / D, d = x % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < PARTS; ++w) M = fmaxf(M, mml[H8 ? w * 8 + h : w * 4 + h].x);
    float O = 0.f, l = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < PARTS; ++w) {
        const int col = H8 ? w * 8 + h : w * 4 + h;
        const float f = exp2f(mml[col].x - M);
        O += f * mo[col * D + d];
        l += f * mml[col].y;
      }
    }
    const size_t rh = (size_t)r * a.Hq + h0 + h;
    if (a.S == 1) {
      a.out[rh * D + d] = __float2bfloat16_rn(l != 0.f ? O * (a.v_factor / l) : 0.f);
      if (a.lse && d == 0) a.lse[rh] = (M + log2f(l) - kPOff) * 0.6931471805599453f;
    } else if (a.S <= kMaxCluster) {
      co[x] = O;
      if (d == 0) cml[h] = make_float2(M, l);
    } else {
      a.part_o[(rh * a.S + split) * D + d] = O * a.v_factor;
      if (d == 0) {
        a.part_ml[(rh * a.S + split) * 2] = M - kPOff;
        a.part_ml[(rh * a.S + split) * 2 + 1] = l;
      }
    }
  }
  if (a.S > 1 && a.S <= kMaxCluster) {
    // ---- merge the cluster: CTA `split` of it combines and writes its share of the elements
    cluster_sync();
    const int per = (heads * D + a.S - 1) / a.S;
    for (int x = split * per + threadIdx.x; x < min(heads * D, (split + 1) * per); x += kWarps * 32) {
      const int h = x / D, d = x % D;
      float M = -INFINITY;
      for (int c = 0; c < a.S; ++c) M = fmaxf(M, ld_cluster(smem_u32(&cml[h].x), c));
      float O = 0.f, l = 0.f;
      if (M != -INFINITY)
        for (int c = 0; c < a.S; ++c) {
          const float f = exp2f(ld_cluster(smem_u32(&cml[h].x), c) - M);
          O += f * ld_cluster(smem_u32(co + x), c);
          l += f * ld_cluster(smem_u32(&cml[h].y), c);
        }
      const size_t rh = (size_t)r * a.Hq + h0 + h;
      a.out[rh * D + d] = __float2bfloat16_rn(l != 0.f ? O * (a.v_factor / l) : 0.f);
      if (a.lse && d == 0) a.lse[rh] = (M + log2f(l) - kPOff) * 0.6931471805599453f;
    }
    cluster_sync();  // no CTA leaves while another still reads its partials
  }
}

// Merge the splits' partial (O, max, sum) of a (row, head) by their log-sum-exp: a warp each, its lanes over
// the splits' weights (at most 64) and then over the dimensions.
constexpr int kMergeWarps = 4;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    q4_merge_kernel(const float* __restrict__ po, const float* __restrict__ pml, int S, long long n,
                    __nv_bfloat16* __restrict__ out, float* __restrict__ lse, const int32_t* cu_q, int B, int Hq) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long rh = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  if (rh >= n || !q4_in_request(cu_q, B, int(rh / Hq))) return;
  const float2* ml = reinterpret_cast<const float2*>(pml) + rh * S;
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 x0 = lane < S ? ml[lane] : none, x1 = lane + 32 < S ? ml[lane + 32] : none;
  constexpr int V = D / 32;  // a lane's dimensions: V lane ..
  using Vec = std::conditional_t<V == 4, float4, float2>;
  const float* p = po + rh * S * D + V * lane;
  Vec ahead[4];  // the first partials, fetched beside the weights
#pragma unroll
  for (int s = 0; s < 4; ++s)
    if (s < S) ahead[s] = *reinterpret_cast<const Vec*>(p + s * D);
  float M = fmaxf(x0.x, x1.x);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float base = M == -INFINITY ? 0.f : M;  // no key at all: every weight is 2^-inf
  const float f0 = exp2f(x0.x - base), f1 = exp2f(x1.x - base);
  float l = f0 * x0.y + f1 * x1.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  float O[V] = {};
  auto add = [&](int s, const Vec& x) {
    const float f = __shfl_sync(0xffffffffu, s < 32 ? f0 : f1, s & 31);
    const float* e = reinterpret_cast<const float*>(&x);
#pragma unroll
    for (int d = 0; d < V; ++d) O[d] += f * e[d];
  };
#pragma unroll
  for (int s = 0; s < 4; ++s)
    if (s < S) add(s, ahead[s]);
#pragma unroll 4
  for (int s = 4; s < S; ++s) add(s, *reinterpret_cast<const Vec*>(p + s * D));
  const float inv = l != 0.f ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(out + rh * D + V * lane);
#pragma unroll
  for (int d = 0; d < V; d += 2) dst[d / 2] = f2_to_bf2(O[d] * inv, O[d + 1] * inv);
  if (lse && lane == 0) lse[rh] = (M + log2f(l)) * 0.6931471805599453f;
}

int q4_heads(int Hq, int Hkv) { return min(Hq / Hkv, 8); }

// Key splits of a unit (query row, KV head, head group): 1, 2, 4, 8 (one cluster) or 16, 32, 64 (workspace).
// The slowest SM carries k = ceil(units S / SMs) CTAs of p = ceil(blocks / S) pages, at most C at a time.  In
// units of the time that a page takes an SM at full rate (0.05 us; 0.07 us with 8 heads): k <= C CTAs take
// (2 k + C) / 3 per page of one, and 25 each to start and end; each further one 40; a cluster 20 (of two
// 40: they may land unevenly, 16 rows of ten documents took 21 us on one GPU and 25 on another), the merge through
// the workspace 50.  Measured, us, S = 1, 2, 4, 8 (chosen: *): 16 rows of 8 KV heads, 4 heads each, 400 keys 9.5*
// 11.0 12.0 12.0, 2000 keys 20.1 18.3 18.0* 25.3, 8000 keys 62 55 42* 49; 64 rows, 8000 keys 130 122* 131 157; 4
// rows, 8000 keys 60 35 21 17*; 16 rows, 8 heads each, 400 keys 10.5* 14.1 21.7 21.6.
struct Splits {
  int S;
  double cost;
};
Splits q4_splits(int rows, int Hq, int Hkv, int max_blocks) {
  const int heads = q4_heads(Hq, Hkv), C = heads == 8 ? 3 : 4;
  const long long units = (long long)rows * (Hq / heads), sms = sm_count();
  Splits best = {1, 0.0};
  for (int S = 1; S <= 64 && S <= max(1, max_blocks / kWarps); S *= 2) {
    const double k = double((units * S + sms - 1) / sms), p = (max_blocks + S - 1) / S, c = min(k, double(C));
    const double cost = (k > C ? p * k : p * (2 * k + C) / 3) + 25 * c + 40 * (k - c) + (S == 2 ? 40 : S > 1 ? 20 : 0) +
                        (S > kMaxCluster ? 50 : 0);
    if (S == 1 || cost < 0.99 * best.cost) best = {S, cost};
  }
  return best;
}

// Decode of wide head groups may run on the tensor-core kernel instead, the group's heads as the rows of one
// tile: the matrix instructions here take 8 heads at a time and dequantise every page once for each 8.  In the
// units above (8 heads) a CTA there takes 45 to start and end, 14 per tile of 128 keys, 35 more for the merge
// of key splits.  Measured, 64 rows of 16 heads of one KV head: 400 keys 10.5 us here, 12.0 there; 1600 keys 18
// and 16; 32 rows of 32 heads, 12 000 keys 74 and 34; one row of 16 heads, 1600 keys 8.9 and 11.9.
bool q4_decode_on_tc(int rows, int Hq, int Hkv, int max_blocks) {
  if (Hq / Hkv < 16 || !q4_use_tc(Hq, Hkv)) return false;
  const int S = q4_tc_splits(rows, Hkv, max_blocks), tiles = (max_blocks + 7) / 8;
  const long long waves = ((long long)rows * Hkv * S + sm_count() - 1) / sm_count();
  const double cost = double(waves) * (45 + 14 * ((tiles + S - 1) / S)) + (S > 1 ? 35 : 0);
  return cost < q4_splits(rows, Hq, Hkv, max_blocks).cost;
}

template <int D, bool H8, int POS>
int launch_q4(const Q4Args& a, int heads, unsigned grid, cudaStream_t st) {
  auto kern = q4_decode_kernel<D, H8, POS>;
  static std::atomic<uint64_t> done{0};
  LAZY_CUDA_TRY(q4_smem_limit(kern, DecL<D, H8>::SMEM, done));
  const int ngrp = a.Hq / a.Hkv / heads;
  if (a.S > 1 && a.S <= kMaxCluster)
    LAZY_CUDA_TRY(launch_pdl_cluster(kern, dim3(grid), dim3(kWarps * 32), DecL<D, H8>::SMEM, st, unsigned(a.S), a,
                                     heads, ngrp));
  else
    LAZY_CUDA_TRY(launch_pdl(kern, dim3(grid), dim3(kWarps * 32), DecL<D, H8>::SMEM, st, a, heads, ngrp));
  return LAZY_OK;
}

template <int D, bool H8>
int launch_q4_pos(const Q4Args& a, int heads, unsigned grid, cudaStream_t st) {
  if (a.pos.kind == kAlibi || a.pos.kind == kNone) return launch_q4<D, H8, kAlibi>(a, heads, grid, st);
  if (a.pos.rotary_dim != D || a.pos.interleaved) return launch_q4<D, H8, kRopeX>(a, heads, grid, st);
  return launch_q4<D, H8, kRope>(a, heads, grid, st);
}

}  // namespace

// Key splits whose partials go through the workspace (1: none do).
static int ws_splits(int rows, int Hq, int Hkv, int max_blocks, bool rows_mode) {
  if (!rows_mode && q4_decode_on_tc(rows, Hq, Hkv, max_blocks)) return q4_tc_splits(rows, Hkv, max_blocks);
  if (rows_mode && q4_use_tc(Hq, Hkv)) return 1;
  const int S = q4_splits(rows, Hq, Hkv, max_blocks).S;
  return S <= kMaxCluster ? 1 : S;
}

size_t q4_ws_bytes(int rows, int Hq, int Hkv, int D, int max_blocks, bool rows_mode) {
  const size_t S = size_t(ws_splits(rows, Hq, Hkv, max_blocks, rows_mode));
  if (S == 1) return 0;
  const size_t po = (size_t)rows * Hq * S * D * 4;
  return (po + 255) / 256 * 256 + (size_t)rows * Hq * S * 8;
}

// Point the partials into the caller's workspace.
static int take_ws(Q4Args& a, int D, bool rows_mode, void* ws, size_t ws_bytes) {
  const size_t need = q4_ws_bytes(a.rows, a.Hq, a.Hkv, D, a.max_blocks, rows_mode);
  if (need == 0) return LAZY_OK;
  if (!ws || ws_bytes < need)
    return fail(LAZY_EINVAL, "workspace too small: need %zu bytes, got %zu", need, ws ? ws_bytes : 0);
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(LAZY_EINVAL, "workspace must be 256-byte aligned");
  const size_t po = (size_t)a.rows * a.Hq * a.S * D * 4;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + (po + 255) / 256 * 256);
  return LAZY_OK;
}

cudaError_t q4_merge(const Q4Args& a, int D, cudaStream_t st) {
  const long long rh = (long long)a.rows * a.Hq;
  const dim3 grid(unsigned((rh + kMergeWarps - 1) / kMergeWarps)), block(kMergeWarps * 32);
  auto kern = D == 128 ? q4_merge_kernel<128> : q4_merge_kernel<64>;
  return launch_pdl(kern, grid, block, 0, st, (const float*)a.part_o, (const float*)a.part_ml, a.S, rh, a.out, a.lse,
                    a.cu_q, a.B, a.Hq);
}

int run_q4_rows(Q4Args& a, int D, bool rows_mode, void* ws, size_t ws_bytes, cudaStream_t st) {
  if ((long long)a.rows * a.Hq > 0x7FFFFFFFll)
    return fail(LAZY_ERANGE, "too many query rows (%d rows, %d heads)", a.rows, a.Hq);
  if (!rows_mode && q4_decode_on_tc(a.rows, a.Hq, a.Hkv, a.max_blocks)) {
    a.S = q4_tc_splits(a.rows, a.Hkv, a.max_blocks);
    int rc = take_ws(a, D, rows_mode, ws, ws_bytes);
    if (rc == LAZY_OK) rc = run_q4_tc(a, D, 1, st);
    if (rc == LAZY_OK && a.S > 1) LAZY_CUDA_TRY(q4_merge(a, D, st));
    return rc;
  }
  const int heads = q4_heads(a.Hq, a.Hkv);
  a.S = q4_splits(a.rows, a.Hq, a.Hkv, a.max_blocks).S;
  int rc = take_ws(a, D, rows_mode, ws, ws_bytes);
  if (rc) return rc;
  const long long ctas = (long long)a.rows * (a.Hq / heads) * a.S;
  if (ctas > 0x7FFFFFFFll) return fail(LAZY_ERANGE, "too many query rows (%d rows, %d heads)", a.rows, a.Hq);
  const unsigned grid = unsigned(ctas);
  if (a.pos.kind == kNone) a.pos.slopes = nullptr;
  if (D == 128)
    rc = heads == 8 ? launch_q4_pos<128, true>(a, heads, grid, st) : launch_q4_pos<128, false>(a, heads, grid, st);
  else
    rc = heads == 8 ? launch_q4_pos<64, true>(a, heads, grid, st) : launch_q4_pos<64, false>(a, heads, grid, st);
  if (rc == LAZY_OK && a.S > kMaxCluster) LAZY_CUDA_TRY(q4_merge(a, D, st));
  return rc;
}

}  // namespace lazykv
