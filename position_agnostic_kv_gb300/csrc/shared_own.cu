// Decode of each request's own keys: the blocks behind those that its group shares (all of them where it
// shares none).
//
// Mathematics: per KV head and 8 of its query heads, S = q_eff K^T with q_eff = R_{m - Delta} q (rotated when a
// page has another Delta than the one before), an online softmax in base 2 per page, O += P V.
//
// One warp streams a run of pages through its own ring of shared-memory stages (TMA boxes, 128-byte swizzle)
// and feeds 16 x 8 x 16 matrix instructions: 8 heads fill half of the 16 rows, so the other half holds the low
// parts.  q_eff and P are each the sum of two bf16 numbers (16 bits of mantissa), rows 0-7 the high and rows
// 8-15 the low ones, and a score or output is the sum of two accumulators of the same thread: the precision
// costs no instruction.  K is exact in bf16.  P leaves the scores' accumulators in the layout of the next
// instruction's first operand.
//
// What bounds it: latency on short lists, then bytes.  64 requests of 33 own keys each, 8 KV heads: 8 to 10 us of a call
// (block words, first pages, one rotation, merge, a chain of dependent loads); 64 requests of up to 1064 keys,
// 515 on average: 38.3 us for 135 MB from cold caches, 3.5 TB/s.  They are 512 blocks, all resident, with one list
// each, so the launch lasts as long as its longest list, twice the average.
#include <cfloat>

#include "shared_decode.cuh"
#include "tcgen05.cuh"

namespace lazykv {

namespace {

using tc::swz;

// Four blocks of 3 warps on an SM: short own lists are a chain of dependent loads, so what counts is how many run at once.
// 64 requests of 33 own tokens / 64 of 532, whole decode steps: 3 blocks of 4 warps 58.7 / 100.9 us, 4 of 3 54.2 / 98.9,
// 6 of 2 56.2 / 101.6.
constexpr int kNW = 3, kStages = 2, kPerSm = 4;
constexpr float kTau = 8.f;  // the running maximum moves when beaten by more than this (base 2)

template <int D>
struct OwnLayout {
  static constexpr int PAGE = kPage * D * 2;
  static constexpr int STAGE = 2 * PAGE;
  static constexpr int Q_OFF = kNW * kStages * STAGE;       // float [8][D]
  static constexpr int SLOT_OFF = Q_OFF + 8 * D * 4;        // int4 [warp][stage] {start, lo, delta, -}
  static constexpr int BAR_OFF = SLOT_OFF + kNW * kStages * 16;
  static constexpr int SMEM = BAR_OFF + kNW * kStages * 8 + 1024;
  // when the pages are done, the stages hold the warps' results: o [warp][8][D], ml [warp][8][2]
  static_assert(kNW * 8 * (D + 2) * 4 <= Q_OFF, "merge buffer");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x = hi + lo in bf16, for two neighbours
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = f2_to_bf2(x, y);
  lo = f2_to_bf2(x - bf_lo(hi), y - bf_hi(hi));
}

template <int D, int POS>
__global__ void __launch_bounds__(kNW * 32, kPerSm) own_kernel(const __grid_constant__ CUtensorMap tmk,
                                                       const __grid_constant__ CUtensorMap tmv, const SharedArgs a) {
  using L = OwnLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sb = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, split = blockIdx.x;
  const int G = a.Hq / a.Hkv, per = (G + 7) / 8;             // head blocks of 8 per KV head
  const int kvh = blockIdx.y / per, h0 = kvh * G + blockIdx.y % per * 8;
  const int nh = min(8, kvh * G + G - h0);
  pdl_wait();
  pdl_trigger();  // the common keys' launch may start: it reads the same inputs and touches other results
  const Share sh = share_of(a, b);
  const int m = a.seq_len[b] - 1;
  const int nb = visible_blocks(m + 1, a.q_start[b], a.doc_blocks[b], a.max_blocks);
  if (split == 0 && blockIdx.y == 0) check_request(a, b, m);
  const int blocks = max(0, nb - sh.blocks), S = own_splits(blocks, a.SB);
  if (split >= S) return;  // uniform for the block
  const int chunk = (blocks + S - 1) / S;
  const int beg = sh.blocks + split * chunk, len = max(0, min(sh.blocks + blocks, beg + chunk) - beg);
  const int wb = beg + warp * len / kNW, n = beg + (warp + 1) * len / kNW - wb;

  float* qs = reinterpret_cast<float*>(sm + L::Q_OFF);
  int4* slots = reinterpret_cast<int4*>(sm + L::SLOT_OFF) + warp * kStages;
  const uint32_t bar0 = sb + L::BAR_OFF + warp * kStages * 8, stage0 = sb + warp * kStages * L::STAGE;
  const uint64_t* mrow = a.meta + (size_t)b * a.max_blocks + wb;
  uint64_t mcur = lane < n ? ldg_u64(mrow + lane) : 0, mnxt = 32 + lane < n ? ldg_u64(mrow + 32 + lane) : 0;
  int mbase = 0;
  if (lane == 0)
    for (int s = 0; s < kStages; ++s) mbar_init(bar0 + 8 * s, 1);
  fence_mbar_init();
  __syncwarp();

  // Page i of the run: the rows that hold a visible key, a prefix of the page, land in the stage's last rows and
  // zeros before them, so rows that hold no key never meet a product.
  auto issue = [&](int i) {
    if (i >= mbase + 32) {
      mcur = mnxt;
      mbase += 32;
      mnxt = mbase + 32 + lane < n ? ldg_u64(mrow + mbase + 32 + lane) : 0;
    }
    const uint64_t w = __shfl_sync(0xffffffffu, mcur, i - mbase);
    if (lane == 0) {
      const int st = i % kStages;
      const int delta = int(word_delta(w)), start = delta + kPage * int(word_pg(w));
      int rows = max(0, min(min(int(word_nvalid(w)), kPage), m - start + 1));
      if (word_page(w) >= uint32_t(a.num_pages)) {
        set_status(a.status, LAZY_STATUS_BAD_PAGE);
        rows = 0;
      }
      const int lo = kPage - rows;
      slots[st] = make_int4(start - lo, lo, delta, 0);
      const uint32_t bar = bar0 + 8 * st;
      if (rows) {
        const int z = int(word_page(w)) * a.Hkv + kvh;
        const uint32_t dst = stage0 + st * L::STAGE;
        mbar_arrive_expect_tx(bar, L::STAGE);
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb) {
          tma_load_page(dst + cb * 2048, &tmk, cb * 64, -lo, z, bar);
          tma_load_page(dst + L::PAGE + cb * 2048, &tmv, cb * 64, -lo, z, bar);
        }
      } else {
        mbar_arrive(bar);
      }
    }
    __syncwarp();
  };
  for (int i = 0; i < min(kStages, n); ++i) issue(i);
  for (int i = threadIdx.x; i < 8 * D; i += kNW * 32)
    qs[i] = i / D < nh ? __bfloat162float(a.q[((size_t)b * a.Hq + h0) * D + i]) * a.pos.scale_log2 : 0.f;
  __syncthreads();

  const int head = lane >> 2, c = lane & 3;  // this thread's row and its pair of columns in the fragments
  const float* qh = qs + head * D;
  float slope = 0.f;
  if constexpr (POS == kAlibi) slope = head < nh ? a.pos.slopes[h0 + head] * 1.4426950408889634f : 0.f;
  uint32_t qa[D / 16][4];
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float m_run = -FLT_MAX, l_run = 0.f;
  int cur = -1;  // Delta that qa holds (none yet)
  bool first = true;

  for (int i = 0; i < n; ++i) {
    const int st = i % kStages;
    if (!mbar_wait(bar0 + 8 * st, uint32_t((i / kStages) & 1))) {
      if (lane == 0) set_status(a.status, LAZY_STATUS_TIMEOUT);
      for (int j = i + 1; j < min(n, i + kStages); ++j) mbar_wait(bar0 + 8 * (j % kStages), uint32_t((j / kStages) & 1));
      break;
    }
    const int4 info = slots[st];
    if (info.y < kPage) {
      if (cur != info.z && (cur < 0 || POS == kRope || POS == kRopeX)) {
        cur = info.z;
        const int dp = m - cur;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int d = 16 * ks + 8 * half + 2 * c;
            float y0 = qh[d], y1 = qh[d + 1];
            if constexpr (POS == kRope) {  // half-split pairs (i, i + D/2) over the whole head
              const bool low = d < D / 2;
              const int f = low ? d : d - D / 2, other = low ? d + D / 2 : d - D / 2;
              float s0, c0, s1, c1;
              turn_sincos_signed(dp, a.pos.turns[f], s0, c0);
              turn_sincos_signed(dp, a.pos.turns[f + 1], s1, c1);
              y0 = y0 * c0 + (low ? -qh[other] : qh[other]) * s0;
              y1 = y1 * c1 + (low ? -qh[other + 1] : qh[other + 1]) * s1;
            } else if constexpr (POS == kRopeX) {
              const int rd = a.pos.rotary_dim, hr = rd / 2;
              if (d < rd) {
                float s0, c0, s1, c1;
                if (a.pos.interleaved) {
                  turn_sincos_signed(dp, a.pos.turns[d / 2], s0, c0);
                  const float x0 = y0;
                  y0 = x0 * c0 - y1 * s0;
                  y1 = x0 * s0 + y1 * c0;
                } else {
                  const bool low = d < hr;
                  const int f = low ? d : d - hr, other = low ? d + hr : d - hr;
                  turn_sincos_signed(dp, a.pos.turns[f], s0, c0);
                  turn_sincos_signed(dp, a.pos.turns[f + 1], s1, c1);
                  y0 = y0 * c0 + (low ? -qh[other] : qh[other]) * s0;
                  y1 = y1 * c1 + (low ? -qh[other + 1] : qh[other + 1]) * s1;
                }
              }
            }
            split2(y0, y1, qa[ks][2 * half], qa[ks][2 * half + 1]);
          }
      }
      // ---- scores of 16 keys: columns 2c, 2c + 1 of two 8-key halves
      const uint32_t sK = stage0 + st * L::STAGE, sV = sK + L::PAGE;
      float s[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k4 = 0; k4 < D / 32; ++k4) {
          const int chunk8 = 4 * k4 + (lane >> 3);
          uint32_t kb[4];
          ldsm4(sK + (chunk8 >> 3) * 2048 + swz(8 * nt + (lane & 7), chunk8 & 7), kb);
          mma16816(acc, qa[2 * k4], kb[0], kb[1]);
          mma16816(acc, qa[2 * k4 + 1], kb[2], kb[3]);
        }
        s[2 * nt] = acc[0] + acc[2];
        s[2 * nt + 1] = acc[1] + acc[3];
      }
      bool need = first;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = (e >> 1) * 8 + 2 * c + (e & 1);
        if constexpr (POS == kAlibi) s[e] += slope * float(info.x + t - m);
        if (t < info.y) s[e] = -INFINITY;
        need |= s[e] > m_run + kTau;
      }
      if (__any_sync(0xffffffffu, need)) {
        first = false;
        float x = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        if (x > m_run) {
          const float alpha = exp2f(m_run - x);
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] *= alpha;
          l_run *= alpha;
          m_run = x;
        }
      }
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = ex2_approx(s[e] - m_run);
      l_run += (p[0] + p[1]) + (p[2] + p[3]);
      uint32_t pa[4];
      split2(p[0], p[1], pa[0], pa[1]);
      split2(p[2], p[3], pa[2], pa[3]);
      // ---- O += P V, 16 columns at a time
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const int chunk8 = 2 * j + (lane >> 4);
        uint32_t vb[4];
        ldsm4t(sV + (chunk8 >> 3) * 2048 + swz((lane & 7) + (lane & 8), chunk8 & 7), vb);
        mma16816(o[2 * j], pa, vb[0], vb[1]);
        mma16816(o[2 * j + 1], pa, vb[2], vb[3]);
      }
    }
    __syncwarp();
    if (i + kStages < n) issue(i + kStages);
  }
  // ---- the warps' results joined by their maxima
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
  __syncthreads();
  float* mo = reinterpret_cast<float*>(sm);  // [warp][8][D]
  float* mml = mo + kNW * 8 * D;             // [warp][8][2]
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
    *reinterpret_cast<float2*>(mo + (warp * 8 + head) * D + 8 * j + 2 * c) =
        make_float2(o[j][0] + o[j][2], o[j][1] + o[j][3]);
  if (c == 0) {
    mml[(warp * 8 + head) * 2] = first ? -INFINITY : m_run;
    mml[(warp * 8 + head) * 2 + 1] = l_run;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nh * D; i += kNW * 32) {
    const int h = i / D, col = i % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kNW; ++w) M = fmaxf(M, mml[(w * 8 + h) * 2]);
    float O = 0.f, Ls = 0.f;
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      const float mw = mml[(w * 8 + h) * 2], f = mw == -INFINITY ? 0.f : exp2f(mw - M);
      O += f * mo[(w * 8 + h) * D + col];
      Ls += f * mml[(w * 8 + h) * 2 + 1];
    }
    const size_t row = (size_t)b * a.Hq + h0 + h, pi = row * (a.SA + a.SB) + a.SA + split;
    if (a.SA + a.SB == 1) {  // nothing to join
      a.out[row * D + col] = __float2bfloat16_rn(Ls == 0.f ? 0.f : O / Ls);
      if (a.lse && col == 0) a.lse[row] = (M + log2f(Ls)) * 0.6931471805599453f;
      continue;
    }
    a.part_o[pi * D + col] = O;
    if (col == 0) {
      a.part_ml[pi * 2] = M;
      a.part_ml[pi * 2 + 1] = Ls;
    }
  }
}

template <int D, int POS>
int launch_own(const SharedArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  auto kern = own_kernel<D, POS>;
  LAZY_CUDA_TRY(smem_limit(kern, OwnLayout<D>::SMEM, done));
  const int per = (a.Hq / a.Hkv + 7) / 8;
  LAZY_CUDA_TRY(launch_pdl(kern, dim3(a.SB, a.Hkv * per, a.B), dim3(kNW * 32), OwnLayout<D>::SMEM, st, mk, mv,
                           a));
  return LAZY_OK;
}

}  // namespace

int run_shared_own(const SharedArgs& a, int D, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  int kind = a.pos.kind == kYarn ? int(kRope) : a.pos.kind;
  if (kind == kRope && (a.pos.rotary_dim != D || a.pos.interleaved)) kind = kRopeX;
  if (D == 128) {
    if (kind == kRope) return launch_own<128, kRope>(a, mk, mv, st);
    if (kind == kRopeX) return launch_own<128, kRopeX>(a, mk, mv, st);
    if (kind == kAlibi) return launch_own<128, kAlibi>(a, mk, mv, st);
    return launch_own<128, kNone>(a, mk, mv, st);
  }
  if (kind == kRope) return launch_own<64, kRope>(a, mk, mv, st);
  if (kind == kRopeX) return launch_own<64, kRopeX>(a, mk, mv, st);
  if (kind == kAlibi) return launch_own<64, kAlibi>(a, mk, mv, st);
  return launch_own<64, kNone>(a, mk, mv, st);
}

}  // namespace lazykv
