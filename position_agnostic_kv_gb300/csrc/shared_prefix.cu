// Decode of the keys that a group of requests shares, read once for all of its rows, on the 5th-generation tensor
// cores.
//
// Mathematics: the rows of a group and KV head are its (request, head) pairs; per 128-key tile S = Q K^T with
// Q = R_m q (each row turned by its own position m) and K = R_Delta k (each page by its document's offset), an online
// softmax in base 2, O += P V.  The result is partial: unnormalised O, maximum and sum per key split, joined with the
// requests' own keys afterwards.
//
// One block per (key split, KV head, 256 rows of a group), 512 threads, one block per SM:
//   warps 0-3 / 4-7  softmax (thread = TMEM lane = row).  With more than 128 rows each warpgroup has a Q tile of its
//              own and sees every key tile; with up to 128 both have the same rows, one the even key tiles and one
//              the odd, and join their results at the end.  Either way step s of the block is key tile s/2 or s
//              against score buffer s % 2, and the products of one buffer run under the other's softmax.
//              Rows are normalised by a power of two each, so that f16 holds any query.
//   warps 8-11 the keys' rotation in place (f16; without rotation only the conversion); a thread owns 8 frequencies of
//              a page's rows and keeps their cosines while Delta stays.
//   warp 12 / 14  block words and TMA copies (64 columns x 16 rows of a page) of keys (3 stages) and of values (2).
//              A page with r < 16 keys is loaded from row r - 16: zeros, then its keys in the last rows.
//   warp 13    TMEM owner and MMA issuer: QK(0) QK(1) | PV(0) QK(2) | PV(1) QK(3) | ...
// TMEM: S0 [0,128), S1 [128,256), O0 [256,384), O1 [384,512); P_i in the first half of S_i, as bf16.
// Every wait is bounded.
//
// Precision: scores, maxima, sums and O are fp32.  A rotated key is rounded to f16 and so is a row's query, 11 bits each,
// because the products take 16 bits and a second part of either would double QK^T.  P is rounded to bf16, 8 bits, because
// both operands of PV have one type and values stay as they are stored; the sum is of the weights before the rounding.
// Random inputs, against 64 bits: 0.0024 relative, of which the bf16 result alone is 0.0017 and P's rounding as much again.
//
// What bounds it: few key tiles per block, each a chain.  64 requests of 4 heads per KV head over 32 000 common keys of 8
// KV heads (131 MB, 34 GFLOP): 39 us of the call's 53 here, 3.4 TB/s; a block has 15 key tiles of two Q tiles, a step per
// Q tile and key tile of ~1600 cycles of softmax, ~1100 of products and ~300 of handshakes, two of them overlapped, so
// 3200 per key tile, with ~10 000 before the first and ~7 000 for the results; the tensor pipe is busy in 44 % of the active cycles.
// Steps (this call): mma.sync with every row in registers 569 -> this kernel 68; Q rows by lanes, results written as whole
// rows, set-up before the launch before has ended 57; own keys before the common ones 54; raw queries by asynchronous
// copies 52.6.  Eight groups of ragged lists: keys' rotation unrolled twice and not eight times 98 -> 92, as the roles'
// loops together miss the instruction cache.  Left out: P handed over by halves, so that the first half's products start
// under the second's exponentials (53.1 as before, groups 94.2 instead of 92.2).
#include <cfloat>
#include <climits>

#include "q4_attn.cuh"
#include "shared_decode.cuh"
#include "tcgen05.cuh"

namespace lazykv {

namespace {

using namespace tc;

constexpr int kM = 128, kN = 128;
constexpr int kPagesPerTile = kN / kPage;
constexpr int kKStages = 3, kVStages = 2;
constexpr int kSlots = 6;  // per-tile metadata: published up to 4 tiles ahead of the softmax's last use
constexpr int kThreads = 512;
constexpr int kRotWarp0 = 8, kKWarp = 12, kMmaWarp = 13, kVWarp = 14;
// Registers per thread: at launch, and after the split (softmax, rotation, the four single warps), which adds up to it.
constexpr int kRegsLaunch = 128, kRegsSoftmax = 184, kRegsRot = 56, kRegsIssue = 88;
static_assert(2 * kRegsSoftmax + kRegsRot + kRegsIssue == 4 * kRegsLaunch, "warpgroup register shares");
constexpr float kTau = 8.0f;

enum : int {
  B_K_FULL = 0,    // [3] K tile landed
  B_K_READY = 3,   // [3] K tile rotated (a lane per warp)
  B_K_FREE = 6,    // [3] every QK^T with the stage done (commit)
  B_V_FULL = 9,    // [2] V tile landed
  B_V_FREE = 11,   // [2] every PV with the stage done (commit)
  B_S_FULL = 13,   // [2] scores written (commit; covers the buffer's PV before)
  B_P_FULL = 15,   // [2] P in TMEM, O rescaled (a lane per warp)
  B_Q_READY = 17,  // Q tiles prepared (a lane per warp)
  B_FINAL = 18,    // all products done (commit)
  NBAR = 19
};

template <int D>
struct Layout {
  static constexpr int BLK = kM * 128;
  static constexpr int TILE = kN * D * 2, QTILE = kM * D * 2;
  static constexpr int K_OFF = 2 * QTILE;
  static constexpr int V_OFF = K_OFF + kKStages * TILE;
  static constexpr int PSTART_OFF = V_OFF + kVStages * TILE;                // int [slot][8] position of stage row 0
  static constexpr int PINFO_OFF = PSTART_OFF + kSlots * kPagesPerTile * 4;  // int2 [slot][8] {Delta, first row with a key}
  static constexpr int FLAG_OFF = PINFO_OFF + kSlots * kPagesPerTile * 8;    // int [slot] every key visible to every row
  static constexpr int TURNS_OFF = FLAG_OFF + kSlots * 8;
  static constexpr int BAR_OFF = TURNS_OFF + (D / 2) * 8;
  static constexpr int EXP_OFF = BAR_OFF + NBAR * 8;  // int8 [256] exponents of the rows' powers of two
  static constexpr int MISC_OFF = EXP_OFF + 2 * kM;
  static constexpr int SMEM = MISC_OFF + 16 + 1024;
};
static_assert(Layout<128>::SMEM <= 227 * 1024, "shared memory budget");

template <int D, int POS>
__global__ void __launch_bounds__(kThreads, 1)
prefix_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const SharedArgs a,
              const int lowest_ex) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sb = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = int(blockIdx.x) % a.SA, pair = int(blockIdx.x) / a.SA, kvh = blockIdx.y, grp = blockIdx.z;
  const int G = a.Hq / a.Hkv;
  const uint32_t sQ0 = sb, sK0 = sb + L::K_OFF, sV0 = sb + L::V_OFF;
  int* pstart = reinterpret_cast<int*>(sm + L::PSTART_OFF);
  int2* pinfo = reinterpret_cast<int2*>(sm + L::PINFO_OFF);
  int* flags = reinterpret_cast<int*>(sm + L::FLAG_OFF);
  unsigned long long* turns = reinterpret_cast<unsigned long long*>(sm + L::TURNS_OFF);
  const uint32_t bar0 = sb + L::BAR_OFF;
  auto BAR = [&](int i) { return bar0 + 8u * uint32_t(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC_OFF + 4);

  if (threadIdx.x == 32 * kKWarp) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmv)) : "memory");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBAR; ++i)
      mbar_init(BAR(i), (i >= B_K_READY && i < B_K_FREE) || (i >= B_P_FULL && i < B_Q_READY) ? 4
                        : i == B_Q_READY                                                     ? 8
                                                                                             : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < D / 2; i += kThreads) turns[i] = a.pos.turns[i];
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // No wait here: own_kernel, the launch before this one, let this one start when it had waited for everything before it, and
  // the two touch different results.  This one waits at its end, so that the launch behind it finds both done.
  const int b0 = max(0, a.group_off[grp]);
  const int nreq = min(min(a.group_off[grp + 1], a.B) - b0, a.max_group);
  const int row0 = pair * 2 * kM, rows = min(2 * kM, nreq * G - row0);
  const int nb = shared_blocks_of(a, grp);
  const int ntiles_all = (nb + kPagesPerTile - 1) / kPagesPerTile, chunk = split_tiles(ntiles_all, a.SA);
  const int t0 = split * chunk, ntiles = min(ntiles_all, t0 + chunk) - t0;
  const bool idle = rows <= 0 || ntiles <= 0;  // uniform for the block
  const bool two = rows > kM;
  const int nsteps = two ? 2 * ntiles : ntiles;

  if (idle) {
  } else if (warp < 8) {
    // ============================ Q preparation, softmax, epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int sl = warp >> 2, r = threadIdx.x & (kM - 1);  // score buffer; row of the tile = TMEM lane
    int8_t* exps = reinterpret_cast<int8_t*>(sm + L::EXP_OFF);
    {
      // Q operands: NC lanes to a row (of the pair's up to 256), a run of rows to a group of lanes, so that the heads of
      // a request share their cosines; f16, 128-byte swizzle.  A power of two per row takes it into [-1, 1], where f16
      // keeps 11 bits of what matters.  The raw rows come into the V stages first, by copies that are all in flight at
      // once: loads row by row wait behind the first K and V tiles of every block (13 400 cycles until Q is ready, so
      // 7 000).  The values' copies start when Q is ready.
      constexpr int NC = POS == kRope ? D / 16 : D / 8, NG = 256 / NC, PER = 2 * kM / NG;
      const int t = threadIdx.x, c = t % NC, n0 = t / NC * PER;
      auto put = [&](int n, int k, const float2 (&y)[4]) {
        st_shared_v4(sQ0 + uint32_t((n >> 7) * L::QTILE + (k >> 3) * L::BLK) + swz(n & 127, k & 7),
                     make_uint4(f2_to_h2(y[0].x, y[0].y), f2_to_h2(y[1].x, y[1].y), f2_to_h2(y[2].x, y[2].y),
                                f2_to_h2(y[3].x, y[3].y)));
      };
      auto unpack = [](uint4 u, float2 (&y)[4]) {
        y[0] = bf2_to_f2(u.x);
        y[1] = bf2_to_f2(u.y);
        y[2] = bf2_to_f2(u.z);
        y[3] = bf2_to_f2(u.w);
      };
      const int rd = POS == kRope ? D : (POS == kRopeX ? a.pos.rotary_dim : 0), hr = rd / 2;
      const bool inter = POS == kRopeX && a.pos.interleaved != 0;
      // this lane's chunk, the one that it turns it against (itself: none), and its first frequency
      const int other = POS == kRope ? c + NC : (inter || 8 * c >= rd ? c : (8 * c < hr ? c + hr / 8 : c - hr / 8));
      const int f0 = POS == kRope ? 8 * c : (inter ? 4 * c : (8 * c < hr ? 8 * c : 8 * c - hr));
      const int nq = two ? 2 * kM : kM;  // rows of the operands
      {
        constexpr int CPR = D / 8, STEP = 256 / CPR;  // 16-byte chunks per row, rows per round of the 256 threads
        const int k = t % CPR;
        int n = t / CPR, rq = (row0 + n) / G, hd = (row0 + n) % G;
        const int step_rq = STEP / G, step_hd = STEP % G;
#pragma unroll 4
        for (; n < nq; n += STEP) {
          const void* src = n < rows ? a.q + ((size_t)(b0 + rq) * a.Hq + kvh * G + hd) * D + 8 * k : a.q;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sV0 + uint32_t(n) * (D * 2) + uint32_t(k) * 16),
                       "l"(src), "r"(n < rows ? 16 : 0) : "memory");
          rq += step_rq;
          hd += step_hd;
          if (hd >= G) {
            hd -= G;
            ++rq;
          }
        }
      }
      // the run's rows belong to at most NC requests: lane c of the group holds the c-th's position
      int req = (row0 + n0) / G, h = (row0 + n0) % G;
      const int req0 = req;
      const uint32_t pos = req0 + c < nreq ? uint32_t(max(a.seq_len[b0 + req0 + c] - 1, 0)) : 0u;
      asm volatile("cp.async.wait_all;" ::: "memory");
      named_sync(1, 2 * kM);
      const int n1 = min(n0 + PER, nq);
      float2 co[4], sn[4];
      uint32_t turned = 0xFFFFFFFFu;  // position that co and sn are of
#pragma unroll 1
      for (int n = n0; n < n1; ++n) {
        float2 x[4], z[4], y[4];
        const uint32_t raw_row = sV0 + uint32_t(n) * (D * 2);
        unpack(ld_shared_v4(raw_row + uint32_t(c) * 16), x);
        unpack(ld_shared_v4(raw_row + uint32_t(other) * 16), z);
        const uint32_t m = __shfl_sync(0xffffffffu, pos, (lane & ~(NC - 1)) | (req - req0));
        if (++h == G) {
          h = 0;
          ++req;
        }
        if ((POS == kRope || POS == kRopeX) && m != turned) {
          turned = m;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i0 = inter ? e : 2 * e;
            if (8 * c < rd || POS == kRope) {
              turn_sincos_fast(m, turns[f0 + i0], sn[e].x, co[e].x);
              if (!inter) turn_sincos_fast(m, turns[f0 + i0 + 1], sn[e].y, co[e].y);
            }
          }
        }
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          top = max3f(top, fabsf(x[e].x), fabsf(x[e].y));
          if (POS == kRope) top = max3f(top, fabsf(z[e].x), fabsf(z[e].y));
        }
#pragma unroll
        for (int o = NC / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int ex = q4_exponent(top, lowest_ex);
        const float inv = __uint_as_float(uint32_t(127 - ex) << 23);
        if (c == 0) exps[n] = int8_t(ex);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = make_float2(x[e].x * inv, x[e].y * inv);
          z[e] = make_float2(z[e].x * inv, z[e].y * inv);
        }
        if constexpr (POS == kRope) {
          float2 y2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 t1 = __fmul2_rn(z[e], sn[e]);
            y[e] = __ffma2_rn(x[e], co[e], make_float2(-t1.x, -t1.y));
            y2[e] = __ffma2_rn(x[e], sn[e], __fmul2_rn(z[e], co[e]));
          }
          put(n, c, y);
          put(n, c + NC, y2);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = x[e];
            if (POS == kRopeX && 8 * c < rd) {
              if (inter)
                y[e] = make_float2(x[e].x * co[e].x - x[e].y * sn[e].x, x[e].x * sn[e].x + x[e].y * co[e].x);
              else
                y[e] = make_float2(x[e].x * co[e].x + (8 * c < hr ? -z[e].x : z[e].x) * sn[e].x,
                                   x[e].y * co[e].y + (8 * c < hr ? -z[e].y : z[e].y) * sn[e].y);
            }
          }
          put(n, c, y);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_Q_READY));
    }
    named_sync(1, 2 * kM);  // the exponents are written
    const int pr = (two ? sl * kM : 0) + r, row = row0 + pr;
    const int b = b0 + row / G, hq = kvh * G + row % G;
    const bool valid = pr < rows;
    const int m_row = valid ? a.seq_len[b] - 1 : -1;
    const float f = a.pos.scale_log2 * __uint_as_float(uint32_t(127 + exps[pr]) << 23);  // scores are the products times this
    float slope = 0.f;
    if constexpr (POS == kAlibi) slope = valid ? a.pos.slopes[hq] * 1.4426950408889634f : 0.f;
    const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t tS = tl + uint32_t(sl * kN), tO = tl + uint32_t(2 * kN + sl * 128);
    const float2 ff = make_float2(f, f);
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int k = 0; ok && 2 * k + sl < nsteps; ++k) {
      const int j = two ? k : 2 * k + sl, slot = j % kSlots;
      const bool got = wait_bar(BAR(B_S_FULL + sl), uint32_t(k & 1), abort_flag, a.status);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      tc_fence_after();
      const bool fast = flags[slot] != 0;
      uint32_t v[kN];
#pragma unroll
      for (int c = 0; c < kN / 32; ++c) tmem_ld32(tS + uint32_t(32 * c), *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
      tmem_wait_ld();
      // ALiBi's bias -slope (m - p), p = pstart + t: slope t on each score, slope (pstart - m) on the page's maximum and
      // on its exponents' offset
      float bpg[kPagesPerTile];
      if constexpr (POS == kAlibi) {
#pragma unroll
        for (int pp = 0; pp < kPagesPerTile; ++pp) {
          bpg[pp] = slope * float(pstart[slot * kPagesPerTile + pp] - m_row);
#pragma unroll
          for (int t = 0; t < kPage; t += 2) {
            float2 x = make_float2(__uint_as_float(v[pp * kPage + t]), __uint_as_float(v[pp * kPage + t + 1]));
            x = __ffma2_rn(x, ff, make_float2(slope * float(t), slope * float(t + 1)));
            v[pp * kPage + t] = __float_as_uint(x.x);
            v[pp * kPage + t + 1] = __float_as_uint(x.y);
          }
        }
      }
      if (!fast) {  // stage row t of a page holds key pstart + t, from row `lo` on
#pragma unroll
        for (int pp = 0; pp < kPagesPerTile; ++pp) {
          const int lo = pinfo[slot * kPagesPerTile + pp].y, hi = m_row - pstart[slot * kPagesPerTile + pp] + 1;
#pragma unroll
          for (int t = 0; t < kPage; ++t)
            if (!(t >= lo && t < hi)) v[pp * kPage + t] = __float_as_uint(-INFINITY);
        }
      }
      float mq[kPagesPerTile];
#pragma unroll
      for (int q = 0; q < kPagesPerTile; ++q) {
        const float* x = reinterpret_cast<const float*>(v + 16 * q);
        float m = max3f(x[0], x[1], x[2]);
#pragma unroll
        for (int e = 3; e < 15; e += 2) m = max3f(m, x[e], x[e + 1]);
        mq[q] = fmaxf(m, x[15]);
        if constexpr (POS == kAlibi) mq[q] += bpg[q];
      }
      float mx = max3f(max3f(mq[0], mq[1], mq[2]), max3f(mq[3], mq[4], mq[5]), fmaxf(mq[6], mq[7]));
      if constexpr (POS != kAlibi) mx *= f;
      const bool need = mx > m_run + kTau;
      const float m_new = need ? mx : m_run;
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int e = 0; e < kN / 2; ++e) {
        float2 x = make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
        if constexpr (POS == kAlibi) {
          const float o = bpg[e / (kPage / 2)] - m_use;
          x = __fadd2_rn(x, make_float2(o, o));
        } else {
          x = __ffma2_rn(x, ff, make_float2(-m_use, -m_use));
        }
        const float2 ev = make_float2(ex2(x.x), ex2(x.y));
        sum4[e & 3] = __fadd2_rn(sum4[e & 3], ev);
        v[e] = f2_to_bf2(ev.x, ev.y);
      }
      const float2 s03 = __fadd2_rn(__fadd2_rn(sum4[0], sum4[1]), __fadd2_rn(sum4[2], sum4[3]));
      const float alpha = (need && m_run != -INFINITY) ? ex2(m_run - m_new) : 1.f;
      l_run = l_run * alpha + (s03.x + s03.y);
      if (__any_sync(0xffffffffu, k > 0 && alpha != 1.f)) {  // O holds the products of the steps before
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + uint32_t(c * 32), o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32(tO + uint32_t(c * 32), o);
        }
      }
      m_run = m_new;
#pragma unroll
      for (int c = 0; c < kN / 64; ++c) tmem_st32(tS + uint32_t(32 * c), *reinterpret_cast<const uint32_t(*)[32]>(v + 32 * c));
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_P_FULL + sl));
    }
    ok = ok && wait_bar(BAR(B_FINAL), 0, abort_flag, a.status);
    // A warp whose wait gave up still meets the others at the barriers below.
    const bool fine = __all_sync(0xffffffffu, ok);
    {
      tc_fence_after();
      // what a row's result is relative to; -inf where it has seen no key (a NaN stays)
      float M = l_run == 0.f ? -INFINITY : (m_run == -INFINITY ? 0.f : m_run), Lt = l_run;
      // Rows go through shared memory (the K and V stages, which no copy or product uses any more; 16-byte chunks
      // swizzled by the row), so that a warp writes whole rows: a thread's own row, 16 bytes at a time, took 8 us.
      const uint32_t stage = sK0 + uint32_t(pr) * (D * 4);
      const size_t pi0 = (size_t)a.SA + a.SB;
      auto stash = [&](int col, const float (&o)[32]) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          st_shared_v4(stage + (uint32_t((col / 4 + q) ^ (r & 7)) << 4),
                       make_uint4(__float_as_uint(o[4 * q]), __float_as_uint(o[4 * q + 1]), __float_as_uint(o[4 * q + 2]),
                                  __float_as_uint(o[4 * q + 3])));
      };
      if (two) {
#pragma unroll 1
        for (int c = 0; c < D / 32 && fine; ++c) {
          float o[32];
          tmem_ld32(tO + uint32_t(c * 32), *reinterpret_cast<uint32_t(*)[32]>(o));
          tmem_wait_ld();
          stash(c * 32, o);
        }
      } else {
        // even and odd tiles joined; each warpgroup takes half of the columns.  (The exchange is in the second Q tile.)
        float2* xml = reinterpret_cast<float2*>(sm + L::QTILE);
        xml[sl * kM + r] = make_float2(M, Lt);
        named_sync(1, 2 * kM);
        const float2 hA = xml[r], hB = xml[kM + r];
        M = fmaxf(hA.x, hB.x);
        const float wA = hA.x == -INFINITY ? 0.f : ex2(hA.x - M), wB = hB.x == -INFINITY ? 0.f : ex2(hB.x - M);
        Lt = (wA != 0.f ? wA * hA.y : 0.f) + (wB != 0.f ? wB * hB.y : 0.f);
#pragma unroll 1
        for (int c = 0; c < D / 64 && fine; ++c) {
          const int col = sl * (D / 2) + c * 32;
          uint32_t oa[32], ob[32];
          tmem_ld32(tl + uint32_t(2 * kN + col), oa);
          tmem_ld32(tl + uint32_t(3 * kN + col), ob);
          tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = (wA != 0.f ? wA * __uint_as_float(oa[e]) : 0.f) + (wB != 0.f ? wB * __uint_as_float(ob[e]) : 0.f);
          stash(col, o);
        }
      }
      if (valid && fine && (two || sl == 0)) {
        const size_t pi = ((size_t)b * a.Hq + hq) * pi0 + split;
        *reinterpret_cast<float2*>(a.part_ml + pi * 2) = make_float2(M, Lt);
      }
      if (two)
        named_sync(1 + sl, kM);
      else
        named_sync(1, 2 * kM);
      constexpr int LPR = D / 4, RPW = 32 / LPR;  // lanes to a row, rows to a warp's store
      constexpr int kRowsPerWarp2 = kM / 4, kRowsPerWarp1 = kM / 8;
      const int n0 = (two ? warp * kRowsPerWarp2 : warp * kRowsPerWarp1) + lane / LPR, c = lane % LPR;
      const int n1 = fine ? min(rows, n0 - lane / LPR + (two ? kRowsPerWarp2 : kRowsPerWarp1)) : 0;
      int hd = (row0 + n0) % G;
      float* to = a.part_o + (((size_t)(b0 + (row0 + n0) / G) * a.Hq + kvh * G + hd) * pi0 + split) * D + 4 * c;
      const size_t step = pi0 * D * RPW, wrap = (size_t)(a.Hq - G) * pi0 * D;  // to the next row's; to the next request's
#pragma unroll 4
      for (int q = n0; q < n1; q += RPW) {
        *reinterpret_cast<uint4*>(to) = ld_shared_v4(sK0 + uint32_t(q) * (D * 4) + (uint32_t(c ^ (q & 7)) << 4));
        to += step;
        for (hd += RPW; hd >= G; hd -= G) to += wrap;
      }
    }
  } else if (warp < kKWarp) {
    // ============================ keys: rotation by the page's Delta, f16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRot));
    const int rt = threadIdx.x - kRotWarp0 * 32;
    const int ps = rt / kPage, l = rt % kPage;  // page slot of the tile, and this thread's part of it
    constexpr int NCP = D / 16;
    bool ok = true;  // once a wait gives up, the thread skips the work but keeps arriving
    float co[8], sn[8];
    int cur = -1;
    // other than half-split rotation of the whole head: one chunk task for all 16 rows of the page (0: rotated chunk
    // pair, 1: chunk of adjacent pairs, 2: a chunk that is only converted, 3: none)
    int kind = 3, chunk8 = 0, part = 0, f0 = 0;
    if constexpr (POS != kRope) {
      const int rd = POS == kRopeX ? a.pos.rotary_dim : 0;
      const int nrot = a.pos.interleaved ? rd / 8 : rd / 16, ntail = (D - rd) / 8;
      if (l < nrot) {
        kind = a.pos.interleaved ? 1 : 0;
        chunk8 = l;
        part = l + rd / 16;
        f0 = a.pos.interleaved ? 4 * l : 8 * l;
      } else if (l < nrot + ntail) {
        kind = 2;
        chunk8 = rd / 8 + (l - nrot);
      }
    }
    for (int j = 0; j < ntiles; ++j) {
      const int s = j % kKStages, slot = j % kSlots;
      if (ok) ok = wait_bar(BAR(B_K_FULL + s), uint32_t((j / kKStages) & 1), abort_flag, a.status);
      const int2 pi = ok ? pinfo[slot * kPagesPerTile + ps] : make_int2(0, kPage);
      const uint32_t sK = sK0 + uint32_t(s * L::TILE);
      if (pi.y < kPage) {
        if constexpr (POS == kRope) {
          const int c = l % NCP, g = l / NCP;
          if (pi.x != cur) {
            cur = pi.x;
#pragma unroll
            for (int e = 0; e < 8; ++e) turn_sincos_fast(uint32_t(pi.x), turns[8 * c + e], sn[e], co[e]);
          }
// (unrolled by 2 and not by 8: every role's code goes through one instruction cache, 98.8 -> 92.2 us for eight groups)
#pragma unroll 2
          for (int i = 0; i < NCP; ++i) {
            const int t = g * NCP + i;
            if (t < pi.y) continue;
            const int r = ps * kPage + t;
            const uint32_t a1 = sK + swz(r, c);
            const uint32_t a2 = D == 128 ? sK + uint32_t(L::BLK) + swz(r, c) : sK + swz(r, c + 4);
            uint4 u1 = ld_shared_v4(a1), u2 = ld_shared_v4(a2);
            uint32_t* p1 = reinterpret_cast<uint32_t*>(&u1);
            uint32_t* p2 = reinterpret_cast<uint32_t*>(&u2);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float2 cv = make_float2(co[2 * w], co[2 * w + 1]), sv = make_float2(sn[2 * w], sn[2 * w + 1]);
              const float2 x1 = bf2_to_f2(p1[w]), x2 = bf2_to_f2(p2[w]);
              const float2 t1 = __fmul2_rn(x2, sv), t2 = __fmul2_rn(x2, cv);
              const float2 y1 = __ffma2_rn(x1, cv, make_float2(-t1.x, -t1.y)), y2 = __ffma2_rn(x1, sv, t2);
              p1[w] = f2_to_h2(y1.x, y1.y);
              p2[w] = f2_to_h2(y2.x, y2.y);
            }
            st_shared_v4(a1, u1);
            st_shared_v4(a2, u2);
          }
        } else {
          auto kaddr = [&](int r, int k) { return sK + uint32_t((k >> 3) * L::BLK) + swz(r, k & 7); };
          if (POS == kRopeX && kind < 2 && pi.x != cur) {
            cur = pi.x;
            const int nf = kind == 0 ? 8 : 4;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < nf) turn_sincos_fast(uint32_t(pi.x), turns[f0 + e], sn[e], co[e]);
          }
#pragma unroll 1
          for (int t = pi.y; t < kPage && kind < 3; ++t) {
            const int r = ps * kPage + t;
            const uint32_t a1 = kaddr(r, chunk8);
            uint4 u1 = ld_shared_v4(a1);
            uint32_t* p1 = reinterpret_cast<uint32_t*>(&u1);
            if (POS == kRopeX && kind == 0) {
              const uint32_t a2 = kaddr(r, part);
              uint4 u2 = ld_shared_v4(a2);
              uint32_t* p2 = reinterpret_cast<uint32_t*>(&u2);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const float2 x1 = bf2_to_f2(p1[w]), x2 = bf2_to_f2(p2[w]);
                p1[w] = f2_to_h2(x1.x * co[2 * w] - x2.x * sn[2 * w], x1.y * co[2 * w + 1] - x2.y * sn[2 * w + 1]);
                p2[w] = f2_to_h2(x1.x * sn[2 * w] + x2.x * co[2 * w], x1.y * sn[2 * w + 1] + x2.y * co[2 * w + 1]);
              }
              st_shared_v4(a2, u2);
            } else if (POS == kRopeX && kind == 1) {
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const float x0 = bf_lo(p1[w]), x1 = bf_hi(p1[w]);
                p1[w] = f2_to_h2(x0 * co[w] - x1 * sn[w], x0 * sn[w] + x1 * co[w]);
              }
            } else {
#pragma unroll
              for (int w = 0; w < 4; ++w) p1[w] = f2_to_h2(bf_lo(p1[w]), bf_hi(p1[w]));
            }
            st_shared_v4(a1, u1);
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_K_READY + s));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    const uint64_t* words = a.meta + (size_t)b0 * a.max_blocks;
    // With ALiBi the newest tiles come first: they hold the rows' maxima, so O is hardly ever rescaled.
    auto tile_of = [&](int j) { return POS == kAlibi ? t0 + ntiles - 1 - j : t0 + j; };
    auto fetch = [&](int j) -> uint64_t {  // lane < 8: the block word of its page slot
      const int jb = tile_of(j) * kPagesPerTile + lane;
      return lane < kPagesPerTile && j < ntiles && jb < nb ? ldg_u64(words + jb) : 0ull;
    };
    auto keys_of = [&](uint64_t w) {  // 0 behind the list and outside the cache
      return word_page(w) < uint32_t(a.num_pages) ? min(int(word_nvalid(w)), kPage) : 0;
    };
    if (warp == kKWarp) {
      // ============================ block words, K copies
      int m_min = INT_MAX;  // of the block's rows
      uint64_t w_next = fetch(0);
      int issued = 0;
      bool ok = true;
      for (int j = 0; j < ntiles && ok; ++j) {
        const int s = j % kKStages, slot = j % kSlots;
        const uint64_t w = w_next;
        w_next = fetch(j + 1);
        const int rows_k = keys_of(w), lo = kPage - rows_k, delta = int(word_delta(w));
        const int start = delta + kPage * int(word_pg(w));
        if (word_page(w) >= uint32_t(a.num_pages)) set_status(a.status, LAZY_STATUS_BAD_PAGE);
        if (j >= kKStages) {
          const bool freed = wait_bar(BAR(B_K_FREE + s), uint32_t((j / kKStages - 1) & 1), abort_flag, a.status);
          ok = __all_sync(0xffffffffu, freed);
          if (!ok) break;
        }
        if (lane < kPagesPerTile) {
          pinfo[slot * kPagesPerTile + lane] = make_int2(delta, lo);
          pstart[slot * kPagesPerTile + lane] = start - lo;
        }
        const uint32_t load = __ballot_sync(0xffffffffu, lane < kPagesPerTile && rows_k > 0);
        if ((load >> lane) & 1u)
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_page(sK0 + uint32_t(s * L::TILE + cb * L::BLK + lane * kPage * 128), &tmk, cb * 64, -lo,
                          int(word_page(w)) * a.Hkv + kvh, BAR(B_K_FULL + s));
        if (j == 0) {
          for (int i = row0 / G + lane; i <= (row0 + rows - 1) / G; i += 32) m_min = min(m_min, a.seq_len[b0 + i] - 1);
#pragma unroll
          for (int o = 16; o; o >>= 1) m_min = min(m_min, __shfl_xor_sync(0xffffffffu, m_min, o));
        }
        const bool all = __all_sync(0xffffffffu, lane >= kPagesPerTile || (rows_k == kPage && start + kPage - 1 <= m_min));
        __syncwarp();
        if (lane == 0) {  // the phase ends with this arrival and the bytes, in either order
          flags[slot] = all;
          mbar_arrive_expect_tx(BAR(B_K_FULL + s), uint32_t(__popc(load)) * kPage * D * 2);
        }
        __syncwarp();
        issued = j + 1;
      }
      if (lane == 0)  // never leave copies in flight
        for (int j = max(0, issued - kKStages); j < issued; ++j) {
          WaitClock clk;
          while (!mbar_test(BAR(B_K_FULL + j % kKStages), uint32_t((j / kKStages) & 1)) && !clk.expired()) {
          }
        }
    } else if (warp == kVWarp) {
      // ============================ V copies
      uint64_t w_next = fetch(0);
      int issued = 0;
      bool ok = wait_bar(BAR(B_Q_READY), 0, abort_flag, a.status);  // the raw queries have left the stages
      ok = __all_sync(0xffffffffu, ok);
      for (int j = 0; j < ntiles && ok; ++j) {
        const int s = j % kVStages;
        const uint64_t w = w_next;
        w_next = fetch(j + 1);
        const int rows_v = keys_of(w), lo = kPage - rows_v;
        if (j >= kVStages) {
          const bool freed = wait_bar(BAR(B_V_FREE + s), uint32_t((j / kVStages - 1) & 1), abort_flag, a.status);
          ok = __all_sync(0xffffffffu, freed);
          if (!ok) break;
        }
        const uint32_t sV = sV0 + uint32_t(s * L::TILE);
        const uint32_t load = __ballot_sync(0xffffffffu, lane < kPagesPerTile && rows_v > 0);
        const uint32_t empty = ~load & ((1u << kPagesPerTile) - 1u);
        if (empty) {  // page slots without keys meet PV with zero weights, and must not hold a NaN
          for (int pp = 0; pp < kPagesPerTile; ++pp) {
            if (!((empty >> pp) & 1u)) continue;
#pragma unroll
            for (int cb = 0; cb < D / 64; ++cb)
#pragma unroll
              for (int i = 0; i < kPage * 8 / 32; ++i)
                st_shared_v4(sV + uint32_t(cb * L::BLK) + swz(pp * kPage + (i * 32 + lane) / 8, (i * 32 + lane) % 8),
                             make_uint4(0, 0, 0, 0));
          }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(BAR(B_V_FULL + s), uint32_t(__popc(load)) * kPage * D * 2);
        __syncwarp();
        if ((load >> lane) & 1u)
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_page(sV + uint32_t(cb * L::BLK + lane * kPage * 128), &tmv, cb * 64, -lo,
                          int(word_page(w)) * a.Hkv + kvh, BAR(B_V_FULL + s));
        __syncwarp();
        issued = j + 1;
      }
      if (lane == 0)
        for (int j = max(0, issued - kVStages); j < issued; ++j) {
          WaitClock clk;
          while (!mbar_test(BAR(B_V_FULL + j % kVStages), uint32_t((j / kVStages) & 1)) && !clk.expired()) {
          }
        }
    } else if (warp == kMmaWarp) {
      // ============================ products (one thread)
      if (elect_one()) {
        constexpr uint32_t IQK = idesc_mma(kM, kN, 0, 1), IPV = idesc_mma(kM, D, 1, 0);
        const uint64_t qd = sdesc(sQ0, 16, 1024), kd = sdesc(sK0, 16, 1024), vd = sdesc(sV0, L::BLK, 1024);
        bool ok = wait_bar(BAR(B_Q_READY), 0, abort_flag, a.status);
        int ks = 0, vs = 0;            // stages of the next QK^T's and PV's tiles
        uint32_t kpar = 0, vpar = 0;
        // The next waits' barriers are asked while products queue, so that the thread goes on at once where they are done.
        bool seen_k = false, seen_p = false, seen_v = false;
        auto qk = [&](int s) -> bool {  // step s: scores into buffer s % 2
          const bool first = !two || !(s & 1), last = !two || (s & 1);
          if (first && !seen_k && !wait_bar(BAR(B_K_READY + ks), kpar, abort_flag, a.status)) return false;
          tc_fence_after();
          const uint64_t k0 = kd + uint64_t(ks * (L::TILE >> 4));
          auto go = [&](uint32_t d, uint64_t q0) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              constexpr uint64_t blk = L::BLK >> 4;
              mma_bf16(d, q0 + (kk >> 2) * blk + (kk & 3) * 2, k0 + (kk >> 2) * blk + (kk & 3) * 2, IQK, kk > 0 ? 1u : 0u);
            }
          };
          if (s & 1)
            go(tmem + kN, two ? qd + (L::QTILE >> 4) : qd);
          else
            go(tmem, qd);
          mma_commit(BAR(B_S_FULL + (s & 1)));
          if (last) {
            mma_commit(BAR(B_K_FREE + ks));
            if (++ks == kKStages) {
              ks = 0;
              kpar ^= 1u;
            }
          }
          return true;
        };
        if (ok) ok = qk(0);
        if (ok && nsteps > 1) ok = qk(1);
        for (int s = 0; s < nsteps && ok; ++s) {
          const bool first = !two || !(s & 1), last = !two || (s & 1);
          ok = (!first || seen_v || wait_bar(BAR(B_V_FULL + vs), vpar, abort_flag, a.status)) &&
               (seen_p || wait_bar(BAR(B_P_FULL + (s & 1)), uint32_t((s >> 1) & 1), abort_flag, a.status));
          if (!ok) break;
          tc_fence_after();
          const uint64_t v0 = vd + uint64_t(vs * (L::TILE >> 4));
          auto go = [&](uint32_t o, uint32_t p) {
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
              mma_ts(o, p + uint32_t(kk * 8), v0 + uint64_t(kk * (16 * 128 >> 4)), IPV, (s > 1 || kk > 0) ? 1u : 0u);
          };
          if (s & 1)
            go(tmem + 3 * kN, tmem + kN);
          else
            go(tmem + 2 * kN, tmem);
          if (last) {
            mma_commit(BAR(B_V_FREE + vs));
            if (++vs == kVStages) {
              vs = 0;
              vpar ^= 1u;
            }
          }
          seen_k = mbar_peek(BAR(B_K_READY + ks), kpar);
          if (s + 2 < nsteps) ok = qk(s + 2);
          seen_v = mbar_peek(BAR(B_V_FULL + vs), vpar);
          seen_p = mbar_peek(BAR(B_P_FULL + ((s + 1) & 1)), uint32_t(((s + 1) >> 1) & 1));
        }
        mma_commit(BAR(B_FINAL));  // every product is done before O is read, and before TMEM goes
        WaitClock clk;
        while (!mbar_test(BAR(B_FINAL), 0) && !clk.expired()) {
        }
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  pdl_trigger();
  pdl_wait();
}

template <int D, int POS>
int launch_prefix(const SharedArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  using L = Layout<D>;
  static std::atomic<uint64_t> done{0};
  static std::atomic<int> regs{0};
  auto kern = prefix_kernel<D, POS>;
  LAZY_CUDA_TRY(smem_limit(kern, L::SMEM, done));
  if (!regs.load(std::memory_order_relaxed)) {
    cudaFuncAttributes fa;
    LAZY_CUDA_TRY(cudaFuncGetAttributes(&fa, kern));
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  // the split of registers is only valid for the number that it was made for
  if (regs.load(std::memory_order_relaxed) != kRegsLaunch)
    return fail(LAZY_ECUDA, "shared decode kernel built with %d registers per thread, expected %d",
                regs.load(std::memory_order_relaxed), kRegsLaunch);
  const long long rows = (long long)a.max_group * (a.Hq / a.Hkv);
  const unsigned pairs = unsigned((rows + 2 * kM - 1) / (2 * kM));
  LAZY_CUDA_TRY(launch_pdl(kern, dim3(unsigned(a.SA) * pairs, a.Hkv, a.n_groups), dim3(kThreads), L::SMEM, st, mk, mv, a,
                           q4_lowest_exponent(a.pos.scale_log2)));
  return LAZY_OK;
}

}  // namespace

// Key splits of the common keys; 0: every request is decoded alone.
int shared_prefix_splits(int B, int n_groups, int max_group, int max_shared, int Hq, int Hkv) {
  if (B <= 0 || n_groups <= 0 || max_group <= 0 || max_shared <= 0) return 0;
  const int sms = sm_count(), tiles = (max_shared + kPagesPerTile - 1) / kPagesPerTile, G = Hq / Hkv;
  // Decoded alone, a page is read once per request and 8 heads, out of the L2 at about 1.8 pages of a head per ns;
  // sharing costs two launches, about 8 us (16 requests over 130 common pages of 8 heads: 28.6 us alone, 16.9 shared;
  // 2 requests over 5 pages of 2 heads: 14.3 and 17.0).
  const long long alone = (long long)B * max_shared * Hkv * ((G + 7) / 8), once = (long long)n_groups * max_shared * Hkv;
  if (alone - once < 8000) return 0;
  const long long rows = (long long)max_group * G, pairs = (rows + 2 * kM - 1) / (2 * kM), units = n_groups * Hkv * pairs;
  // A shared page takes a block as long as two pages alone, and its start and results as long as 120: groups of two or of few
  // common pages are faster alone, where the requests alone are one wave of blocks.  (32 / 8 heads, 32 groups of 2 requests
  // over 260 common pages: alone 109.2 us, shared 134.8; 16 of 4 over 30: 25.2, 34.4; over 260: 92.8, 81.5.  More waves: 32 / 32
  // heads, 6 groups of 2 over 600: 249.5, 186.0.)
  const long long lists = (long long)B * Hkv * ((G + 7) / 8), splits = (3ll * sms + lists - 1) / lists;
  if (lists * splits <= 4ll * sms && alone < 2 * once + 120 * units) return 0;
  // Time of a launch in key tiles: waves of blocks, each its tiles, and its start and results, as long as 6 tiles of two
  // Q tiles or 12 of one; then the join, with every split.  (16 requests as above, splits 4 / 6 / 9 / 17: 19.9, 17.8,
  // 16.9, 22.2 us; 32 requests of 32 heads over 94 tiles of one KV head, splits 16 / 24 / 38: 28.2, 25.6, 30.4.)
  const bool two = rows > kM;
  const long long start = two ? 600 : 1200, join = two ? 15 : 30;  // hundredths of a tile
  long long best = 0;
  int S = 1;
  for (int s = 1; s <= 64 && s <= tiles; ++s) {
    const long long t = ((units * s + sms - 1) / sms) * (100ll * ((tiles + s - 1) / s) + start) + join * s;
    if (s == 1 || t < best) {
      best = t;
      S = s;
    }
  }
  return S;
}

int run_shared_prefix(const SharedArgs& a, int D, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  int kind = a.pos.kind == kYarn ? int(kRope) : a.pos.kind;
  if (kind == kRope && (a.pos.rotary_dim != D || a.pos.interleaved)) kind = kRopeX;
  if (D == 128) {
    if (kind == kRope) return launch_prefix<128, kRope>(a, mk, mv, st);
    if (kind == kRopeX) return launch_prefix<128, kRopeX>(a, mk, mv, st);
    if (kind == kAlibi) return launch_prefix<128, kAlibi>(a, mk, mv, st);
    return launch_prefix<128, kNone>(a, mk, mv, st);
  }
  if (kind == kRope) return launch_prefix<64, kRope>(a, mk, mv, st);
  if (kind == kRopeX) return launch_prefix<64, kRopeX>(a, mk, mv, st);
  if (kind == kAlibi) return launch_prefix<64, kAlibi>(a, mk, mv, st);
  return launch_prefix<64, kNone>(a, mk, mv, st);
}

}  // namespace lazykv
