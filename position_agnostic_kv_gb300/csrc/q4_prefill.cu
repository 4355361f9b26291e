// Causal prefill over the 4-bit paged cache on the 5th-generation tensor cores.
//
// Mathematics: per KV head, S = (R_m q)(R_Delta k)^T for every query row (a query head of a token at
// position m) and visible key, an online softmax in base 2 over 128-key tiles, O += P V.
//
// One CTA per (request, KV head, 256 query rows = two 128-row Q tiles, rows = (token, head) pairs), 512
// threads, one CTA per SM.  Roles:
//   warps 0-3 / 4-7  softmax of Q tile 0 / 1 (thread = TMEM lane = row): the Q operand (rotated by m,
//              normalised by a power of two per row, f16, 128-byte swizzle), then per tile the scores from
//              TMEM, mask, running maximum (moved only when beaten by more than 8), P back to TMEM over S
//              as f16, held as 2^(s - max + 7); the epilogue.
//   warps 8-11 keys: each tile's packed pages (9 D bytes of keys each) become the f16 operand.  Code
//              times scale is exact in f16; the rotation by the page's Delta then rounds cos, sin, one
//              product and the sum to f16 (2^-11 each: 2 instructions per value against 3.5 through
//              fp32; the 4-bit codes themselves are off by up to 2^-3 of a group's maximum).  A thread owns
//              8 frequencies (two runs of 8 dimensions) of 8 rows of a page; the packed pages lie 9 D + pad
//              bytes apart, so that its word loads meet no bank conflicts.
//   warps 14-15 values: the same, exact in f16; even and odd groups store their rows in opposite order,
//              against bank conflicts.  A weight of 0 does not hide a NaN from a product, so NaN scales become 0
//              before the conversion (while it waits for its stage), and the first position of one in each 16
//              columns is noted: at the end the rows at or behind it, which are those that see it, become
//              NaN there.
//   warp 12    producer: block words four tiles at a time, asynchronous 16-byte copies into a ring of packed
//              keys (2 stages, KH 4) and one of packed values (1, KH 2).
//   warp 13    TMEM owner and MMA issuer: QK0(j) QK1(j) | PV0(j) QK0(j+1) PV1(j) QK1(j+1) | ...
// Both f16 rings have 2 stages, filled a tile ahead.  TMEM: S0 [0,128), S1 [128,256), O0 [256,384),
// O1 [384,512); P_i in the first half of S_i.
// With one live Q tile S0 and S1 double-buffer its scores; in launches whose CTAs all have one (KH) the two
// softmax warpgroups each take half of every tile's keys and merge in the epilogue.
//
// What bounds it: the softmax, one exponential and ~4 other instructions per score: 128 scores of a row take
// ~2100 of a tile's ~3800 cycles, the products of both Q tiles 2048, and the two overlap in part (the scores
// of one Q tile are computed while the other's are waited for).  KH waits for its keys' role.  The packed
// cache, 18 D / 16 bytes per key and head, comes out of the L2.  8 x 64 queries of 64 heads (8 KV heads) over
// 10 300 keys: 159 us, 1083 TFLOP/s; 32 x 32 queries of 32 heads of one KV head over 12 000 keys, ALiBi: 223
// us, 903 TFLOP/s; 16 x 32 queries of 32 heads over 2000 keys (KH): 32 us, 528 TFLOP/s; 1600 tokens of one
// document: 38 us.
// Measured and left out: dequantisation of both operands by one warpgroup 232 us (first shape), scores in
// halves of a tile with two buffers per Q tile 176 (second shape 200), values only in halves 171 (201), an
// MMA thread per Q tile 229 (291).  Replacing NaN scales during the conversion (a minimum per pair) 161 (220)
// and 33.5 against 34.0 for the decode of wide head groups.  Every wait is bounded.
#include <cfloat>
#include <climits>

#include "q4_attn.cuh"
#include "tcgen05.cuh"

namespace lazykv {

namespace tcq {

using namespace tc;

constexpr int kM = 128, kQT = 2, kN = 128;
constexpr int kPagesPerTile = kN / kPage;
constexpr int kSlots = 8;  // per-tile metadata: published up to 7 tiles ahead of the softmax's last use
constexpr int kThreads = 512;
constexpr int kDeqWarp0 = 8, kProdWarp = 12, kMmaWarp = 13, kValWarp0 = 14;
constexpr int kRegsLaunch = 128;
// Registers per thread after the re-split: softmax, keys, and the warpgroup of producer, MMA and values; they
// add up to the launch's.  (176, 72, 88) takes 163 us for the first shape above, (168, 72, 104) 160.  KH's
// softmax holds half a row of scores; its keys' role has registers for two steps at once (below).
template <bool KH> struct Regs {
  static constexpr int softmax = KH ? 144 : 176, deq = KH ? 104 : 56, issue = KH ? 120 : 104;
  static_assert(2 * softmax + deq + issue == 4 * kRegsLaunch, "warpgroup register shares");
};
constexpr float kTau = 8.0f, kPOff = 7.0f;

enum : int {
  B_PK_FULL = 0,   // [4] packed keys landed (the producer's 32 lanes, and its lane 0 for the metadata)
  B_PK_FREE = 4,   // [4] packed keys read (128 arrivals)
  B_PV_FULL = 8,   // [2] packed values landed
  B_PV_FREE = 10,  // [2] packed values read (64)
  B_K_READY = 12,  // [2] K operand written (128)
  B_K_FREE = 14,   // [2] every QK^T of the stage done (commit)
  B_V_READY = 16,  // [2] V operand written (64)
  B_V_FREE = 18,   // [2] every PV of the stage done (commit)
  B_S_FULL = 20,   // [2] per Q tile (one live tile: per S buffer): S written (commit)
  B_P_FULL = 22,   // [2] P in TMEM, O rescaled (32 per warp that holds rows)
  B_Q_READY = 24,  // Q operands written (256)
  B_FINAL = 25,    // all MMAs done (commit)
  B_PV_DONE = 26,  // one live Q tile: a tile's PV done (commit)
  NBAR = 27
};

template <int D>
struct Layout {
  static constexpr int BLK = kM * 128;
  static constexpr int TILE = kN * D * 2;
  static constexpr int QTILE = kM * D * 2;
  static constexpr int PKS = D == 128 ? 1184 : 656;  // bytes between packed key pages (9 D + pad)
  static constexpr int PVS = 9 * D;
  // in the second Q tile (KH): {max, sum} [2][128], stage 1 of the packed values, stages 2 and 3 of the keys
  static constexpr int XML_OFF = QTILE;
  static constexpr int PV1_OFF = XML_OFF + 2 * kM * 8;
  static constexpr int PK2_OFF = PV1_OFF + kPagesPerTile * PVS;
  static constexpr int Q_END = PK2_OFF + 2 * kPagesPerTile * PKS;
  static constexpr int K_OFF = ((Q_END > kQT * QTILE ? Q_END : kQT * QTILE) + 1023) / 1024 * 1024;
  static constexpr int V_OFF = K_OFF + 2 * TILE;
  static constexpr int PK_OFF = V_OFF + 2 * TILE;
  static constexpr int PV_OFF = PK_OFF + 2 * kPagesPerTile * PKS;
  static constexpr int PSTART_OFF = PV_OFF + kPagesPerTile * PVS;              // int [slot][8] first key position
  static constexpr int PINFO_OFF = PSTART_OFF + kSlots * kPagesPerTile * 4;    // int2 [slot][8] {Delta, rows}
  static constexpr int FLAG_OFF = PINFO_OFF + kSlots * kPagesPerTile * 8;      // int [slot] every key visible
  static constexpr int TURNS_OFF = FLAG_OFF + kSlots * 8;
  static constexpr int BAR_OFF = TURNS_OFF + (D / 2) * 8;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  // int [D / 16] first key with a NaN in 16 columns, [1] in any; [4] {first query row and head, tokens, m_min}
  static constexpr int NANPOS_OFF = MISC_OFF + 16;
  static constexpr int SMEM = NANPOS_OFF + (D / 16 + 5) * 4 + 1024;
};
static_assert(Layout<128>::SMEM <= 227 * 1024, "shared memory budget");

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// One lane of a converged warp.  The MMA thread is chosen this way and not by `lane == 0`: in a branch that
// elect.sync guards the compiler keeps descriptors and addresses in uniform registers, and issuing a product
// costs 11 cycles instead of 50 (64 with a descriptor built for each: as long as the product takes).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int D, int POS, bool KH>
__global__ void __launch_bounds__(kThreads, 1) q4_prefill_kernel(const Q4Args a, int nmp, int long_first) {
  using L = Layout<D>;
  using Q = Q4<D>;
  constexpr bool kRotate = (POS == kRope || POS == kRopeX);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // block order: (request, head) outermost, or (few of those) the longest query blocks first
  const int split = int(blockIdx.x) % a.S;
  int u = int(blockIdx.x) / a.S, mp, g, b;
  if (long_first) {
    const int bg = u % (a.B * a.Hkv);
    mp = nmp - 1 - u / (a.B * a.Hkv);
    g = bg % a.Hkv;
    b = bg / a.Hkv;
  } else {
    mp = u % nmp;
    u /= nmp;
    g = u % a.Hkv;
    b = u / a.Hkv;
  }
  pdl_wait();
  const int G = a.Hq / a.Hkv;
  const int tpt = kM / G;  // tokens per Q tile
  const int qs = a.q_start[b];
  const bool dec = a.seq_len != nullptr;
  const int q0 = dec ? b : a.cu_q[b];
  const int Lq = dec ? 1 : a.cu_q[b + 1] - q0;
  const int mbase = dec ? a.seq_len[b] - 1 : qs;
  const int tok0 = mp * kQT * tpt;
  if (tok0 >= Lq) return;  // uniform for the CTA, before any barrier or TMEM use
  const int nq = (!KH && tok0 + tpt < Lq) ? 2 : 1;
  const int ntok = min((KH ? 1 : kQT) * tpt, Lq - tok0);
  // warps of each Q tile that hold rows (a short question leaves some without): the others only write Q
  const int live0 = (min(ntok, tpt) * G + 31) / 32, live1 = (max(ntok - tpt, 0) * G + 31) / 32;
  const int m_min = mbase + tok0, m_max = mbase + tok0 + ntok - 1;
  const int rel = m_max - qs;
  int nb = max(0, a.doc_blocks[b]) + (rel >= 0 ? rel / kPage + 1 : 0);
  if (nb > a.max_blocks) {
    if (threadIdx.x == 0) set_status(a.status, LAZY_STATUS_BAD_ROW);
    nb = a.max_blocks;
  }
  const int ntiles_all = (nb + kPagesPerTile - 1) / kPagesPerTile;
  const int chunk = (ntiles_all + a.S - 1) / a.S;
  const int t0 = split * chunk;
  const int ntiles = min(ntiles_all, t0 + chunk) - t0;
  if (ntiles <= 0) {  // nothing to see: a neutral partial, or (no split) an empty row
    for (int i = threadIdx.x; i < ntok * G; i += blockDim.x) {
      const size_t rh = (size_t)(q0 + tok0 + i / G) * a.Hq + g * G + i % G;
      if (a.S > 1) {
        a.part_ml[(rh * a.S + split) * 2] = -INFINITY;
        a.part_ml[(rh * a.S + split) * 2 + 1] = 0.f;
        for (int c = 0; c < D; ++c) a.part_o[(rh * a.S + split) * D + c] = 0.f;
      } else {
        for (int c = 0; c < D; ++c) a.out[rh * D + c] = __float2bfloat16_rn(0.f);
        if (a.lse) a.lse[rh] = -INFINITY;
      }
    }
    return;
  }

  const uint32_t sQ0 = sb, sK0 = sb + L::K_OFF, sV0 = sb + L::V_OFF;
  int* pstart = reinterpret_cast<int*>(sm + L::PSTART_OFF);
  int2* pinfo = reinterpret_cast<int2*>(sm + L::PINFO_OFF);
  int* flags = reinterpret_cast<int*>(sm + L::FLAG_OFF);
  unsigned long long* turns = reinterpret_cast<unsigned long long*>(sm + L::TURNS_OFF);
  const uint32_t bar0 = sb + L::BAR_OFF;
  auto BAR = [&](int i) { return bar0 + 8u * uint32_t(i); };
  // Stages of packed keys and values.  KH has room for more where the second Q tile would lie, and needs
  // them: its tiles are half as long, and a stage's copy takes about as long as a tile.
  constexpr int kPK = KH ? 4 : 2, kPV = KH ? 2 : 1;
  auto PKS = [&](int j) {
    const int s = j % kPK;
    return sb + uint32_t(KH && s >= 2 ? L::PK2_OFF : L::PK_OFF) + uint32_t((s & 1) * kPagesPerTile * L::PKS);
  };
  auto PVS = [&](int j) { return KH && (j & 1) ? sb + uint32_t(L::PV1_OFF) : sb + uint32_t(L::PV_OFF); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC_OFF + 4);

  volatile int* nanpos = reinterpret_cast<volatile int*>(sm + L::NANPOS_OFF);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPK; ++s) {
      mbar_init(BAR(B_PK_FULL + s), 33);
      mbar_init(BAR(B_PK_FREE + s), 128);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(BAR(B_K_READY + s), 128);
      mbar_init(BAR(B_K_FREE + s), 1);
      mbar_init(BAR(B_V_READY + s), 64);
      mbar_init(BAR(B_V_FREE + s), 1);
      mbar_init(BAR(B_S_FULL + s), 1);
      mbar_init(BAR(B_P_FULL + s), 32 * (KH ? 2 * live0 : s == 1 && nq == 2 ? live1 : live0));
      mbar_init(BAR(B_PV_FULL + s), 33);
      mbar_init(BAR(B_PV_FREE + s), 64);
    }
    mbar_init(BAR(B_Q_READY), 2 * 128);
    mbar_init(BAR(B_FINAL), 1);
    mbar_init(BAR(B_PV_DONE), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x >= 32 && threadIdx.x <= 32 + D / 16) nanpos[threadIdx.x - 32] = INT_MAX;
  if (threadIdx.x == 64) {
    nanpos[D / 16 + 1] = q0 + tok0;
    nanpos[D / 16 + 2] = g * G;
    nanpos[D / 16 + 3] = ntok;
    nanpos[D / 16 + 4] = m_min;
  }
  if constexpr (kRotate)
    for (int i = threadIdx.x; i < D / 2; i += blockDim.x) turns[i] = a.pos.turns[i];
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 8) {
    // ============================ Q operand, softmax and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<KH>::softmax));
    const int qt = warp >> 2;  // the warpgroup's Q tile, or (KH) its half of the keys
    const int r = threadIdx.x & (kM - 1);
    const int token = tok0 + (KH ? 0 : qt * tpt) + r / G;
    const int h = g * G + r % G;
    const bool valid = token < Lq && r < tpt * G;
    const int m_row = valid ? mbase + token : -1;
    float rf;  // score -> base-2 logit
    {
      // KH: both warpgroups write the one Q tile, each the chunks (pairs) of one parity
      const uint32_t sQ = sQ0 + uint32_t(KH ? 0 : qt * L::QTILE);
      auto qaddr = [&](int k) { return sQ + uint32_t((k >> 3) * L::BLK) + swz(r, k & 7); };
      const int rd = kRotate ? a.pos.rotary_dim : 0, hr = rd / 2;
      const int half = kRotate && !a.pos.interleaved ? hr / 8 : 0;  // chunk k is rotated with chunk k + half
      // whole rows by neighbouring lanes into place (a row per lane would touch 32 lines at once); KH: each
      // warpgroup half of the rows
      constexpr int CH = D / 8, RL = 32 / CH;  // chunks of a row, rows at a time
      constexpr int NR = KH ? 16 : 32;
      const int recip = (65536 + G - 1) / G;  // row * recip >> 16 = row / G for rows and G up to 128
      const int tbase = tok0 + (KH ? 0 : qt * tpt), lim = min(tpt, Lq - tbase) * G;
      uint4 in[NR / RL];
#pragma unroll
      for (int i = 0; i < NR / RL; ++i) {
        const int row = 32 * (warp & 3) + (KH ? 16 * qt : 0) + i * RL + lane / CH;
        const int tok = row * recip >> 16;
        const size_t at = ((size_t)(q0 + tbase + tok) * a.Hq + g * G + row - tok * G) * D;
        in[i] = row < lim ? *reinterpret_cast<const uint4*>(a.q + at + lane % CH * 8) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < NR / RL; ++i) {
        const int row = 32 * (warp & 3) + (KH ? 16 * qt : 0) + i * RL + lane / CH, k = lane % CH;
        st_shared_v4(sQ + uint32_t((k >> 3) * L::BLK) + swz(row, k & 7), in[i]);
      }
      if (KH) named_sync(1, 2 * kM);
      else __syncwarp();
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const uint4 x = ld_shared_v4(qaddr(k));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(xs[e] & 0x7FFFu, (xs[e] >> 16) & 0x7FFFu));
      }
      if (KH) named_sync(1, 2 * kM);  // both have read every row: it may be rotated in place
      const int ex = q4_exponent(__uint_as_float(top << 16), a.lowest_ex);
      rf = a.qk_log2 * __uint_as_float(uint32_t(127 + ex) << 23);
      const float sc = __uint_as_float(uint32_t(127 - ex) << 23);
      auto pack = [&](const float (&y)[8]) {
        return make_uint4(f2_to_h2(y[0] * sc, y[1] * sc), f2_to_h2(y[2] * sc, y[3] * sc),
                          f2_to_h2(y[4] * sc, y[5] * sc), f2_to_h2(y[6] * sc, y[7] * sc));
      };
      auto unpack = [](uint4 x, float (&y)[8]) {
        y[0] = bf_lo(x.x); y[1] = bf_hi(x.x); y[2] = bf_lo(x.y); y[3] = bf_hi(x.y);
        y[4] = bf_lo(x.z); y[5] = bf_hi(x.z); y[6] = bf_lo(x.w); y[7] = bf_hi(x.w);
      };
      constexpr int step = KH ? 2 : 1;
      const int first = KH ? qt : 0;
      if constexpr (kRotate) {
        const uint32_t m = uint32_t(max(m_row, 0));
        const bool in_table = a.pos.table != nullptr && m < uint32_t(a.pos.max_pos);
        const float* tab = in_table ? a.pos.table + (size_t)m * rd : nullptr;
        auto csf = [&](int i, float (&sn)[4], float (&co)[4]) {  // frequencies i .. i + 3
          if (tab) {
#pragma unroll
            for (int e = 0; e < 4; ++e) co[e] = tab[i + e], sn[e] = tab[hr + i + e];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) turn_sincos_fast(m, turns[i + e], sn[e], co[e]);
          }
        };
        float sn[4], co[4];
        if (!a.pos.interleaved) {
#pragma unroll 1
          for (int c = first; c < half; c += step) {
            float x1[8], x2[8], y1[8], y2[8];
            unpack(ld_shared_v4(qaddr(c)), x1);
            unpack(ld_shared_v4(qaddr(c + half)), x2);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (e % 4 == 0) csf(c * 8 + e, sn, co);
              y1[e] = x1[e] * co[e % 4] - x2[e] * sn[e % 4];
              y2[e] = x1[e] * sn[e % 4] + x2[e] * co[e % 4];
            }
            st_shared_v4(qaddr(c), pack(y1));
            st_shared_v4(qaddr(c + half), pack(y2));
          }
        } else {
#pragma unroll 1
          for (int k = first; k < rd / 8; k += step) {
            float x[8], y[8];
            unpack(ld_shared_v4(qaddr(k)), x);
            csf(k * 4, sn, co);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              y[2 * w] = x[2 * w] * co[w] - x[2 * w + 1] * sn[w];
              y[2 * w + 1] = x[2 * w] * sn[w] + x[2 * w + 1] * co[w];
            }
            st_shared_v4(qaddr(k), pack(y));
          }
        }
      }
#pragma unroll 1
      for (int k = rd / 8 + (KH ? (rd / 8 + qt) & 1 : 0); k < D / 8; k += step) {
        float x[8];
        unpack(ld_shared_v4(qaddr(k)), x);
        st_shared_v4(qaddr(k), pack(x));
      }
      fence_async_smem();
      mbar_arrive(BAR(B_Q_READY));
    }
    const int live = KH || qt == 0 ? live0 : live1;
    float2* xml = reinterpret_cast<float2*>(sm + L::XML_OFF);
    if ((warp & 3) < live) {
      bool ok = true;
      const float2 rf2 = make_float2(rf, rf);
      float slope = 0.f;
      if constexpr (POS == kAlibi)
        if (a.pos.slopes && valid) slope = a.pos.slopes[h] * 1.4426950408889634f;
      const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
      const uint32_t tO = tl + uint32_t(2 * kN + qt * 128);
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < ntiles && ok; ++j) {
        const int slot = j % kSlots;
        const int buf = nq == 2 ? qt : (j & 1);
        const uint32_t tS = tl + uint32_t(buf * kN);
        const bool got_s =
            wait_bar(BAR(B_S_FULL + buf), uint32_t(nq == 2 ? (j & 1) : ((j >> 1) & 1)), abort_flag, a.status);
        if (!__all_sync(0xffffffffu, got_s)) { ok = false; break; }
        tc_fence_after();
        const bool fast = flags[slot * 2] != 0;
        constexpr int NK = KH ? kN / 2 : kN, NPG = NK / kPage;
        const int pg0 = KH ? NPG * qt : 0;
        uint32_t v[NK];
#pragma unroll
        for (int c = 0; c < NK / 32; ++c)
          tmem_ld32(tS + uint32_t(pg0 * kPage + 32 * c), *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
        tmem_wait_ld();
        // ALiBi: the scores become logits here, the per-key part slope t of the bias added; its per-page
        // part slope (pstart - m) goes onto the page's maximum and exponent offset
        float bpg[NPG];
        if constexpr (POS == kAlibi) {
#pragma unroll
          for (int pp = 0; pp < NPG; ++pp) {
            bpg[pp] = slope * float(pstart[slot * kPagesPerTile + pg0 + pp] - m_row);
#pragma unroll
            for (int t = 0; t < kPage; t += 2) {
              float2 x = make_float2(__uint_as_float(v[pp * kPage + t]), __uint_as_float(v[pp * kPage + t + 1]));
              x = __ffma2_rn(x, rf2, make_float2(slope * float(t), slope * float(t + 1)));
              v[pp * kPage + t] = __float_as_uint(x.x);
              v[pp * kPage + t + 1] = __float_as_uint(x.y);
            }
          }
        }
        if (!fast) {  // row t of a page holds key p = pstart + t; visible iff t < rows and p <= m
#pragma unroll
          for (int pp = 0; pp < NPG; ++pp) {
            const int hi = min(pinfo[slot * kPagesPerTile + pg0 + pp].y,
                               m_row - pstart[slot * kPagesPerTile + pg0 + pp] + 1);
#pragma unroll
            for (int t = 0; t < kPage; ++t)
              if (t >= hi) v[pp * kPage + t] = __float_as_uint(-INFINITY);
          }
        }
        float mq[NPG];
#pragma unroll
        for (int q = 0; q < NPG; ++q) {
          const float* x = reinterpret_cast<const float*>(v + 16 * q);
          float m = max3f(x[0], x[1], x[2]);
#pragma unroll
          for (int e = 3; e < 15; e += 2) m = max3f(m, x[e], x[e + 1]);
          mq[q] = fmaxf(m, x[15]);
          if constexpr (POS == kAlibi) mq[q] += bpg[q];
        }
        float mx;
        if constexpr (KH)
          mx = max3f(max3f(mq[0], mq[1], mq[2]), mq[3], mq[3]);
        else
          mx = max3f(max3f(mq[0], mq[1], mq[2]), max3f(mq[3], mq[4], mq[5]), fmaxf(mq[6], mq[7]));
        if constexpr (POS != kAlibi) mx *= rf;  // rf > 0
        const bool need = mx > m_run + kTau;
        const float m_new = need ? mx : m_run;
        const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
        float2 mneg[NPG];
#pragma unroll
        for (int pp = 0; pp < NPG; ++pp) {
          const float o = POS == kAlibi ? bpg[pp] - m_use + kPOff : kPOff - m_use;
          mneg[pp] = make_float2(o, o);
        }
        float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                          make_float2(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < NK / 2; ++e) {
          float2 x = make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
          if constexpr (POS == kAlibi)
            x = __fadd2_rn(x, mneg[e / (kPage / 2)]);
          else
            x = __ffma2_rn(x, rf2, mneg[e / (kPage / 2)]);
          const float2 ev = make_float2(ex2(x.x), ex2(x.y));
          sum4[e & 3] = __fadd2_rn(sum4[e & 3], ev);
          v[e] = f2_to_h2(ev.x, ev.y);
        }
        const float2 s01 = __fadd2_rn(sum4[0], sum4[1]), s23 = __fadd2_rn(sum4[2], sum4[3]);
        const float2 s03 = __fadd2_rn(s01, s23);
        const float sum = s03.x + s03.y;
        const float alpha = (j > 0 && need && m_run != -INFINITY) ? ex2(m_run - m_new) : 1.f;
        l_run = (j == 0) ? sum : l_run * alpha + sum;
        if (nq == 1 && j > 0) {  // S of tile j was issued before PV of tile j - 1: the rescale waits for it
          const bool got_pv = wait_bar(BAR(B_PV_DONE), uint32_t((j - 1) & 1), abort_flag, a.status);
          if (!__all_sync(0xffffffffu, got_pv)) { ok = false; break; }
          tc_fence_after();
        }
        if (__any_sync(0xffffffffu, j > 0 && alpha != 1.f)) {
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
        for (int c = 0; c < NK / 64; ++c)
          tmem_st32(tS + uint32_t(pg0 * kPage + 32 * c), *reinterpret_cast<const uint32_t(*)[32]>(v + 32 * c));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR(B_P_FULL + buf));
      }
      const bool got_last = ok && wait_bar(BAR(B_FINAL), 0, abort_flag, a.status);
      const size_t rh = (size_t)(q0 + token) * a.Hq + h;
      const size_t pi = rh * a.S + split;
      // 32 output columns of this row: scaled partials (S > 1) or the bf16 result
      auto store = [&](int col, const float (&o)[32]) {
        if (a.S > 1) {
          float4* dst = reinterpret_cast<float4*>(a.part_o + pi * D + col);
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4) dst[q4] = make_float4(o[4 * q4], o[4 * q4 + 1], o[4 * q4 + 2], o[4 * q4 + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(a.out + rh * D + col);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
            dst[q4] = make_uint4(f2_to_bf2(o[8 * q4], o[8 * q4 + 1]), f2_to_bf2(o[8 * q4 + 2], o[8 * q4 + 3]),
                                 f2_to_bf2(o[8 * q4 + 4], o[8 * q4 + 5]), f2_to_bf2(o[8 * q4 + 6], o[8 * q4 + 7]));
        }
      };
      auto store_ml = [&](float M, float l) {
        if (a.S > 1) {
          a.part_ml[pi * 2] = l != 0.f ? M - kPOff : -INFINITY;
          a.part_ml[pi * 2 + 1] = l;
        } else if (a.lse) {
          a.lse[rh] = (M + log2f(l) - kPOff) * 0.6931471805599453f;
        }
      };
      if constexpr (KH) {
        // the key halves' partial softmaxes, merged by their maxima and sums (exchanged in the unused
        // second Q tile); each warpgroup writes half of the columns
        xml[qt * kM + r] = make_float2(l_run != 0.f ? m_run : -INFINITY, l_run);
        named_sync(1, 64 * live0);
        const float2 mine = xml[qt * kM + r], other = xml[(qt ^ 1) * kM + r];
        const float2 hA = qt == 0 ? mine : other, hB = qt == 0 ? other : mine;
        const float M = fmaxf(hA.x, hB.x);
        const float wA = hA.y != 0.f ? ex2(hA.x - M) : 0.f, wB = hB.y != 0.f ? ex2(hB.x - M) : 0.f;
        const float Lt = wA * hA.y + wB * hB.y;
        if (__all_sync(0xffffffffu, got_last)) {
          tc_fence_after();
          const float inv = a.S > 1 ? a.v_factor : (Lt != 0.f ? a.v_factor / Lt : 0.f);
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            const int col = qt * (D / 2) + c * 32;
            uint32_t oa[32], ob[32];
            tmem_ld32(tl + uint32_t(2 * kN + col), oa);
            tmem_ld32(tl + uint32_t(3 * kN + col), ob);
            tmem_wait_ld();
            float o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = (wA * __uint_as_float(oa[e]) + wB * __uint_as_float(ob[e])) * inv;
            if (valid) store(col, o);
          }
          if (valid && qt == 0) store_ml(M, Lt);
        }
      } else if (__all_sync(0xffffffffu, got_last)) {
        tc_fence_after();
        const float inv = a.S > 1 ? a.v_factor : (l_run != 0.f ? a.v_factor / l_run : 0.f);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t oa[32];
          tmem_ld32(tO + uint32_t(c * 32), oa);
          tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(oa[e]) * inv;
          if (valid) store(c * 32, o);
        }
        if (valid) store_ml(m_run, l_run);
      }
    }
  } else if (warp < kProdWarp) {
    // ============================ dequantisation
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<KH>::deq));
    const int rt = threadIdx.x - kDeqWarp0 * 32;
    const int ps = rt / kPage, l = rt % kPage;  // page slot, thread of the page
    constexpr int NCP = D / 16;                 // runs of 8 dimensions in half a row
    bool ok = true;  // once a wait gives up, the thread skips work but keeps arriving
    uint32_t co[4], sn[4], nsn[4];  // f16 pairs
    int cur_delta = -1;
    int g_kind = 3, g_chunk = 0, g_part = 0, g_f0 = 0;
    if constexpr (POS == kRopeX) {
      // one task per thread, all 16 rows: a rotated chunk pair (kind 0), an interleaved chunk (1), or a
      // chunk beyond rotary_dim (2)
      const int rd = a.pos.rotary_dim;
      const int nrot = a.pos.interleaved ? rd / 8 : rd / 16, ntail = (D - rd) / 8;
      if (l < nrot) {
        g_kind = a.pos.interleaved ? 1 : 0;
        g_chunk = l;
        g_part = l + rd / 16;
        g_f0 = a.pos.interleaved ? 4 * l : 8 * l;
      } else if (l < nrot + ntail) {
        g_kind = 2;
        g_chunk = rd / 8 + (l - nrot);
      }
    }
    auto keys = [&](int j) {
      const int s = j & 1, slot = j % kSlots;
      if (ok) ok = wait_bar(BAR(B_PK_FULL + j % kPK), uint32_t((j / kPK) & 1), abort_flag, a.status);
      if (ok && j >= 2) ok = wait_bar(BAR(B_K_FREE + s), uint32_t(((j >> 1) - 1) & 1), abort_flag, a.status);
      const int2 pi = ok ? pinfo[slot * kPagesPerTile + ps] : make_int2(0, 0);
      if (pi.y > 0) {  // rows past the page's keys are converted too (their scores are masked)
        const uint32_t src = PKS(j) + uint32_t(ps * L::PKS);
        const uint32_t sK = sK0 + uint32_t(s * L::TILE);
        if constexpr (POS != kRopeX) {
          constexpr int HG = 16 / NCP;  // row groups
          const int c = l % NCP, hg = l / NCP;
          if constexpr (POS == kRope) {
            if (pi.x != cur_delta) {
              cur_delta = pi.x;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                float s0, c0, s1, c1;
                turn_sincos_fast(uint32_t(pi.x), turns[8 * c + 2 * w], s0, c0);
                turn_sincos_fast(uint32_t(pi.x), turns[8 * c + 2 * w + 1], s1, c1);
                co[w] = f2_to_h2(c0, c1);
                sn[w] = f2_to_h2(s0, s1);
                nsn[w] = f2_to_h2(-s0, -s1);
              }
            }
          }
          // Two rows (r7, r7 + 8) a time, the next ones' words loaded ahead.  The loop stays rolled: five
          // roles run different code at once, and unrolled they miss the instruction cache (a third of
          // all stalls).  KH, which waits for its keys, takes two steps at once (31.3 us against 33.7 rolled
          // and 31.9 with all four; 16 x 32 queries of 32 heads over 2000 keys).
          constexpr int NI = 8 / HG;
          const uint32_t wsrc = src + hg * (D / 2) + c * 4;
          const uint32_t ssrc = src + Q::KS + (D == 128 ? (hg * 4 + (c >> 2)) * 4 : (hg * 4 + (c >> 1)) * 2);
          auto load = [&](int i, uint32_t (&w)[6]) {  // codes of both rows, first run and its partner; scales
            const uint32_t x = wsrc + i * HG * (D / 2);
            w[0] = ld_shared_u32(x);
            w[1] = ld_shared_u32(x + D / 4);
            w[2] = ld_shared_u32(x + 4 * D);
            w[3] = ld_shared_u32(x + 4 * D + D / 4);
            const uint32_t y = ssrc + i * HG * (D == 128 ? 16 : 8);
            w[4] = D == 128 ? ld_shared_u32(y) : ld_shared_u16(y);
            w[5] = D == 128 ? ld_shared_u32(y + 8) : ld_shared_u16(y + 4);
          };
          // D = 128: a word holds two groups of row r7, then of r7 + 8; D = 64: one group of each
          const uint32_t sel_a = D == 128 ? ((c >> 1) & 1 ? 0x3232u : 0x1010u) : 0x1010u;
          const uint32_t sel_b = D == 128 ? sel_a : 0x3232u;
          uint32_t nxt[6];
          load(0, nxt);
          // rows r7 + 8 lie 1024 bytes on, equally swizzled
#pragma unroll (KH ? 2 : 1)
          for (int i = 0; i < NI; ++i) {
            uint32_t cur[6];
#pragma unroll
            for (int e = 0; e < 6; ++e) cur[e] = nxt[e];
            if (i + 1 < NI) load(i + 1, nxt);
            const uint32_t a1 = sK + swz(ps * kPage + hg + HG * i, c);
            const uint32_t a2 = (D == 128) ? a1 + uint32_t(L::BLK) : sK + swz(ps * kPage + hg + HG * i, c + 4);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t sel = hh ? sel_b : sel_a;
              auto two = [&](uint32_t w) { return e4m3x2_to_h2(D == 128 && hh ? w >> 16 : w & 0xFFFFu); };
              const uint32_t sc1 = __byte_perm(two(cur[4]), 0, sel), sc2 = __byte_perm(two(cur[5]), 0, sel);
              uint32_t x1[4], x2[4];
              e2m1x8_to_h2(cur[2 * hh], x1);
              e2m1x8_to_h2(cur[2 * hh + 1], x2);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t p1 = hmul2(x1[w], sc1), p2 = hmul2(x2[w], sc2);
                if constexpr (POS == kRope) {
                  x1[w] = hfma2(p2, nsn[w], hmul2(p1, co[w]));  // x1 c - x2 s
                  x2[w] = hfma2(p2, co[w], hmul2(p1, sn[w]));   // x1 s + x2 c
                } else {
                  x1[w] = p1;
                  x2[w] = p2;
                }
              }
              st_shared_v4(a1 + hh * 1024, make_uint4(x1[0], x1[1], x1[2], x1[3]));
              st_shared_v4(a2 + hh * 1024, make_uint4(x2[0], x2[1], x2[2], x2[3]));
            }
          }
        } else {
          auto chunk8 = [&](int t, int k, uint32_t (&x)[4]) {  // 8 scaled values: row t, dimensions 8k ..
            e2m1x8_to_h2(ld_shared_u32(src + t * (D / 2) + k * 4), x);
            const uint32_t sc = __byte_perm(e4m3x2_to_h2(ld_shared_u8(src + Q::k_scale(t, k >> 1))), 0, 0x1010);
#pragma unroll
            for (int w = 0; w < 4; ++w) x[w] = hmul2(x[w], sc);
          };
          auto put = [&](int t, int k, const uint32_t (&x)[4]) {
            st_shared_v4(sK + uint32_t((k >> 3) * L::BLK) + swz(ps * kPage + t, k & 7),
                         make_uint4(x[0], x[1], x[2], x[3]));
          };
          if (g_kind < 2 && pi.x != cur_delta) {
            cur_delta = pi.x;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              float s0, c0, s1, c1;
              if (g_kind == 0) {
                turn_sincos_fast(uint32_t(pi.x), turns[g_f0 + 2 * w], s0, c0);
                turn_sincos_fast(uint32_t(pi.x), turns[g_f0 + 2 * w + 1], s1, c1);
                co[w] = f2_to_h2(c0, c1);
                sn[w] = f2_to_h2(s0, s1);
                nsn[w] = f2_to_h2(-s0, -s1);
              } else {
                turn_sincos_fast(uint32_t(pi.x), turns[g_f0 + w], s0, c0);
                co[w] = f2_to_h2(c0, c0);
                sn[w] = f2_to_h2(-s0, s0);
              }
            }
          }
#pragma unroll 1
          for (int t = 0; t < kPage && g_kind < 3; ++t) {
            uint32_t x1[4], x2[4];
            chunk8(t, g_chunk, x1);
            if (g_kind == 0) {
              chunk8(t, g_part, x2);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t p1 = x1[w], p2 = x2[w];
                x1[w] = hfma2(p2, nsn[w], hmul2(p1, co[w]));
                x2[w] = hfma2(p2, co[w], hmul2(p1, sn[w]));
              }
              put(t, g_part, x2);
            } else if (g_kind == 1) {  // pairs inside a register: (x0 c - x1 s, x1 c + x0 s)
#pragma unroll
              for (int w = 0; w < 4; ++w)
                x1[w] = hfma2(__byte_perm(x1[w], 0, 0x1032), sn[w], hmul2(x1[w], co[w]));
            }
            put(t, g_chunk, x1);
          }
        }
      }
      fence_async_smem();
      mbar_arrive(BAR(B_PK_FREE + j % kPK));
      mbar_arrive(BAR(B_K_READY + s));
    };
    for (int j = 0; j < ntiles; ++j) keys(j);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<KH>::issue));
    if (warp == kProdWarp) {
      // ============================ block words and copies: K0 K1 V0 K2 V1 ... (KH: K0 K1 K2 V0 K3 V1 ...)
      const uint64_t* mrow = a.meta + (size_t)b * a.max_blocks;
      // ALiBi visits the tiles newest first: the first tile then fixes each row's running maximum
      auto tile_of = [&](int j) { return POS == kAlibi ? t0 + ntiles - 1 - j : t0 + j; };
      // block words of four tiles at a time, one per lane, fetched four tiles before they are needed (a load
      // takes about as long as a tile)
      auto fetch = [&](int j) -> uint64_t {
        j += lane / kPagesPerTile;
        const int jb = tile_of(j) * kPagesPerTile + lane % kPagesPerTile;
        return (j < ntiles && jb < nb) ? ldg_u64(mrow + jb) : 0ull;
      };
      uint64_t words = 0, words_next = fetch(0);
      const int page = lane >> 2;  // the lane's page of a tile
      const uint8_t* ahead[kPK] = {};  // this lane's blocks of the tiles whose values are to come (null: none)
      // Half a block (keys or values) by four lanes, 16 bytes a time: 9 D / 64 instructions per tile.  One bulk
      // copy per page would be issued lane by lane, at 84 cycles each: 1340 of a tile's 2700.
      auto copy = [&](uint32_t dst, const uint8_t* src, uint32_t full) {
        if (src) {
#pragma unroll
          for (int i = 0; i < Q::VC / 64; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + uint32_t(64 * i + 16 * (lane & 3))),
                         "l"(src + 64 * i + 16 * (lane & 3))
                         : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(full);  // releases the tile's metadata too
      };
      auto issue_k = [&](int j) -> bool {
        const int slot = j % kSlots;
        const uint32_t full = BAR(B_PK_FULL + j % kPK);
        if (j % 4 == 0) {
          words = words_next;
          words_next = fetch(j + 4);
        }
        const uint64_t w = __shfl_sync(0xffffffffu, words, j % 4 * kPagesPerTile + page);
        int rows = 0, start = 0, delta = 0;
        const int jb = tile_of(j) * kPagesPerTile + page;
        const uint8_t* blk = nullptr;
        if (jb < nb) {
          delta = int(word_delta(w));
          start = delta + kPage * int(word_pg(w));
          rows = q4_rows(w, m_max);
          if (word_page(w) >= uint32_t(a.num_pages)) {
            set_status(a.status, LAZY_STATUS_BAD_PAGE);
            rows = 0;
          }
          if (rows > 0) blk = a.cache + ((size_t)word_page(w) * a.Hkv + g) * Q::BYTES;
        }
        if (j >= kPK) {
          const bool freed = wait_bar(BAR(B_PK_FREE + j % kPK), uint32_t((j / kPK - 1) & 1), abort_flag, a.status);
          if (!__all_sync(0xffffffffu, freed)) return false;
        }
        if ((lane & 3) == 0) {
          pinfo[slot * kPagesPerTile + page] = make_int2(delta, rows);
          pstart[slot * kPagesPerTile + page] = start;
        }
        // every key visible to every row: full pages that end at or before the first row's position
        const int seen = __all_sync(0xffffffffu, rows == kPage && start + kPage - 1 <= m_min);
        if (lane == 0) flags[slot * 2] = seen;
        copy(PKS(j) + uint32_t(page * L::PKS), blk, full);
        ahead[kPK - 1] = blk;
        return true;
      };
      auto issue_v = [&](int j) -> bool {
        const uint32_t full = BAR(B_PV_FULL + j % kPV);
        if (j >= kPV) {
          const bool freed = wait_bar(BAR(B_PV_FREE + j % kPV), uint32_t((j / kPV - 1) & 1), abort_flag, a.status);
          if (!__all_sync(0xffffffffu, freed)) return false;
        }
        const uint8_t* blk = ahead[0];
        copy(PVS(j) + uint32_t(page * L::PVS), blk ? blk + Q::VC : nullptr, full);
        return true;
      };
      bool ok = true;
      for (int i = 0; i < kPK - 1 + ntiles && ok; ++i) {  // keys of tile i, values of tile i - (kPK - 1)
        const int j = i - (kPK - 1);
#pragma unroll
        for (int e = 0; e < kPK - 1; ++e) ahead[e] = ahead[e + 1];
        if (KH && j >= 0) ok = issue_v(j);
        if (ok && i < ntiles) ok = issue_k(i);
        if (!KH && ok && j >= 0) ok = issue_v(j);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // never leave copies in flight
    } else if (warp == kMmaWarp) {
      // ============================ MMA issue (one thread)
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      if (elect_one()) {
        const uint64_t dQ = sdesc(sQ0, 16, 1024), dK = sdesc(sK0, 16, 1024), dV = sdesc(sV0, L::BLK, 1024);
        // no carry out of the address field: shared addresses end below 2^18
        auto at = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };
        constexpr uint32_t IQK = idesc_mma(kM, kN, 0, 1);
        constexpr uint32_t IPV = idesc_mma(kM, D, 1, 1);
        bool ok = wait_bar(BAR(B_Q_READY), 0, abort_flag, a.status);
        auto wait = [&](int bar, int phase) -> bool {
          return wait_bar(BAR(bar), uint32_t(phase & 1), abort_flag, a.status);
        };
        auto qk = [&](int qt, int j, int buf) {  // S_buf = Q_qt K_j^T
          const uint64_t d = at(dK, uint32_t((j & 1) * L::TILE)), e = at(dQ, uint32_t(qt * L::QTILE));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = uint32_t((kk >> 2) * L::BLK + (kk & 3) * 32);
            mma_bf16(tm + uint32_t(buf * kN), at(e, off), at(d, off), IQK, kk > 0 ? 1u : 0u);
          }
          mma_commit(BAR(B_S_FULL + buf));
        };
        auto pv = [&](int qt, int jj) {  // O_qt += P_qt V_jj
          const uint64_t d = at(dV, uint32_t((jj & 1) * L::TILE));
#pragma unroll
          for (int kk = 0; kk < kN / 16; ++kk)
            mma_ts(tm + uint32_t(2 * kN + qt * 128), tm + uint32_t(qt * kN + kk * 8),
                   at(d, uint32_t(kk * 16 * 128)), IPV, (jj > 0 || kk > 0) ? 1u : 0u);
        };
        if (nq == 1) {
          // one live Q tile: QK(0) QK(1) | PV(0) QK(2) | PV(1) ...
          auto qk1 = [&](int j) -> bool {
            if (!wait(B_K_READY + (j & 1), j >> 1)) return false;
            tc_fence_after();
            qk(0, j, j & 1);
            mma_commit(BAR(B_K_FREE + (j & 1)));
            return true;
          };
          if (ok) ok = qk1(0);
          if (ok && ntiles > 1) ok = qk1(1);
          for (int j = 0; j < ntiles && ok; ++j) {
            ok = wait(B_P_FULL + (j & 1), j >> 1) && wait(B_V_READY + (j & 1), j >> 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t d = at(dV, uint32_t((j & 1) * L::TILE));
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk) {
              const int hk = KH ? kk / 4 : 0;
              const uint32_t pcol = uint32_t((j & 1) * kN + (KH ? 64 * hk + (kk % 4) * 8 : kk * 8));
              mma_ts(tm + uint32_t((2 + hk) * kN), tm + pcol, at(d, uint32_t(kk * 16 * 128)),
                     IPV, (j > 0 || kk > (KH ? 4 * hk : 0)) ? 1u : 0u);
            }
            mma_commit(BAR(B_PV_DONE));
            mma_commit(BAR(B_V_FREE + (j & 1)));
            if (j + 2 < ntiles) ok = qk1(j + 2);
          }
        } else {
          if (ok) ok = wait(B_K_READY, 0);
          if (ok) {
            tc_fence_after();
            qk(0, 0, 0);
            qk(1, 0, 1);
            mma_commit(BAR(B_K_FREE));
          }
          for (int j = 1; j < ntiles && ok; ++j) {
            const int s = j & 1, sp = (j - 1) & 1;
            ok = wait(B_P_FULL, j - 1) && wait(B_V_READY + sp, (j - 1) >> 1);
            if (!ok) break;
            tc_fence_after();
            pv(0, j - 1);
            ok = wait(B_K_READY + s, j >> 1);
            if (!ok) break;
            tc_fence_after();
            qk(0, j, 0);
            ok = wait(B_P_FULL + 1, j - 1);
            if (!ok) break;
            tc_fence_after();
            pv(1, j - 1);
            mma_commit(BAR(B_V_FREE + sp));
            qk(1, j, 1);
            mma_commit(BAR(B_K_FREE + s));
          }
          if (ok) {
            const int jl = ntiles - 1;
            ok = wait(B_P_FULL, jl) && wait(B_V_READY + (jl & 1), jl >> 1);
            if (ok) {
              tc_fence_after();
              pv(0, jl);
              ok = wait(B_P_FULL + 1, jl);
            }
            if (ok) {
              tc_fence_after();
              pv(1, jl);
              mma_commit(BAR(B_V_FREE + (jl & 1)));
            }
          }
        }
        // every MMA must be complete before TMEM is released (and before the epilogue reads O)
        mma_commit(BAR(B_FINAL));
        WaitClock clk;
        while (!mbar_test(BAR(B_FINAL), 0) && !clk.expired()) {
        }
      }
      __syncwarp();
    } else if (warp >= kValWarp0) {
      // ============================ values: packed -> f16, 8 threads per page
      const int rt = threadIdx.x - kValWarp0 * 32;
      const int ps = rt >> 3, l = rt & 7, t = l & 3;
      bool ok = true;
      for (int j = 0; j < ntiles; ++j) {
        const int s = j & 1, slot = j % kSlots;
        if (ok) ok = wait_bar(BAR(B_PV_FULL + j % kPV), uint32_t((j / kPV) & 1), abort_flag, a.status);
        const uint32_t src = PVS(j) + uint32_t(ps * L::PVS);
        const uint32_t csrc = src + (l >> 2) * 64 + t * 16, ssrc = src + 8 * D + (D == 128 ? l >> 2 : 0) * 16 + t * 4;
        // rows without a key (and page slots without a page) become zeros: their scales are replaced by 0
        const int rr = (ok ? pinfo[slot * kPagesPerTile + ps].y : 0) - 2 * t;
        const uint32_t keep = (rr > 0 ? 0xFFu : 0u) | (rr > 1 ? 0xFF00u : 0u) | (rr > 8 ? 0xFF0000u : 0u) |
                              (rr > 9 ? 0xFF000000u : 0u);  // scale bytes: rows 2t, 2t + 1, 2t + 8, 2t + 9
        if (a.seq_len == nullptr) {  // a decode's one row sees every key that is kept
          constexpr uint32_t step = D == 128 ? 32 : 16;  // between this thread's scale words
          auto nan_bits = [](uint32_t sw) { return ((sw & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; };  // 0x7F, 0xFF
          uint32_t any = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) any |= nan_bits(ld_shared_u32(ssrc + k * step) & keep);
          if (any) {
            const int page0 = pstart[slot * kPagesPerTile + ps];
            int* first = const_cast<int*>(nanpos);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              const uint32_t sw = ld_shared_u32(ssrc + k * step), bits = nan_bits(sw & keep);
              if (bits == 0) continue;
              const int byte = (__ffs(int(bits)) - 1) >> 3, p = page0 + 2 * t + (byte & 1) + (byte >> 1) * 8;
              atomicMin(first + (D == 128 ? (l >> 2) + 2 * k : k), p);
              atomicMin(first + D / 16, p);
              st_shared_u32(ssrc + k * step, sw & ~((bits >> 7) * 0xFFu));  // D = 64: the same by both lanes
            }
          }
        }
        if (ok && j >= 2) ok = wait_bar(BAR(B_V_FREE + s), uint32_t(((j >> 1) - 1) & 1), abort_flag, a.status);
        if (ok) {
          const uint32_t sV = sV0 + uint32_t(s * L::TILE);
          auto put = [&](int row, int cb, int ch, uint32_t codes, uint32_t scale) {
            uint32_t x[4];
            e2m1x8_to_h2(codes, x);
            st_shared_v4(sV + uint32_t(cb * L::BLK) + swz(ps * kPage + row, ch),
                         make_uint4(hmul2(x[0], scale), hmul2(x[1], scale), hmul2(x[2], scale), hmul2(x[3], scale)));
          };
          if constexpr (D == 128) {
            // groups q = l / 4 + 2 k; odd ones store their odd row first: no two lanes share a bank
            const int odd = l >> 2;
            const uint32_t sela = odd ? 0x3232 : 0x1010, selb = odd ? 0x1010 : 0x3232;
            uint4 n0 = ld_shared_v4(csrc), n1 = ld_shared_v4(csrc + 512);
            uint32_t ns = ld_shared_u32(ssrc);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              const uint4 x[2] = {n0, n1};
              const uint32_t sw = ns & keep;
              if (k < 3) {
                n0 = ld_shared_v4(csrc + (k + 1) * 128);
                n1 = ld_shared_v4(csrc + (k + 1) * 128 + 512);
                ns = ld_shared_u32(ssrc + (k + 1) * 32);
              }
              const int q = odd + 2 * k, ch = (2 * q) & 7;
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t hs = e4m3x2_to_h2(half ? sw >> 16 : sw & 0xFFFFu);
                const uint32_t a0 = odd ? x[half].z : x[half].x, a1 = odd ? x[half].w : x[half].y;
                const uint32_t b0 = odd ? x[half].x : x[half].z, b1 = odd ? x[half].y : x[half].w;
                const uint32_t sa = __byte_perm(hs, 0, sela), sc = __byte_perm(hs, 0, selb);
                const int ra = half * 8 + 2 * t + odd, rb = half * 8 + 2 * t + 1 - odd;
                put(ra, q >> 2, ch, a0, sa);
                put(rb, q >> 2, ch, b0, sc);
                put(ra, q >> 2, ch + 1, a1, sa);
                put(rb, q >> 2, ch + 1, b1, sc);
              }
            }
          } else {
            uint4 n0 = ld_shared_v4(csrc);
            uint32_t ns = ld_shared_u32(ssrc);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {  // runs of 8 dimensions gd = l / 4 + 2 k
              const uint4 x = n0;
              const uint32_t sw = ns & keep;
              if (k < 3) {
                n0 = ld_shared_v4(csrc + (k + 1) * 128);
                ns = ld_shared_u32(ssrc + (k + 1) * 16);
              }
              const int gd = (l >> 2) + 2 * k;
              const uint32_t h0 = e4m3x2_to_h2(sw & 0xFFFFu), h1 = e4m3x2_to_h2(sw >> 16);
              put(2 * t, 0, gd, x.x, __byte_perm(h0, 0, 0x1010));
              put(2 * t + 1, 0, gd, x.y, __byte_perm(h0, 0, 0x3232));
              put(2 * t + 8, 0, gd, x.z, __byte_perm(h1, 0, 0x1010));
              put(2 * t + 9, 0, gd, x.w, __byte_perm(h1, 0, 0x3232));
            }
          }
        }
        fence_async_smem();
        mbar_arrive(BAR(B_PV_FREE + j % kPV));
        mbar_arrive(BAR(B_V_READY + s));
      }
      __syncwarp();
    }
  }

  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  // NaN over the columns where a row sees one (the row's sizes come out of shared memory: kept in registers they
  // would be spilled by every role)
  if (warp < 8 && nanpos[D / 16] != INT_MAX) {
    const int G = a.Hq / a.Hkv, r0 = nanpos[D / 16 + 1], h0 = nanpos[D / 16 + 2], m0 = nanpos[D / 16 + 4];
    const int n = nanpos[D / 16 + 3] * G * D;
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += 256) {
      const int c = i % D, t = i / D / G, h = i / D % G;
      if (m0 + t < nanpos[c / 16]) continue;
      const size_t rh = (size_t)(r0 + t) * a.Hq + h0 + h;
      if (a.S > 1)
        a.part_o[(rh * a.S + int(blockIdx.x) % a.S) * D + c] = NAN;
      else
        a.out[rh * D + c] = __float2bfloat16_rn(NAN);
    }
  }
}

}  // namespace tcq

namespace {

template <int D, int POS, bool KH>
int launch_q4_tc(const Q4Args& a, int max_q, cudaStream_t st) {
  using L = tcq::Layout<D>;
  auto kern = tcq::q4_prefill_kernel<D, POS, KH>;
  // the setmaxnreg split is only valid for a launch with exactly kRegsLaunch registers per thread
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    LAZY_CUDA_TRY(cudaFuncGetAttributes(&fa, kern));
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != tcq::kRegsLaunch)
    return fail(LAZY_ECUDA, "4-bit prefill kernel built with %d registers per thread, expected %d", regs.load(),
                tcq::kRegsLaunch);
  static std::atomic<uint64_t> done{0};
  LAZY_CUDA_TRY(q4_smem_limit(kern, L::SMEM, done));
  const int rows_tok = tcq::kQT * (tcq::kM / (a.Hq / a.Hkv));
  const long long nmp = ((long long)max_q + rows_tok - 1) / rows_tok;
  const long long pairs = (long long)a.B * a.Hkv;
  if (pairs > 0x7FFFFFFFll || nmp * a.S > 0x7FFFFFFFll / pairs)
    return fail(LAZY_ERANGE, "too many query rows (B=%d, max_q=%d)", a.B, max_q);
  LAZY_CUDA_TRY(launch_pdl(kern, dim3(unsigned(pairs * nmp * a.S)), dim3(tcq::kThreads), L::SMEM, st, a, int(nmp),
                           int(pairs < sm_count())));
  return LAZY_OK;
}

template <bool KH>
int dispatch_q4_tc(int D, int kind, const Q4Args& a, int max_q, cudaStream_t st) {
  if (D == 128) {
    if (kind == kRope) return launch_q4_tc<128, kRope, KH>(a, max_q, st);
    if (kind == kRopeX) return launch_q4_tc<128, kRopeX, KH>(a, max_q, st);
    return launch_q4_tc<128, kAlibi, KH>(a, max_q, st);
  }
  if (kind == kRope) return launch_q4_tc<64, kRope, KH>(a, max_q, st);
  if (kind == kRopeX) return launch_q4_tc<64, kRopeX, KH>(a, max_q, st);
  return launch_q4_tc<64, kAlibi, KH>(a, max_q, st);
}

}  // namespace

// The tensor-core kernel holds whole tokens in 128-row tiles, the rest of the rows empty.
bool q4_use_tc(int Hq, int Hkv) { return Hq / Hkv <= tcq::kM; }

// Key splits of a decode on it: one wave of CTAs, at least two tiles of 128 keys each.
int q4_tc_splits(int B, int Hkv, int max_blocks) {
  const int tiles = (max_blocks + tcq::kPagesPerTile - 1) / tcq::kPagesPerTile;
  const long long units = (long long)B * Hkv;
  return int(max(1ll, min(min((long long)sm_count() / max(units, 1ll), tiles / 2ll), 64ll)));
}

int run_q4_tc(Q4Args& a, int D, int max_q, cudaStream_t st) {
  int kind = a.pos.kind == kYarn ? kRope : a.pos.kind;
  if (kind == kRope && (a.pos.rotary_dim != D || a.pos.interleaved)) kind = kRopeX;
  if (kind == kNone) {  // no rotation and no bias: the ALiBi kernel with slope 0
    kind = kAlibi;
    a.pos.slopes = nullptr;
  }
  // every CTA has one live Q tile: its keys are shared by the two softmax warpgroups
  if (a.seq_len || max_q <= tcq::kM / (a.Hq / a.Hkv)) return dispatch_q4_tc<true>(D, kind, a, max_q, st);
  return dispatch_q4_tc<false>(D, kind, a, max_q, st);
}

}  // namespace lazykv
