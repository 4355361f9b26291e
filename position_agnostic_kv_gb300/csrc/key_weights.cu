// The attention weight that every cached key receives: w_k = sum over query rows i and heads h of
// 2^(s_ihk - lse_ih), s in base 2.
//
// One product per tile of 128 keys and block of up to 128 query rows: S = K Q^T, keys x rows, on the 5th-generation
// tensor cores.  With the keys as its rows a score's lane is its key, so a thread adds up one key's weights and no
// lane talks to another; keys go from the cache into the product as they are (a key's rotation is undone on the
// query's side: Q = R_{m - Delta} q, prepared anew for every document), so a row of K that holds no key spoils
// nothing but a sum that is not written.
//
// Precision: the weights are fp32 results and their sums are kept over many steps, so the scores are not rounded to
// 16 bits: K is exact in bf16, and a query value is the sum of three bf16 numbers (24 bits) in blocks of up to 32
// rows, of two (16 bits) in larger ones, where the rows' errors average out.  Against 64 bits: 1e-7 to 1e-6 relative.
//
// Work is cut into equal parts, one per SM, in the order request, KV head, group of row blocks, page; a part is a
// sequence of items (a run of up to 32 pages of one document against one block of rows), and a tile is 8 pages of it.
// Roles of a block (640 threads, one block per SM):
//   warps 0-7   weights: two warpgroups, thread = key.  More than 32 rows: both read each tile, half of the columns
//               each; fewer: every second tile each.  2^(s - lse) per row, sums in registers.
//   warps 8-15  Q operands (two buffers): turned, scaled, split into bf16 parts, 128-byte swizzle.
//   warp 16     the items, from the block words.
//   warps 17-18 TMA copies of K, 64 columns x 16 rows of a page each (3 to 6 tiles in flight).
//   warp 19     products (one thread).
// A second launch adds the KV heads' and groups' sums in a fixed order, so results repeat bit for bit.
//
// What bounds it: with one row per head (a decode step) the keys' bytes: 16 requests of 32 033 keys, 8 KV heads, 176 us,
// 6.0 TB/s, some 3 of them for adding up the heads' sums.  With many rows the roles share the SM's issue slots and no one
// of them is the limit: 8 x 32 rows of 64 heads over 10 304 keys 94.5 us, 456 TFLOP/s, a tile ~2000 cycles, of which the
// products (two passes of 16 bits) take 1024; when it was 103, it was 94 with a quarter of the preparation, 92 without
// exponentials and 101 with half of the products.  One question of 800 tokens over 2400 keys 52.5, some 7 of them before the
// first product and 3 for the sums.
// Steps (this case; a decode step's in brackets): handshakes per run of pages and not per tile 123 -> 113 us [-];
// copies, planning and preparation by warps of their own 132 [298 -> 227]; the parts of a query in one product of
// concatenated columns [227 -> 181]; four score buffers 110 -> 104; the share's ends found in one pass over the requests
// without 64-bit divisions (2 us sooner at the first tile), code for few and for many rows apart, sums that read the lists
// before they wait 104 -> 94.5 [182 -> 176].  Left out: registers split between the roles (any spill goes to
// the L2, as shared memory leaves no L1: 167), four warpgroups of readers (112), pages prefetched into the L2 (111 [203]), 32
// columns at a time (105), the next 16 scores' load ahead of the exponentials (103 where 96.6), preparation by four warps
// (105, 67 instead of 60 for the one question), the sums' launch let go early (103 where 100.7, 63.8 where 59.1), an
// operand's first row made before its buffer is free (96.6, 55.5 where 53.7).
#include <algorithm>
#include <climits>

#include "shared_decode.cuh"
#include "tcgen05.cuh"

namespace lazykv {

namespace {

using namespace tc;

constexpr int kTile = 128, kPagesPerTile = kTile / kPage;  // keys per tile: the rows of a product
constexpr int kRows = 128;                                  // most query rows per block: its columns
constexpr int kRowsAlibi = 64;                              // (ALiBi keeps two more numbers per row)
constexpr int kGroups = 8;                                  // most groups of row blocks
constexpr int kPrepWarps = 8, kPrep = 32 * kPrepWarps;
constexpr int kCopyWarps = 2;
constexpr int kPrepWarp0 = 8, kPlanWarp = kPrepWarp0 + kPrepWarps, kCopyWarp0 = kPlanWarp + 1,
              kMmaWarp = kCopyWarp0 + kCopyWarps, kThreads = 32 * (kMmaWarp + 1);
constexpr int kMaxStages = 6, kSlots = 4, kLse = 4;
// A set of log-sum-exps is written anew kLse operands later, and so at least kLse items behind the last item that reads it;
// an item is published when the one kSlots before it is done with by every reading warp.
static_assert(kSlots <= kLse, "log-sum-exps are overwritten while they are read");
constexpr int kRun = 32;     // pages per item
constexpr int kFew = 32;     // up to so many rows a query value is three bf16 numbers (24 bits), else two (16)
constexpr int kScore = 128, kBufs = 4;  // columns of a score buffer, buffers

struct Args {
  const __nv_bfloat16* q;
  const float* lse;
  const int32_t* cu_q;
  const int32_t* seq_len;
  const int32_t* q_start;
  const int32_t* doc_blocks;
  const uint64_t* meta;
  float* part;  // [groups][Hkv][B][16 max_blocks]
  float* weights;
  uint32_t* status;
  int B, max_blocks, Hq, Hkv, num_pages, window, accumulate, groups;
  int rows;             // columns of the Q buffers: query rows per block at most, a multiple of 16
  int most;             // rows per head of a request at most (the call's bound)
  int sums;             // per group: 2 in blocks of many rows (each warpgroup has a part of the columns)
  int stages;           // K tiles in flight
  PosParams pos;
};

// What a request's weights take: its window's rows, the row blocks and their groups, its list.
struct Request {
  int nb, docs, n, first, m0;  // visible blocks, document blocks; rows per head, the first of them, its position
  int R, nrb, size, rgc; // rows per KV head, blocks of `size` rows, groups of row blocks
};
__device__ __forceinline__ Request request_of(const Args& a, int b) {
  Request r;
  const int lo = a.cu_q[b], hi = a.cu_q[b + 1], len = a.seq_len[b];
  r.n = max(0, hi - lo);
  if (a.window > 0) r.n = min(r.n, a.window);
  r.n = min(r.n, a.most);
  r.nb = visible_blocks(len, a.q_start[b], a.doc_blocks[b], a.max_blocks);
  r.docs = a.doc_blocks[b];
  r.first = hi - r.n;
  r.m0 = len - r.n;
  r.R = r.nb > 0 ? r.n * (a.Hq / a.Hkv) : 0;
  r.nrb = (r.R + a.rows - 1) / a.rows;
  r.size = r.nrb ? ((r.R + r.nrb - 1) / r.nrb + 15) / 16 * 16 : 16;
  r.nrb = (r.R + r.size - 1) / r.size;
  r.rgc = min(r.nrb, a.groups);
  return r;
}
// group g covers row blocks [group_start(g), group_start(g + 1))
__device__ __forceinline__ int group_start(const Request& r, int g) {  // up to 8 x 2^27
  return int(uint32_t(g) * uint32_t(r.nrb) / uint32_t(r.rgc));
}
// x / d where the quotient is a small number: an estimate and its correction (x, d >= 0)
__device__ __forceinline__ int small_quotient(long long x, long long d) {
  int q = int(__fdividef(float(x), float(d)));
  while (q * d > x) --q;
  while ((q + 1) * d <= x) ++q;
  return q;
}

enum : int { F_END = 1, F_NEWQ = 2, F_MASK = 4 };
struct Item {  // a run of pages of one document against one block of query rows: tiles of 8 pages
  uint8_t flags, np, rg, rows;  // np list blocks; group; query rows (of the request's) from r0 on
  int b, j0, kvh;               // first list block
  int r0, delta, m0, first;     // position of row 0's token, its query row
  int qn, pg0, stored;          // number of the Q operand; first page's index; pages up to this position have a sum
  uint32_t page[kRun];          // physical page << 8 | keys (0: none)
};
static_assert(sizeof(Item) == 172, "the layout below counts on it");

enum : int {
  B_META = 0,                      // [kSlots] item published (1)
  B_QOK = B_META + kSlots,         // [kSlots] its Q operand is ready (a lane per warp)
  B_DONE = B_QOK + kSlots,         // [kSlots] item finished (a lane per reading warp)
  B_SFULL = B_DONE + kSlots,       // [kBufs] a tile's scores written (commit)
  B_SFREE = B_SFULL + kBufs,       // [kBufs] scores read (a lane per reading warp)
  B_QFREE = B_SFREE + kBufs,           // [2] products with the Q buffer done (commit)
  B_FINAL = B_QFREE + 2,
  B_KFULL = B_FINAL + 1,           // [stages] K tile landed (a lane per copying warp)
  NBAR_FIXED = B_KFULL             // then [stages] products with the stage done (commit)
};

template <int D>
struct WLayout {
  static constexpr int TILE = kTile * D * 2, KBLK = kTile * 128;
  static constexpr int LIMIT = 227 * 1024;
  __host__ __device__ static constexpr int parts(int rows) { return rows <= kFew ? 3 : 2; }
  __host__ __device__ static constexpr int qbuf(int rows) { return parts(rows) * rows * D * 2; }
  __host__ __device__ static constexpr int ring(int rows, bool alibi) { return kLse * rows * 4 * (alibi ? 3 : 1); }
  __host__ static int smem(int rows, int st, bool alibi) {
    return st * TILE + 2 * qbuf(rows) + ring(rows, alibi) + kSlots * int(sizeof(Item)) + (NBAR_FIXED + 2 * st) * 8 + 8;
  }
  __host__ static int stages(int rows, bool alibi) {  // at least 3 (D 128, 128 rows: 3)
    int n = kMaxStages;
    while (smem(rows, n, alibi) > LIMIT) --n;
    return n;
  }
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// Waits for the thread's loads; the values are used behind it.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// Eight values in bf16, and what that leaves of them.
__device__ __forceinline__ uint4 round8(const float2 (&y)[4]) {
  return make_uint4(f2_to_bf2(y[0].x, y[0].y), f2_to_bf2(y[1].x, y[1].y), f2_to_bf2(y[2].x, y[2].y),
                    f2_to_bf2(y[3].x, y[3].y));
}
__device__ __forceinline__ void less8(float2 (&y)[4], uint4 part) {
  const uint32_t h[4] = {part.x, part.y, part.z, part.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = __ffma2_rn(bf2_to_f2(h[i]), make_float2(-1.f, -1.f), y[i]);
}
__device__ __forceinline__ void unpack8(uint4 u, float2 (&y)[4]) {
  y[0] = bf2_to_f2(u.x);
  y[1] = bf2_to_f2(u.y);
  y[2] = bf2_to_f2(u.z);
  y[3] = bf2_to_f2(u.w);
}
// Where a block's share of the work begins or ends: total work is cut into equal parts in the order request,
// KV head, group of row blocks, list block; a list block costs one unit per row block.
struct Place {
  int b, kvh, rg, page;
};

template <int D, int POS, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
weights_kernel(const __grid_constant__ CUtensorMap tmk, const Args a) {
  using L = WLayout<D>;
  constexpr bool kAl = POS == kAlibi;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NS = a.stages, rows = a.rows, G = a.Hq / a.Hkv;
  // Blocks of many rows: both warpgroups read each tile's scores, half of the columns each (their sums stay
  // apart); of few rows: every second tile each.
  constexpr bool split = SPLIT;  // rows > kFew
  const uint32_t QBUF = uint32_t(L::qbuf(rows)), QPART = uint32_t(rows) * 128, QBLK = QPART * L::parts(rows);
  const uint32_t sK = sb, sQ = sb + NS * L::TILE;
  uint8_t* const tail = sm + NS * L::TILE + 2 * QBUF;
  float* ring = reinterpret_cast<float*>(tail);  // [kLse][rows] -lse (ALiBi: and slope, position)
  const uint32_t bar0 = smem_u32(tail + L::ring(rows, kAl));
  const int B_KFREE = B_KFULL + NS;
  Item* items = reinterpret_cast<Item*>(tail + L::ring(rows, kAl) + (NBAR_FIXED + 2 * NS) * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(items + kSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto BAR = [&](int i) { return bar0 + 8u * uint32_t(i); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < NBAR_FIXED + 2 * NS; ++i)
      mbar_init(BAR(i), i >= B_QOK && i < B_DONE                                            ? kPrepWarps
                        : i >= B_DONE && i < B_SFULL                                          ? 8
                        : i >= B_SFREE && i < B_QFREE                                        ? (split ? 8 : 4)
                        : i >= B_KFULL && i < B_KFREE                                        ? kCopyWarps
                                                                                             : 1);
    *abort_flag = (sb & 1023u) ? 1 : 0;  // the operands' swizzle goes by addresses
    if (sb & 1023u) set_status(a.status, LAZY_STATUS_TIMEOUT);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = *abort_flag == 0;

  if (warp < 8) {
    // ============================ weights: a thread owns a key of a tile
    const int wg = warp >> 2, row = threadIdx.x & 127;  // TMEM lane = key of the tile
    uint32_t tile = 0;  // of this block's tiles
    for (int i = 0; ok; ++i) {
      const Item& it = items[i % kSlots];
      bool got = wait_bar(BAR(B_META + i % kSlots), uint32_t((i / kSlots) & 1), abort_flag, a.status);
      if (!__all_sync(0xffffffffu, got)) break;
      const int flags = it.flags, np = it.np;
      if (flags & F_END) break;
      const int n16 = (it.rows + 15) / 16, stored = it.stored, delta = it.delta, pg0 = it.pg0, m0 = it.m0, r0 = it.r0;
      const float* lse = ring + (it.qn % kLse) * rows * (kAl ? 3 : 1);
      float* to = a.part + ((((size_t)(split ? 2 * it.rg + wg : it.rg) * a.Hkv + it.kvh) * a.B + it.b) * a.max_blocks +
                            it.j0) * kPage + row;
      for (int j = 0; j < np; j += kPagesPerTile, ++tile) {
        const int buf = int(tile % kBufs);
        if (!split && (buf & 1) != wg) continue;
        const int mine = j + row / kPage, start = delta + kPage * (pg0 + mine), p = start + row % kPage;
        float old = 0.f;
        if (stored >= 0 && mine < np && start <= stored) old = to[j * kPage];  // this thread's own, of the row block before
        got = wait_bar(BAR(B_SFULL + buf), (tile / kBufs) & 1u, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tS = tmem + (uint32_t(32 * (warp & 3)) << 16) + uint32_t(buf * kScore);
        int n0 = 0;  // rows from n0 on see the key
        if (flags & F_MASK) {
          const long long see = (long long)(p - m0) * G - r0;
          n0 = int(see < 0 ? 0 : (see > kRows ? kRows : see));
        }
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const bool masked = flags & F_MASK;
        const int keys = mine < np && n0 < int(it.rows) ? int(it.page[mine] & 0xFFu) : 0;  // 0 too for a key that no row sees
        const int cut = split ? (n16 + 1) / 2 : 0, c1 = split && wg == 0 ? cut : n16;
        constexpr int PARTS = split ? 1 : 3;  // columns that a score is the sum of (of many rows the products add them up)
        uint32_t u[PARTS][16];
        auto load = [&](int c) {
#pragma unroll
          for (int e = 0; e < PARTS; ++e) tmem_ld16(tS + uint32_t(e * rows + 16 * c), u[e]);
        };
        int c = split && wg ? cut : 0;
#pragma unroll 1
        for (; c < c1; ++c) {  // 16 scores: acc += 2^(s - lse)
          const float* l = lse + 16 * c;
          float4 l4[4];  // negative log-sum-exps
          auto lses = [&]() {
#pragma unroll
            for (int e = 0; e < 4; ++e) l4[e] = *reinterpret_cast<const float4*>(l + 4 * e);
          };
          load(c);
          if constexpr (split) lses();
#pragma unroll
          for (int e = 0; e < PARTS; ++e) tmem_wait_ld16(u[e]);
          if constexpr (!split) lses();
          float2 x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            auto part = [&](int i) { return make_float2(__uint_as_float(u[i][2 * e]), __uint_as_float(u[i][2 * e + 1])); };
            x[e] = part(0);
            if constexpr (!split) x[e] = __fadd2_rn(x[e], __fadd2_rn(part(1), part(2)));
            if constexpr (kAl) {
              const float *sl = l + rows + 2 * e, *mm = sl + rows;
              x[e].x = fmaf(sl[0], float(p) - mm[0], x[e].x);
              x[e].y = fmaf(sl[1], float(p) - mm[1], x[e].y);
            }
            x[e] = __fadd2_rn(x[e], e & 1 ? make_float2(l4[e / 2].z, l4[e / 2].w) : make_float2(l4[e / 2].x, l4[e / 2].y));
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (16 * c + 2 * e < n0) x[e].x = -INFINITY;
              if (16 * c + 2 * e + 1 < n0) x[e].y = -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e & 3] = __fadd2_rn(acc[e & 3], make_float2(ex2(x[e].x), ex2(x[e].y)));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_SFREE + buf));
        if (mine < np) {
          const float w = row % kPage < keys ? ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) + ((acc[2].x + acc[2].y) + (acc[3].x + acc[3].y)) : 0.f;
          to[j * kPage] = old + w;
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_DONE + i % kSlots));
    }
  } else if (warp < kPlanWarp) {
    // ============================ Q operands: rows turned by m - Delta, scaled, split into two or three bf16 numbers
    const int t = threadIdx.x - kPrepWarp0 * 32;
    for (int i = 0; ok; ++i) {
      const int sl = i % kSlots;
      bool got = wait_bar(BAR(B_META + sl), uint32_t((i / kSlots) & 1), abort_flag, a.status);
      if (!__all_sync(0xffffffffu, got)) break;
      const Item& it = items[sl];
      const int flags = it.flags;
      if (flags & F_END) break;
      if (flags & F_NEWQ) {
        const int qn = it.qn, buf = qn & 1, nr = it.rows;
        const int n16 = (nr + 15) / 16 * 16, r0 = it.r0, delta = it.delta, kvh = it.kvh;
        float* lse = ring + (qn % kLse) * rows * (kAl ? 3 : 1);
        float l = -INFINITY, sl2 = 0.f;  // an empty column weighs nothing
        if (t < nr) {
          const int r = r0 + t, h = kvh * G + r % G;
          l = a.lse[(size_t)(it.first + r / G) * a.Hq + h] * -1.4426950408889634f;
          if (l == INFINITY) l = -INFINITY;  // nor does a row that saw nothing
          if constexpr (kAl) sl2 = a.pos.slopes[h] * 1.4426950408889634f;
        }
        // the buffer's last products are done
        auto buffer_free = [&]() -> bool {
          const bool g = qn < 2 || wait_bar(BAR(B_QFREE + buf), uint32_t(((qn >> 1) - 1) & 1), abort_flag, a.status);
          if (!__all_sync(0xffffffffu, g)) return false;
          if (t < n16) {
            lse[t] = l;
            if constexpr (kAl) {
              lse[rows + t] = sl2;
              lse[2 * rows + t] = float(it.m0 + (r0 + t) / G);
            }
          }
          return true;
        };
        const uint32_t q0 = sQ + uint32_t(buf) * QBUF;
        auto put = [&](int n, int k, float2 (&y)[4]) {  // chunk k (8 dimensions) of column n
          const uint32_t at = q0 + uint32_t(k >> 3) * QBLK + swz(n, k & 7);
          uint4 u = round8(y);
          st_shared_v4(at, u);
          less8(y, u);
          u = round8(y);
          st_shared_v4(at + QPART, u);
          if (!split) {
            less8(y, u);
            st_shared_v4(at + 2 * QPART, round8(y));
          }
        };
        const float sc = a.pos.scale_log2;
        // query row of column n, head `h` of the token's `token`; null behind the last
        auto src = [&](int n, int token, int h) {
          return n < nr ? reinterpret_cast<const uint4*>(a.q + ((size_t)(it.first + token) * a.Hq + kvh * G + h) * D)
                        : nullptr;
        };
        const uint4 zero = make_uint4(0, 0, 0, 0);
        if constexpr (POS == kRope) {  // half-split pairs over the whole head: a thread owns a chunk and its partner
          constexpr int NC = D / 16, NG = kPrep / NC;
          const int c = t % NC, per = (n16 + NG - 1) / NG, n0 = t / NC * per;
          float2 co[4], sn[4], ns[4];  // times the scale
          int token = (r0 + n0) / G, h = (r0 + n0) % G;
          int tk = token, hh = h;  // of the row that is loaded next, one ahead of the one in use
          uint4 raw[2];
          auto load = [&](int e) {
            const uint4* s = e < per ? src(n0 + e, tk, hh) : nullptr;
            raw[0] = s ? s[c] : zero;
            raw[1] = s ? s[c + NC] : zero;
            if (++hh == G) {
              hh = 0;
              ++tk;
            }
          };
          load(0);
          bool turn = true;  // the token has changed
          ok = buffer_free();
          const int n1 = ok ? min(n0 + per, n16) : n0;
#pragma unroll 1
          for (int n = n0; n < n1; ++n) {
            float2 x1[4], x2[4], y1[4], y2[4];
            unpack8(raw[0], x1);
            unpack8(raw[1], x2);
            load(n + 1 - n0);
            if (turn) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                turn_sincos_signed(it.m0 + token - delta, a.pos.turns[8 * c + 2 * e], sn[e].x, co[e].x);
                turn_sincos_signed(it.m0 + token - delta, a.pos.turns[8 * c + 2 * e + 1], sn[e].y, co[e].y);
                co[e] = make_float2(co[e].x * sc, co[e].y * sc);
                sn[e] = make_float2(sn[e].x * sc, sn[e].y * sc);
                ns[e] = make_float2(-sn[e].x, -sn[e].y);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y1[e] = __ffma2_rn(x1[e], co[e], __fmul2_rn(x2[e], ns[e]));
              y2[e] = __ffma2_rn(x1[e], sn[e], __fmul2_rn(x2[e], co[e]));
            }
            put(n, c, y1);
            put(n, c + NC, y2);
            turn = ++h == G;
            if (turn) {
              h = 0;
              ++token;
            }
          }
        } else {
          // A thread owns one chunk of its rows and, with half-split pairs, reads the one that it is turned against.
          constexpr int NC = D / 8, NG = kPrep / NC;
          const int k = t % NC, per = (n16 + NG - 1) / NG, n0 = t / NC * per;
          const int rd = POS == kRopeX ? a.pos.rotary_dim : 0, hr = rd / 2;
          const bool inter = a.pos.interleaved != 0, still = 8 * k >= rd, low = 8 * k < hr;
          const int other = still || inter ? k : (low ? k + hr / 8 : k - hr / 8);
          const int f0 = inter ? 4 * k : (low ? 8 * k : 8 * k - hr);
          float2 co[4], sn[4];  // times the scale; sn with the sign of the partner's product
          int token = (r0 + n0) / G, h = (r0 + n0) % G;
          int tk = token, hh = h;  // of the row that is loaded next, one ahead of the one in use
          uint4 raw[2];
          auto load = [&](int e) {
            const uint4* s = e < per ? src(n0 + e, tk, hh) : nullptr;
            raw[0] = s ? s[k] : zero;
            raw[1] = s && other != k ? s[other] : zero;
            if (++hh == G) {
              hh = 0;
              ++tk;
            }
          };
          load(0);
          bool turn = true;  // the token has changed
          ok = buffer_free();
          const int n1 = ok ? min(n0 + per, n16) : n0;
#pragma unroll 1
          for (int n = n0; n < n1; ++n) {
            float2 x[4], z[4], y[4];
            unpack8(raw[0], x);
            unpack8(raw[1], z);
            load(n + 1 - n0);
            if (turn && !still) {
              const int dp = it.m0 + token - delta;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (inter) {  // one angle per pair of neighbours
                  turn_sincos_signed(dp, a.pos.turns[f0 + e], sn[e].y, co[e].x);
                  co[e].x = co[e].y = co[e].x * sc;
                  sn[e].y *= sc;
                  sn[e].x = -sn[e].y;
                } else {
                  turn_sincos_signed(dp, a.pos.turns[f0 + 2 * e], sn[e].x, co[e].x);
                  turn_sincos_signed(dp, a.pos.turns[f0 + 2 * e + 1], sn[e].y, co[e].y);
                  co[e] = make_float2(co[e].x * sc, co[e].y * sc);
                  sn[e] = low ? make_float2(-sn[e].x * sc, -sn[e].y * sc) : make_float2(sn[e].x * sc, sn[e].y * sc);
                }
              }
            }
            turn = ++h == G;
            if (turn) {
              h = 0;
              ++token;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (still) {
                y[e] = make_float2(x[e].x * sc, x[e].y * sc);
              } else {
                const float2 p = inter ? make_float2(x[e].y, x[e].x) : z[e];  // the partners
                y[e] = __ffma2_rn(x[e], co[e], __fmul2_rn(p, sn[e]));
              }
            }
            put(n, k, y);
          }
        }
        fence_async_smem();
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_QOK + sl));
    }
  } else if (warp == kPlanWarp) {
    // ============================ the block's share of the work, item by item
    long long total = 0;
    Request r = {};  // of request b0 + lane
    long long c = 0;
    auto count = [&](int b0) {
      c = 0;
      if (b0 + lane < a.B) {
        r = request_of(a, b0 + lane);
        c = (long long)r.nb * r.nrb * a.Hkv;
      }
    };
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      count(b0);
      long long all = c;
#pragma unroll
      for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      total += all;
    }
    // the share [total * block / blocks, total * (block + 1) / blocks)
    const uint32_t grid = gridDim.x, bid = blockIdx.x;
    const long long each = (total >> 32) ? total / grid : (long long)(uint32_t(total) / grid);
    const uint32_t rest = uint32_t(total - each * grid);
    const long long x0 = each * bid + rest * bid / grid, x1 = each * (bid + 1) + rest * (bid + 1) / grid;
    Place at = {a.B, 0, 0, 0}, end = at;
    int known = -1;  // request that `r` is of
    if (x0 < x1) {
      Request mine = {};
      long long base = 0;
      int left = x1 < total ? 2 : 1;  // places to find
      for (int b0 = 0; b0 < a.B && left; b0 += 32) {
        if (a.B > 32) count(b0);
        long long up = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, up, o);
          if (lane >= o) up += y;
        }
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          const long long x = (e ? x1 : x0) - base;
          const bool here = x >= up - c && x < up;
          const uint32_t in = __ballot_sync(0xffffffffu, here);
          if (!in || (e && x1 == total)) continue;
          Place at_lane = {};
          if (here) {
            const long long y = x - (up - c), one = (long long)r.nb * r.nrb;
            at_lane.kvh = small_quotient(y, one);
            const long long z = y - at_lane.kvh * one;
            const int rb = small_quotient(z, r.nb);
            int g = small_quotient((long long)rb * r.rgc, r.nrb);
            while (group_start(r, g + 1) <= rb) ++g;
            const int first = group_start(r, g);
            at_lane.rg = g;
            at_lane.page = small_quotient(z - (long long)first * r.nb, group_start(r, g + 1) - first);
          }
          const int l = __ffs(in) - 1;
          Place& to = e ? end : at;
          to = {b0 + l, __shfl_sync(0xffffffffu, at_lane.kvh, l), __shfl_sync(0xffffffffu, at_lane.rg, l),
                __shfl_sync(0xffffffffu, at_lane.page, l)};
          if (e == 0) {
            known = b0 + l;
            mine = {__shfl_sync(0xffffffffu, r.nb, l),  __shfl_sync(0xffffffffu, r.docs, l),  __shfl_sync(0xffffffffu, r.n, l),
                    __shfl_sync(0xffffffffu, r.first, l), __shfl_sync(0xffffffffu, r.m0, l),  __shfl_sync(0xffffffffu, r.R, l),
                    __shfl_sync(0xffffffffu, r.nrb, l), __shfl_sync(0xffffffffu, r.size, l),  __shfl_sync(0xffffffffu, r.rgc, l)};
          }
          --left;
        }
        base += __shfl_sync(0xffffffffu, up, 31);
      }
      r = mine;
    }
    int i = 0, qn = -1;
    auto slot_free = [&](int j) -> bool {
      const bool got = j < kSlots || wait_bar(BAR(B_DONE + j % kSlots), uint32_t((j / kSlots - 1) & 1), abort_flag, a.status);
      return __all_sync(0xffffffffu, got);
    };
    auto before = [](const Place& p, const Place& e) {
      return p.b != e.b ? p.b < e.b : p.kvh != e.kvh ? p.kvh < e.kvh : p.rg != e.rg ? p.rg < e.rg : p.page < e.page;
    };
    while (ok && before(at, end)) {
      if (at.b != known) r = request_of(a, known = at.b);
      if (r.R == 0) {
        at = {at.b + 1, 0, 0, 0};
        continue;
      }
      const bool same = at.b == end.b && at.kvh == end.kvh && at.rg == end.rg;
      const int p1 = same ? end.page : r.nb, rb0 = group_start(r, at.rg), rb1 = group_start(r, at.rg + 1);
      const uint64_t* words = a.meta + (size_t)at.b * a.max_blocks;
      int wbase = at.page;
      auto fetch = [&](int p) -> uint64_t { return p + lane < p1 ? ldg_u64(words + p + lane) : 0; };
      uint64_t win = fetch(wbase), next = fetch(wbase + 32);  // 64 words from wbase on
      int delta = -1, last_rb = -1;  // of the Q operand
      for (int p = at.page; p < p1 && ok;) {
        if (p >= wbase + 32) {
          wbase += 32;
          win = next;
          next = fetch(wbase + 32);
        }
        const int wi = p - wbase + lane;
        const uint64_t w_here = __shfl_sync(0xffffffffu, win, wi & 31), w_next = __shfl_sync(0xffffffffu, next, wi & 31);
        const uint64_t w = wi < 32 ? w_here : w_next;
        const int d = int(word_delta(w)), d0 = __shfl_sync(0xffffffffu, d, 0);
        const int pg0 = __shfl_sync(0xffffffffu, int(word_pg(w)), 0), start = d + kPage * int(word_pg(w));
        // a run: consecutive pages of one document
        const uint32_t run = __ballot_sync(0xffffffffu, p + lane < p1 && d == d0 && int(word_pg(w)) == pg0 + lane);
        const int len = ~run ? __ffs(~run) - 1 : 32;
        int nv = min(int(word_nvalid(w)), kPage);
        if (lane < len && word_page(w) >= uint32_t(a.num_pages)) {
          set_status(a.status, LAZY_STATUS_BAD_PAGE);
          nv = 0;
        }
        const uint32_t page = nv > 0 ? word_page(w) << 8 | uint32_t(nv) : 0u;
        // every row block of the group over the run, while its pages are in the L2
        for (int rb = rb0; rb < rb1 && ok; ++rb) {
          const int r0 = rb * r.size, nr = min(r.size, r.R - r0);
          const int m_lo = r.m0 + r0 / G, m_hi = r.m0 + (r0 + nr - 1) / G;
          const uint32_t seen = __ballot_sync(0xffffffffu, lane < len && start <= m_hi);
          const int np = ~seen ? __ffs(~seen) - 1 : 32;  // pages that some row of the block sees
          if (np == 0) continue;
          const bool newq = rb != last_rb || (d0 != delta && (POS == kRope || POS == kRopeX));
          delta = d0;
          last_rb = rb;
          if (newq) ++qn;
          ok = slot_free(i);
          if (!ok) break;
          Item& it = items[i % kSlots];
          it.page[lane] = lane < np ? page : 0u;
          if (lane == 0) {
            it.flags = uint8_t((newq ? F_NEWQ : 0) | (d0 + kPage * (pg0 + np) - 1 > m_lo ? F_MASK : 0));
            it.np = uint8_t(np);
            it.rg = uint8_t(at.rg);
            it.rows = uint8_t(nr);
            it.b = at.b;
            it.j0 = p;
            it.kvh = at.kvh;
            it.r0 = r0;
            it.delta = d0;
            it.m0 = r.m0;
            it.first = r.first;
            it.qn = qn;
            it.pg0 = pg0;
            it.stored = rb > rb0 ? r.m0 + (r0 - 1) / G : INT_MIN;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_META + i % kSlots));
          ++i;
        }
        p += len;
      }
      at = {at.b, at.kvh, at.rg + 1, 0};
      if (at.rg == r.rgc) at = {at.b, at.kvh + 1, 0, 0};
      if (at.kvh == a.Hkv) at = {at.b + 1, 0, 0, 0};
    }
    if (ok && slot_free(i) && lane == 0) {
      items[i % kSlots].flags = F_END;
      mbar_arrive(BAR(B_META + i % kSlots));
    }
  } else if (warp < kMmaWarp) {
    // ============================ copies: each warp takes every second page of a tile (a copy costs its issuer ~75 cycles)
    const int part = warp - kCopyWarp0;
    int tiles = 0, st = 0;
    uint32_t phase = 1;  // parity of the stage's last use (none: passes at once)
    for (int i = 0; ok; ++i) {
      const int sl = i % kSlots;
      bool got = wait_bar(BAR(B_META + sl), uint32_t((i / kSlots) & 1), abort_flag, a.status);
      if (!__all_sync(0xffffffffu, got)) break;
      const Item& it = items[sl];
      if (it.flags & F_END) break;
      const int np = it.np, kvh = it.kvh;
      for (int j = 0; j < np; j += kPagesPerTile) {
        const uint32_t pg = lane < kPagesPerTile && lane % kCopyWarps == part && j + lane < np ? it.page[j + lane] : 0u;
        const uint32_t load = __ballot_sync(0xffffffffu, pg != 0);
        got = wait_bar(BAR(B_KFREE + st), phase, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(BAR(B_KFULL + st), uint32_t(__popc(load)) * kPage * D * 2);
        __syncwarp();
        if (pg)
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_page(sK + uint32_t(st * L::TILE + cb * L::KBLK + lane * kPage * 128), &tmk, cb * 64, 0,
                          int(pg >> 8) * a.Hkv + kvh, BAR(B_KFULL + st));
        __syncwarp();
        ++tiles;
        if (++st == NS) {
          st = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0)  // never leave copies in flight
      for (int j = max(0, tiles - NS); j < tiles; ++j) {
        WaitClock clk;
        while (*abort_flag && !mbar_test(BAR(B_KFULL + j % NS), uint32_t((j / NS) & 1)) && !clk.expired()) {
        }
      }
  } else if (warp == kMmaWarp) {
    // ============================ products (one thread): S = K Q^T by the parts of Q, keys x query rows
    if (elect_one()) {
      // Descriptors are built from launch constants and counters alone, and a branch chooses the Q buffer, so that
      // they stay in uniform registers.
      const uint64_t kd = sdesc(sK, 16, 1024), qd0 = sdesc(sQ, 16, 1024), qd1 = sdesc(sQ + QBUF, 16, 1024);
      // Blocks of few rows: one product for the three parts of a query, side by side, which reads the keys once (16
      // columns cost what 64 do: the keys' 4 KB from shared memory).  Of many: a product per part, into one sum, so that
      // four score buffers fit.
      const int passes = split ? 2 : 1, cols = split ? rows : 3 * rows;
      const uint32_t idesc = idesc_mma(kTile, 16, 0, 0) + (uint32_t(cols / 16 * 2 - 2) << 17);
      const uint64_t qblk = QBLK >> 4, qpart = QPART >> 4;
      auto products = [&](uint32_t d, uint64_t k0, uint64_t q0) {
#pragma unroll 1
        for (int part = 0; part < passes; ++part, q0 += qpart)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16(d, k0 + uint64_t(((kk >> 2) * L::KBLK + (kk & 3) * 32) >> 4), q0 + (kk >> 2) * qblk + (kk & 3) * 2, idesc,
                     part || kk ? 1u : 0u);
      };
      int st = 0, newest = -1;
      uint32_t tile = 0, kpar = 0;
      bool seen_k = false, seen_s = true;  // the next tile's barriers, asked for while this one's products queue
      for (int i = 0; ok; ++i) {
        const int sl = i % kSlots;
        ok = wait_bar(BAR(B_META + sl), uint32_t((i / kSlots) & 1), abort_flag, a.status);
        if (!ok) break;
        const int flags = items[sl].flags, np = items[sl].np;
        if (flags & F_END) break;
        if (flags & F_NEWQ) {
          // Nothing needs this wait (the ring of log-sum-exps is guarded by the items' slots): a new operand begins when
          // the readers are at most two tiles behind.  Without it 8 x 32 rows over 10 304 keys take 95.9 us instead of
          // 94.2, one question of 800 tokens 52.1 instead of 52.6.
          if (tile >= 3) {
            const uint32_t t = tile - 3;
            ok = wait_bar(BAR(B_SFREE + int(t % kBufs)), (t / kBufs) & 1u, abort_flag, a.status);
            if (!ok) break;
          }
          if (newest >= 0) mma_commit(BAR(B_QFREE + (newest & 1)));
          ++newest;
        }
        ok = wait_bar(BAR(B_QOK + sl), uint32_t((i / kSlots) & 1), abort_flag, a.status);
        for (int j = 0; j < np && ok; j += kPagesPerTile, ++tile) {
          const int buf = int(tile % kBufs);
          ok = (seen_k || wait_bar(BAR(B_KFULL + st), kpar, abort_flag, a.status)) &&
               (seen_s || wait_bar(BAR(B_SFREE + buf), (tile / kBufs) & 1u ^ 1u, abort_flag, a.status));
          if (!ok) break;
          tc_fence_after();
          const uint64_t k0 = kd + uint64_t(st * (L::TILE >> 4));
          if (newest & 1)
            products(tmem + uint32_t(buf * kScore), k0, qd1);
          else
            products(tmem + uint32_t(buf * kScore), k0, qd0);
          mma_commit(BAR(B_SFULL + buf));
          mma_commit(BAR(B_KFREE + st));
          if (++st == NS) {
            st = 0;
            kpar ^= 1u;
          }
          seen_k = mbar_peek(BAR(B_KFULL + st), kpar);
          seen_s = mbar_peek(BAR(B_SFREE + int((tile + 1) % kBufs)), ((tile + 1) / kBufs) & 1u ^ 1u);
        }
      }
      mma_commit(BAR(B_FINAL));  // every product is done before TMEM goes
      WaitClock clk;
      while (!mbar_test(BAR(B_FINAL), 0) && !clk.expired()) {
      }
    }
    __syncwarp();
  }

  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Adds the parts of a key: groups of row blocks, KV heads, in a fixed order.  A thread owns 4 keys of a page; SL threads
// share their parts where a launch would leave SMs idle (one request of 2400 keys with 80 parts: 62.2 us by 1, 56.1 by 2, 54.6
// by 4, 53.6 by 8; 16 requests of 32 033 keys with 8 parts: 177, 179, 183, 187).  A page has parts of
// the groups with a row that sees its first key; they hold 0 where a key is not there or not seen.
constexpr int kSumThreads = 256;
template <int SL>
__global__ void __launch_bounds__(kSumThreads) weights_sum_kernel(const Args a) {
  constexpr int KEYS = 4 * kSumThreads / SL;
  __shared__ float4 share[SL][SL > 1 ? KEYS / 4 : 1];
  // What comes before the first wait reads what was there before the weights' launch: it waited for that itself before it
  // let this one start.
  const int b = blockIdx.y, N = a.max_blocks * kPage, quad = threadIdx.x % (KEYS / 4), slice = threadIdx.x / (KEYS / 4);
  const size_t n = (size_t)a.B * N;
  const Request r = request_of(a, b);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const int rows = a.cu_q[b + 1] - a.cu_q[b];
    if ((a.window > 0 ? min(rows, a.window) : rows) > a.most ||
        (r.R > 0 && list_too_long(a.seq_len[b] - 1, a.q_start[b], a.doc_blocks[b], a.max_blocks)))
      set_status(a.status, LAZY_STATUS_BAD_ROW);
  }
  const int per = a.sums * a.Hkv, G = a.Hq / a.Hkv, last = r.rgc * per;
  for (int i0 = blockIdx.x * KEYS; i0 < N; i0 += gridDim.x * KEYS) {  // the same rounds for every thread
    const int i = i0 + 4 * quad, j = i / kPage;
    const size_t at = (size_t)b * N + i;
    float old[4] = {0.f, 0.f, 0.f, 0.f};
    int g0 = r.rgc;  // the first group with a row that sees the page
    if (i < N) {
      if (a.accumulate && slice == 0)
#pragma unroll
        for (int e = 0; e < 4; ++e) old[e] = a.weights[at + e];
      if (r.R > 0 && j < r.nb) {
        const uint64_t w = a.meta[(size_t)b * a.max_blocks + j];
        const int p = int(word_delta(w)) + kPage * int(word_pg(w));
        g0 = 0;
        while (g0 < r.rgc && p > r.m0 + (min(r.R, group_start(r, g0 + 1) * r.size) - 1) / G) ++g0;
      }
    }
    pdl_wait();
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int e = g0 * per + slice; e < last; e += SL) {
      const float4 x = *reinterpret_cast<const float4*>(a.part + (size_t)e * n + at);
      t.x += x.x;
      t.y += x.y;
      t.z += x.z;
      t.w += x.w;
    }
    if constexpr (SL > 1) {
      share[slice][quad] = t;
      __syncthreads();
      if (slice == 0)
#pragma unroll
        for (int e = 1; e < SL; ++e) {
          const float4 x = share[e][quad];
          t.x += x.x;
          t.y += x.y;
          t.z += x.z;
          t.w += x.w;
        }
      __syncthreads();
    }
    if (i < N && slice == 0) {
      a.weights[at] = old[0] + t.x;
      a.weights[at + 1] = old[1] + t.y;
      a.weights[at + 2] = old[2] + t.z;
      a.weights[at + 3] = old[3] + t.w;
    }
  }
  pdl_wait();
  pdl_trigger();
}

// Partial sums of a key and KV head, at most, of a call with up to R rows per KV head: one where they fit a block of few
// rows, else two (each reading warpgroup's columns) for every group of row blocks, and blocks hold 64 (ALiBi) or 128 rows.
// The workspace has room for so many whatever the positional kind, and a call makes no more groups than that.
long long sums_of(long long R) {
  return R <= kFew ? 1 : 2 * std::min<long long>(kGroups, (R + kRowsAlibi - 1) / kRowsAlibi);
}

int most_rows(bool alibi, long long R) {
  const long long m = alibi ? kRowsAlibi : kRows, x = (R + 15) / 16 * 16;
  return int(x < 16 ? 16 : (x < m ? x : m));
}
template <int D, int POS, bool SPLIT>
int launch_weights(Args& a, const CUtensorMap& mk, cudaStream_t st) {
  using L = WLayout<D>;
  static std::atomic<uint64_t> done{0};
  auto kern = weights_kernel<D, POS, SPLIT>;
  LAZY_CUDA_TRY(smem_limit(kern, L::LIMIT, done));
  a.stages = L::stages(a.rows, POS == kAlibi);
  // A block's share is at least about a tile.
  const long long shares = (long long)a.B * a.Hkv * ((a.max_blocks + kPagesPerTile - 1) / kPagesPerTile) * a.groups;
  const int grid = int(std::min<long long>(shares, sm_count()));
  LAZY_CUDA_TRY(launch_pdl(kern, dim3(grid), dim3(kThreads), L::smem(a.rows, a.stages, POS == kAlibi), st, mk,
                           a));
  return LAZY_OK;
}
template <int D, int POS>
int launch_weights(Args& a, const CUtensorMap& mk, cudaStream_t st) {
  return a.rows > kFew ? launch_weights<D, POS, true>(a, mk, st) : launch_weights<D, POS, false>(a, mk, st);
}

}  // namespace

int check_shared_call(const char* what, int B, int max_blocks, int Hq, int Hkv, int D, int num_pages, float scale,
                      const lazy_pos_cfg* cfg, PosParams* pos, const void* meta, std::initializer_list<const void*> ptrs,
                      std::initializer_list<const void*> ints) {
  if (B < 0 || max_blocks <= 0 || Hq <= 0 || Hkv <= 0 || num_pages <= 0)
    return fail(LAZY_EINVAL, "%s: bad sizes (B=%d max_blocks=%d Hq=%d Hkv=%d num_pages=%d)", what, B, max_blocks, Hq,
                Hkv, num_pages);
  if (D != 64 && D != 128) return fail(LAZY_EINVAL, "%s: head_dim must be 64 or 128, got %d", what, D);
  if (Hq % Hkv) return fail(LAZY_EINVAL, "%s: Hq (%d) must be a multiple of Hkv (%d)", what, Hq, Hkv);
  if (num_pages > (1 << 24)) return fail(LAZY_ERANGE, "%s: num_pages above 2^24", what);
  if (max_blocks > (1 << 26)) return fail(LAZY_ERANGE, "%s: lists above 2^26 blocks", what);
  if (B > 65535 || Hkv > 65535) return fail(LAZY_ERANGE, "%s: B and Hkv must be below 65536", what);
  if (!(scale >= 0.f && scale <= 3.0e38f))
    return fail(LAZY_EINVAL, "%s: scale must be positive (or 0 for the default)", what);
  const int rc = prepare_pos(cfg, Hq, D, scale, pos);
  if (rc) return rc;
  if (!(pos->scale_log2 >= 0x1p-60f && pos->scale_log2 <= 0x1p60f))
    return fail(LAZY_EINVAL, "%s: scale must lie in [2^-60, 2^60]", what);
  if (B == 0) return LAZY_OK;
  for (const void* p : ints)
    if (!p) return fail(LAZY_EINVAL, "%s: NULL pointer", what);
  for (const void* p : ptrs) {
    if (!p) return fail(LAZY_EINVAL, "%s: NULL pointer", what);
    if (reinterpret_cast<uintptr_t>(p) & 15u) return fail(LAZY_EINVAL, "%s: tensors must be 16-byte aligned", what);
  }
  if (!meta) return fail(LAZY_EINVAL, "%s: NULL pointer", what);
  if (reinterpret_cast<uintptr_t>(meta) & 7u) return fail(LAZY_EINVAL, "%s: meta must be 8-byte aligned", what);
  return LAZY_OK;
}

int check_workspace(const char* what, const void* ws, size_t got, size_t need) {
  if (!need) return LAZY_OK;
  if (!ws || got < need) return fail(LAZY_EINVAL, "%s: workspace too small: need %zu bytes, got %zu", what, need, got);
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(LAZY_EINVAL, "%s: workspace must be 256-byte aligned", what);
  return LAZY_OK;
}

size_t key_weights_ws_bytes(int rows, int B, int max_blocks, int Hq, int Hkv) {
  return (size_t)sums_of((long long)rows * (Hq / Hkv)) * Hkv * B * max_blocks * kPage * 4;
}

}  // namespace lazykv

using namespace lazykv;

extern "C" int lazy_attn_key_weights(const void* q, const float* lse, const int32_t* cu_q, const int32_t* seq_len,
                                     const int32_t* q_start, const int32_t* doc_blocks, const uint64_t* meta, int B,
                                     int max_blocks, int total_q, int max_q, int window, const void* k_cache,
                                     int num_pages, int Hq, int Hkv, int D, float scale, const lazy_pos_cfg* cfg,
                                     int accumulate, float* weights, void* ws, size_t ws_bytes, void* stream) {
  const char* what = "lazy_attn_key_weights";
  Args a = {};
  if (total_q < 0 || max_q < 0 || window < 0) return fail(LAZY_EINVAL, "%s: bad total_q, max_q or window", what);
  int rc = check_shared_call(what, B, max_blocks, Hq, Hkv, D, num_pages, scale, cfg, &a.pos, meta, {k_cache},
                             {cu_q, seq_len, q_start, doc_blocks, weights});
  if (rc) return rc;
  if (B > 0 && total_q > 0 && (!q || !lse)) return fail(LAZY_EINVAL, "%s: NULL pointer", what);
  if (reinterpret_cast<uintptr_t>(q) & 15u) return fail(LAZY_EINVAL, "%s: tensors must be 16-byte aligned", what);
  if ((uint64_t)num_pages * Hkv > 0x7fffffffull) return fail(LAZY_ERANGE, "%s: num_pages * Hkv above 2^31", what);
  rc = check_workspace(what, ws, ws_bytes, B > 0 ? key_weights_ws_bytes(total_q, B, max_blocks, Hq, Hkv) : 0);
  if (!rc) rc = check_device();
  if (rc || B == 0) return rc;
  CUtensorMap mk;
  rc = cache_tensor_map(&mk, k_cache, num_pages, Hkv, D);
  if (rc) return rc;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lse = lse;
  a.cu_q = cu_q;
  a.seq_len = seq_len;
  a.q_start = q_start;
  a.doc_blocks = doc_blocks;
  a.meta = meta;
  a.part = static_cast<float*>(ws);
  a.weights = weights;
  a.status = status_word();
  a.B = B;
  a.max_blocks = max_blocks;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.num_pages = num_pages;
  a.window = window;
  a.accumulate = accumulate;
  long long n = std::min(max_q, total_q);
  if (window > 0) n = std::min<long long>(n, window);
  const bool alibi = a.pos.kind == kAlibi;
  a.rows = most_rows(alibi, n * (Hq / Hkv));
  a.most = int(n);
  a.sums = a.rows <= kFew ? 1 : 2;
  // Row blocks in one block's share, so that it still has runs of 32 pages: a Q operand then serves four tiles, and a
  // run's pages are read from memory once for all of them.  The more groups, the more parts to add.
  const long long nrb = (n * (Hq / Hkv) + a.rows - 1) / a.rows;
  const long long per = std::max(1ll, nrb * max_blocks * B * Hkv / (32ll * sm_count()));
  a.groups = int(std::min(sums_of((long long)total_q * (Hq / Hkv)) / a.sums, std::max(1ll, (nrb + per - 1) / per)));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int kind = a.pos.kind == kYarn ? int(kRope) : a.pos.kind;
  if (kind == kRope && (a.pos.rotary_dim != D || a.pos.interleaved)) kind = kRopeX;
  if (total_q > 0) {
    if (D == 128)
      rc = kind == kRope    ? launch_weights<128, kRope>(a, mk, st)
           : kind == kRopeX ? launch_weights<128, kRopeX>(a, mk, st)
           : kind == kAlibi ? launch_weights<128, kAlibi>(a, mk, st)
                            : launch_weights<128, kNone>(a, mk, st);
    else
      rc = kind == kRope    ? launch_weights<64, kRope>(a, mk, st)
           : kind == kRopeX ? launch_weights<64, kRopeX>(a, mk, st)
           : kind == kAlibi ? launch_weights<64, kAlibi>(a, mk, st)
                            : launch_weights<64, kNone>(a, mk, st);
    if (rc) return rc;
  }
  int slices = 1;
  auto sum_blocks = [&]() { return ((long long)max_blocks * kPage * slices + 4 * kSumThreads - 1) / (4 * kSumThreads); };
  while (slices < 8 && sum_blocks() * B < sm_count() && a.groups * a.sums * Hkv >= 8 * slices) slices *= 2;
  void (*const sum)(const Args) = slices == 1   ? weights_sum_kernel<1>
                                  : slices == 2 ? weights_sum_kernel<2>
                                  : slices == 4 ? weights_sum_kernel<4>
                                                : weights_sum_kernel<8>;
  const dim3 sums(int(std::min<long long>(sum_blocks(), 65535)), B);
  if (total_q > 0) {
    LAZY_CUDA_TRY(launch_pdl(sum, sums, dim3(kSumThreads), 0, st, a));
  } else {  // what comes before has to end first
    sum<<<sums, dim3(kSumThreads), 0, st>>>(a);
    LAZY_CUDA_TRY(cudaGetLastError());
  }
  return LAZY_OK;
}
