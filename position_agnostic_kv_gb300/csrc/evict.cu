// Eviction inside a context: the plan (which keys stay, where they go) and the rows' copies.
//
// A stored key is R_j k with j its position in the document, and attention applies R_Delta per page: the row
// a key lies in does not enter.  So keys of one document may move between pages with its Delta as plain row
// copies, and what attention computes over the keys that stay does not change.
//
// The plan's floor is a microsecond or less of bytes; it is a chain of scans, counts and block-wide meetings: 16 lists of
// 32 000 keys 20 us, one of 2000 keys 9 (the host's share of a call included).  The copies read and write every row once:
// 32 000 rows of 8 heads, 262 MB, 41 us, 94 % of the measured copy rate.
#include <algorithm>

#include "common.cuh"

namespace lazykv {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kWarps = kPlanThreads / 32;
constexpr uint32_t kProtected = 0xFFFFFFFFu;

// Whole numbers in the order of the weights: NaN lowest (0), then -inf ... +inf (0xFF800000); -0 equals 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct PlanArgs {
  const float* weights;
  const uint64_t* meta;
  const int32_t* doc_blocks;
  const int32_t* keep;
  const int32_t* dst_pages;
  uint64_t* new_meta;
  int32_t* new_doc_blocks;
  int32_t* src_slot;
  int32_t* dst_slot;
  float* new_weights;
  uint32_t* status;
  int first, recent, max_dst, max_blocks, num_pages;
  int cluster;  // blocks of threads per request
};

// Where a stretch of blocks leaves the packing: whether a document starts in it, the kept keys before its
// first start, the new blocks of the documents that begin and end in it, and the kept keys since its last start.
struct Packed {
  int starts, head, blocks, tail;
};
__device__ __forceinline__ int pages_of(int keys) { return (keys + kPage - 1) / kPage; }
__device__ __forceinline__ Packed join(Packed a, Packed b) {
  Packed r;
  r.starts = a.starts | b.starts;
  r.head = a.starts ? a.head : a.head + b.head;
  r.blocks = a.blocks + b.blocks + (a.starts && b.starts ? pages_of(a.tail + b.head) : 0);
  r.tail = b.starts ? b.tail : a.tail + (a.starts ? b.head : 0);
  return r;
}
__device__ __forceinline__ Packed shfl_up(Packed p, int n) {
  Packed r;
  r.starts = __shfl_up_sync(0xffffffffu, p.starts, n);
  r.head = __shfl_up_sync(0xffffffffu, p.head, n);
  r.blocks = __shfl_up_sync(0xffffffffu, p.blocks, n);
  r.tail = __shfl_up_sync(0xffffffffu, p.tail, n);
  return r;
}

// Sum over the threads before this one; `total` gets the block's.
__device__ __forceinline__ int scan_before(int x, int* buf, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) buf[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = buf[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    buf[lane] = w;
  }
  __syncthreads();
  total = buf[kWarps - 1];
  const int r = v - x + (warp ? buf[warp - 1] : 0);
  __syncthreads();
  return r;
}

// The scan of `me` over the threads: what lies before this thread, and the whole.
__device__ __forceinline__ Packed scan_packed(Packed me, Packed* pbuf, Packed& whole) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Packed inc = me;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Packed y = shfl_up(inc, o);
    if (lane >= o) inc = join(y, inc);
  }
  if (lane == 31) pbuf[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    Packed x = pbuf[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Packed y = shfl_up(x, o);
      if (lane >= o) x = join(y, x);
    }
    pbuf[lane] = x;
  }
  __syncthreads();
  Packed pre = shfl_up(inc, 1);
  if (lane == 0) pre = Packed{0, 0, 0, 0};
  if (warp > 0) pre = join(pbuf[warp - 1], pre);
  whole = pbuf[kWarps - 1];
  return pre;
}

// The new word of list block `blk` with its document's kept keys [16 pg, 16 pg + rows).
__device__ __forceinline__ void put_word(const PlanArgs& a, uint64_t* new_meta, const int32_t* pages, int blk, int pg,
                                         int rows, uint32_t delta) {
  const int page = blk < a.max_dst ? pages[blk] : -1;
  const bool bad = page < 0 || page >= a.num_pages;
  if (bad) set_status(a.status, LAZY_STATUS_BAD_PAGE);
  new_meta[blk] = uint64_t(bad ? 0 : rows) | uint64_t(pg) << 5 | uint64_t(delta) << 16 | uint64_t(bad ? 0 : page) << 40;
}

constexpr int kMaxCluster = 8;
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// An int of the same shared variable in block `rank` of the cluster.
__device__ __forceinline__ int peer_int(const int* p, int rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ int2 peer_int2(const int* p, int rank) {
  uint32_t at;
  int2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}

// Lists of up to 64 IT C document blocks: a cluster of C blocks of threads per request, each with 64 IT list blocks and
// their ordered weights in registers (key 1024 i + t of its part is thread t's i-th).  The keep-th largest is found in
// digits of 11, 11 and 10 bits (the first takes sign, exponent and two bits of fraction, which spreads weights over
// enough counters); every block adds up the cluster's counters.  Kept keys are 16 bits per list block; a scan over the
// list blocks then gives each the place of its first kept key in the new list.
template <int IT>
__global__ void __launch_bounds__(kPlanThreads, 1) evict_plan_short_kernel(const PlanArgs a) {
  constexpr int kBlocks = 64 * IT, kPer = (kBlocks + kPlanThreads - 1) / kPlanThreads;
  constexpr int kBins = 2048;
  __shared__ __align__(8) int hists[2][kBins];
  __shared__ int buf[kWarps];
  __shared__ Packed pbuf[kWarps];
  __shared__ __align__(8) int share[6];  // what the cluster's other blocks read: keys, equals, packing
  __shared__ int place[kBlocks];       // keys before the block; then the new place of its first kept key
  __shared__ int base[kBlocks];        // first new block of its document
  __shared__ uint16_t stays[kBlocks];  // kept keys
  __shared__ uint32_t s_prefix;
  __shared__ int s_left, s_same;
  const int C = a.cluster, b = blockIdx.x / C, rank = blockIdx.x % C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int all_t = rank * kPlanThreads + tid, all_n = C * kPlanThreads;  // of the cluster's threads
  pdl_wait();
  pdl_trigger();
  const size_t MB = a.max_blocks;
  const uint64_t* meta = a.meta + b * MB;
  const float* w = a.weights + b * MB * kPage;
  uint64_t* new_meta = a.new_meta + b * MB;
  float* new_w = a.new_weights + b * MB * kPage;
  const int32_t* pages = a.dst_pages + (size_t)b * a.max_dst;
  int32_t* src = a.src_slot + (size_t)b * a.max_dst * kPage;
  int32_t* dst = a.dst_slot + (size_t)b * a.max_dst * kPage;
  const int nd = min(max(a.doc_blocks[b], 0), a.max_blocks);
  const int want = a.keep[b];
  const int j0 = rank * kBlocks;  // this block's first list block
  uint32_t v[IT];  // the weights, all loads in flight at once; then their ordered values, 0 where no key lies, NaN 1
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = j0 * kPage + i * kPlanThreads + tid;
    v[i] = k < nd * kPage ? __float_as_uint(w[k]) : 0u;
  }
  // this thread's list blocks: kPer consecutive ones, so that scans over the threads are scans over the list
  uint64_t word[kPer + 2];  // and a neighbour on either side
#pragma unroll
  for (int e = 0; e < kPer + 2; ++e) {
    const int j = j0 + tid * kPer + e - 1;
    word[e] = tid * kPer + e - 1 <= kBlocks && j >= 0 && j < nd ? meta[j] : 0;
  }
  for (int i = all_t; i < a.max_dst * kPage; i += all_n) src[i] = dst[i] = -1;
  if (want < 0) {  // the same for the whole cluster
    for (int i = all_t; i < a.max_blocks; i += all_n) new_meta[i] = meta[i];
    for (int i = all_t; i < a.max_blocks * kPage; i += all_n) new_w[i] = w[i];
    if (all_t == 0) a.new_doc_blocks[b] = nd;
    return;
  }
  if (tid == 0) {
    s_prefix = 0;
    if (rank == 0 && a.doc_blocks[b] > a.max_blocks) set_status(a.status, LAZY_STATUS_BAD_ROW);
  }

  int nv[kPer], mine = 0, total;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    nv[e] = tid * kPer + e < kBlocks ? min(int(word_nvalid(word[e + 1])), kPage) : 0;
    mine += nv[e];
  }
  int before = scan_before(mine, buf, total);
  // Sum of share[k] over the blocks before this one; `sum` gets the cluster's.
  auto across = [&](int k, int& sum) {
    int pre = 0;
    sum = 0;
    if (C == 1) {
      sum = share[k];
      return 0;
    }
    int x[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) x[r] = r < C ? peer_int(&share[k], r) : 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      pre += r < rank ? x[r] : 0;
      sum += x[r];
    }
    return pre;
  };
  auto meet = [&] {
    if (C == 1) __syncthreads(); else cluster_sync();
  };
  if (tid == 0) share[0] = total;
  meet();
  before += across(0, total);
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int j = tid * kPer + e;
    if (j < kBlocks) {
      place[j] = before;
      stays[j] = uint16_t(nv[e]);
    }
    before += nv[e];
  }
  const int keep = min(want, total);
  __syncthreads();

#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int j = (i * kPlanThreads + tid) / kPage, t = tid % kPage, nth = place[j] + t;
    const uint32_t x = nth < a.first || nth >= total - a.recent ? kProtected : max(order_of(__uint_as_float(v[i])), 1u);
    v[i] = t < stays[j] ? x : 0u;
  }

  // ---- the keep-th largest value, `limit`, of which `ties` equals stay
  int ties = keep;
  uint32_t limit = 0;
  if (keep > 0) {
#pragma unroll
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0), bins = round == 2 ? 1024 : kBins;
      const uint32_t mask = round == 0 ? 0u : 0xFFFFFFFFu << (round == 1 ? 21 : 10);
      int* hist = hists[round & 1];  // (the other blocks have read the last but one by now)
      hist[tid] = hist[tid + 1024] = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < IT; ++i)
        if (v[i] != 0 && (v[i] & mask) == limit) atomicAdd(&hist[(v[i] >> shift) & (bins - 1)], 1);
      meet();
      // thread t holds the digits bins - 1 - 2 t and the one below
      const int d = kBins - 1 - 2 * tid;
      int c0 = 0, c1 = 0;
      if (C == 1) {
        c0 = d < bins ? hist[d] : 0;
        c1 = d < bins ? hist[d - 1] : 0;
      } else if (d < bins) {
        int2 x[kMaxCluster];  // all loads in flight at once
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) x[r] = r < C ? peer_int2(&hist[d - 1], r) : make_int2(0, 0);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          c0 += x[r].y;
          c1 += x[r].x;
        }
      }
      int all;
      const int above = scan_before(c0 + c1, buf, all);
      if (above < ties && ties <= above + c0 + c1) {
        const bool second = ties > above + c0;
        s_prefix = limit | uint32_t(second ? d - 1 : d) << shift;
        s_left = ties - above - (second ? c0 : 0);
        s_same = second ? c1 : c0;
      }
      __syncthreads();
      limit = s_prefix;
      ties = s_left;
    }
  }

  // ---- who stays, 16 bits per list block; among equals the earlier in the list
  int* counts = hists[1];  // (round 2 used the other)
  int same_before = 0;
  if (keep > 0 && s_same != ties) {  // (uniform) not all of them: count the equals before each warp's keys
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const uint32_t eq = __ballot_sync(0xffffffffu, v[i] == limit);
      if (lane == 0) counts[i * kWarps + warp] = __popc(eq);
    }
    __syncthreads();
    int sum;
    const int c = tid < IT * kWarps ? counts[tid] : 0, c_before = scan_before(c, buf, sum);
    if (tid < IT * kWarps) counts[tid] = c_before;
    if (tid == 0) share[1] = sum;
    meet();
    same_before = across(1, sum);
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    bool stay = keep > 0 && v[i] >= limit && v[i] != 0;
    if (keep > 0 && s_same != ties) {
      const uint32_t eq = __ballot_sync(0xffffffffu, v[i] == limit);
      if (v[i] == limit) stay = same_before + counts[i * kWarps + warp] + __popc(eq & ((1u << lane) - 1u)) < ties;
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, stay);
    const int j = (i * kPlanThreads + tid) / kPage;
    if (lane % kPage == 0) stays[j] = uint16_t(bits >> lane);
  }
  __syncthreads();

  // ---- packing, document by document
  uint32_t kept[kPer];
  bool starts[kPer], ends[kPer];
  Packed me = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int jl = tid * kPer + e, j = j0 + jl;
    const bool here = jl < kBlocks && j < nd;
    const uint32_t delta = word_delta(word[e + 1]);
    kept[e] = here ? __popc(uint32_t(stays[jl])) : 0;
    starts[e] = here && (j == 0 || word_delta(word[e]) != delta);
    ends[e] = here && (j + 1 == nd || word_delta(word[e + 2]) != delta);
    if (starts[e]) me = join(me, Packed{1, 0, 0, 0});
    if (me.starts) me.tail += kept[e]; else me.head += kept[e];
  }
  Packed whole;
  Packed pre = scan_packed(me, pbuf, whole);
  if (tid == 0) {
    share[2] = whole.starts;
    share[3] = whole.head;
    share[4] = whole.blocks;
    share[5] = whole.tail;
  }
  meet();
  if (C > 1) {
    Packed of[kMaxCluster], all = {0, 0, 0, 0}, lower = all;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < C) {
        const int2 p = peer_int2(&share[2], r), q = peer_int2(&share[4], r);
        of[r] = Packed{p.x, p.y, q.x, q.y};
      }
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < C) {
        if (r == rank) lower = all;
        all = join(all, of[r]);
      }
    pre = join(lower, pre);
    whole = all;
  }
  const int nn = whole.blocks + (whole.starts ? pages_of(whole.tail) : 0);  // document blocks of the new list
  int first_block = pre.starts ? pre.blocks : 0, run = pre.starts ? pre.tail : 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int j = tid * kPer + e;
    if (starts[e]) {
      first_block += pages_of(run);
      run = 0;
    }
    if (j < kBlocks) {
      place[j] = first_block * kPage + run;
      base[j] = first_block;
    }
    run += kept[e];
    if (ends[e] && run % kPage)
      put_word(a, new_meta, pages, first_block + run / kPage, run / kPage, run % kPage, word_delta(word[e + 1]));
  }

  // ---- the rest of the new list: the query segment's blocks and weights, and zeros
  for (int i = all_t; i < nn * kPage; i += all_n) new_w[i] = 0.f;
  for (int i = all_t + nn; i < a.max_blocks; i += all_n) new_meta[i] = i - nn + nd < a.max_blocks ? meta[i - nn + nd] : 0;
  for (int i = all_t + nn * kPage; i < a.max_blocks * kPage; i += all_n)
    new_w[i] = i + (nd - nn) * kPage < a.max_blocks * kPage ? w[i + (nd - nn) * kPage] : 0.f;
  if (all_t == 0) a.new_doc_blocks[b] = nn;
  meet();  // (also: no block leaves while another reads from it)

  // ---- kept keys: slots, weights, and the words of full pages
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int j = (i * kPlanThreads + tid) / kPage, t = tid % kPage;
    const uint32_t bits = stays[j];
    if (!((bits >> t) & 1u)) continue;
    const int at = place[j] + __popc(bits & ((1u << t) - 1u)), blk = at / kPage, row = at % kPage;
    const uint64_t here = meta[j0 + j];
    const int page = blk < a.max_dst ? pages[blk] : -1;
    if (page >= 0 && page < a.num_pages) {
      src[at] = int(word_page(here)) * kPage + t;
      dst[at] = page * kPage + row;
      new_w[at] = w[j0 * kPage + i * kPlanThreads + tid];
    }
    if (row == kPage - 1) put_word(a, new_meta, pages, blk, blk - base[j], kPage, word_delta(here));
  }
}

// Longer lists.  One block of threads per request.  Thread t owns a run of consecutive list blocks, so that prefix sums over
// the threads are prefix sums over the list.  The keep-th largest weight is found digit by digit (8 bits of
// the ordered value at a time, counts in shared memory); keys above it stay, and as many of its equals as are
// needed, in list order.
__global__ void __launch_bounds__(kPlanThreads) evict_plan_kernel(const PlanArgs a) {
  __shared__ int hist[256];
  __shared__ int buf[kWarps];
  __shared__ Packed pbuf[kWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const size_t MB = a.max_blocks;
  const uint64_t* meta = a.meta + b * MB;
  const float* w = a.weights + b * MB * kPage;
  uint64_t* new_meta = a.new_meta + b * MB;
  float* new_w = a.new_weights + b * MB * kPage;
  const int32_t* pages = a.dst_pages + (size_t)b * a.max_dst;
  int32_t* src = a.src_slot + (size_t)b * a.max_dst * kPage;
  int32_t* dst = a.dst_slot + (size_t)b * a.max_dst * kPage;
  const int nd = min(max(a.doc_blocks[b], 0), a.max_blocks);
  const int want = a.keep[b];
  for (int i = tid; i < a.max_dst * kPage; i += kPlanThreads) src[i] = dst[i] = -1;
  if (want < 0) {
    for (int i = tid; i < a.max_blocks; i += kPlanThreads) new_meta[i] = meta[i];
    for (int i = tid; i < a.max_blocks * kPage; i += kPlanThreads) new_w[i] = w[i];
    if (tid == 0) a.new_doc_blocks[b] = nd;
    return;
  }

  const int per = (nd + kPlanThreads - 1) / kPlanThreads;
  const int beg = min(nd, tid * per), end = min(nd, beg + per);
  int mine = 0, total;
  for (int j = beg; j < end; ++j) mine += min(int(word_nvalid(meta[j])), kPage);
  const int before = scan_before(mine, buf, total);
  const int keep = min(want, total);
  auto value = [&](int j, int t, int rank) -> uint32_t {
    return rank < a.first || rank >= total - a.recent ? kProtected : order_of(w[(size_t)j * kPage + t]);
  };

  // ---- the keep-th largest value: s_prefix, of which s_left equals stay
  if (tid == 0) {
    s_prefix = 0;
    s_left = keep;
  }
  if (keep > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      int rank = before;
      for (int j = beg; j < end; ++j) {
        const int nv = min(int(word_nvalid(meta[j])), kPage);
        for (int t = 0; t < nv; ++t, ++rank) {
          const uint32_t v = value(j, t, rank);
          if ((v & mask) == prefix) atomicAdd(&hist[(v >> shift) & 255], 1);
        }
      }
      __syncthreads();
      if (warp == 0) {  // lane l holds digits 255 - 8 l downwards
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
        int up = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, up, o);
          if (lane >= o) up += y;
        }
        int left = s_left - (up - sum);
        __syncwarp();
        if (left > 0 && left <= sum) {
          int i = 0;
          while (left > c[i]) left -= c[i++];
          s_prefix = prefix | uint32_t(255 - 8 * lane - i) << shift;
          s_left = left;
        }
      }
      __syncthreads();
    }
  }
  __syncthreads();
  const uint32_t limit = s_prefix;
  const int ties = keep > 0 ? s_left : 0;

  // ---- how many equals come before this thread's blocks
  int same = 0, all_same;
  {
    int rank = before;
    for (int j = beg; j < end; ++j) {
      const int nv = min(int(word_nvalid(meta[j])), kPage);
      for (int t = 0; t < nv; ++t, ++rank) same += value(j, t, rank) == limit;
    }
  }
  const int same_before = scan_before(same, buf, all_same);

  // ---- packing: kept keys per document
  auto walk = [&](auto&& on_start, auto&& on_key, auto&& on_end) {
    int rank = before, tie = same_before;
    for (int j = beg; j < end; ++j) {
      const uint64_t word = meta[j];
      if (j == 0 || word_delta(meta[j - 1]) != word_delta(word)) on_start();
      const int nv = min(int(word_nvalid(word)), kPage);
      for (int t = 0; t < nv; ++t, ++rank) {
        const uint32_t v = value(j, t, rank);
        const bool stays = keep > 0 && (v > limit || (v == limit && tie++ < ties));
        if (stays) on_key(j, t, word);
      }
      if (j + 1 == nd || word_delta(meta[j + 1]) != word_delta(word)) on_end(word);
    }
  };
  Packed me = {0, 0, 0, 0};
  walk([&] {
    me = join(me, Packed{1, 0, 0, 0});
  }, [&](int, int, uint64_t) {
    if (me.starts) ++me.tail; else ++me.head;
  }, [](uint64_t) {});
  Packed whole;
  const Packed pre = scan_packed(me, pbuf, whole);
  const int nn = whole.blocks + (whole.starts ? pages_of(whole.tail) : 0);  // document blocks of the new list

  // ---- the rest of the new list: the query segment's blocks and weights, and zeros
  for (int i = tid; i < nn * kPage; i += kPlanThreads) new_w[i] = 0.f;
  for (int i = tid + nn; i < a.max_blocks; i += kPlanThreads) new_meta[i] = i - nn + nd < a.max_blocks ? meta[i - nn + nd] : 0;
  for (int i = tid + nn * kPage; i < a.max_blocks * kPage; i += kPlanThreads)
    new_w[i] = i + (nd - nn) * kPage < a.max_blocks * kPage ? w[i + (nd - nn) * kPage] : 0.f;
  if (tid == 0) {
    a.new_doc_blocks[b] = nn;
    if (a.doc_blocks[b] > a.max_blocks) set_status(a.status, LAZY_STATUS_BAD_ROW);
  }
  __syncthreads();

  // ---- kept keys: slots, weights, words
  int base = pre.blocks, run = pre.tail;  // new blocks before the document, kept keys of it so far
  if (!pre.starts) base = run = 0;
  auto put = [&](int rows, uint64_t word) {  // of the page that holds the document's kept key `run - 1`
    put_word(a, new_meta, pages, base + (run - 1) / kPage, (run - 1) / kPage, rows, word_delta(word));
  };
  walk([&] {
    base += pages_of(run);
    run = 0;
  }, [&](int j, int t, uint64_t word) {
    const int blk = base + run / kPage, row = run % kPage;
    ++run;
    const int page = blk < a.max_dst ? pages[blk] : -1;
    if (page >= 0 && page < a.num_pages) {
      src[blk * kPage + row] = int(word_page(word)) * kPage + t;
      dst[blk * kPage + row] = page * kPage + row;
      new_w[(size_t)blk * kPage + row] = w[(size_t)j * kPage + t];
    }
    if (row == kPage - 1) put(kPage, word);
  }, [&](uint64_t word) {
    if (run % kPage) put(run % kPage, word);
  });
}

// A warp copies one row of every head, keys and values: D / 8 lanes to a row, 16 bytes a lane.
template <int D>
__global__ void __launch_bounds__(256) kv_move_kernel(const int32_t* __restrict__ src_slot,
                                                      const int32_t* __restrict__ dst_slot, int T, int Hkv,
                                                      uint4* k_cache, uint4* v_cache, int num_pages, uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  constexpr int LPR = D / 8, HPS = 32 / LPR;  // lanes per row, heads per step
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= T) return;
  const int from = src_slot[i], to = dst_slot[i];
  if (from < 0 || to < 0) return;
  if (from >= num_pages * kPage || to >= num_pages * kPage) {
    if (lane == 0) set_status(status, LAZY_STATUS_BAD_SLOT);
    return;
  }
  const int h0 = lane / LPR, c = lane % LPR;
  const size_t at = (size_t)(from / kPage) * Hkv * kPage * LPR + (from % kPage) * LPR + c;
  const size_t go = (size_t)(to / kPage) * Hkv * kPage * LPR + (to % kPage) * LPR + c;
  for (int h = h0; h < Hkv; h += HPS) {
    const uint4 k = k_cache[at + (size_t)h * kPage * LPR], v = v_cache[at + (size_t)h * kPage * LPR];
    k_cache[go + (size_t)h * kPage * LPR] = k;
    v_cache[go + (size_t)h * kPage * LPR] = v;
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

}  // namespace lazykv

using namespace lazykv;

extern "C" int lazy_evict_plan(const float* weights, const uint64_t* meta, const int32_t* doc_blocks,
                               const int32_t* keep, int first, int recent, const int32_t* dst_pages, int max_dst,
                               int B, int max_blocks, int num_pages, const lazy_pos_cfg* cfg, uint64_t* new_meta,
                               int32_t* new_doc_blocks, int32_t* src_slot, int32_t* dst_slot, float* new_weights,
                               void* stream) {
  const char* what = "lazy_evict_plan";
  if (B < 0 || max_blocks <= 0 || max_dst <= 0 || num_pages <= 0)
    return fail(LAZY_EINVAL, "%s: bad sizes (B=%d max_blocks=%d max_dst=%d num_pages=%d)", what, B, max_blocks, max_dst,
                num_pages);
  if (first < 0 || recent < 0) return fail(LAZY_EINVAL, "%s: first and recent must not be negative", what);
  if (num_pages > (1 << 24)) return fail(LAZY_ERANGE, "%s: num_pages above 2^24", what);
  if (B > (1 << 24)) return fail(LAZY_ERANGE, "%s: B above 2^24", what);
  if (max_blocks > (1 << 26) || max_dst > (1 << 26)) return fail(LAZY_ERANGE, "%s: lists above 2^26 blocks", what);
  if (!cfg) return fail(LAZY_EINVAL, "%s: pos cfg is NULL", what);
  if (cfg->kind < LAZY_POS_ROPE || cfg->kind > LAZY_POS_NONE)
    return fail(LAZY_EINVAL, "%s: unknown positional kind %d", what, cfg->kind);
  if (cfg->kind == LAZY_POS_ALIBI)
    return fail(LAZY_EINVAL, "%s: with ALiBi a key's position is its row's, so keys cannot be packed", what);
  if (B > 0) {
    if (!weights || !meta || !doc_blocks || !keep || !dst_pages || !new_meta || !new_doc_blocks || !src_slot || !dst_slot ||
        !new_weights)
      return fail(LAZY_EINVAL, "%s: NULL pointer", what);
    if (!aligned(meta, 8) || !aligned(new_meta, 8)) return fail(LAZY_EINVAL, "%s: meta must be 8-byte aligned", what);
    if (meta == new_meta || weights == new_weights)
      return fail(LAZY_EINVAL, "%s: the new list and weights cannot take the place of the old", what);
  }
  int rc = check_device();
  if (rc || B == 0) return rc;
  PlanArgs a = {weights,  meta,     doc_blocks,  keep,          dst_pages, new_meta, new_doc_blocks, src_slot,
                dst_slot, new_weights, status_word(), first,    recent,    max_dst,  max_blocks,     num_pages, 1};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Keys a thread and blocks of threads a list.  Few keys a thread shorten the block's chain of loops, more blocks make
  // its meetings dearer: 16 lists of 2000 blocks take 32 us with one block of 32 keys a thread each, 26 with two of 16, 20
  // with four of 8 and 39 with eight of 4 (clusters of eight whole SMs do not all fit at once).
  auto clusters = [&](int per) {  // blocks of `per` list blocks each, a power of two
    int c = 1;
    while (c * per < max_blocks) c *= 2;
    return c;
  };
  const int its = max_blocks <= 256 ? 4 : max_blocks <= 8 * 512 && (long long)B * clusters(512) <= 2 * sm_count() ? 8 : 16;
  if (max_blocks <= 8 * 1024) {
    auto kern = its == 4 ? evict_plan_short_kernel<4> : its == 8 ? evict_plan_short_kernel<8> : evict_plan_short_kernel<16>;
    a.cluster = clusters(64 * its);
    LAZY_CUDA_TRY(launch_pdl_cluster(kern, dim3((unsigned)B * a.cluster), dim3(kPlanThreads), 0, st, a.cluster, a));
  } else {
    LAZY_CUDA_TRY(launch_pdl(evict_plan_kernel, dim3(B), dim3(kPlanThreads), 0, st, a));
  }
  return LAZY_OK;
}

extern "C" int lazy_kv_move(const int32_t* src_slot, const int32_t* dst_slot, int T, int Hkv, int D, void* k_cache,
                            void* v_cache, int num_pages, void* stream) {
  const char* what = "lazy_kv_move";
  if (T < 0 || Hkv <= 0 || num_pages <= 0)
    return fail(LAZY_EINVAL, "%s: bad sizes (T=%d Hkv=%d num_pages=%d)", what, T, Hkv, num_pages);
  if (D != 64 && D != 128) return fail(LAZY_EINVAL, "%s: head_dim must be 64 or 128, got %d", what, D);
  if (num_pages > (1 << 24)) return fail(LAZY_ERANGE, "%s: num_pages above 2^24", what);
  if (T > 0x7fffffff - 7) return fail(LAZY_ERANGE, "%s: T must be below 2^31 - 7", what);  // (8 rows to a block of threads)
  if (T > 0) {
    if (!src_slot || !dst_slot || !k_cache || !v_cache) return fail(LAZY_EINVAL, "%s: NULL pointer", what);
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return fail(LAZY_EINVAL, "%s: caches must be 16-byte aligned", what);
  }
  int rc = check_device();
  if (rc || T == 0) return rc;
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3((T + 7) / 8), dim3(256), 0, static_cast<cudaStream_t>(stream), src_slot, dst_slot, T,
                      Hkv, static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), num_pages, status_word());
  };
  LAZY_CUDA_TRY(D == 128 ? go(kv_move_kernel<128>) : go(kv_move_kernel<64>));
  return LAZY_OK;
}
