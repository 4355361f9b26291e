// Arguments of the decode over lists that share their first documents.
#pragma once

#include <cuda.h>  // CUtensorMap

#include "share.cuh"

namespace lazykv {

struct SharedArgs {
  const __nv_bfloat16* q;
  const int32_t* seq_len;
  const int32_t* q_start;
  const int32_t* doc_blocks;
  const uint64_t* meta;
  const int32_t* group_off;
  const int32_t* shared_blocks;
  int n_groups, max_group, max_shared, B, max_blocks, num_pages, Hq, Hkv;
  __nv_bfloat16* out;
  float* lse;
  // partial results, [B][Hq][SA + SB] of them: SA from the common keys, SB from each request's own
  float* part_o;   // [...][D] unnormalised
  float* part_ml;  // [...][2] base-2 maximum and sum
  int SA, SB;
  uint32_t* status;
  PosParams pos;
};

// Where a request's common keys end: group g (-1: none), and the blocks of its list that its group's launch
// has taken.  Every kernel of a call goes by this.
struct Share {
  int g, blocks;
};
__device__ __forceinline__ int shared_blocks_of(const SharedArgs& a, int g) {
  return min(min(max(a.shared_blocks[g], 0), a.max_shared), a.max_blocks);
}
__device__ __forceinline__ Share share_of(const SharedArgs& a, int b) {
  if (a.SA == 0 || b < a.group_off[0] || b >= a.group_off[a.n_groups]) return {-1, 0};
  int lo = 0;  // last group with group_off[g] <= b; up to 31 by one load of the warp (every lane has the same b)
  if (a.n_groups <= 31) {
    const int lane = threadIdx.x & 31;
    const bool at = lane < a.n_groups && a.group_off[lane] <= b;
    lo = 31 - __clz(int(__ballot_sync(0xffffffffu, at)));
  } else {
    int hi = a.n_groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.group_off[mid] <= b) lo = mid; else hi = mid;
    }
  }
  if (b - a.group_off[lo] >= a.max_group) return {-1, 0};
  return {lo, shared_blocks_of(a, lo)};
}

// Reports a list that is longer than max_blocks, and a group or its common blocks above the call's bounds (a block of
// threads per request).
__device__ __forceinline__ void check_request(const SharedArgs& a, int b, int m) {
  bool bad = threadIdx.x == 0 && m >= 0 && list_too_long(m, a.q_start[b], a.doc_blocks[b], a.max_blocks);
  for (int g = threadIdx.x; b == 0 && g < a.n_groups; g += blockDim.x)
    bad |= a.group_off[g + 1] - a.group_off[g] > a.max_group || a.shared_blocks[g] > a.max_shared;
  if (bad) set_status(a.status, LAZY_STATUS_BAD_ROW);
}

// Key splits: of the common keys (in tiles of 8 blocks), and of a request's own blocks.
__device__ __forceinline__ int split_tiles(int tiles, int S) { return (tiles + S - 1) / S; }
__device__ __forceinline__ int own_splits(int blocks, int SB) { return min(SB, max(1, (blocks + 31) / 32)); }

int cache_tensor_map(CUtensorMap* map, const void* base, int num_pages, int Hkv, int D);
int run_shared_own(const SharedArgs& a, int D, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st);
int run_shared_prefix(const SharedArgs& a, int D, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st);
int shared_prefix_splits(int B, int n_groups, int max_group, int max_shared, int Hq, int Hkv);

// 3-D tiled load (column x, row y inside the page, page-head z) of a box of 64 columns x 16 rows.  y may be
// negative: the rows before row 0 are outside the tensor and arrive as zeros; the transaction counts the
// whole box.  x is a multiple of 64 elements.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

}  // namespace lazykv
