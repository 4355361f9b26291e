// Arguments of the attention kernels over the 4-bit cache.
#pragma once

#include <algorithm>
#include <atomic>
#include <cmath>

#include "q4.cuh"

namespace lazykv {

struct Q4Args {
  const __nv_bfloat16* q;
  const int32_t* seq_len;     // decode: [B]; null for prefill
  const int32_t* cu_q;        // prefill: [B + 1]; null for decode
  const int32_t* q_start;
  const int32_t* doc_blocks;
  const uint64_t* meta;
  const uint8_t* cache;       // [num_pages][Hkv][18 D]
  int num_pages, B, max_blocks, Hq, Hkv, rows;
  float qk_log2;              // softmax scale * log2(e) * k factor: scores in base-2 units
  int lowest_ex;              // q4_lowest_exponent(qk_log2)
  float v_factor;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;              // [rows][Hq][S][D] unnormalised partial outputs (S > 1)
  float* part_ml;             // [rows][Hq][S][2] their base-2 maximum and sum
  int S;                      // key splits
  uint32_t* status;
  PosParams pos;
};

// Whether a query row belongs to a request (decode: every row does).  A batch padded to a fixed number of rows
// has some behind the last sequence; their outputs stay as they were.
__device__ __forceinline__ bool q4_in_request(const int32_t* cu_q, int B, int r) {
  return cu_q == nullptr || (r >= cu_q[0] && r < cu_q[B]);
}

// Query row -> request b and absolute position m; number of blocks nb that m can see.
struct Q4Row {
  int b, m, nb;
};
template <bool ROWS>
__device__ __forceinline__ Q4Row q4_row(const Q4Args& a, int r) {
  Q4Row w;
  if constexpr (ROWS) {
    int lo = 0, hi = a.B;  // last b with cu_q[b] <= r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_q[mid] <= r) lo = mid; else hi = mid;
    }
    w.b = lo;
    w.m = a.q_start[lo] + (r - a.cu_q[lo]);
  } else {
    w.b = r;
    w.m = a.seq_len[r] - 1;
  }
  const int rel = w.m - a.q_start[w.b];  // negative: the request has no token of its own yet
  w.nb = max(0, a.doc_blocks[w.b]) + (rel >= 0 ? rel / kPage + 1 : 0);
  return w;
}

// Rows of a block that hold a key visible to position m (a prefix of the page).
__device__ __forceinline__ int q4_rows(uint64_t w, int m) {
  const int start = int(word_delta(w) + kPage * word_pg(w));
  return max(0, min(min(int(word_nvalid(w)), kPage), m - start + 1));
}

// Exponent ex of the power of two that normalises a query row whose largest magnitude is `top`: the row
// times 2^-ex lies in [-1, 1].  Rows below 2^lowest keep ex = 0 and become zeros (infinities and NaN too, and
// pass through): a sum of D products with keys below 2^12 times the score factor is then below 2^-100.
__device__ __forceinline__ int q4_exponent(float top, int lowest) {
  const int ex = int(__float_as_uint(top) >> 23) - 126;
  return ex < lowest || ex > 128 ? 0 : min(ex, 126);
}
// The lowest exponent that leaves 2^-ex, and the score factor times 2^ex, normal numbers.
inline int q4_lowest_exponent(float qk_log2) { return std::max(-126, -120 - std::ilogb(qk_log2)); }

// Set a kernel's dynamic shared memory limit, once per device (`done`: one bit per device, per kernel).
template <typename F>
inline cudaError_t q4_smem_limit(F kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

bool q4_use_tc(int Hq, int Hkv);
int q4_tc_splits(int B, int Hkv, int max_blocks);
cudaError_t q4_merge(const Q4Args& a, int D, cudaStream_t st);
int run_q4_tc(Q4Args& a, int D, int max_q, cudaStream_t st);
int run_q4_rows(Q4Args& a, int D, bool rows_mode, void* ws, size_t ws_bytes, cudaStream_t st);
size_t q4_ws_bytes(int rows, int Hq, int Hkv, int D, int max_blocks, bool rows_mode);

}  // namespace lazykv
