// What the calls over shared lists and the key weights have in common (host checks, sizes).
#pragma once

#include <atomic>
#include <cmath>

#include "common.cuh"

namespace lazykv {

// Set a kernel's dynamic shared memory limit, once per device (`done`: one bit per device, per kernel).
template <typename F>
inline cudaError_t smem_limit(F kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Sizes, pointers and the score factor of an attention call over a bf16 cache; `ptrs` may not be null and lie on
// 16-byte boundaries, `ints` may not be null.
int check_shared_call(const char* what, int B, int max_blocks, int Hq, int Hkv, int D, int num_pages, float scale,
                      const lazy_pos_cfg* cfg, PosParams* pos, const void* meta, std::initializer_list<const void*> ptrs,
                      std::initializer_list<const void*> ints);
int check_workspace(const char* what, const void* ws, size_t got, size_t need);

__device__ __forceinline__ bool mbar_peek(uint32_t bar, uint32_t parity) {  // asks, and never waits
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}

// sin and cos of p * theta for a signed position difference p.
__device__ __forceinline__ void turn_sincos_signed(int p, unsigned long long turns, float& s, float& c) {
  const unsigned long long frac = (unsigned long long)(long long)p * turns;
  __sincosf(float(int(uint32_t(frac >> 32))) * 1.4629180792671596e-9f, &s, &c);  // * pi * 2^-31 -> [-pi, pi)
}

// Blocks of a request's list that its last token can see; 0 for an idle request.
__device__ __forceinline__ int visible_blocks(int seq_len, int q_start, int doc_blocks, int max_blocks) {
  if (seq_len <= 0) return 0;
  const int own = seq_len - q_start;  // keys of its query segment
  const long long nb = (long long)max(doc_blocks, 0) + (own > 0 ? (own + kPage - 1) / kPage : 0);
  return int(nb < max_blocks ? nb : max_blocks);
}
// A token at position m of the query segment sees more blocks than a list has words.
__device__ __forceinline__ bool list_too_long(int m, int q_start, int doc_blocks, int max_blocks) {
  return m >= q_start && (long long)doc_blocks + (m - q_start) / kPage + 1 > max_blocks;
}

}  // namespace lazykv
