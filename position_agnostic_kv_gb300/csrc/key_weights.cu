// The attention weight that every cached key receives: w_k = sum over query rows i and heads h of
// 2^(s_ihk - lse_ih), s in base 2.
#include "share.cuh"

namespace lazykv {

namespace {

struct Args {
  const __nv_bfloat16* q;
  const float* lse;
  const int32_t* cu_q;
  const int32_t* seq_len;
  const int32_t* q_start;
  const int32_t* doc_blocks;
  const uint64_t* meta;
  const __nv_bfloat16* k_cache;
  float* part;  // [Hkv][B][16 max_blocks]
  float* weights;
  uint32_t* status;
  int B, max_blocks, Hq, Hkv, num_pages, window, accumulate;
  PosParams pos;
};

// One block of 128 threads per (list block, KV head, request): 8 threads to a key.
template <int D>
__global__ void __launch_bounds__(128) weights_kernel(const Args a) {
  __shared__ float qs[D], qr[D];
  pdl_wait();
  pdl_trigger();
  const int j = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int G = a.Hq / a.Hkv, key = tid / 8, c0 = tid % 8 * (D / 8);
  const int nb = visible_blocks(a.seq_len[b], a.q_start[b], a.doc_blocks[b], a.max_blocks);
  float sum = 0.f;
  if (j < nb) {
    const uint64_t w = a.meta[(size_t)b * a.max_blocks + j];
    const int delta = int(word_delta(w)), p = delta + kPage * int(word_pg(w)) + key;
    const uint32_t page = word_page(w);
    if (page < uint32_t(a.num_pages)) {
      const __nv_bfloat16* k = a.k_cache + (((size_t)page * a.Hkv + kvh) * kPage + key) * D + c0;
      const int hi = a.cu_q[b + 1], n = a.window > 0 ? min(a.window, hi - a.cu_q[b]) : hi - a.cu_q[b];
      const bool rotary = a.pos.kind == kRope || a.pos.kind == kYarn;
      const int hr = a.pos.rotary_dim / 2;
      for (int i = 0; i < n * G; ++i) {
        const int row = hi - n + i / G, h = kvh * G + i % G, m = a.seq_len[b] - (hi - row);
        __syncthreads();
        for (int d = tid; d < D; d += 128) qs[d] = __bfloat162float(a.q[((size_t)row * a.Hq + h) * D + d]);
        __syncthreads();
        for (int d = tid; d < D; d += 128) {
          float y = qs[d];
          if (rotary && d < 2 * hr) {
            const int f = a.pos.interleaved ? d / 2 : d % hr, other = a.pos.interleaved ? d ^ 1 : (d < hr ? d + hr : d - hr);
            float sn, cs;
            turn_sincos_signed(m - delta, a.pos.turns[f], sn, cs);
            y = y * cs + (other > d ? -qs[other] : qs[other]) * sn;
          }
          qr[d] = y * a.pos.scale_log2;
        }
        __syncthreads();
        float s = 0.f;
        if (key < int(word_nvalid(w)) && p <= m)
          for (int e = 0; e < D / 8; ++e) s += __bfloat162float(k[e]) * qr[c0 + e];
        for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (a.pos.kind == kAlibi) s += a.pos.slopes[h] * 1.4426950408889634f * float(p - m);
        const float lse = a.lse[(size_t)row * a.Hq + h];
        if (key < int(word_nvalid(w)) && p <= m && lse != -INFINITY) sum += exp2f(s - lse * 1.4426950408889634f);
      }
    } else if (tid == 0) {
      set_status(a.status, LAZY_STATUS_BAD_PAGE);
    }
  }
  if (tid % 8 == 0) a.part[(((size_t)kvh * a.B + b) * a.max_blocks + j) * kPage + key] = sum;
}

// Adds the KV heads' parts in order.
__global__ void __launch_bounds__(256) weights_sum_kernel(const float* __restrict__ part, int Hkv, size_t n,
                                                          int accumulate, float* __restrict__ weights) {
  pdl_wait();
  pdl_trigger();
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = accumulate ? weights[i] : 0.f;
  float t = 0.f;
  for (int h = 0; h < Hkv; ++h) t += part[h * n + i];
  weights[i] = s + t;
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

size_t key_weights_ws_bytes(int B, int Hkv, int max_blocks) { return (size_t)Hkv * B * max_blocks * kPage * 4; }

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
  rc = check_workspace(what, ws, ws_bytes, key_weights_ws_bytes(B, Hkv, max_blocks));
  if (!rc) rc = check_device();
  if (rc || B == 0) return rc;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lse = lse;
  a.cu_q = cu_q;
  a.seq_len = seq_len;
  a.q_start = q_start;
  a.doc_blocks = doc_blocks;
  a.meta = meta;
  a.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
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
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(max_blocks, Hkv, B);
  LAZY_CUDA_TRY(D == 128 ? launch_pdl(weights_kernel<128>, grid, dim3(128), 0, st, a)
                         : launch_pdl(weights_kernel<64>, grid, dim3(128), 0, st, a));
  const size_t n = (size_t)B * max_blocks * kPage;
  if ((n + 255) / 256 > 0x7fffffffu) return fail(LAZY_ERANGE, "%s: more than 2^39 weights", what);
  LAZY_CUDA_TRY(launch_pdl(weights_sum_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, st,
                           (const float*)a.part, Hkv, n, accumulate, weights));
  return LAZY_OK;
}
