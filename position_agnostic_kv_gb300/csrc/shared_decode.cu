// Decode of a batch whose requests share their first documents: entry point, and the join of the partial
// results of the common keys and of each request's own.
#include <algorithm>

#include "shared_decode.cuh"

namespace lazykv {

namespace {

// A row's partial results joined by their maxima: out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.  One block of
// kJoinWarps warps per row; every warp takes the maxima and sums (its lanes up to 4 each), then every
// kJoinWarps-th result.  Its bytes are the partial results, 20 MB for 64 requests of 32 heads with 19 each: 11 us from
// cold caches, 7 of the call's 52 after the kernels that wrote them, half of it the launch and the first loads.  With 2
// warps 53.5 (32 heads of one KV head: 27.1 instead of 25.5), with 8 57.5; waiting before the lists are read 53.4.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const SharedArgs a) {
  constexpr int V = D / 32;  // columns per lane
  __shared__ float part[kJoinWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hq = blockIdx.x, b = blockIdx.y;
  const size_t row = (size_t)b * a.Hq + hq, at = row * (a.SA + a.SB);
  // The lists are as they were before the call's first launch, which waited for what came before it.
  const Share sh = share_of(a, b);
  const int tiles = (sh.blocks + 7) / 8, chunk = tiles ? split_tiles(tiles, a.SA) : 1, na = (tiles + chunk - 1) / chunk;
  const int nb = visible_blocks(a.seq_len[b], a.q_start[b], a.doc_blocks[b], a.max_blocks);
  const int n = na + own_splits(max(0, nb - sh.blocks), a.SB);
  pdl_wait();
  pdl_trigger();
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + at;
  auto index = [&](int s) { return s < na ? s : a.SA + s - na; };
  float2 mine[4];
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int s = 32 * e + lane;
    mine[e] = s < n ? ml[index(s)] : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, mine[e].x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float f[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[e] = mine[e].x == -INFINITY ? 0.f : exp2f(mine[e].x - M);
    if (f[e] != 0.f) L += f[e] * mine[e].y;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  float O[V];
#pragma unroll
  for (int c = 0; c < V; ++c) O[c] = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll 8
    for (int s = 32 * e + warp; s < min(n, 32 * e + 32); s += kJoinWarps) {
      const float g = __shfl_sync(0xffffffffu, f[e], s & 31);
      const float* o = a.part_o + (at + index(s)) * D + lane * V;
      float x[V];
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(o);
      else
        *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(o);
      if (g != 0.f)  // a split that saw no key counts for nothing, whatever it holds
#pragma unroll
        for (int c = 0; c < V; ++c) O[c] += g * x[c];
    }
#pragma unroll
  for (int c = 0; c < V; ++c) part[warp][lane * V + c] = O[c];
  __syncthreads();
  const int c = 2 * threadIdx.x;
  if (c < D) {
    float y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      y0 += part[w][c];
      y1 += part[w][c + 1];
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;  // (a NaN stays)
    *reinterpret_cast<uint32_t*>(a.out + row * D + c) = f2_to_bf2(y0 * inv, y1 * inv);
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = (M + log2f(L)) * 0.6931471805599453f;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct Sizes {
  int SA, SB;
  size_t o_bytes, bytes;
};

Sizes sizes_of(int B, int n_groups, int max_group, int max_shared, int max_blocks, int Hq, int Hkv, int D) {
  Sizes s;
  max_shared = std::min(max_shared, max_blocks);
  max_group = std::min(max_group, B);
  s.SA = shared_prefix_splits(B, n_groups, max_group, max_shared, Hq, Hkv);
  // Own blocks: three blocks of threads per SM (four fit), runs of at least 32 blocks a split.  64 requests in 8 groups, 64 /
  // 8 heads, 2 own documents of 512 keys: 89.7 us, with four times as many splits 92.9; 16 requests with 10: 82.0 and 90.5
  // (two per SM 86.0, the quotient rounded down 85.9); 32 requests with 20, 32 / 8 heads: 264.7, 265.7 (rounded down 302).
  const int own = max_blocks - (s.SA ? max_shared : 0);
  const long long units = (long long)B * Hkv * ((Hq / Hkv + 7) / 8), slots = 3ll * sm_count();
  long long sb = std::min<long long>((slots + units - 1) / units, (own + 31) / 32);
  s.SB = int(std::max(1ll, std::min(64ll, sb)));
  const size_t n = s.SA + s.SB > 1 ? (size_t)B * Hq * (s.SA + s.SB) : 0;  // one result is the row's
  s.o_bytes = (n * D * 4 + 255) / 256 * 256;
  s.bytes = s.o_bytes + n * 8;
  return s;
}

}  // namespace

// Tensor map of a paged cache: columns (D) x rows of a page (16) x page-heads; boxes of 64 x 16 x 1, 128-byte
// swizzle, zeros outside.
int cache_tensor_map(CUtensorMap* map, const void* base, int num_pages, int Hkv, int D) {
  static std::atomic<EncodeFn> encode{nullptr};
  EncodeFn fn = encode.load(std::memory_order_acquire);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return fail(LAZY_ECUDA, "cuTensorMapEncodeTiled is unavailable");
    fn = reinterpret_cast<EncodeFn>(p);
    encode.store(fn, std::memory_order_release);
  }
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(kPage), cuuint64_t(num_pages) * cuuint64_t(Hkv)};
  const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(kPage) * D * 2};
  const cuuint32_t box[3] = {64, kPage, 1}, estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? LAZY_OK : fail(LAZY_ECUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
}

}  // namespace lazykv

using namespace lazykv;

static bool bad_sizes(int B, int n_groups, int max_group, int max_shared, int max_blocks, int Hq, int Hkv, int D) {
  return B < 0 || n_groups < 0 || max_group < 0 || max_shared < 0 || max_blocks <= 0 || Hq <= 0 || Hkv <= 0 ||
         Hq % Hkv || (D != 64 && D != 128);
}

extern "C" size_t lazy_decode_shared_workspace_size(int B, int n_groups, int max_group, int max_shared, int max_blocks,
                                                    int Hq, int Hkv, int D) {
  if (bad_sizes(B, n_groups, max_group, max_shared, max_blocks, Hq, Hkv, D) || B == 0) return 0;
  return sizes_of(B, n_groups, max_group, max_shared, max_blocks, Hq, Hkv, D).bytes;
}

extern "C" int lazy_attn_decode_shared(const void* q, const int32_t* seq_len, const int32_t* q_start,
                                       const int32_t* doc_blocks, const uint64_t* meta, const int32_t* group_off,
                                       const int32_t* shared_blocks, int n_groups, int max_group, int max_shared, int B,
                                       int max_blocks, const void* k_cache, const void* v_cache, int num_pages, int Hq,
                                       int Hkv, int D, float scale, const lazy_pos_cfg* cfg, void* out, float* lse,
                                       void* ws, size_t ws_bytes, void* stream) {
  const char* what = "lazy_attn_decode_shared";
  SharedArgs a = {};
  if (n_groups < 0 || max_group < 0 || max_shared < 0)
    return fail(LAZY_EINVAL, "%s: bad sizes (n_groups=%d max_group=%d max_shared=%d)", what, n_groups, max_group,
                max_shared);
  if (n_groups > 65535) return fail(LAZY_ERANGE, "%s: n_groups must be below 65536", what);
  int rc = check_shared_call(what, B, max_blocks, Hq, Hkv, D, num_pages, scale, cfg, &a.pos, meta,
                             {k_cache, v_cache, q, out}, {seq_len, q_start, doc_blocks});
  if (rc) return rc;
  if (B > 0 && n_groups > 0 && (!group_off || !shared_blocks)) return fail(LAZY_EINVAL, "%s: NULL pointer", what);
  if (Hkv * ((Hq / Hkv + 7) / 8) > 65535) return fail(LAZY_ERANGE, "%s: too many heads", what);
  if ((uint64_t)num_pages * Hkv > 0x7fffffffull) return fail(LAZY_ERANGE, "%s: num_pages * Hkv above 2^31", what);
  rc = check_device();
  if (rc || B == 0) return rc;
  const Sizes z = sizes_of(B, n_groups, max_group, max_shared, max_blocks, Hq, Hkv, D);
  rc = check_workspace(what, ws, ws_bytes, z.bytes);
  if (rc) return rc;
  CUtensorMap mk, mv;
  rc = cache_tensor_map(&mk, k_cache, num_pages, Hkv, D);
  if (!rc) rc = cache_tensor_map(&mv, v_cache, num_pages, Hkv, D);
  if (rc) return rc;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.seq_len = seq_len;
  a.q_start = q_start;
  a.doc_blocks = doc_blocks;
  a.meta = meta;
  a.group_off = group_off;
  a.shared_blocks = shared_blocks;
  a.n_groups = n_groups;
  a.max_group = std::min(max_group, B);
  a.max_shared = std::min(max_shared, max_blocks);
  a.B = B;
  a.max_blocks = max_blocks;
  a.num_pages = num_pages;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + z.o_bytes);
  a.SA = z.SA;
  a.SB = z.SB;
  a.status = status_word();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = run_shared_own(a, D, mk, mv, st);
  if (!rc && a.SA > 0) rc = run_shared_prefix(a, D, mk, mv, st);
  if (rc || a.SA + a.SB == 1) return rc;
  const dim3 grid(Hq, B);
  LAZY_CUDA_TRY(D == 128 ? launch_pdl(join_kernel<128>, grid, dim3(32 * kJoinWarps), 0, st, a)
                         : launch_pdl(join_kernel<64>, grid, dim3(32 * kJoinWarps), 0, st, a));
  return LAZY_OK;
}
