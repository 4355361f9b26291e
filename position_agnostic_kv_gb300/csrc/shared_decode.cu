// Decode of a batch whose requests share their first documents: entry point, and the join of the partial
// results of the common keys and of each request's own.
#include <algorithm>

#include "shared_decode.cuh"

namespace lazykv {

namespace {

// A row's partial results joined by their maxima: out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
template <int D>
__global__ void __launch_bounds__(D) join_kernel(const SharedArgs a) {
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x, b = blockIdx.y, col = threadIdx.x;
  const Share sh = share_of(a, b);
  const int tiles = (sh.blocks + 7) / 8;
  const int na = tiles ? (tiles + split_tiles(tiles, a.SA) - 1) / split_tiles(tiles, a.SA) : 0;
  const int nb = visible_blocks(a.seq_len[b], a.q_start[b], a.doc_blocks[b], a.max_blocks);
  const int no = own_splits(max(0, nb - sh.blocks), a.SB);
  const size_t row = (size_t)b * a.Hq + h, at = row * (a.SA + a.SB);
  float M = -INFINITY;
  for (int i = 0; i < na + no; ++i) M = fmaxf(M, a.part_ml[2 * (at + (i < na ? i : a.SA + i - na))]);
  float O = 0.f, L = 0.f;
  if (M != -INFINITY)
    for (int i = 0; i < na + no; ++i) {
      const size_t s = at + (i < na ? i : a.SA + i - na);
      const float ms = a.part_ml[2 * s];
      if (ms == -INFINITY) continue;
      const float f = exp2f(ms - M);
      O += f * a.part_o[s * D + col];
      L += f * a.part_ml[2 * s + 1];
    }
  a.out[row * D + col] = __float2bfloat16_rn(L > 0.f ? O / L : (L == 0.f ? 0.f : O + L));
  if (a.lse && col == 0) a.lse[row] = (M + log2f(L)) * 0.6931471805599453f;
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
  s.SA = shared_prefix_splits(n_groups, max_group, max_shared, Hq, Hkv);
  // Own blocks: enough warps for about four waves, runs of at least 32 blocks a split.
  const int own = max_blocks - (s.SA ? max_shared : 0);
  const long long units = (long long)B * Hkv * ((Hq / Hkv + 7) / 8), slots = 3ll * sm_count();
  long long sb = std::min<long long>((4 * slots + units - 1) / units, (own + 31) / 32);
  s.SB = int(std::max(1ll, std::min(64ll, sb)));
  const size_t n = (size_t)B * Hq * (s.SA + s.SB);
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
  if (a.SA > 0) rc = run_shared_prefix(a, D, mk, mv, st);
  if (!rc) rc = run_shared_own(a, D, mk, mv, a.SA > 0, st);
  if (rc) return rc;
  const dim3 grid(Hq, B);
  LAZY_CUDA_TRY(D == 128 ? launch_pdl(join_kernel<128>, grid, dim3(128), 0, st, a)
                         : launch_pdl(join_kernel<64>, grid, dim3(64), 0, st, a));
  return LAZY_OK;
}
