// extern "C" entry points of the attention over the 4-bit cache: argument checks and dispatch.
// Everything that can be refused without a GPU is refused before the device is looked at.
#include "q4_attn.cuh"

using namespace lazykv;

static int check_q4(const char* what, int B, int max_blocks, int Hq, int Hkv, int D, int num_pages, const void* cache,
                    const void* q, const void* out, const void* meta, const void* q_start, const void* doc_blocks,
                    float scale, float k_scale, float v_scale, float* kf, float* vf) {
  if (B < 0 || max_blocks <= 0 || Hq <= 0 || Hkv <= 0 || num_pages <= 0)
    return fail(LAZY_EINVAL, "%s: bad sizes (B=%d max_blocks=%d Hq=%d Hkv=%d num_pages=%d)", what, B, max_blocks, Hq,
                Hkv, num_pages);
  if (D != 64 && D != 128) return fail(LAZY_EINVAL, "%s: head_dim must be 64 or 128, got %d", what, D);
  if (Hq % Hkv) return fail(LAZY_EINVAL, "%s: Hq (%d) must be a multiple of Hkv (%d)", what, Hq, Hkv);
  const int G = Hq / Hkv;
  if (G > 8 && G % 8) return fail(LAZY_EINVAL, "%s: Hq/Hkv = %d: above 8 it must be a multiple of 8", what, G);
  if (G < 8 && (G & (G - 1))) return fail(LAZY_EINVAL, "%s: Hq/Hkv = %d must be a power of two below 8", what, G);
  if (num_pages > (1 << 24)) return fail(LAZY_ERANGE, "%s: num_pages above 2^24", what);
  if (!(scale >= 0.f && scale <= 3.0e38f))
    return fail(LAZY_EINVAL, "%s: scale must be positive (or 0 for the default)", what);
  if (!q4_factor(k_scale, kf) || !q4_factor(v_scale, vf))
    return fail(LAZY_EINVAL, "%s: k_scale and v_scale must be powers of two in [2^-32, 2^32] (or 0 for 1)", what);
  if (B == 0) return LAZY_OK;
  if (!cache || !q || !out || !meta || !q_start || !doc_blocks) return fail(LAZY_EINVAL, "%s: NULL pointer", what);
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!al(cache) || !al(q) || !al(out)) return fail(LAZY_EINVAL, "%s: tensors must be 16-byte aligned", what);
  if (reinterpret_cast<uintptr_t>(meta) & 7u) return fail(LAZY_EINVAL, "%s: meta must be 8-byte aligned", what);
  return LAZY_OK;
}

// Scores are products of f16 operands times this factor and a row's power of two, which must not leave fp32.
static int check_factor(const char* what, float scale_log2, float kf) {
  if (scale_log2 * kf >= 0x1p-60f && scale_log2 * kf <= 0x1p60f) return LAZY_OK;
  return fail(LAZY_EINVAL, "%s: scale times k_scale must lie in [2^-60, 2^60]", what);
}

static void fill_args(Q4Args& a, const void* q, const int32_t* q_start, const int32_t* doc_blocks,
                      const uint64_t* meta, int B, int max_blocks, const void* cache, int num_pages, int Hq, int Hkv,
                      float kf, float vf, void* out, float* lse) {
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_start = q_start;
  a.doc_blocks = doc_blocks;
  a.meta = meta;
  a.cache = static_cast<const uint8_t*>(cache);
  a.num_pages = num_pages;
  a.B = B;
  a.max_blocks = max_blocks;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.qk_log2 = a.pos.scale_log2 * kf;
  a.lowest_ex = q4_lowest_exponent(a.qk_log2);
  a.v_factor = vf;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.S = 1;
  a.status = status_word();
}

extern "C" int lazy_attn_decode_q4(const void* q, const int32_t* seq_len, const int32_t* q_start,
                                   const int32_t* doc_blocks, const uint64_t* meta, int B, int max_blocks,
                                   const void* kv_cache, int num_pages, int Hq, int Hkv, int D, float scale,
                                   float k_scale, float v_scale, const lazy_pos_cfg* cfg, void* out, float* lse,
                                   void* ws, size_t ws_bytes, void* stream) {
  Q4Args a = {};
  float kf, vf;
  int rc = check_q4("lazy_attn_decode_q4", B, max_blocks, Hq, Hkv, D, num_pages, kv_cache, q, out, meta, q_start,
                    doc_blocks, scale, k_scale, v_scale, &kf, &vf);
  if (rc) return rc;
  if (B > 0 && !seq_len) return fail(LAZY_EINVAL, "lazy_attn_decode_q4: seq_len is NULL");
  rc = prepare_pos(cfg, Hq, D, scale, &a.pos);
  if (!rc) rc = q4_check_table("lazy_attn_decode_q4", a.pos);
  if (!rc) rc = check_factor("lazy_attn_decode_q4", a.pos.scale_log2, kf);
  if (rc) return rc;
  rc = check_device();
  if (rc || B == 0) return rc;
  fill_args(a, q, q_start, doc_blocks, meta, B, max_blocks, kv_cache, num_pages, Hq, Hkv, kf, vf, out, lse);
  a.seq_len = seq_len;
  a.rows = B;
  return run_q4_rows(a, D, false, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int lazy_attn_prefill_q4(const void* q, const int32_t* cu_q, const int32_t* q_start,
                                    const int32_t* doc_blocks, const uint64_t* meta, int B, int max_blocks,
                                    int total_q, int max_q, const void* kv_cache, int num_pages, int Hq, int Hkv,
                                    int D, float scale, float k_scale, float v_scale, const lazy_pos_cfg* cfg,
                                    void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  Q4Args a = {};
  float kf, vf;
  if (total_q < 0 || max_q < 0) return fail(LAZY_EINVAL, "lazy_attn_prefill_q4: bad total_q / max_q");
  int rc = check_q4("lazy_attn_prefill_q4", total_q == 0 ? 0 : B, max_blocks, Hq, Hkv, D, num_pages, kv_cache, q, out,
                    meta, q_start, doc_blocks, scale, k_scale, v_scale, &kf, &vf);
  if (rc) return rc;
  if (B > 0 && total_q > 0 && !cu_q) return fail(LAZY_EINVAL, "lazy_attn_prefill_q4: cu_q is NULL");
  rc = prepare_pos(cfg, Hq, D, scale, &a.pos);
  if (!rc) rc = q4_check_table("lazy_attn_prefill_q4", a.pos);
  if (!rc) rc = check_factor("lazy_attn_prefill_q4", a.pos.scale_log2, kf);
  if (rc) return rc;
  rc = check_device();
  if (rc || B <= 0 || total_q == 0) return rc;
  fill_args(a, q, q_start, doc_blocks, meta, B, max_blocks, kv_cache, num_pages, Hq, Hkv, kf, vf, out, lse);
  a.cu_q = cu_q;
  a.rows = total_q;
  if (max_q > total_q) max_q = total_q;  // any upper bound will do; no request has more rows than there are
  if (q4_use_tc(Hq, Hkv)) return max_q > 0 ? run_q4_tc(a, D, max_q, static_cast<cudaStream_t>(stream)) : LAZY_OK;
  return run_q4_rows(a, D, true, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}
