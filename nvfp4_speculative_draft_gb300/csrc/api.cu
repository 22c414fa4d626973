// api.cu -- the C ABI: argument validation on the host, then the launchers.
// Nothing here allocates, synchronises or keeps state beyond a cached SM count.

#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"

namespace nvfp4 {

int sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev >= 0 && dev < 64 && cached[dev] > 0) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 1;
  if (dev >= 0 && dev < 64) cached[dev] = n;
  return n;
}

namespace {
struct OccEntry {
  int dev;
  const void* func;
  int threads;
  size_t smem;
  int occ;
};
std::mutex g_occ_mutex;
OccEntry g_occ[256];
int g_nocc = 0;
long g_occ_asked = 0;  // queries that the table did not answer
}  // namespace

int occupancy(const void* func, int threads, size_t smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(g_occ_mutex);
  for (int i = 0; i < g_nocc; ++i)
    if (g_occ[i].dev == dev && g_occ[i].func == func && g_occ[i].threads == threads &&
        g_occ[i].smem == smem)
      return g_occ[i].occ;
  ++g_occ_asked;
  int maxopt = 0;
  if (cudaDeviceGetAttribute(&maxopt, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
    return 0;
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, func) != cudaSuccess) return 0;
  const int limit = maxopt - (int)attr.sharedSizeBytes;  // dynamic + static <= opt-in maximum
  if (limit < 0 || smem > (size_t)limit) return 0;
  if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, limit) != cudaSuccess)
    return 0;
  int occ = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, func, threads, smem) != cudaSuccess)
    return 0;
  if (g_nocc < 256) g_occ[g_nocc++] = OccEntry{dev, func, threads, smem, occ};
  return occ;
}

}  // namespace nvfp4

#ifdef NVFP4_TEST_WITHHOLD
// Test build: how many occupancy queries went to the runtime so far.
extern "C" long nvfp4_test_occupancy_asked() {
  std::lock_guard<std::mutex> lock(nvfp4::g_occ_mutex);
  return nvfp4::g_occ_asked;
}
#endif

namespace nvfp4 {

int check_weight(const nvfp4_weight* w) {
  if (w == nullptr || w->packed == nullptr || w->scales == nullptr || w->global_scale == nullptr)
    return NVFP4_ERR_NULL;
  if (w->n < 1 || w->k < 32 || w->k % 32 != 0) return NVFP4_ERR_SHAPE;
  if (w->n * (w->k / 2) >= (int64_t)1 << 32) return NVFP4_ERR_SHAPE;  // 32-bit offsets
  if (!aligned16(w->packed) || (reinterpret_cast<uintptr_t>(w->scales) & 1u) ||
      (reinterpret_cast<uintptr_t>(w->global_scale) & 3u))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

int check_fp8_weight(const fp8w_weight* w) {
  if (w == nullptr || w->codes == nullptr || w->row_scale == nullptr) return NVFP4_ERR_NULL;
  if (w->n < 1 || w->k < 32 || w->k % 32 != 0) return NVFP4_ERR_SHAPE;
  if (w->n * w->k >= (int64_t)1 << 32) return NVFP4_ERR_SHAPE;  // 32-bit offsets
  if (!aligned16(w->codes) || (reinterpret_cast<uintptr_t>(w->row_scale) & 3u)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

int check_fp8b_act(const fp8b_act* a) {
  if (a == nullptr || a->codes == nullptr || a->scales == nullptr) return NVFP4_ERR_NULL;
  if (a->m < 1 || a->m > 0x7FFFFFFF || a->k < 16 || a->k % 16 != 0 || a->k > 0x7FFFFFFF ||
      a->ld < a->k || a->ld_scales < a->m)
    return NVFP4_ERR_SHAPE;
  if (!aligned16(a->codes) || a->ld % 16 != 0 || !aligned4(a->scales)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

int check_segments(const w4a16_act_segment* seg, int nseg, int m, int64_t k) {
  if (seg == nullptr) return NVFP4_ERR_NULL;
  if (nseg < 1 || nseg > 2) return NVFP4_ERR_SHAPE;
  if (m < 1 || m > W4A16_GEMV_MAX_M) return NVFP4_ERR_SHAPE;
  if (k > W4A16_GEMV_MAX_K) return NVFP4_ERR_SHAPE;
  int64_t total = 0;
  for (int s = 0; s < nseg; ++s) {
    if (seg[s].x == nullptr) return NVFP4_ERR_NULL;
    if (seg[s].k_seg < 32 || seg[s].k_seg % 32 != 0) return NVFP4_ERR_SHAPE;
    if (seg[s].ld < seg[s].k_seg) return NVFP4_ERR_SHAPE;
    if (seg[s].ld % 8 != 0 || !aligned16(seg[s].x)) return NVFP4_ERR_ALIGN;
    if (seg[s].gamma != nullptr && !aligned16(seg[s].gamma)) return NVFP4_ERR_ALIGN;
    if (seg[s].gamma != nullptr && !(seg[s].eps >= 0.0f)) return NVFP4_ERR_SHAPE;
    if (seg[s].row_index != nullptr) {
      if (reinterpret_cast<uintptr_t>(seg[s].row_index) & 3u) return NVFP4_ERR_ALIGN;
      if (seg[s].index_rows < 1) return NVFP4_ERR_SHAPE;
    }
    total += seg[s].k_seg;
  }
  if (total != k) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

bool encode_tiled(CUtensorMap* map, CUtensorMapDataType type, cuuint32_t rank, void* addr,
                  const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                  const cuuint32_t* elem_strides, CUtensorMapSwizzle swizzle) {
  static std::mutex mu;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (fn == nullptr) {
      void* ptr = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                           &q) == cudaSuccess &&
          q == cudaDriverEntryPointSuccess)
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }
  }
  if (fn == nullptr) return false;
  return fn(map, type, rank, addr, dims, strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace nvfp4

namespace {

using nvfp4::aligned16;
using nvfp4::aligned4;
using nvfp4::check_fp8b_act;
using nvfp4::check_fp8_weight;
using nvfp4::check_segments;
using nvfp4::check_weight;

cudaStream_t stream_of(const nvfp4_exec* ex) {
  return ex ? reinterpret_cast<cudaStream_t>(ex->stream) : nullptr;
}
int32_t* status_of(const nvfp4_exec* ex) { return ex ? ex->dev_status : nullptr; }

// Argument checks and launch shared by the two weight formats' _ex calls.
int gemv_argmax_ex(const w4a16_act_segment* seg, int nseg, int m, const WeightRef& wr, float* logits,
                   int64_t ld_logits, int32_t* argmax, float* logprob, const int32_t* mask,
                   int64_t ld_mask, const nvfp4_exec* ex) {
  const WeightRef* w = &wr;
  int rc = check_segments(seg, nseg, m, w->k);
  if (rc) return rc;
  if (argmax == nullptr) return NVFP4_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(argmax) & 3u) ||
      (logits != nullptr && (reinterpret_cast<uintptr_t>(logits) & 3u)) ||
      (logprob != nullptr && (reinterpret_cast<uintptr_t>(logprob) & 3u)) ||
      (mask != nullptr && (reinterpret_cast<uintptr_t>(mask) & 3u)))
    return NVFP4_ERR_ALIGN;
  if (logits != nullptr && ld_logits < w->n) return NVFP4_ERR_SHAPE;
  if (mask != nullptr && ld_mask < (w->n + 31) / 32) return NVFP4_ERR_SHAPE;
  if (w->n > 0x7FFFFFFFLL) return NVFP4_ERR_SHAPE;
  if (ex == nullptr || ex->workspace == nullptr || ex->workspace_bytes < W4A16_ARGMAX_EX_WS_BYTES ||
      !aligned16(ex->workspace))
    return NVFP4_ERR_WORKSPACE;
  return launch_gemv(seg, nseg, m, wr, logits, NVFP4_DTYPE_F32, ld_logits, true, argmax,
                     ex->workspace, ex->workspace_bytes, status_of(ex), stream_of(ex), logprob, mask,
                     ld_mask);
}

bool rows_aligned(const attn_rows& r) {
  return aligned16(r.data) && r.ld_token % 8 == 0 && r.ld_head % 8 == 0;
}
bool pages_aligned(const kv_pages& r) {
  return aligned16(r.data) && r.ld_page % 8 == 0 && r.ld_token % 8 == 0 && r.ld_head % 8 == 0;
}
// A stride in the range of a TMA descriptor (2^40 bytes).
bool strides_fit(int64_t a, int64_t b, int64_t c) {
  const int64_t most = (int64_t)1 << 39;
  return a >= 0 && a < most && b >= 0 && b < most && c >= 0 && c < most;
}

// Argument checks that the two attention calls share.
int attention(const paged_attention_input& in, const attn_rows* out, const nvfp4_exec* ex) {
  if (out == nullptr) return NVFP4_ERR_NULL;
  if (in.tokens < 0 || in.tokens >= 0x7FFFFFFF - 512 || in.batch < 0 || in.batch >= 1 << 20 || in.kv_heads < 1 ||
      in.heads < 1 || in.heads % in.kv_heads != 0 || in.heads / in.kv_heads > 128 || in.heads >= 1 << 20 ||
      (in.dim != 64 && in.dim != 128 && in.dim != 256) || !(in.scale - in.scale == 0.0f))
    return NVFP4_ERR_SHAPE;
  if (in.tokens == 0 || in.batch == 0) return NVFP4_OK;
  if (in.q.data == nullptr || in.k.data == nullptr || in.v.data == nullptr || in.cu == nullptr || out->data == nullptr)
    return NVFP4_ERR_NULL;
  if (!strides_fit(in.q.ld_token, in.q.ld_head, 0) || !strides_fit(in.k.ld_page, in.k.ld_token, in.k.ld_head) ||
      !strides_fit(in.v.ld_page, in.v.ld_token, in.v.ld_head))
    return NVFP4_ERR_SHAPE;
  if (!rows_aligned(in.q) || !pages_aligned(in.k) || !pages_aligned(in.v) || !rows_aligned(*out) || !aligned4(in.cu))
    return NVFP4_ERR_ALIGN;
  if (ex == nullptr || ex->workspace == nullptr || ex->workspace_bytes < ATTENTION_WS_BYTES ||
      (reinterpret_cast<uintptr_t>(ex->workspace) & 31u))
    return NVFP4_ERR_WORKSPACE;
  return launch_attention(&in, out, ex->workspace, status_of(ex), stream_of(ex));
}

}  // namespace

extern "C" {

int nvfp4_quantize(const void* w_bf16, int64_t n, int64_t k, uint8_t* packed, uint8_t* scales,
                   float* global_scale, float* absmax, const nvfp4_exec* ex) {
  if (w_bf16 == nullptr || packed == nullptr || scales == nullptr || global_scale == nullptr)
    return NVFP4_ERR_NULL;
  if (n < 1 || k < 32 || k % 32 != 0) return NVFP4_ERR_SHAPE;
  if (!aligned16(w_bf16) || !aligned16(packed) || (reinterpret_cast<uintptr_t>(global_scale) & 3u))
    return NVFP4_ERR_ALIGN;
  uint32_t* word = reinterpret_cast<uint32_t*>(absmax);
  if (word == nullptr) {
    if (ex == nullptr || ex->workspace == nullptr || ex->workspace_bytes < NVFP4_QUANTIZE_WS_BYTES ||
        !aligned16(ex->workspace))
      return NVFP4_ERR_WORKSPACE;
    word = reinterpret_cast<uint32_t*>(ex->workspace);
  } else if (reinterpret_cast<uintptr_t>(absmax) & 3u) {
    return NVFP4_ERR_ALIGN;
  }
  return launch_quantize(w_bf16, n, k, packed, scales, global_scale, word, status_of(ex),
                         stream_of(ex));
}

int w4a16_gemv(const w4a16_act_segment* seg, int nseg, int m, const nvfp4_weight* w, void* y,
               int y_dtype, int64_t ldy, const nvfp4_exec* ex) {
  int rc = check_weight(w);
  if (rc) return rc;
  rc = check_segments(seg, nseg, m, w->k);
  if (rc) return rc;
  if (y == nullptr) return NVFP4_ERR_NULL;
  if (y_dtype != NVFP4_DTYPE_F32 && y_dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_DTYPE;
  if (ldy < w->n) return NVFP4_ERR_SHAPE;
  const uintptr_t ya = reinterpret_cast<uintptr_t>(y);
  if ((y_dtype == NVFP4_DTYPE_F32 && (ya & 3u)) || (ya & 1u)) return NVFP4_ERR_ALIGN;
  return launch_gemv(seg, nseg, m, ref_of(w), y, y_dtype, ldy, false, nullptr,
                     ex != nullptr ? ex->workspace : nullptr, ex != nullptr ? ex->workspace_bytes : 0,
                     status_of(ex), stream_of(ex));
}

int w4a16_gemv_argmax(const w4a16_act_segment* seg, int nseg, int m, const nvfp4_weight* w,
                      float* logits, int64_t ld_logits, int32_t* argmax, const nvfp4_exec* ex) {
  int rc = check_weight(w);
  if (rc) return rc;
  rc = check_segments(seg, nseg, m, w->k);
  if (rc) return rc;
  if (argmax == nullptr) return NVFP4_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(argmax) & 3u) ||
      (logits != nullptr && (reinterpret_cast<uintptr_t>(logits) & 3u)))
    return NVFP4_ERR_ALIGN;
  if (logits != nullptr && ld_logits < w->n) return NVFP4_ERR_SHAPE;
  if (w->n > 0x7FFFFFFFLL) return NVFP4_ERR_SHAPE;
  if (ex == nullptr || ex->workspace == nullptr || ex->workspace_bytes < W4A16_ARGMAX_WS_BYTES ||
      !aligned16(ex->workspace))
    return NVFP4_ERR_WORKSPACE;
  return launch_gemv(seg, nseg, m, ref_of(w), logits, NVFP4_DTYPE_F32, ld_logits, true, argmax,
                     ex->workspace, ex->workspace_bytes, status_of(ex), stream_of(ex));
}

int w4a16_gemv_argmax_ex(const w4a16_act_segment* seg, int nseg, int m, const nvfp4_weight* w,
                         float* logits, int64_t ld_logits, int32_t* argmax, float* logprob,
                         const int32_t* mask, int64_t ld_mask, const nvfp4_exec* ex) {
  int rc = check_weight(w);
  if (rc) return rc;
  return gemv_argmax_ex(seg, nseg, m, ref_of(w), logits, ld_logits, argmax, logprob, mask, ld_mask, ex);
}

int fp8w_gemv_argmax_ex(const w4a16_act_segment* seg, int nseg, int m, const fp8w_weight* w,
                        float* logits, int64_t ld_logits, int32_t* argmax, float* logprob,
                        const int32_t* mask, int64_t ld_mask, const nvfp4_exec* ex) {
  int rc = check_fp8_weight(w);
  if (rc) return rc;
  return gemv_argmax_ex(seg, nseg, m, ref_of(w), logits, ld_logits, argmax, logprob, mask, ld_mask, ex);
}

int w4a16_gemm(const void* a_bf16, int64_t m, int64_t lda, const nvfp4_weight* w, void* c_bf16,
               int64_t ldc, const nvfp4_exec* ex) {
  int rc = check_weight(w);
  if (rc) return rc;
  if (a_bf16 == nullptr || c_bf16 == nullptr) return NVFP4_ERR_NULL;
  if (m < 1 || w->n % 128 != 0 || w->k % 64 != 0 || lda < w->k || ldc < w->n)
    return NVFP4_ERR_SHAPE;
  if (!aligned16(a_bf16) || !aligned16(c_bf16) || lda % 8 != 0 || ldc % 8 != 0 ||
      (reinterpret_cast<uintptr_t>(w->scales) & 3u))
    return NVFP4_ERR_ALIGN;
  return launch_gemm(a_bf16, m, lda, w, c_bf16, ldc, ex ? ex->workspace : nullptr,
                     ex ? ex->workspace_bytes : 0, status_of(ex), stream_of(ex));
}

int fp8w_quantize(const void* w_bf16, int64_t n, int64_t k, uint8_t* codes, float* row_scale,
                  const nvfp4_exec* ex) {
  if (w_bf16 == nullptr || codes == nullptr || row_scale == nullptr) return NVFP4_ERR_NULL;
  if (n < 1 || k < 32 || k % 32 != 0 || n * k >= (int64_t)1 << 32) return NVFP4_ERR_SHAPE;
  if (!aligned16(w_bf16) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(row_scale) & 3u))
    return NVFP4_ERR_ALIGN;
  return launch_fp8_quantize(w_bf16, n, k, codes, row_scale, status_of(ex), stream_of(ex));
}

int fp8w_gemv(const w4a16_act_segment* seg, int nseg, int m, const fp8w_weight* w, void* y,
              int y_dtype, int64_t ldy, const nvfp4_exec* ex) {
  int rc = check_fp8_weight(w);
  if (rc) return rc;
  rc = check_segments(seg, nseg, m, w->k);
  if (rc) return rc;
  if (y == nullptr) return NVFP4_ERR_NULL;
  if (y_dtype != NVFP4_DTYPE_F32 && y_dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_DTYPE;
  if (ldy < w->n) return NVFP4_ERR_SHAPE;
  const uintptr_t ya = reinterpret_cast<uintptr_t>(y);
  if ((y_dtype == NVFP4_DTYPE_F32 && (ya & 3u)) || (ya & 1u)) return NVFP4_ERR_ALIGN;
  return launch_gemv(seg, nseg, m, ref_of(w), y, y_dtype, ldy, false, nullptr,
                     ex != nullptr ? ex->workspace : nullptr, ex != nullptr ? ex->workspace_bytes : 0,
                     status_of(ex), stream_of(ex));
}

int fp8w_gemv_argmax(const w4a16_act_segment* seg, int nseg, int m, const fp8w_weight* w,
                     float* logits, int64_t ld_logits, int32_t* argmax, const nvfp4_exec* ex) {
  int rc = check_fp8_weight(w);
  if (rc) return rc;
  rc = check_segments(seg, nseg, m, w->k);
  if (rc) return rc;
  if (argmax == nullptr) return NVFP4_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(argmax) & 3u) ||
      (logits != nullptr && (reinterpret_cast<uintptr_t>(logits) & 3u)))
    return NVFP4_ERR_ALIGN;
  if (logits != nullptr && ld_logits < w->n) return NVFP4_ERR_SHAPE;
  if (w->n > 0x7FFFFFFFLL) return NVFP4_ERR_SHAPE;
  if (ex == nullptr || ex->workspace == nullptr || ex->workspace_bytes < W4A16_ARGMAX_WS_BYTES ||
      !aligned16(ex->workspace))
    return NVFP4_ERR_WORKSPACE;
  return launch_gemv(seg, nseg, m, ref_of(w), logits, NVFP4_DTYPE_F32, ld_logits, true,
                     argmax, ex->workspace, ex->workspace_bytes, status_of(ex), stream_of(ex));
}

int fp8b_quantize(const void* w_bf16, int64_t n, int64_t k, int64_t ld, uint8_t* codes,
                  float* scales, const nvfp4_exec* ex) {
  if (w_bf16 == nullptr || codes == nullptr || scales == nullptr) return NVFP4_ERR_NULL;
  if (n < 1 || k < 16 || k % 16 != 0 || ld < k || n > 0x7FFFFFFF || k > 0x7FFFFFFF)
    return NVFP4_ERR_SHAPE;
  if (!aligned16(w_bf16) || !aligned16(codes) || !aligned4(scales) || ld % 8 != 0)
    return NVFP4_ERR_ALIGN;
  return launch_fp8b_quantize(w_bf16, n, k, ld, codes, scales, status_of(ex), stream_of(ex));
}

int fp8b_rmsnorm(const fp8b_norm_input* in, const fp8b_act* out, const nvfp4_exec* ex) {
  if (in == nullptr || in->x == nullptr) return NVFP4_ERR_NULL;
  int rc = check_fp8b_act(out);
  if (rc) return rc;
  const int64_t k = out->k;
  if (k > FP8B_MAX_K) return NVFP4_ERR_SHAPE;
  if (in->ld_x < k || (in->residual != nullptr && in->ld_residual < k) ||
      (in->residual_out != nullptr && in->ld_residual_out < k) ||
      (in->gamma != nullptr && !(in->eps >= 0.0f)))
    return NVFP4_ERR_SHAPE;
  if (!aligned16(in->x) || !aligned16(in->residual) || !aligned16(in->residual_out) ||
      !aligned16(in->gamma) || in->ld_x % 8 != 0 ||
      (in->residual != nullptr && in->ld_residual % 8 != 0) ||
      (in->residual_out != nullptr && in->ld_residual_out % 8 != 0))
    return NVFP4_ERR_ALIGN;
  return launch_fp8b_rmsnorm(in, out, status_of(ex), stream_of(ex));
}

int fp8b_gemm(const fp8b_act* a, const fp8b_weight* w, void* c, int c_dtype, int64_t ldc,
              const nvfp4_exec* ex) {
  if (w == nullptr || w->codes == nullptr || w->scales == nullptr || c == nullptr)
    return NVFP4_ERR_NULL;
  int rc = check_fp8b_act(a);
  if (rc) return rc;
  if (c_dtype != NVFP4_DTYPE_F32 && c_dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_DTYPE;
  if (w->n < 1 || w->n > 0x7FFFFFFF || w->k != a->k || ldc < w->n) return NVFP4_ERR_SHAPE;
  if (!aligned16(w->codes) || !aligned4(w->scales) ||
      (reinterpret_cast<uintptr_t>(c) & (c_dtype == NVFP4_DTYPE_F32 ? 3u : 1u)))
    return NVFP4_ERR_ALIGN;
  return launch_fp8b_gemm(a, w, c, c_dtype, ldc, status_of(ex), stream_of(ex));
}

int spec_verify(const spec_verify_input* in, int32_t* out_tokens, int64_t ld_out,
                int32_t* accepted, const nvfp4_exec* ex) {
  if (in == nullptr || in->target == nullptr || in->sample_u == nullptr || out_tokens == nullptr ||
      accepted == nullptr || (in->g > 0 && (in->tokens == nullptr || in->accept_u == nullptr)))
    return NVFP4_ERR_NULL;
  if (in->dtype != NVFP4_DTYPE_F32 && in->dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_DTYPE;
  if (in->batch < 1 || in->g < 0 || in->g > SPEC_MAX_DRAFT || in->vocab < 1 ||
      in->vocab > SPEC_MAX_VOCAB || in->ld_target_seq < 0 || in->ld_target_pos < 0 ||
      ld_out < in->g + 1)
    return NVFP4_ERR_SHAPE;
  if (in->g > 0 && (in->ld_tokens < in->g || in->ld_accept_u < in->g)) return NVFP4_ERR_SHAPE;
  if (in->g > 0 && in->draft != nullptr &&
      (in->draft_vocab < 1 || in->draft_vocab > in->vocab || in->ld_draft_seq < 0 ||
       in->ld_draft_pos < 0))
    return NVFP4_ERR_SHAPE;
  const uintptr_t each = in->dtype == NVFP4_DTYPE_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(in->target) & each) ||
      (reinterpret_cast<uintptr_t>(in->draft) & each) || !aligned4(in->tokens) ||
      !aligned4(in->num_draft) || !aligned4(in->accept_u) || !aligned4(in->sample_u) ||
      !aligned4(out_tokens) || !aligned4(accepted))
    return NVFP4_ERR_ALIGN;
  return launch_spec_verify(in, out_tokens, ld_out, accepted, status_of(ex), stream_of(ex));
}

int kv_plan(const kv_plan_input* in, const kv_plan_output* out, const nvfp4_exec* ex) {
  if (in == nullptr || out == nullptr || in->free_count == nullptr || out->cu_new == nullptr)
    return NVFP4_ERR_NULL;
  if (in->batch < 0 || in->batch > KV_PLAN_MAX_BATCH || in->page_size < 1 || in->page_size > KV_MAX_PAGE ||
      in->tokens < 0 || in->tokens > 0x7FFFFFFF || in->free_capacity < 0 || in->free_capacity > 0x7FFFFFFF)
    return NVFP4_ERR_SHAPE;
  if ((in->batch > 0 && (in->lens == nullptr || in->num_new == nullptr || in->block_table == nullptr ||
                         out->kv_lens == nullptr)) ||
      (in->free_capacity > 0 && in->free_pages == nullptr) ||
      (in->tokens > 0 && (out->positions == nullptr || out->slots == nullptr)))
    return NVFP4_ERR_NULL;
  if (in->batch > 0 && (in->max_pages < 1 || in->max_pages > in->ld_table || in->max_pages > 0x7FFFFFFF))
    return NVFP4_ERR_SHAPE;
  if (!aligned4(in->lens) || !aligned4(in->num_new) || !aligned4(in->held) || !aligned4(in->block_table) ||
      !aligned4(in->free_pages) || !aligned4(in->free_count) || !aligned4(out->cu_new) || !aligned4(out->kv_lens) ||
      !aligned4(out->positions) || !aligned4(out->slots) || !aligned4(out->held) || !aligned4(out->free_count))
    return NVFP4_ERR_ALIGN;
  return launch_kv_plan(in, out, status_of(ex), stream_of(ex));
}

int rope_kv_write(const rope_kv_input* in, const rope_kv_output* out, const nvfp4_exec* ex) {
  if (in == nullptr || out == nullptr) return NVFP4_ERR_NULL;
  if (in->tokens < 0 || in->tokens > 0x7FFFFFFF || in->heads < 1 || in->heads >= 1 << 20 || in->kv_heads < 1 ||
      in->kv_heads >= 1 << 20 || in->dim < 16 || in->dim % 16 != 0 || in->dim > ROPE_MAX_DIM || in->rot_dim < 16 ||
      in->rot_dim % 16 != 0 || in->rot_dim > in->dim || in->axes < 1 || in->axes > 256 ||
      (in->ld_positions < in->tokens && in->ld_positions != 0))
    return NVFP4_ERR_SHAPE;
  const bool cached = in->k_cache.data != nullptr;
  if (cached != (in->v_cache.data != nullptr)) return NVFP4_ERR_NULL;
  if (cached && (in->pages < 1 || in->page_size < 1 || in->page_size > KV_MAX_PAGE ||
                 in->pages > 0x7FFFFFFF / in->page_size))
    return NVFP4_ERR_SHAPE;
  if (in->tokens == 0) return NVFP4_OK;
  if (in->q.data == nullptr || in->k.data == nullptr || in->positions == nullptr || in->turns == nullptr ||
      out->q.data == nullptr || (cached && (in->v.data == nullptr || in->slots == nullptr)))
    return NVFP4_ERR_NULL;
  if (!rows_aligned(in->q) || !rows_aligned(in->k) || (cached && !rows_aligned(in->v)) || !rows_aligned(out->q) ||
      (out->k.data != nullptr && !rows_aligned(out->k)) || !pages_aligned(in->k_cache) ||
      !pages_aligned(in->v_cache) || !aligned4(in->positions) || !aligned4(in->slots) ||
      (reinterpret_cast<uintptr_t>(in->turns) & 7u))
    return NVFP4_ERR_ALIGN;
  return launch_rope_kv_write(in, out, status_of(ex), stream_of(ex));
}

int prompt_attention(const prompt_attention_input* in, const attn_rows* out, const nvfp4_exec* ex) {
  if (in == nullptr) return NVFP4_ERR_NULL;
  paged_attention_input a = {};
  a.q = in->q;
  a.k = kv_pages{in->k.data, 0, in->k.ld_token, in->k.ld_head};
  a.v = kv_pages{in->v.data, 0, in->v.ld_token, in->v.ld_head};
  a.pages = 1;
  a.page_size = in->tokens;
  a.cu = in->cu;
  a.tokens = in->tokens;
  a.batch = in->batch;
  a.heads = in->heads;
  a.kv_heads = in->kv_heads;
  a.dim = in->dim;
  a.scale = in->scale;
  return attention(a, out, ex);
}

int paged_attention(const paged_attention_input* in, const attn_rows* out, const nvfp4_exec* ex) {
  if (in == nullptr) return NVFP4_ERR_NULL;
  if (in->pages < 1 || in->pages > 0x7FFFFFFF || in->page_size < 16 || in->page_size % 16 != 0 ||
      in->page_size > KV_MAX_PAGE)
    return NVFP4_ERR_SHAPE;
  if (in->batch > 0 && (in->max_pages < 1 || in->max_pages > in->ld_table || in->max_pages > 0x7FFFFFFF))
    return NVFP4_ERR_SHAPE;
  if (in->batch > 0 && in->tokens > 0 && (in->block_table == nullptr || in->kv_lens == nullptr))
    return NVFP4_ERR_NULL;
  if (!aligned4(in->block_table) || !aligned4(in->kv_lens)) return NVFP4_ERR_ALIGN;
  return attention(*in, out, ex);
}

}  // extern "C"
