// attention.cu -- causal attention with grouped heads over packed prompts and over the
// paged cache.
//
// One warp per (query, head): scores by shuffles, the softmax's maximum and sum carried
// along, everything in FP32.
#include "common.cuh"

namespace {

constexpr int kThreads = 256;

struct Params {
  paged_attention_input in;
  attn_rows out;
  int32_t* dev_status;
};

template <int D>
__global__ void __launch_bounds__(kThreads) attention_kernel(const __grid_constant__ Params p) {
  constexpr int E = D / 32;
  const paged_attention_input& in = p.in;
  const int lane = threadIdx.x & 31;
  nvfp4::wait_for_previous_kernel();
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = item / in.heads, head = item % in.heads, kv_head = head / (in.heads / in.kv_heads);
  if (row >= in.tokens) return;
  // the sequence of the row
  int64_t seq = -1, begin = 0, end = 0;
  for (int64_t s = 0; s < in.batch; ++s) {
    if (in.cu[s] < 0 || in.cu[s + 1] > in.tokens || in.cu[s] > in.cu[s + 1] ||
        (in.block_table != nullptr && in.kv_lens[s] > in.max_pages * in.page_size))
      nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
    const int64_t a = min(max((int64_t)in.cu[s], (int64_t)0), in.tokens), b = min((int64_t)in.cu[s + 1], in.tokens);
    if (row >= a && row < b) {
      seq = s;
      begin = a;
      end = b;
      break;
    }
  }
  if (seq < 0) return;
  int64_t len = end - begin;
  if (in.block_table != nullptr) len = min((int64_t)in.kv_lens[seq], in.max_pages * in.page_size);
  const int64_t seen = min(len, len - (end - begin) + (row - begin) + 1);
  const __nv_bfloat16* q = (const __nv_bfloat16*)in.q.data + row * in.q.ld_token + head * in.q.ld_head;
  float qv[E], o[E], m = -INFINITY, l = 0.0f;
  for (int e = 0; e < E; ++e) {
    qv[e] = __bfloat162float(q[lane + 32 * e]) * in.scale;
    o[e] = 0.0f;
  }
  for (int64_t j = 0; j < seen; ++j) {
    int64_t page = 0, at = begin + j;
    if (in.block_table != nullptr) {
      page = in.block_table[seq * in.ld_table + j / in.page_size];
      at = j % in.page_size;
      if (page < 0 || page >= in.pages) {
        nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
        page = -1;
      }
    }
    const __nv_bfloat16* k = (const __nv_bfloat16*)in.k.data + page * in.k.ld_page + at * in.k.ld_token + kv_head * in.k.ld_head;
    const __nv_bfloat16* v = (const __nv_bfloat16*)in.v.data + page * in.v.ld_page + at * in.v.ld_token + kv_head * in.v.ld_head;
    float s = 0.0f;
    if (page >= 0)
      for (int e = 0; e < E; ++e) s += qv[e] * __bfloat162float(k[lane + 32 * e]);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    const float next = fmaxf(m, s), keep = __expf(m - next), w = __expf(s - next);
    l = l * keep + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + (page >= 0 ? w * __bfloat162float(v[lane + 32 * e]) : 0.0f);
    m = next;
  }
  __nv_bfloat16* out = (__nv_bfloat16*)p.out.data + row * p.out.ld_token + head * p.out.ld_head;
  for (int e = 0; e < E; ++e) out[lane + 32 * e] = __float2bfloat16_rn(l > 0.0f ? o[e] / l : 0.0f);
}

}  // namespace

int launch_attention(const paged_attention_input* in, const attn_rows* out, void* workspace, int32_t* dev_status,
                     cudaStream_t stream) {
  (void)workspace;
  Params p{*in, *out, dev_status};
  const int64_t blocks = nvfp4::cdiv(in->tokens * in->heads, kThreads / 32);
  if (blocks > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  const void* kern = in->dim == 64 ? (const void*)attention_kernel<64>
                                   : in->dim == 128 ? (const void*)attention_kernel<128> : (const void*)attention_kernel<256>;
  void* args[] = {&p};
  return nvfp4::launch_dependent(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, 1, args) == cudaSuccess
             ? NVFP4_OK
             : NVFP4_ERR_CUDA;
}
