// kv_cache.cu -- the paged KV cache: which pages a batch's new tokens go to, and the
// write of their rotated keys and their values.
#include <cooperative_groups.h>

#include "common.cuh"

namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------- plan
//
// Per sequence: n new tokens behind len cached ones, need = ceil((len + n) / page)
// pages, extra = max(0, need - held) of them from the top of the free stack, in the
// order of the sequences.  Two prefix sums over the batch (tokens, then extra pages)
// give every token its row and every new page its place; both are formed by each CTA
// of one cluster for itself, in shared memory, and tokens and pages are then shared
// out evenly, each finding its sequence by bisection.  All reads that an in-place call
// overwrites come before the cluster's barrier, all writes behind it.
//
// What bounds it is the chain of dependent steps (launch, the lengths' load, two prefix
// sums, bisection, the table's load), not the bytes: 24 requests of up to 6 tokens take
// 4.2 us, 1000 of up to 400 (a chunk in eight of them) 8.8 us.

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

struct PlanParams {
  kv_plan_input in;
  kv_plan_output out;
  int page_shift;  // log2 of the page size, or -1
  int32_t* dev_status;
};

// Exclusive prefix sums of each thread's value over the CTA; total to all.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T sum = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
    if (lane >= d) sum += o;
  }
  __syncthreads();  // the sums of the scan before are read
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  T before = lane < kPlanWarps ? warp_sums[lane] : 0;  // (every warp sums the warps' sums)
  total = before;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xFFFFFFFFu, total, d);
    if (lane >= d) total += o;
  }
  before = __shfl_sync(0xFFFFFFFFu, total - before, warp);
  total = __shfl_sync(0xFFFFFFFFu, total, 31);
  return before + sum - v;
}

// The smallest of the CTA's values.
__device__ __forceinline__ int64_t block_min(int64_t v, int64_t* warp_values) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = min(v, (int64_t)__shfl_xor_sync(0xFFFFFFFFu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_values[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warp_values[threadIdx.x & 31];
#pragma unroll
  for (int d = 16; d; d >>= 1) v = min(v, (int64_t)__shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}

// Last s in [0, batch) with start[s] <= i (start ascends, start[0] <= i).
__device__ __forceinline__ int find_sequence(const int32_t* start, int batch, int32_t i) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

static_assert(kPlanWarps == 32, "a lane a warp");

__global__ void __launch_bounds__(kPlanThreads, 1) kv_plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int32_t plan_smem[];
  __shared__ int64_t sums64[kPlanWarps];
  const int batch = (int)p.in.batch, page = (int)p.in.page_size;
  const int64_t tokens = p.in.tokens, width = p.in.max_pages;
  // per sequence: first token, first extra page, cached length, held pages; -1 - held where
  // refused (until then: new tokens, need, cached length, held pages)
  int32_t* const s_token = plan_smem;
  int32_t* const s_page = plan_smem + batch;
  int32_t* const s_len = plan_smem + 2 * batch;
  int32_t* const s_held = plan_smem + 3 * batch;
  auto pages_of = [&](uint32_t n) { return p.page_shift >= 0 ? n >> p.page_shift : n / (uint32_t)page; };
  nvfp4::wait_for_previous_kernel();

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  int64_t left = *p.in.free_count;
  int error = 0;
  if (left < 0 || left > p.in.free_capacity) {
    error = NVFP4_ERR_INDEX;
    left = left < 0 ? 0 : p.in.free_capacity;
  }
  // each thread a run of neighbouring sequences
  const int run = (batch + kPlanThreads - 1) / kPlanThreads;
  const int first = min(batch, (int)threadIdx.x * run), last = min(batch, first + run);
  int64_t mine = 0;
  for (int s = first; s < last; ++s) {
    // (plain loads: lens and held may be outputs of this call, and of the one before it on the
    // stream, which the read-only path does not allow for)
    const int32_t n = max(p.in.num_new[s], 0), len = max(p.in.lens[s], 0);
    s_token[s] = n;
    s_len[s] = len;
    // (a count that is given stays what it is, past the table's row too: those pages are not lost)
    s_held[s] = p.in.held != nullptr ? max(p.in.held[s], 0)
                                     : (int32_t)min((int64_t)pages_of((uint32_t)len + (uint32_t)page - 1u), width);
    mine += n;
  }
  int64_t total;
  int64_t at = block_scan<int64_t>(mine, sums64, total);
  const int32_t used = (int32_t)min(total, tokens);
  // pages wanted by the sequences that fit their table's row and the tokens; -1: does not fit
  int64_t extra = 0;
  {
    int64_t start = at;
    for (int s = first; s < last; ++s) {
      const int32_t n = s_token[s], held = s_held[s];
      int32_t want = 0;
      if (n > 0) {
        const uint32_t length = (uint32_t)s_len[s] + (uint32_t)n;  // (two int32: no overflow)
        const int64_t need = length <= 0x7FFFFFFFu ? pages_of(length + (uint32_t)page - 1u) : (int64_t)width + 1;
        want = need > width || start + n > tokens ? -1 : (int32_t)max(need - held, (int64_t)0);
        start += n;
      }
      s_page[s] = want;
      if (want > 0) extra += want;
    }
  }
  int64_t all_extra;
  int64_t upto = block_scan<int64_t>(extra, sums64, all_extra);
  int64_t taken = 0;  // pages taken by this thread's run, counted from the stack's top
  for (int s = first; s < last; ++s) {
    const int32_t want = s_page[s], n = s_token[s], e = max(want, 0);
    const bool ok = want >= 0 && (e == 0 || upto + e <= left);
    s_token[s] = (int32_t)min(at, tokens);
    s_page[s] = (int32_t)min(upto, left);
    if (!ok) {
      s_held[s] = -1 - s_held[s];
      error = NVFP4_ERR_PAGES;
    }
    at += n;
    upto += e;
    if (ok && e > 0) taken = upto;
  }
  if (error) nvfp4::report(p.dev_status, error);
  // the most that any sequence took up to (its prefix counts those before it, which all got theirs)
  taken = -block_min(-taken, sums64);
  cluster.sync();

  const int me = rank * kPlanThreads + (int)threadIdx.x, step = ranks * kPlanThreads;
  for (int s = me; s < batch; s += step) {
    const int32_t next = s + 1 < batch ? s_token[s + 1] : used;
    const int32_t held = s_held[s] < 0 ? -1 - s_held[s] : s_held[s];
    const int64_t n = s_held[s] < 0 ? 0 : next - s_token[s];
    const int64_t kv = s_len[s] + n, need = n > 0 ? pages_of((uint32_t)kv + (uint32_t)page - 1u) : 0;
    p.out.cu_new[s + 1] = next;
    p.out.kv_lens[s] = (int32_t)kv;
    if (p.out.held != nullptr) p.out.held[s] = (int32_t)max((int64_t)held, need);
  }
  if (me == 0) {
    p.out.cu_new[0] = 0;
    if (p.out.free_count != nullptr) *p.out.free_count = (int32_t)(left - taken);
  }
  const int32_t* top = p.in.free_pages + left - 1;
  for (int64_t f = me; f < taken; f += step) {
    const int s = find_sequence(s_page, batch, (int32_t)f);
    p.in.block_table[s * p.in.ld_table + s_held[s] + (f - s_page[s])] = top[-f];
  }
  for (int64_t i = me; i < tokens; i += step) {
    int32_t position = 0, slot = -1;
    if (i < used) {
      const int s = find_sequence(s_token, batch, (int32_t)i);
      const int64_t at_kv = (int64_t)s_len[s] + (i - s_token[s]);
      position = (int32_t)min(at_kv, (int64_t)0x7FFFFFFF);
      const int32_t held = s_held[s];
      if (held >= 0) {
        const int32_t entry = (int32_t)pages_of((uint32_t)position);
        const int32_t id = entry < held ? p.in.block_table[s * p.in.ld_table + entry]
                                        : top[-((int64_t)s_page[s] + entry - held)];
        const int64_t where = (int64_t)id * page + (position - entry * page);
        if (id >= 0 && where <= 0x7FFFFFFF)
          slot = (int32_t)where;
        else
          nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
      }
    }
    p.out.positions[i] = position;
    p.out.slots[i] = slot;
  }
}

// ------------------------------------------------------------------ rotary
//
// Pair i of a head, elements i and half + i:  (x, y) -> (x cos t - y sin t, x sin t + y cos t),
// t = position[axis(i)] frequency(i).  The frequency is held as turns per position in
// 64-bit fixed point: position times it wraps around to the fraction of a turn exactly,
// however far the position (a binary32 angle at position 100 000 is off by 0.004).
// The sines of a CTA's tokens are formed once, in shared memory; FP32 arithmetic, one
// rounding to BF16.
//
// HBM bounds it: 16384 tokens of 40 / 8 heads of 128 take 71 us, 6.6 TB/s (0.98 of a copy's
// rate).  Few tokens are a launch and a load's latency: one token 1.9 us, 315 tokens 3.1 us.

constexpr int kRopeThreads = 256;

struct RopeParams {
  rope_kv_input in;
  rope_kv_output out;
  int32_t* dev_status;
};

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint4& v) {
  asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Eight pairs: a = elements 8 i.., b = elements half + 8 i..; cs: cosines and sines of two of the
// pairs, then of the next two `items` further on (so that neighbouring threads read neighbouring
// words).
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float4* cs, int items) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 t = cs[j * items];
    const float x0 = __uint_as_float(x[j] << 16), x1 = __uint_as_float(x[j] & 0xFFFF0000u);
    const float y0 = __uint_as_float(y[j] << 16), y1 = __uint_as_float(y[j] & 0xFFFF0000u);
    x[j] = pack_bf16(x0 * t.x - y0 * t.y, x1 * t.z - y1 * t.w);
    y[j] = pack_bf16(x0 * t.y + y0 * t.x, x1 * t.w + y1 * t.z);
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(y[0], y[1], y[2], y[3]);
}

// A CTA takes TOKENS tokens (and a share of their vectors), a thread the same vectors of all of
// them: their loads are in flight together, the first ones while the sines are formed.
template <int TOKENS>
__global__ void __launch_bounds__(kRopeThreads) rope_kv_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) float2 angles[TOKENS][ROPE_MAX_DIM / 2];
  __shared__ int64_t k_at[TOKENS], v_at[TOKENS];
  const rope_kv_input& in = p.in;
  const int half = (int)in.rot_dim / 2, dim = (int)in.dim;
  const int64_t t0 = (int64_t)blockIdx.x * TOKENS;
  const int count = (int)min(in.tokens - t0, (int64_t)TOKENS);
  const bool cached = in.k_cache.data != nullptr;
  // items: 16 elements of a (token, head): the two ends of eight pairs, or two neighbouring vectors
  const int per_head = dim / 16, rot_items = half / 8;
  const int q_heads = (int)in.heads, k_heads = q_heads + (int)in.kv_heads;
  const int all = k_heads + (cached ? (int)in.kv_heads : 0);
  const int items = all * per_head, step = kRopeThreads * (int)gridDim.y;

  const __nv_bfloat16* src = nullptr;  // of token t0
  int64_t ld_src = 0;
  int h = 0, i = 0, lo = 0, hi = 0;
  uint4 a[TOKENS], b[TOKENS];
  auto locate = [&](int w) {
    h = w / per_head;
    i = w - h * per_head;
    const bool turn = i < rot_items && h < k_heads;
    lo = turn ? 8 * i : h < k_heads ? 2 * half + 16 * (i - rot_items) : 16 * i;
    hi = lo + (turn ? half : 8);
    const attn_rows& r = h < q_heads ? in.q : h < k_heads ? in.k : in.v;
    const int head = h < q_heads ? h : h < k_heads ? h - q_heads : h - k_heads;
    ld_src = r.ld_token;
    src = (const __nv_bfloat16*)r.data + t0 * ld_src + head * r.ld_head;
  };
  auto load = [&]() {
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
      if (t < count) {
        a[t] = load16(src + t * ld_src + lo);
        b[t] = load16(src + t * ld_src + hi);
      }
    }
  };
  int w = (int)blockIdx.y * kRopeThreads + (int)threadIdx.x;
  if (w < items) locate(w);
  nvfp4::wait_for_previous_kernel();
  if (w < items) load();
  for (int x = threadIdx.x; x < count * half; x += kRopeThreads) {
    const int t = x / half, j = x - t * half;
    const int axis = in.axis != nullptr ? in.axis[j] : 0;
    const int64_t position = nvfp4::ld_ro(in.positions + (axis < in.axes ? axis : 0) * in.ld_positions + t0 + t);
    const uint64_t turns = (uint64_t)position * in.turns[j];
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    angles[t][2 * (j % 8 / 2 * rot_items + j / 8) + j % 2] = make_float2(c, s);
  }
  if (cached && (int)threadIdx.x < count) {
    const int32_t slot = nvfp4::ld_ro(in.slots + t0 + threadIdx.x);
    const int32_t page = slot / (int32_t)in.page_size, off = slot - page * (int32_t)in.page_size;
    const bool ok = slot >= 0 && page < in.pages;
    if (slot >= 0 && !ok) nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
    k_at[threadIdx.x] = ok ? page * in.k_cache.ld_page + off * in.k_cache.ld_token : -1;
    v_at[threadIdx.x] = ok ? page * in.v_cache.ld_page + off * in.v_cache.ld_token : -1;
  }
  __syncthreads();
  while (w < items) {
    const bool turn = i < rot_items && h < k_heads;
    // where it goes: a tensor's rows (not what an in-place call leaves as it is), the cache's pages
    const attn_rows& r = h < q_heads ? p.out.q : p.out.k;
    const int head = h < q_heads ? h : h < k_heads ? h - q_heads : h - k_heads;
    __nv_bfloat16* dst = nullptr;
    if (h < k_heads && r.data != nullptr) {
      dst = (__nv_bfloat16*)r.data + t0 * r.ld_token + head * r.ld_head;
      if (!turn && dst == src) dst = nullptr;
    }
    const kv_pages& c = h < k_heads ? in.k_cache : in.v_cache;
    const int64_t* slots = h < k_heads ? k_at : v_at;
    const bool caching = cached && h >= q_heads;
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
      if (t >= count) continue;
      if (turn) rotate(a[t], b[t], reinterpret_cast<const float4*>(angles[t]) + i, rot_items);
      if (dst != nullptr) {
        store16(dst + t * r.ld_token + lo, a[t]);
        store16(dst + t * r.ld_token + hi, b[t]);
      }
      if (caching && slots[t] >= 0) {
        __nv_bfloat16* at = (__nv_bfloat16*)c.data + slots[t] + head * c.ld_head;
        store16(at + lo, a[t]);
        store16(at + hi, b[t]);
      }
    }
    w += step;
    if (w < items) {
      locate(w);
      load();
    }
  }
}

}  // namespace

int launch_kv_plan(const kv_plan_input* in, const kv_plan_output* out, int32_t* dev_status, cudaStream_t stream) {
  PlanParams p{*in, *out, -1, dev_status};
  for (int i = 0; i < 17; ++i)
    if (in->page_size == (int64_t)1 << i) p.page_shift = i;
  const size_t smem = (size_t)in->batch * 16;
  // (asked for the largest batch, whatever this one's: one entry of the table that all calls share)
  if (nvfp4::occupancy((const void*)kv_plan_kernel, kPlanThreads, (size_t)KV_PLAN_MAX_BATCH * 16) < 1)
    return NVFP4_ERR_CUDA;
  // One CTA while each thread has two tokens at most, else a cluster of eight: 200 requests of 5
  // tokens 5.2 us (a cluster 5.5), 1000 of 1 6.1 (6.4); 400 of 5 6.6 (5.8), 1000 of 8 13.5 (6.4).
  const unsigned ranks = in->tokens + in->batch <= 2 * kPlanThreads ? 1 : 8;
  void* args[] = {&p};
  return nvfp4::launch_dependent((const void*)kv_plan_kernel, dim3(ranks), dim3(kPlanThreads), smem, stream, ranks,
                                 args) == cudaSuccess
             ? NVFP4_OK
             : NVFP4_ERR_CUDA;
}

int launch_rope_kv_write(const rope_kv_input* in, const rope_kv_output* out, int32_t* dev_status,
                         cudaStream_t stream) {
  RopeParams p{*in, *out, dev_status};
  // Four tokens a CTA where that leaves each SM one; fewer tokens one by one, their vectors over
  // several CTAs.  32 / 8 heads of 128: 608 tokens 4.0 us (one by one 4.6), 2432 9.3 (12.1), 16384
  // 61 (83); 315 tokens one by one 3.2 (3.9).
  const bool many = in->tokens >= (int64_t)4 * nvfp4::sm_count();
  const int64_t groups = many ? nvfp4::cdiv(in->tokens, 4) : in->tokens;
  if (groups > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  const int64_t items = (in->heads + (in->k_cache.data != nullptr ? 2 : 1) * in->kv_heads) * (in->dim / 16);
  const int64_t parts = many ? 1 : nvfp4::cdiv(items, kRopeThreads);
  void* args[] = {&p};
  const void* kern = many ? (const void*)rope_kv_kernel<4> : (const void*)rope_kv_kernel<1>;
  return nvfp4::launch_dependent(kern, dim3((unsigned)groups, (unsigned)(parts < 64 ? parts : 64)), dim3(kRopeThreads), 0,
                                 stream, 1, args) == cudaSuccess
             ? NVFP4_OK
             : NVFP4_ERR_CUDA;
}
