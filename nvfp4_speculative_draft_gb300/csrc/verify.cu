// verify.cu -- speculative verification: which drafted tokens the target keeps,
// and the token sampled after them, from given uniform numbers.
//
//   accept draft i while u_i q_i(d_i) < p_i(d_i);  a = accepted
//   w_j = max(p_a(j) - q_a(j), 0) after a refusal, p_a(j) when all were accepted
//   token = min { j : w_0 + ... + w_j > r W },  W = sum w
//
// One thread-block cluster per sequence.  Every CTA finds a for itself (a few
// gathers), then sums w over its contiguous share of the row, one contiguous
// segment per warp; the totals are exchanged through distributed shared memory,
// every CTA forms the same prefix sums in the same order, and the one CTA whose
// share crosses r W narrows its crossing segment (in cache by now) until a single
// warp finds the index in 32 vectors.  So a row is read from memory once, there is
// no workspace and no atomic, and nothing depends on timing.
//
// Precision: with 150 000 tokens the borders between neighbouring tokens lie
// about 2^-17 W apart, so sums in binary32 would pick a neighbour now and then.
// p - q is kept exactly as the sum of two binary32 words, a lane's running sum as
// two words (the rounding errors of the additions are added up beside it, Knuth's
// two-sum), and segment totals are joined in binary64: off by about 2^-46 of W.
// Binary64 adds for every element would be slower than memory on this chip (its
// rate is a 64th of binary32's).

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct VerifyParams {
  const void* target;
  const void* draft;
  int64_t ld_ts, ld_tp, ld_ds, ld_dp;
  int64_t draft_vocab, vocab;
  const int32_t* tokens;
  int64_t ld_tok;
  const int32_t* num_draft;
  const float* accept_u;
  int64_t ld_u;
  const float* sample_u;
  int32_t* out;
  int64_t ld_out;
  int32_t* accepted;
  int32_t* dev_status;
  int g;
};

__device__ __forceinline__ float load_one(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// One 16-byte vector of a row (VE = 4 or 8 elements), as binary32.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int VE = 4, kUnroll = 4;
  uint4 raw;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w)
                 : "l"(p));
  }
  __device__ __forceinline__ void load_elements(const float* p) {
    raw = make_uint4(__float_as_uint(__ldg(p)), __float_as_uint(__ldg(p + 1)),
                     __float_as_uint(__ldg(p + 2)), __float_as_uint(__ldg(p + 3)));
  }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = __uint_as_float(raw.x);
    f[1] = __uint_as_float(raw.y);
    f[2] = __uint_as_float(raw.z);
    f[3] = __uint_as_float(raw.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int VE = 8, kUnroll = 2;
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w)
                 : "l"(p));
  }
  __device__ __forceinline__ void load_elements(const __nv_bfloat16* p) {
    const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (uint32_t)__ldg(u + 2 * j) | (uint32_t)__ldg(u + 2 * j + 1) << 16;
    raw = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(u[j] << 16);
      f[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
  }
};

// The rows of one sequence's decision, and how its weights are formed.
template <typename T>
struct Rows {
  const T* p;     // target row
  const T* q;     // draft row or nullptr
  int vocab;      // elements of p (at most 2^30: all indices of a row fit in 32 bits)
  int qn;         // elements of q (0 without)
  int skip;       // greedy: the refused token, whose weight is max(p - 1, 0); else -1
  int mis;        // elements from the 16-byte boundary at or before p to p
  bool qvec;      // q has the same misalignment: it can be read as vectors too
};

// A sum in two words, s + c.
struct Sum {
  float s, c;
  __device__ __forceinline__ void add(float hi, float lo) {  // two-sum of s and hi
    const float t = s + hi;
    const float z = t - s;
    c += ((s - (t - z)) + (hi - z)) + lo;
    s = t;
  }
  __device__ __forceinline__ double value() const { return (double)s + (double)c; }
};

__device__ __forceinline__ Sum warp_sum(Sum v) {  // the same value and order in every lane
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const float s = __shfl_xor_sync(0xFFFFFFFFu, v.s, d), c = __shfl_xor_sync(0xFFFFFFFFu, v.c, d);
    v.add(s, c);
  }
  return v;
}

// Inclusive prefix over the first N lanes (a power of two), binary64.
template <int N>
__device__ __forceinline__ double prefix(double v, int lane) {
#pragma unroll
  for (int d = 1; d < N; d <<= 1) {
    const double o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// w = max(p - q, 0) as an unevaluated sum hi + lo; 0 for what is not finite.
__device__ __forceinline__ void weight(float p, float q, float& hi, float& lo, bool& bad) {
  const float d = p - q;  // two-sum of p and -q: d + e = p - q exactly
  const float b = d - p;
  const float e = (p - (d - b)) + (-q - b);
  const bool fin = fabsf(d) < __int_as_float(0x7F800000);
  bad = bad || !fin;
  const bool pos = fin && d > 0.0f;
  hi = pos ? d : 0.0f;
  lo = pos ? e : 0.0f;
}

// Vector v of the row is its elements v VE - mis + (0..VE-1).  inner: it lies
// wholly in the target row, wholly in or wholly past the draft's, and clear of
// the refused token; the others (a few per row) are read element by element.
template <typename T>
__device__ __forceinline__ bool inner(const Rows<T>& r, int i) {
  constexpr int VE = Vec<T>::VE;
  return i >= 0 && i + VE <= r.vocab && (i >= r.qn || i + VE <= r.qn) &&
         !(r.skip >= i && r.skip < i + VE);
}
template <typename T>
__device__ __forceinline__ void edge_weight(const Rows<T>& r, int i, float& hi, float& lo,
                                            bool& bad) {
  hi = lo = 0.0f;
  if (i >= 0 && i < r.vocab) {
    const float q = i == r.skip ? 1.0f : i < r.qn ? load_one(r.q + i) : 0.0f;
    weight(load_one(r.p + i), q, hi, lo, bad);
  }
}

// One lane's sum of the weights of vectors v, v + step, ... below end.
template <typename T>
__device__ __forceinline__ Sum lane_sum(const Rows<T>& r, int v, int end, int step, bool& bad) {
  constexpr int VE = Vec<T>::VE, U = Vec<T>::kUnroll;
  Sum sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // two chains of dependent additions
  for (; v < end; v += U * step) {
    Vec<T> a[U], b[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // all loads first
      const int vv = v + u * step, i = vv * VE - r.mis;
      in[u] = vv < end && inner(r, i);
      if (in[u]) {
        a[u].load(r.p + i);
        if (i < r.qn) {
          if (r.qvec)
            b[u].load(r.q + i);
          else
            b[u].load_elements(r.q + i);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int vv = v + u * step, i = vv * VE - r.mis;
      if (in[u]) {
        float p[VE], q[VE];
        a[u].get(p);
        if (i < r.qn) {
          b[u].get(q);
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            float hi, lo;
            weight(p[j], q[j], hi, lo, bad);
            sum[j & 1].add(hi, lo);
          }
        } else {
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const bool fin = fabsf(p[j]) < __int_as_float(0x7F800000);
            bad = bad || !fin;
            sum[j & 1].add(fin ? fmaxf(p[j], 0.0f) : 0.0f, 0.0f);
          }
        }
      } else if (vv < end) {
#pragma unroll 1
        for (int j = 0; j < VE; ++j) {
          float hi, lo;
          edge_weight(r, i + j, hi, lo, bad);
          sum[0].add(hi, lo);
        }
      }
    }
  }
  sum[0].add(sum[1].s, sum[1].c);
  return sum[0];
}

// The part (lane c < N holding part c's sum) that t falls into: the first whose
// prefix upto exceeds t, or the last with any mass; -1 without mass.
__device__ __forceinline__ int pick(double mine, double upto, double t) {
  const unsigned over = __ballot_sync(0xFFFFFFFFu, mine > 0.0 && upto > t);
  const unsigned any = __ballot_sync(0xFFFFFFFFu, mine > 0.0);
  return over != 0u ? __ffs(over) - 1 : 31 - __clz(any);  // (31 - clz(0) = -1)
}
// The prefix before part `who`.
__device__ __forceinline__ double before(double upto, int who, double base) {
  const double v = __shfl_sync(0xFFFFFFFFu, upto, who > 0 ? who - 1 : 0);
  return who > 0 ? v : base;
}

// One warp: the first index among vectors [v0, v1) whose running sum from base
// exceeds t; the last one with a weight where rounding leaves none.  First over
// lanes with equal contiguous shares, then over the elements of one share.
constexpr int kFindElements = 64;  // most elements of a lane's share
template <typename T>
__device__ int find_index(const Rows<T>& r, int v0, int v1, double base, double t,
                              int lane) {
  constexpr int VE = Vec<T>::VE;
  const int share = (v1 - v0 + 31) / 32;
  bool bad = false;
  const int mv = min(v1, v0 + lane * share);
  const double mine = lane_sum(r, mv, min(v1, mv + share), 1, bad).value();
  const double upto = base + prefix<32>(mine, lane);
  const int who = pick(mine, upto, t);
  if (who < 0) return 0;
  base = before(upto, who, base);
  const int e0 = (v0 + who * share) * VE - r.mis, e1 = min(v1, v0 + (who + 1) * share) * VE - r.mis;
  int last = 0;
  for (int e = e0; e < e1; e += 32) {
    float hi = 0.0f, lo = 0.0f;
    if (e + lane < e1) edge_weight(r, e + lane, hi, lo, bad);
    const double w = (double)hi + (double)lo;
    const double run = base + prefix<32>(w, lane);
    const int at = pick(w, run, t);
    if (at >= 0) last = e + at;
    base = __shfl_sync(0xFFFFFFFFu, run, 31);
    if (__any_sync(0xFFFFFFFFu, w > 0.0 && run > t)) break;
  }
  return last;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) spec_verify_kernel(const __grid_constant__ VerifyParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int64_t seq = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ Sum part[kWarps];    // the warps' sums
  __shared__ double cta_sum[2];   // this CTA's, read by the others; one per pass
  __shared__ int s_accepted, s_owner, s_part;

  const T* target = reinterpret_cast<const T*>(p.target) + seq * p.ld_ts;
  const T* draft = p.draft != nullptr ? reinterpret_cast<const T*>(p.draft) + seq * p.ld_ds : nullptr;
  const int32_t* tokens = p.tokens + seq * p.ld_tok;
  int num = p.g;
  if (p.num_draft != nullptr) {
    num = __ldg(p.num_draft + seq);
    if (num < 0) return;  // absent: the same in every CTA of the cluster
    if (num > p.g) {
      num = p.g;
      if (rank == 0 && threadIdx.x == 0) nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
    }
  }
  if (warp == 0) {  // the first refusal
    int a = num;
    for (int i0 = 0; i0 < p.g; i0 += 32) {
      const int i = i0 + lane;
      bool refuse = false;
      if (i < p.g) {  // (loads before the comparison with num, which is on its way too)
        const int64_t d = __ldg(tokens + i);
        const float u = __ldg(p.accept_u + seq * p.ld_u + i);
        const bool known = d >= 0 && d < p.vocab;
        if (i < num) {
          refuse = true;
          if (known) {
            const float pd = load_one(target + i * p.ld_tp + d);
            const float qd = draft == nullptr    ? 1.0f
                             : d < p.draft_vocab ? load_one(draft + i * p.ld_dp + d)
                                                 : 0.0f;
            refuse = !((double)u * (double)qd < (double)pd);  // 48 bits: the product is exact
          } else if (rank == 0) {
            nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
          }
        }
      }
      const unsigned b = __ballot_sync(0xFFFFFFFFu, refuse);
      if (b != 0u) {
        a = i0 + __ffs(b) - 1;
        break;
      }
      if (i0 + 32 >= num) break;
    }
    if (lane == 0) s_accepted = a;
    if (rank == 0) {  // everything but the sampled token
      for (int i = lane; i <= p.g; i += 32)
        if (i != a) p.out[seq * p.ld_out + i] = i < a ? __ldg(tokens + i) : -1;
      if (lane == 0) p.accepted[seq] = a;
    }
  }
  __syncthreads();
  const int a = s_accepted;
  const bool refused = a < num;

  Rows<T> r;
  r.p = target + a * p.ld_tp;
  r.vocab = (int)p.vocab;
  r.q = refused && draft != nullptr ? draft + a * p.ld_dp : nullptr;
  r.qn = r.q != nullptr ? (int)p.draft_vocab : 0;
  r.skip = refused && draft == nullptr ? __ldg(tokens + a) : -1;
  r.mis = (int)((reinterpret_cast<uintptr_t>(r.p) & 15u) / sizeof(T));
  r.qvec = ((reinterpret_cast<uintptr_t>(r.q) ^ reinterpret_cast<uintptr_t>(r.p)) & 15u) == 0;

  constexpr int VE = Vec<T>::VE;
  const int nvec = (r.vocab + r.mis + VE - 1) / VE;
  const int per_cta = (nvec + ranks - 1) / ranks;
  int v0 = min(nvec, rank * per_cta), v1 = min(nvec, v0 + per_cta);

  bool bad = false;
  double t = 0.0, base = 0.0;  // warp 0: r W, and the prefix before the part at hand
  int per = (v1 - v0 + kWarps - 1) / kWarps;  // vectors of a warp's segment
  auto sum_parts = [&]() {
    const int w0 = min(v1, v0 + warp * per);
    const Sum mine = warp_sum(lane_sum(r, w0 + lane, min(v1, w0 + per), 32, bad));
    if (lane == 0) part[warp] = mine;
    __syncthreads();
  };
  for (int pass = 0; pass < 2; ++pass) {
    sum_parts();
    double mine = 0.0, upto = 0.0;  // warp 0: of the CTA's parts
    if (warp == 0) {
      mine = lane < kWarps ? part[lane].value() : 0.0;
      upto = prefix<kWarps>(mine, lane);
      if (lane == kWarps - 1) cta_sum[pass] = upto;
    }
    cluster.sync();
    if (warp == 0) {  // the CTA that t falls into, the same in every CTA; there, the part
      const double c = lane < ranks ? *cluster.map_shared_rank(&cta_sum[pass], lane) : 0.0;
      const double cupto = prefix<kMaxCluster>(c, lane);
      t = (double)__ldg(p.sample_u + seq) * __shfl_sync(0xFFFFFFFFu, cupto, ranks - 1);
      if (t < 0.0) t = 0.0;
      const int owner = pick(c, cupto, t);
      if (owner == rank) {
        base = before(cupto, owner, 0.0);
        upto += base;
        const int w = max(pick(mine, upto, t), 0);
        base = before(upto, w, base);
        if (lane == 0) s_part = w;
      }
      if (lane == 0) s_owner = owner;
    }
    __syncthreads();
    if (s_owner >= 0 || pass == 1 || (r.qn == 0 && r.skip < 0)) break;
    r.q = nullptr;  // nothing is left of p - q: sample p
    r.qn = 0;
    r.skip = -1;
  }
  if (s_owner < 0) {
    if (rank == 0 && threadIdx.x == 0) p.out[seq * p.ld_out + a] = 0;
  } else if (rank == s_owner) {
    while (true) {  // narrow [v0, v1) to the segment that t falls into
      v0 = min(v1, v0 + s_part * per);
      v1 = min(v1, v0 + per);
      if (v1 - v0 <= 32 * (kFindElements / VE)) break;
      per = (v1 - v0 + kWarps - 1) / kWarps;
      sum_parts();
      if (warp == 0) {
        const double mine = lane < kWarps ? part[lane].value() : 0.0;
        const double upto = base + prefix<kWarps>(mine, lane);
        const int w = max(pick(mine, upto, t), 0);
        base = before(upto, w, base);
        if (lane == 0) s_part = w;
      }
      __syncthreads();
    }
    if (warp == 0) {
      const int j = find_index(r, v0, v1, base, t, lane);
      if (lane == 0) p.out[seq * p.ld_out + a] = j;
    }
  }
  if (bad) nvfp4::report(p.dev_status, NVFP4_ERR_NONFINITE);
  cluster.sync();  // no CTA leaves while another may still read its sum
}

}  // namespace

int launch_spec_verify(const spec_verify_input* in, int32_t* out_tokens, int64_t ld_out,
                       int32_t* accepted, int32_t* dev_status, cudaStream_t stream) {
  VerifyParams p;
  p.target = in->target;
  p.draft = in->g > 0 ? in->draft : nullptr;
  p.ld_ts = in->ld_target_seq;
  p.ld_tp = in->ld_target_pos;
  p.ld_ds = in->ld_draft_seq;
  p.ld_dp = in->ld_draft_pos;
  p.draft_vocab = in->draft_vocab;
  p.vocab = in->vocab;
  p.tokens = in->tokens;
  p.ld_tok = in->ld_tokens;
  p.num_draft = in->num_draft;
  p.accept_u = in->accept_u;
  p.ld_u = in->ld_accept_u;
  p.sample_u = in->sample_u;
  p.out = out_tokens;
  p.ld_out = ld_out;
  p.accepted = accepted;
  p.dev_status = dev_status;
  p.g = (int)in->g;
  // CTAs per sequence: as many as keep about two CTAs on every SM, while each
  // still has a few thousand tokens to read
  const int64_t sms = nvfp4::sm_count();
  int ranks = 1;
  while (ranks < kMaxCluster && in->batch * ranks < 2 * sms && in->vocab / (2 * ranks) >= 2048) ranks *= 2;
  if (in->batch > 0x7FFFFFFF / ranks) return NVFP4_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(in->batch * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = in->dtype == NVFP4_DTYPE_F32
                            ? cudaLaunchKernelEx(&cfg, spec_verify_kernel<float>, p)
                            : cudaLaunchKernelEx(&cfg, spec_verify_kernel<__nv_bfloat16>, p);
  return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
