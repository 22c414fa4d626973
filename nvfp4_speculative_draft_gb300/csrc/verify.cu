// verify.cu -- speculative verification: which drafted tokens the target keeps,
// and the token sampled after them, from given uniform numbers.
//
//   accept draft i while u_i q_i(d_i) < p_i(d_i);  a = accepted
//   w_j = max(p_a(j) - q_a(j), 0) after a refusal, p_a(j) when all were accepted
//   token = min { j : w_0 + ... + w_j > r W },  W = sum w
//
// One thread-block cluster per sequence.  Every CTA finds a for itself (a few
// gathers), then sums w over its contiguous share of the row, one contiguous
// segment per warp and one part of it per eight lanes; the warps' sums are exchanged
// through distributed shared memory, every CTA forms the same prefix sums in the
// same order, and the one CTA whose segment crosses r W narrows it (in cache by now)
// to the index.  So a row is read from memory once, there is no workspace and no
// atomic, and nothing depends on timing.
//
// Precision: with 150 000 tokens the borders between neighbouring tokens lie
// about 2^-17 W apart, so sums in binary32 would pick a neighbour now and then.
// p - q is kept exactly as the sum of two binary32 words, and all sums are carried
// in two words (the rounding errors of the additions are added up beside them,
// Knuth's two-sum): off by about 2^-46 of W.  Binary64 is not used: the SM's one
// binary64 unit takes 16 cycles a warp instruction.
//
// What bounds it: for large batches HBM (256 sequences of 151936 FP32 probabilities,
// ragged drafts, 55.7 us; every sequence's target row and the draft rows of those that
// refuse are about 250 MB, 4.5 TB/s, 0.66 of the measured copy; 121 us with sums joined in
// binary64 and 512 threads a CTA); for few sequences the chain of dependent steps, each a
// load's or a shuffle's latency: one sequence of 32768 5.8 us, of which launch about 2,
// finding the refusal 0.8, the sums 2, their exchange 1 and the search 1.3 (17 us with one
// CTA).  16 CTAs a sequence or 512 threads are no faster.

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;  // four CTAs an SM: one's dependent steps hide behind another's loads
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kLaneParts = kMaxCluster * kWarps / 32;  // most segments that a lane looks at
constexpr int kGroupLanes = 8, kGroups = 32 / kGroupLanes;  // parts of a warp's segment
constexpr int kShare = 4;  // vectors of a lane's share that is searched element by element

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
  int g, log_ranks;
};

using nvfp4::ld_ro;

__device__ __forceinline__ float load_one(const float* p) { return ld_ro(p); }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) {
  return __uint_as_float(ld_ro(reinterpret_cast<const unsigned short*>(p)) << 16);
}

// Packed binary32 pairs.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void halves(uint64_t v, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {  // b (-1) + a: one rounding
  return fma2(b, 0xBF800000BF800000ull, a);
}
// The bits of v where the matching half of d is not negative, else +0.
__device__ __forceinline__ uint64_t where_positive(uint64_t d, uint64_t v) {
  uint32_t d0, d1, v0, v1;
  halves(d, d0, d1);
  halves(v, v0, v1);
  return pair(v0 & ~(uint32_t)((int32_t)d0 >> 31), v1 & ~(uint32_t)((int32_t)d1 >> 31));
}

// One 16-byte vector of a row (VE = 4 or 8 elements), as binary32 pairs.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int VE = 4;
  uint4 raw;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w)
                 : "l"(p));
  }
  __device__ __forceinline__ void load_elements(const float* p) {
    raw = make_uint4(__float_as_uint(ld_ro(p)), __float_as_uint(ld_ro(p + 1)),
                     __float_as_uint(ld_ro(p + 2)), __float_as_uint(ld_ro(p + 3)));
  }
  __device__ __forceinline__ void get(uint64_t (&f)[2]) const {
    f[0] = pair(raw.x, raw.y);
    f[1] = pair(raw.z, raw.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int VE = 8;
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
    for (int j = 0; j < 4; ++j) w[j] = ld_ro(u + 2 * j) | ld_ro(u + 2 * j + 1) << 16;
    raw = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void get(uint64_t (&f)[4]) const {
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = pair(u[j] << 16, u[j] & 0xFFFF0000u);
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
  __device__ __forceinline__ void add(Sum o) { add(o.s, o.c); }
  // The same value with s the rounded sum, so that sums compare word by word.
  __device__ __forceinline__ Sum normal() const {
    const float t = s + c;
    return Sum{t, c - (t - s)};
  }
};
__device__ __forceinline__ bool greater(Sum a, Sum b) {  // both normal
  return a.s > b.s || (a.s == b.s && a.c > b.c);
}
__device__ __forceinline__ Sum shuffle(Sum v, int lane) {
  return Sum{__shfl_sync(0xFFFFFFFFu, v.s, lane), __shfl_sync(0xFFFFFFFFu, v.c, lane)};
}
// Inclusive prefix over the lanes.
__device__ __forceinline__ Sum prefix(Sum v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float s = __shfl_up_sync(0xFFFFFFFFu, v.s, d), c = __shfl_up_sync(0xFFFFFFFFu, v.c, d);
    if (lane >= d) v.add(s, c);
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

// Two running sums in two words each (even and odd elements), and a word that turns
// NaN with the first value that is not finite.
struct Sum2 {
  uint64_t s, c, nan;
  __device__ __forceinline__ void add_positive(uint64_t d) {  // + max(d, 0)
    nan = fma2(d, 0ull, nan);
    const uint64_t hi = where_positive(d, d);
    const uint64_t t = add2(s, hi), z = sub2(t, s);
    c = add2(c, add2(sub2(s, sub2(t, z)), sub2(hi, z)));
    s = t;
  }
  __device__ __forceinline__ void add_difference(uint64_t p, uint64_t q) {  // + max(p - q, 0)
    const uint64_t d = sub2(p, q), b = sub2(d, p);
    const uint64_t e = sub2(sub2(p, sub2(d, b)), add2(q, b));
    nan = fma2(d, 0ull, nan);
    const uint64_t hi = where_positive(d, d), lo = where_positive(d, e);
    const uint64_t t = add2(s, hi), z = sub2(t, s);
    c = add2(c, add2(add2(sub2(s, sub2(t, z)), sub2(hi, z)), lo));
    s = t;
  }
};

// One lane's sum of the weights of vectors v, v + step, ... below end, element by
// element: where a value is not finite.
template <typename T>
__device__ __noinline__ Sum lane_sum_checked(Rows<T> r, int v, int end, int step, int32_t* dev_status) {
  Sum sum{0.0f, 0.0f};
  bool bad = false;
  for (; v < end; v += step)
    for (int j = 0; j < Vec<T>::VE; ++j) {
      float hi, lo;
      edge_weight(r, v * Vec<T>::VE - r.mis + j, hi, lo, bad);
      sum.add(hi, lo);
    }
  if (bad) nvfp4::report(dev_status, NVFP4_ERR_NONFINITE);
  return sum;
}

// One lane's sum of the weights of vectors first, first + step, ... below end.  (Not
// inlined: both uses share the code, which a short kernel fetches for the first time.)
template <typename T, int EL>
__device__ __noinline__ Sum lane_sum(Rows<T> r, int first, int end, int step, int32_t* dev_status) {
  constexpr int VE = Vec<T>::VE, U = EL / VE;  // vectors of each row in flight
  Sum2 sum{0ull, 0ull, 0ull};
  Sum edge{0.0f, 0.0f};
  bool edge_bad = false;
  Vec<T> a[U], b[U];
  auto load = [&](int v) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int vv = v + u * step, i = vv * VE - r.mis;
      if (vv < end && inner(r, i)) {
        a[u].load(r.p + i);
        if (i < r.qn) {
          if (r.qvec)
            b[u].load(r.q + i);
          else
            b[u].load_elements(r.q + i);
        }
      }
    }
  };
  load(first);
  for (int v = first; v < end; v += U * step) {
    uint64_t p[U][VE / 2], q[U][VE / 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      a[u].get(p[u]);
      b[u].get(q[u]);
    }
    load(v + U * step);  // the next vectors are on their way during the arithmetic
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int vv = v + u * step, i = vv * VE - r.mis;
      if (vv < end && inner(r, i)) {
        if (i < r.qn) {
#pragma unroll
          for (int j = 0; j < VE / 2; ++j) sum.add_difference(p[u][j], q[u][j]);
        } else {
#pragma unroll
          for (int j = 0; j < VE / 2; ++j) sum.add_positive(p[u][j]);
        }
      } else if (vv < end) {
#pragma unroll 1
        for (int j = 0; j < VE; ++j) {
          float hi, lo;
          edge_weight(r, i + j, hi, lo, edge_bad);
          edge.add(hi, lo);
        }
      }
    }
  }
  uint32_t n0, n1;
  halves(sum.nan, n0, n1);
  if (__uint_as_float(n0) + __uint_as_float(n1) != 0.0f)  // NaN
    return lane_sum_checked(r, first, end, step, dev_status);
  if (edge_bad) nvfp4::report(dev_status, NVFP4_ERR_NONFINITE);
  uint32_t s0, s1, c0, c1;
  halves(sum.s, s0, s1);
  halves(sum.c, c0, c1);
  edge.add(__uint_as_float(s0), __uint_as_float(c0));
  edge.add(__uint_as_float(s1), __uint_as_float(c1));
  return edge;
}

// The lane whose part t falls into: the first whose prefix upto exceeds t, or the
// last with any mass; -1 without mass.
__device__ __forceinline__ int pick(Sum mine, Sum upto, Sum t) {
  const unsigned over = __ballot_sync(0xFFFFFFFFu, mine.s > 0.0f && greater(upto.normal(), t));
  const unsigned any = __ballot_sync(0xFFFFFFFFu, mine.s > 0.0f);
  return over != 0u ? __ffs(over) - 1 : 31 - __clz(any);  // (31 - clz(0) = -1)
}
// The same among N parts that every lane holds, or that shared memory does; base becomes the prefix
// before the part.
template <int N>
__device__ __forceinline__ int pick_among(const Sum* parts, Sum t, Sum& base) {
  Sum run = base, at = base;
  int who = -1;
  bool found = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!found && parts[i].s > 0.0f) {
      who = i;
      at = run;
    }
    run.add(parts[i]);
    found = found || (parts[i].s > 0.0f && greater(run.normal(), t));
  }
  base = at;
  return who;
}
__device__ __forceinline__ Sum plus(Sum a, Sum b) {
  a.add(b);
  return a;
}
// The prefix before lane `who`, base and the inclusive prefixes given.
__device__ __forceinline__ Sum before(Sum upto, int who, Sum base) {
  const Sum v = shuffle(upto, who > 0 ? who - 1 : 0);
  return who > 0 ? v : base;
}

// One warp: the first index among vectors [v0, v1) (a few) whose running sum from
// base exceeds t; the last one with a weight where rounding leaves none.
template <typename T>
__device__ int find_index(const Rows<T>& r, int v0, int v1, Sum base, Sum t, int lane) {
  constexpr int VE = Vec<T>::VE;
  bool bad = false;  // (reported by the sums)
  const int e0 = v0 * VE - r.mis, e1 = v1 * VE - r.mis;
  int last = 0;
  for (int e = e0; e < e1; e += 32) {
    Sum w{0.0f, 0.0f};
    if (e + lane < e1) edge_weight(r, e + lane, w.s, w.c, bad);
    const Sum run = plus(base, prefix(w, lane));
    const int at = pick(w, run, t);
    if (at >= 0) last = e + at;
    if (__any_sync(0xFFFFFFFFu, w.s > 0.0f && greater(run.normal(), t))) break;
    base = shuffle(run, 31);
  }
  return last;
}

__device__ __forceinline__ bool below(float u, float q, float p) {  // u q < p, exactly
  const float h = u * q;
  if (h < 0x1p-60f) return (double)u * (double)q < (double)p;
  return h < p || (h == p && fmaf(u, q, -h) < 0.0f);
}

// EL: elements of a row that a lane has in flight; CTAS: CTAs an SM.
template <typename T, int EL, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) spec_verify_kernel(const __grid_constant__ VerifyParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = 1 << p.log_ranks, rank = (int)blockIdx.x & (ranks - 1);
  const int64_t seq = (int)blockIdx.x >> p.log_ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ Sum warp_part[2][kWarps];        // the warps' sums, read by the other CTAs; per pass
  __shared__ Sum group_part[kWarps][kGroups];  // of their parts
  __shared__ Sum find_part[kWarps];
  __shared__ Sum s_base, s_target;
  __shared__ int s_accepted, s_token, s_owner, s_part, s_v0, s_v1;

  const T* target = reinterpret_cast<const T*>(p.target) + seq * p.ld_ts;
  const T* draft = p.draft != nullptr ? reinterpret_cast<const T*>(p.draft) + seq * p.ld_ds : nullptr;
  const int32_t* tokens = p.tokens + seq * p.ld_tok;
  nvfp4::wait_for_previous_kernel();
  int num = p.g;
  if (p.num_draft != nullptr) {
    num = ld_ro(p.num_draft + seq);
    if (num < 0) return;  // absent: the same in every CTA of the cluster
    if (num > p.g) {
      num = p.g;
      if (rank == 0 && threadIdx.x == 0) nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
    }
  }
  if (warp == 0) {  // the first refusal
    int a = num, d = -1;
    for (int i0 = 0; i0 < num; i0 += 32) {
      const int i = i0 + lane;
      bool refuse = false;
      if (i < num) {
        d = ld_ro(tokens + i);
        const float u = ld_ro(p.accept_u + seq * p.ld_u + i);
        refuse = true;
        if (d >= 0 && d < p.vocab) {
          const float pd = load_one(target + i * p.ld_tp + d);
          const float qd = draft == nullptr    ? 1.0f
                           : d < p.draft_vocab ? load_one(draft + i * p.ld_dp + d)
                                               : 0.0f;
          refuse = !below(u, qd, pd);
        } else if (rank == 0) {
          nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
        }
      }
      const unsigned b = __ballot_sync(0xFFFFFFFFu, refuse);
      if (b != 0u) {
        a = i0 + __ffs(b) - 1;
        d = __shfl_sync(0xFFFFFFFFu, d, a - i0);
        break;
      }
    }
    if (lane == 0) {
      s_accepted = a;
      s_token = d;  // the refused one
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
  r.skip = refused && draft == nullptr ? s_token : -1;
  r.mis = (int)((reinterpret_cast<uintptr_t>(r.p) & 15u) / sizeof(T));
  r.qvec = ((reinterpret_cast<uintptr_t>(r.q) ^ reinterpret_cast<uintptr_t>(r.p)) & 15u) == 0;

  // vectors of the row: shares of CTAs, segments of warps, parts of eight lanes
  constexpr int VE = Vec<T>::VE;
  const int nvec = (r.vocab + r.mis + VE - 1) / VE;
  const int per_cta = (nvec + ranks - 1) >> p.log_ranks;
  const int c0 = min(nvec, rank * per_cta), c1 = min(nvec, c0 + per_cta);
  const int per_warp = (c1 - c0 + kWarps - 1) / kWarps, per = (per_warp + kGroups - 1) / kGroups;
  auto segment = [&](int w) { return min(c1, c0 + w * per_warp); };
  for (int pass = 0; pass < 2; ++pass) {
    const int w1 = segment(warp + 1), g0 = min(w1, segment(warp) + lane / kGroupLanes * per);
    Sum sum = lane_sum<T, EL>(r, g0 + lane % kGroupLanes, min(w1, g0 + per), kGroupLanes, p.dev_status);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      if (d == kGroupLanes && lane % kGroupLanes == 0) group_part[warp][lane / kGroupLanes] = sum;
      sum.add(__shfl_xor_sync(0xFFFFFFFFu, sum.s, d), __shfl_xor_sync(0xFFFFFFFFu, sum.c, d));
    }
    if (lane == 0) warp_part[pass][warp] = sum;
    if (pass == 0 && rank == 0 && warp == 0) {  // the outputs but for the sampled token
      for (int i = lane; i <= p.g; i += 32)
        if (i != a) p.out[seq * p.ld_out + i] = i < a ? ld_ro(tokens + i) : -1;
      if (lane == 0) p.accepted[seq] = a;
    }
    if (ranks > 1)
      cluster.sync();
    else
      __syncthreads();
    if (warp == 0) {
      // the segment that t falls into, the same in every CTA: a lane has n segments
      const int n = (ranks * kWarps + 31) / 32;
      Sum mine{0.0f, 0.0f}, parts[kLaneParts];
#pragma unroll
      for (int i = 0; i < kLaneParts; ++i) {
        const int s = lane * n + i;
        parts[i] = Sum{0.0f, 0.0f};
        if (i < n && s < ranks * kWarps)
          parts[i] = *cluster.map_shared_rank(&warp_part[pass][s % kWarps], s / kWarps);
      }
#pragma unroll
      for (int i = 0; i < kLaneParts; ++i) mine.add(parts[i]);
      const Sum upto = prefix(mine, lane), all = shuffle(upto, 31).normal();
      const float u = ld_ro(p.sample_u + seq), h = u * all.s;
      Sum t = Sum{h, fmaf(u, all.s, -h) + u * all.c}.normal();
      if (t.s < 0.0f) t = Sum{0.0f, 0.0f};
      const int who = pick(mine, upto, t);
      Sum base = before(upto, who, Sum{0.0f, 0.0f});
#pragma unroll
      for (int i = 0; i < kLaneParts; ++i) parts[i] = shuffle(parts[i], max(who, 0));
      const int s = max(who, 0) * n + max(pick_among<kLaneParts>(parts, t, base), 0);
      const int owner = who < 0 ? -1 : s / kWarps, w = s % kWarps;
      if (owner == rank) {  // and the part of it
        const int gp = max(pick_among<kGroups>(group_part[w], t, base), 0);
        const int g0 = min(segment(w + 1), segment(w) + gp * per);
        if (lane == 0) {
          s_v0 = g0;
          s_v1 = min(segment(w + 1), g0 + per);
          s_base = base;
          s_target = t;
        }
      }
      if (lane == 0) s_owner = owner;
    }
    __syncthreads();
    if (s_owner >= 0 || pass == 1 || (r.qn == 0 && r.skip < 0)) break;
    r.q = nullptr;  // nothing is left of p - q: sample p
    r.qn = 0;
    r.skip = -1;
  }
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  if (s_owner < 0) {
    if (rank == 0 && threadIdx.x == 0) p.out[seq * p.ld_out + a] = 0;
  } else if (rank == s_owner) {
    // Narrow the part: each thread (of one warp where that is enough) sums a contiguous
    // share, and the share that t falls into is next.
    while (true) {
      const int v0 = s_v0, v1 = s_v1;
      const bool one = v1 - v0 <= 32 * kShare;
      const int threads = one ? 32 : kThreads;
      if (one && warp > 0) break;
      const int share = (v1 - v0 + threads - 1) / threads;
      const int mv = min(v1, v0 + (int)threadIdx.x * share), me = min(v1, mv + share);
      const Sum mine = lane_sum<T, EL>(r, mv, me, 1, nullptr);
      Sum upto = prefix(mine, lane);
      bool mine_next = warp == 0;
      if (!one) {
        if (lane == 31) find_part[warp] = upto;
        __syncthreads();
        if (threadIdx.x == 0) {
          Sum base = s_base;
          s_part = max(pick_among<kWarps>(find_part, s_target, base), 0);
          s_base = base;
        }
        __syncthreads();
        mine_next = warp == s_part;
      }
      if (mine_next) {
        const Sum base = s_base, t = s_target;
        upto = plus(base, upto);
        const int who = max(pick(mine, upto, t), 0);
        const Sum b = before(upto, who, base);
        const int f0 = __shfl_sync(0xFFFFFFFFu, mv, who), f1 = __shfl_sync(0xFFFFFFFFu, me, who);
        if (share <= kShare) {
          const int j = find_index(r, f0, f1, b, t, lane);
          if (lane == 0) p.out[seq * p.ld_out + a] = j;
        } else if (lane == 0) {
          s_v0 = f0;
          s_v1 = f1;
          s_base = b;
        }
      }
      if (share <= kShare) break;
      __syncthreads();
    }
  }
  // no CTA leaves while another may still read its sums
  if (ranks > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
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
  // CTAs per sequence: as many as are resident at once (four an SM), while each still
  // has 2048 tokens to read.  256 sequences of 151936 FP32 probabilities, ragged drafts:
  // 2 CTAs 55 us, 1 CTA 74, 4 CTAs 59, 8 CTAs 64; one sequence of 32768: 8 CTAs 6.4 us,
  // 1 CTA 11.5.
  const int64_t sms = nvfp4::sm_count();
  int log_ranks = 0;
  while ((2 << log_ranks) <= kMaxCluster && in->batch << (log_ranks + 1) <= 4 * sms &&
         in->vocab >> (log_ranks + 1) >= 2048)
    ++log_ranks;
  const int ranks = 1 << log_ranks;
  if (in->batch > 0x7FFFFFFF / ranks) return NVFP4_ERR_SHAPE;
  p.log_ranks = log_ranks;
  // Few CTAs: twice the registers each, and for BF16 twice the loads in flight (one
  // sequence 6.2 -> 5.8 us; another doubling is slower, 13.5 us against 11.5 for 24 x 151936).
  const bool few = in->batch * ranks <= 2 * sms, f32 = in->dtype == NVFP4_DTYPE_F32;
  const void* kern = f32 ? (few ? (const void*)spec_verify_kernel<float, 8, 2>
                                : (const void*)spec_verify_kernel<float, 8, 4>)
                         : (few ? (const void*)spec_verify_kernel<__nv_bfloat16, 16, 2>
                                : (const void*)spec_verify_kernel<__nv_bfloat16, 8, 4>);
  void* args[] = {&p};
  return nvfp4::launch_dependent(kern, dim3((unsigned)(in->batch * ranks)), dim3(kThreads), 0, stream,
                                 (unsigned)ranks, args) == cudaSuccess
             ? NVFP4_OK
             : NVFP4_ERR_CUDA;
}
