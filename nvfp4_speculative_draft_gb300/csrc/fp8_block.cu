// fp8_block.cu -- block-scaled FP8 (E4M3): the load-time weight quantiser (one
// FP32 scale per 128 x 128 block) and the activation path, residual addition +
// RMSNorm + quantisation in one pass (one scale per row and 128 columns).
//
//     s = fl32(amax / 448),   c = E4M3_RNE_SATFINITE(fl32(x / s))
//
// Both are bound by HBM: every input element is read once and held in registers
// between the maximum and its codes, every output written once.  Codes come from the
// quotient's one correction step (e4m3.cuh).

#include "e4m3.cuh"

namespace {

using namespace nvfp4::e4m3;

constexpr int kBlock = 128;  // rows and columns of a weight block, columns of a row group

// ------------------------------------------------------------ weights
//
// One CTA per 128 x 128 block: thread t holds the eight 16-byte vectors of rows
// t/16 + 16 i, columns 8 (t % 16).., so a warp's load covers two rows x 256 bytes and
// a CTA has 32 KB in flight.  Bound by HBM (3 bytes an element) once the quotients
// cost few instructions: 151936 x 5120 takes 362 us, 6.45 TB/s, 0.95 of the measured
// copy; with a rounding test and a division in doubt it took 432, with a second
// correction step of the quotient 404.  Measured and not kept: a persistent CTA with
// a TMA ring of blocks (390 us even without the quotients), 512 threads a block (377),
// four CTAs an SM (392).
constexpr int kQThreads = 256;
constexpr int kQVecs = kBlock * kBlock / 8 / kQThreads;  // vectors of a thread

__global__ void __launch_bounds__(kQThreads, 3)
fp8b_quantize_kernel(const uint4* __restrict__ w, int64_t n, int64_t k, int64_t ldv,
                     uint2* __restrict__ codes, float* __restrict__ scales, int64_t kblocks,
                     int32_t* dev_status) {
  __shared__ uint32_t red[kQThreads / 32];
  const int64_t bn = blockIdx.x / kblocks, bk = blockIdx.x % kblocks;
  const int64_t col = bk * (kBlock / 8) + (threadIdx.x & 15);
  const int64_t row0 = bn * kBlock + (threadIdx.x >> 4);
  const bool colok = col < k / 8;
  uint4 v[kQVecs];
  uint32_t m2 = 0u;
  nvfp4::wait_for_previous_kernel();
#pragma unroll
  for (int i = 0; i < kQVecs; ++i) {
    const int64_t r = row0 + (kQThreads / 16) * i;
    v[i] = colok && r < n ? ld_u4(w + r * ldv + col) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kQVecs; ++i) m2 = __vmaxu2(m2, mag_max8(v[i]));
  uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = 0u;
#pragma unroll
  for (int i = 0; i < kQThreads / 32; ++i) m = max(m, red[i]);
  const Scale sc = scale_of(__uint_as_float(m << 16));
  if (threadIdx.x == 0) {
    scales[blockIdx.x] = sc.s;
    if (m >= 0x7F80u) nvfp4::report(dev_status, NVFP4_ERR_NONFINITE);
  }
#pragma unroll
  for (int i = 0; i < kQVecs; ++i) {
    const int64_t r = row0 + (kQThreads / 16) * i;
    if (colok && r < n) codes[r * (k / 8) + col] = codes_of(v[i], sc);
  }
}

// -------------------------------------------------------- activations
//
// T threads per row (a multiple of 32), thread t holding the 8-element vectors
// t, t + T, ...: sixteen neighbouring threads hold one 128-column group, whose
// maximum four shuffles give.  blockDim = (T, rows per CTA).  Without gamma the
// groups are independent, and a row is split over gridDim.y CTAs.
//
// Bound by HBM (7 bytes an element with the residual) while it stays below about 20
// instructions an element, hence the packed FP32 and BF16 arithmetic; 32 registers
// keep 2048 threads on an SM.  8192 x 5120 with residual and gamma takes 44.6 to
// 45.8 us, 6.44 TB/s, 0.95 of the measured copy at least (72.5 us with scalar arithmetic, divisions and
// one vector a thread; a CTA that walks over rows with the next row's loads in flight
// is slower, 55 us).  One row of 5120: 2.4 us, mostly the launch.
struct NormParams {
  const uint4* x;
  const uint4* residual;
  uint4* residual_out;
  const uint4* gamma;
  uint2* codes;
  float* scales;
  int64_t ldx, ldr, ldo, ldc;  // in vectors of 8
  int64_t lds, m;
  int nvec;  // k / 8
  float eps, inv_k;
  int32_t* dev_status;
};

// bf16(fl32(a + b)), each half: fl32(a + b) keeps every bit that decides the
// rounding to BF16 (a and b have 8 bits each), so one rounding gives the same.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// max(m, |a|, |b|), NaN if any is
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

constexpr int kNormMaxThreads = 1024;

// Squares below 2^-126 lose bits and below 2^-150 everything: at most 2^-150 each, so
// nothing of a mean (with eps) of 2^-100 or more.  A row below it, which needs an eps
// below it, is summed again times 2^96: its largest value is then below 2^46 sqrt(k) and
// BF16's smallest 2^-37, so squares, sums and products are normal, and no scaling rounds.
// y = h / sqrt(mean + eps) is the same for both factors.
constexpr float kTinyVar = 0x1p-100f;
constexpr uint32_t kTinyScale = 0x6F806F80u;  // 2^96, twice

// 32 registers a thread; 64 where each holds four vectors.  TINY: eps < kTinyVar, so that
// a row may be tiny (8192 x 5120 with that in it, 45.1 us; without, 44.6).
template <int V, int MAXT, bool TINY>
__global__ void __launch_bounds__(MAXT, (V == 4 ? 1024 : 2048) / MAXT)
fp8b_rmsnorm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[1 + TINY][kNormMaxThreads / 32];
  const int T = blockDim.x, t = threadIdx.x, lane = t & 31;
  const int c0 = blockIdx.y * V * T + t;  // the thread's first vector
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.m;
  uint4 h[V];
  nvfp4::wait_for_previous_kernel();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * T;
    // not the read-only path: residual_out may be x or residual
    h[i] = live && c < p.nvec ? p.x[row * p.ldx + c] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.residual != nullptr) {
    uint4 r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + i * T;
      r[i] = live && c < p.nvec ? p.residual[row * p.ldr + c] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      h[i] = make_uint4(add_bf16x2(h[i].x, r[i].x), add_bf16x2(h[i].y, r[i].y),
                        add_bf16x2(h[i].z, r[i].z), add_bf16x2(h[i].w, r[i].w));
  }
  if (p.residual_out != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + i * T;
      if (live && c < p.nvec) p.residual_out[row * p.ldo + c] = h[i];
    }
  }
  float rstd = 1.0f;
  bool bad = false;
  if (p.gamma != nullptr) {
    const int warps = T / 32;
    auto warp_squares = [&]() {
      uint64_t ss2 = 0ull;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint64_t f[4];
        pairs_of(h[i], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) ss2 = fma_f32x2(f[j], f[j], ss2);
      }
      float ss, s1;
      unpack_f32x2(ss2, ss, s1);
      ss += s1;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
      return ss;
    };
    auto total = [&](const float* mine) {
      float ss = 0.0f;
      for (int w = 0; w < warps; ++w) ss += mine[w];  // the same order in every thread
      return ss;
    };
    const float ws = warp_squares();
    float* mine = part[0] + threadIdx.y * warps;
    if (lane == 0) mine[t >> 5] = ws;
    bool any_tiny = false;
    if constexpr (TINY)  // (a warp's squares are no more than its row's: all of a tiny row's warps say so)
      any_tiny = __syncthreads_or(fmaf(ws, p.inv_k, p.eps) < kTinyVar);
    else
      __syncthreads();
    const float ss = total(mine);
    bad = !(ss < __int_as_float(0x7F800000));
    float var = fmaf(ss, p.inv_k, p.eps);
    if (TINY && any_tiny) {
      const bool tiny = var < kTinyVar;  // the same in all threads of a row
      if (tiny) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          h[i] = make_uint4(mul_bf16x2(h[i].x, kTinyScale), mul_bf16x2(h[i].y, kTinyScale),
                            mul_bf16x2(h[i].z, kTinyScale), mul_bf16x2(h[i].w, kTinyScale));
      }
      const float scaled = warp_squares();
      mine = part[TINY] + threadIdx.y * warps;
      if (lane == 0) mine[t >> 5] = scaled;
      __syncthreads();
      if (tiny) var = fmaf(total(mine), p.inv_k, p.eps * 0x1p96f * 0x1p96f);
    }
    rstd = var > 0.0f ? rsqrtf(var) : 0.0f;  // an all-zero row with eps 0
  }
  const uint64_t rstd2 = f32x2_splat(rstd);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * T;
    const bool ok = live && c < p.nvec;
    uint64_t y[4];
    pairs_of(h[i], y);
    if (p.gamma != nullptr) {
      uint64_t g[4];
      pairs_of(ok ? ld_u4(p.gamma + c) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mul_f32x2(mul_f32x2(y[j], rstd2), g[j]);
    }
    float mag = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      unpack_f32x2(y[j], a, b);
      mag = max_abs(mag, a, b);
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) mag = max_abs(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, d), 0.0f);
    bad = bad || !(mag < __int_as_float(0x7F800000));
    const Scale sc = scale_of(mag);
    if (ok) {
      p.codes[row * p.ldc + c] = codes_of(y, sc);
      if ((lane & 15) == 0) p.scales[(int64_t)(c >> 4) * p.lds + row] = sc.s;
    }
  }
  if (live && bad) nvfp4::report(p.dev_status, NVFP4_ERR_NONFINITE);
}

template <int V, int MAXT, bool TINY>
int launch_norm_as(const NormParams& p, int T, cudaStream_t stream) {
  const int rows = T >= 256 ? 1 : 256 / T;  // of a CTA
  const int64_t grid = nvfp4::cdiv(p.m, rows);
  const unsigned cols = p.gamma != nullptr ? 1u : (unsigned)nvfp4::cdiv(p.nvec, V * T);
  void* args[] = {const_cast<NormParams*>(&p)};
  return nvfp4::launch_dependent((const void*)fp8b_rmsnorm_kernel<V, MAXT, TINY>, dim3((unsigned)grid, cols), dim3(T, rows), 0,
                                 stream, 1, args) == cudaSuccess
             ? NVFP4_OK
             : NVFP4_ERR_CUDA;
}
template <int V, int MAXT>
int launch_norm(const NormParams& p, int T, cudaStream_t stream) {
  return p.gamma != nullptr && p.eps < kTinyVar ? launch_norm_as<V, MAXT, true>(p, T, stream)
                                                : launch_norm_as<V, MAXT, false>(p, T, stream);
}

}  // namespace

int launch_fp8b_quantize(const void* w, int64_t n, int64_t k, int64_t ld, uint8_t* codes,
                         float* scales, int32_t* dev_status, cudaStream_t stream) {
  const int64_t kb = nvfp4::cdiv(k, kBlock), blocks = nvfp4::cdiv(n, kBlock) * kb;
  if (blocks > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  const uint4* wv = reinterpret_cast<const uint4*>(w);
  uint2* cv = reinterpret_cast<uint2*>(codes);
  int64_t ldv = ld / 8, kbv = kb;
  void* args[] = {&wv, &n, &k, &ldv, &cv, &scales, &kbv, &dev_status};
  return nvfp4::launch_dependent((const void*)fp8b_quantize_kernel, dim3((unsigned)blocks), dim3(kQThreads), 0, stream, 1,
                                 args) == cudaSuccess
             ? NVFP4_OK
             : NVFP4_ERR_CUDA;
}

int launch_fp8b_rmsnorm(const fp8b_norm_input* in, const fp8b_act* out, int32_t* dev_status,
                        cudaStream_t stream) {
  NormParams p;
  p.x = reinterpret_cast<const uint4*>(in->x);
  p.residual = reinterpret_cast<const uint4*>(in->residual);
  p.residual_out = reinterpret_cast<uint4*>(in->residual_out);
  p.gamma = reinterpret_cast<const uint4*>(in->gamma);
  p.codes = reinterpret_cast<uint2*>(out->codes);
  p.scales = out->scales;
  p.ldx = in->ld_x / 8;
  p.ldr = in->ld_residual / 8;
  p.ldo = in->ld_residual_out / 8;
  p.ldc = out->ld / 8;
  p.lds = out->ld_scales;
  p.m = out->m;
  p.nvec = (int)(out->k / 8);
  p.eps = in->eps;
  p.inv_k = 1.0f / (float)out->k;
  p.dev_status = dev_status;
  const int warps = (int)nvfp4::cdiv(p.nvec, 32);  // one vector per thread
  if (p.gamma == nullptr) return launch_norm<1, 256>(p, warps < 8 ? warps * 32 : 256, stream);
  // A row on as many threads as it has vectors while rows are few (2.4 us against 2.65
  // for one row of 5120); two vectors per thread once there are rows for every SM's
  // 2048 threads (8192 rows: 45.4 us against 57.9); four where 1024 threads would not
  // reach otherwise.
  const bool many = p.m > 2 * nvfp4::sm_count();
  const int v = p.nvec > 2048 ? 4 : p.nvec > 1024 || (many && p.nvec > 256) ? 2 : 1;
  const int T = (int)nvfp4::cdiv(warps, v) * 32;
  if (v == 4) return launch_norm<4, 1024>(p, T, stream);
  if (v == 2) return launch_norm<2, 1024>(p, T, stream);
  // (compiled for 256 threads: 100000 x 512 58.4 us against 59.9)
  return T <= 256 ? launch_norm<1, 256>(p, T, stream) : launch_norm<1, 1024>(p, T, stream);
}
