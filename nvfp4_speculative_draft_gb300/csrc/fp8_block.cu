// fp8_block.cu -- block-scaled FP8 (E4M3): the load-time weight quantiser (one
// FP32 scale per 128 x 128 block) and the activation path, residual addition +
// RMSNorm + quantisation in one pass (one scale per row and 128 columns).
//
//     s = fl32(amax / 448),   c = E4M3_RNE_SATFINITE(fl32(x / s))
//
// Both are bound by HBM: every input element is read once and held in registers
// between the maximum and its codes, every output written once.  The correctly
// rounded quotient's code comes from the rounding test of e4m3.cuh.

#include "e4m3.cuh"

namespace {

using namespace nvfp4::e4m3;

constexpr int kBlock = 128;  // rows and columns of a weight block, columns of a row group

// ------------------------------------------------------------ weights
//
// One CTA per 128 x 128 block: thread t holds the eight 16-byte vectors of rows
// t/16 + 16 i, columns 8 (t % 16).., so a warp's load covers two rows x 256
// bytes and a CTA has 32 KB in flight.
constexpr int kQThreads = 256;

__global__ void __launch_bounds__(kQThreads)
fp8b_quantize_kernel(const uint4* __restrict__ w, int64_t n, int64_t k, int64_t ldv,
                     uint2* __restrict__ codes, float* __restrict__ scales, int64_t kblocks,
                     int32_t* dev_status) {
  __shared__ uint32_t red[kQThreads / 32];
  const int64_t bn = blockIdx.x / kblocks, bk = blockIdx.x % kblocks;
  const int64_t col = bk * (kBlock / 8) + (threadIdx.x & 15);
  const int64_t row0 = bn * kBlock + (threadIdx.x >> 4);
  const bool colok = col < k / 8;
  uint4 v[8];
  uint32_t m2 = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = row0 + 16 * i;
    v[i] = colok && r < n ? ld_u4(w + r * ldv + col) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, mag_max8(v[i]));
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
  for (int i = 0; i < 8; ++i) {
    const int64_t r = row0 + 16 * i;
    if (colok && r < n) codes[r * (k / 8) + col] = codes_of(v[i], sc.s, sc.fast, sc.rlo, sc.rhi);
  }
}

// -------------------------------------------------------- activations
//
// T threads per row (a multiple of 32), thread t holding the 8-element vectors
// t, t + T, ...: sixteen neighbouring threads hold one 128-column group, whose
// maximum four shuffles give.  blockDim = (T, rows per CTA).
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
  float eps;
  int32_t* dev_status;
};

__device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(u[j] << 16);
    f[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {  // bf16(fl32(a + b)), each half
  const __nv_bfloat162 r =
      __floats2bfloat162_rn(__uint_as_float(a << 16) + __uint_as_float(b << 16),
                            __uint_as_float(a & 0xFFFF0000u) + __uint_as_float(b & 0xFFFF0000u));
  return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr int kNormMaxThreads = 1024;

template <int V>
__global__ void __launch_bounds__(kNormMaxThreads)
fp8b_rmsnorm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[kNormMaxThreads / 32];
  const int T = blockDim.x, t = threadIdx.x, lane = t & 31;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.m;
  uint4 h[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    // not the read-only path: residual_out may be x or residual
    h[i] = live && c < p.nvec ? p.x[row * p.ldx + c] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.residual != nullptr) {
    uint4 r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
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
      const int c = t + i * T;
      if (live && c < p.nvec) p.residual_out[row * p.ldo + c] = h[i];
    }
  }
  float rstd = 1.0f;
  bool bad = false;
  if (p.gamma != nullptr) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      unpack(h[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    const int warps = T / 32;
    float* mine = part + threadIdx.y * warps;
    if (lane == 0) mine[t >> 5] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int w = 0; w < warps; ++w) ss += mine[w];  // the same order in every thread
    bad = !(ss < __int_as_float(0x7F800000));
    const float var = __fdiv_rn(ss, (float)(p.nvec * 8)) + p.eps;
    rstd = var > 0.0f ? __fdiv_rn(1.0f, __fsqrt_rn(var)) : 0.0f;  // an all-zero row with eps 0
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    const bool ok = live && c < p.nvec;
    float y[8];
    unpack(h[i], y);
    if (p.gamma != nullptr) {
      float g[8];
      unpack(ok ? ld_u4(p.gamma + c) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = (y[j] * rstd) * g[j];
    }
    uint32_t mag = 0u;  // magnitudes as bit patterns: NaN and infinity are the largest
#pragma unroll
    for (int j = 0; j < 8; ++j) mag = max(mag, __float_as_uint(y[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, d));
    bad = bad || mag >= 0x7F800000u;
    const Scale sc = scale_of(__uint_as_float(mag));
    if (ok) {
      p.codes[row * p.ldc + c] = codes_of(y, sc.s, sc.fast, sc.rlo, sc.rhi);
      if ((lane & 15) == 0) p.scales[(int64_t)(c >> 4) * p.lds + row] = sc.s;
    }
  }
  if (live && bad) nvfp4::report(p.dev_status, NVFP4_ERR_NONFINITE);
}

}  // namespace

int launch_fp8b_quantize(const void* w, int64_t n, int64_t k, int64_t ld, uint8_t* codes,
                         float* scales, int32_t* dev_status, cudaStream_t stream) {
  const int64_t kb = nvfp4::cdiv(k, kBlock), blocks = nvfp4::cdiv(n, kBlock) * kb;
  if (blocks > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  fp8b_quantize_kernel<<<(unsigned)blocks, kQThreads, 0, stream>>>(
      reinterpret_cast<const uint4*>(w), n, k, ld / 8, reinterpret_cast<uint2*>(codes), scales, kb,
      dev_status);
  return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
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
  p.dev_status = dev_status;
  const int v = p.nvec <= 1024 ? 1 : p.nvec <= 2048 ? 2 : 4;
  const int T = (int)nvfp4::cdiv(nvfp4::cdiv(p.nvec, v), 32) * 32;
  const int rows = T >= 256 ? 1 : 256 / T;
  const int64_t grid = nvfp4::cdiv(p.m, rows);
  if (grid > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  const dim3 block(T, rows);
  if (v == 1)
    fp8b_rmsnorm_kernel<1><<<(unsigned)grid, block, 0, stream>>>(p);
  else if (v == 2)
    fp8b_rmsnorm_kernel<2><<<(unsigned)grid, block, 0, stream>>>(p);
  else
    fp8b_rmsnorm_kernel<4><<<(unsigned)grid, block, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
