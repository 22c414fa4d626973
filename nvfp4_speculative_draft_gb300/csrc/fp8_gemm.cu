// fp8_gemm.cu -- block-scaled FP8 (W8A8) product on the 5th-generation tensor
// cores (sm_103a), one kernel from one token to prefill sizes.
//
//   C[m, n] = sum_b sa[b][m] sw[n/128][b] D_b[n, m],  D_b = sum_{i in block b} w[n, i] a[m, i]
//
// The weights are the MMA's M operand (128 rows: one scale block, so the weight
// scale is one number per K block of a tile) and TN tokens its N operand, TN from
// 16 to 256 chosen per call.  D_b is formed by four kind::f8f6f4 MMAs (K = 32 each)
// into one of a ring of TMEM buffers; the epilogue warps take every D_b out of
// TMEM and add it, times its scales, to FP32 accumulators in registers (one packed
// FMA per two elements), while the tensor core forms the next.
//   warp 0   TMA producer: per K block 128 x 128 weight codes and TN x 128
//            activation codes (128-byte swizzle; past n, m and k read as 0);
//   warp 1   allocates TMEM; one thread issues the MMAs, committing each stage to
//            its "empty" barrier and each D_b to its "full" barrier;
//   warp 2   forms the TN products sa sw of each K block in shared memory, loads
//            four K blocks ahead in registers;
//   warps 4..  epilogue: lane = weight row (TMEM lane), columns = tokens.
// Few output tiles: a cluster of S CTAs splits K, each CTA leaves its partial tile
// in shared memory and adds a share of the columns over the S partials in rank
// order (distributed shared memory), so results do not depend on timing.
// Every wait is bounded (2 s of globaltimer): one that runs out records
// NVFP4_ERR_TIMEOUT in the caller's status word and the CTA unwinds.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "tc.cuh"

namespace {

using namespace nvfp4::tc;
namespace cg = cooperative_groups;

constexpr int kRows = 128;               // weight rows of a tile = rows of a scale block
constexpr int kK = 128;                  // K block: one swizzled 128-byte row of codes
constexpr int kWBytes = kRows * kK;      // 16 KB
constexpr int kSmemRing = 196 * 1024;    // ring of stages, with room for what follows it
constexpr int kScalePrefetch = 4;        // K blocks of activation scales in flight

template <int TN>
struct Tile {
  static constexpr int kEpiWarps = TN > 128 ? 8 : 4;
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kCols = TN / (kEpiWarps / 4);  // columns of one epilogue warp
  static constexpr int kStageBytes = kWBytes + TN * kK;
  static constexpr int kStages = kSmemRing / kStageBytes < 10 ? kSmemRing / kStageBytes : 10;
  static constexpr int kBufs = TN >= 256 ? 2 : TN >= 64 ? 4 : 8;  // TMEM ring
  static constexpr int kTmemCols = TN * kBufs;
  static constexpr int kScaleBytes = kBufs * TN * 4;
  static constexpr bool kSplit = TN <= 64;  // K may be split over a cluster
  static constexpr int kBars = 2 * kStages + 3 * kBufs + 1;
  static constexpr size_t kSmemBytes =
      1024 + (size_t)kStages * kStageBytes + kScaleBytes + 8 * kBars + 16;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM");
  static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1 KB");
  static_assert(TN * 512 <= kStages * kStageBytes, "the partial tile reuses the ring");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct Params {
  const float* sa;
  int64_t lds;
  const float* sw;
  void* c;
  int64_t ldc;
  int64_t m, n;
  int kblocks, mtiles, items;
  int32_t* dev_status;
};

template <typename Out>
__device__ __forceinline__ Out cast(float x);
template <>
__device__ __forceinline__ float cast<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 cast<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// p + ld, opaque to the compiler: it would form all of a tile's addresses first, in
// registers that the accumulators need.
template <typename Out>
__device__ __forceinline__ Out* next_token(Out* p, int64_t ld) {
  asm volatile("add.s64 %0, %0, %1;" : "+l"(p) : "l"(ld * (int64_t)sizeof(Out)));
  return p;
}

template <int TN, typename Out>
__global__ void __launch_bounds__(Tile<TN>::kThreads, 1)
fp8b_gemm_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
                 const __grid_constant__ Params p) {
  using L = Tile<TN>;
  constexpr int kStages = L::kStages, kBufs = L::kBufs;
  constexpr uint32_t kIdesc = idesc_e4m3(kRows, TN);
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  unsigned char* const smem = smem_raw + (ring - raw);
  float* const scale_buf = reinterpret_cast<float*>(smem + kStages * L::kStageBytes);
  const uint32_t bars = ring + kStages * L::kStageBytes + L::kScaleBytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto tmem_full = [&](int b) { return bars + 8u * (2 * kStages + b); };
  auto tmem_empty = [&](int b) { return bars + 8u * (2 * kStages + kBufs + b); };
  auto scale_full = [&](int b) { return bars + 8u * (2 * kStages + 2 * kBufs + b); };
  const uint32_t drain_bar = bars + 8u * (L::kBars - 1);
  uint32_t* tmem_slot =
      reinterpret_cast<uint32_t*>(smem + kStages * L::kStageBytes + L::kScaleBytes + 8 * L::kBars);
  volatile uint32_t* abort = tmem_slot + 1;

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // items of this cluster: first, first + step, ... (one only where K is split)
  const int first = (int)blockIdx.x / ranks, step = (int)gridDim.x / ranks;
  const int my_items = first < p.items ? (p.items - 1 - first) / step + 1 : 0;
  const int kb0 = (int)((int64_t)p.kblocks * rank / ranks);
  const int nk = (int)((int64_t)p.kblocks * (rank + 1) / ranks) - kb0;
  const int total = my_items * nk;  // K blocks streamed through the ring

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(tmem_full(b), 1);
      mbar_init(tmem_empty(b), L::kEpiWarps);
      mbar_init(scale_full(b), 1);
    }
    mbar_init(drain_bar, 1);
    *abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(L::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int issued = 0;  // stages filled (TMA producer)

  if (warp < 4) {
  // TN = 256: the epilogue's two warpgroups take registers that the first has no
  // use for (128 x 88 + 256 x 208 = 384 x 168, what the block was launched with).
  if constexpr (L::kEpiWarps == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    if (lane == 0) {
      int g = 0;
      bool ok = true;
      for (int it = 0; it < my_items && ok; ++it) {
        const int item = first + it * step;
        const int m0 = item % p.mtiles * TN, n0 = item / p.mtiles * kRows;
        for (int kb = 0; kb < nk; ++kb, ++g) {
          const int s = g % kStages, r = g / kStages;
          if (r > 0 && !mbar_wait(empty(s), (r - 1) & 1, abort, p.dev_status)) {
            ok = false;
            break;
          }
          issued = g + 1;
          if (nvfp4::kWithhold && blockIdx.x == 0 && g == 0) continue;  // test build: never issued
          const uint32_t dst = ring + (uint32_t)(s * L::kStageBytes);
          mbar_arrive_expect_tx(full(s), L::kStageBytes);
          tma_load_2d(dst, &tmap_w, (kb0 + kb) * kK, n0, full(s));
          tma_load_2d(dst + kWBytes, &tmap_a, (kb0 + kb) * kK, m0, full(s));
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      for (int g = 0; g < total; ++g) {
        const int s = g % kStages, b = g % kBufs;
        if (g >= kBufs && !mbar_wait(tmem_empty(b), (g / kBufs - 1) & 1, abort, p.dev_status)) break;
        if (!mbar_wait(full(s), (g / kStages) & 1, abort, p.dev_status)) break;
        tc_fence_after();
        const uint32_t src = ring + (uint32_t)(s * L::kStageBytes);
        const uint64_t wd = smem_desc(src), ad = smem_desc(src + kWBytes);
        const uint32_t d = tmem + (uint32_t)(b * TN);
#pragma unroll
        for (int kk = 0; kk < kK / 32; ++kk)
          mma_f8(d, wd + 2 * kk, ad + 2 * kk, kIdesc, kk > 0 ? 1u : 0u);
        mma_commit(empty(s));
        mma_commit(tmem_full(b));
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- scales
    constexpr int kPer = TN >= 32 ? TN / 32 : 1;
    float sa[kScalePrefetch][kPer], sw[kScalePrefetch];
    int lit = 0, lkb = 0;  // load cursor
    auto load = [&](int i) {
      const int item = first + lit * step;
      const int64_t m0 = (int64_t)(item % p.mtiles) * TN;
      const int64_t kb = kb0 + lkb;
      sw[i] = __ldg(p.sw + (int64_t)(item / p.mtiles) * p.kblocks + kb);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int64_t t = m0 + 32 * j + lane;
        sa[i][j] = t < p.m ? __ldg(p.sa + kb * p.lds + t) : 0.0f;
      }
      if (++lkb == nk) {
        lkb = 0;
        ++lit;
      }
    };
#pragma unroll
    for (int i = 0; i < kScalePrefetch; ++i)
      if (i < total) load(i);
    bool ok = true;
    for (int g0 = 0; g0 < total && ok; g0 += kScalePrefetch) {
#pragma unroll
      for (int i = 0; i < kScalePrefetch; ++i) {
        const int g = g0 + i;
        if (g < total && ok) {
          const int b = g % kBufs;
          float v[kPer];
#pragma unroll
          for (int j = 0; j < kPer; ++j) v[j] = sa[i][j] * sw[i];
          if (g + kScalePrefetch < total) load(i);
          ok = g < kBufs || mbar_wait(tmem_empty(b), (g / kBufs - 1) & 1, abort, p.dev_status);
          if (ok) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
              if (TN >= 32 || lane < TN) scale_buf[b * TN + 32 * j + lane] = v[j];
            __syncwarp();
            if (lane == 0) mbar_arrive(scale_full(b));
          }
        }
      }
    }
  }
  } else {
    if constexpr (L::kEpiWarps == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // -------------------------------------------------------------- epilogue
    constexpr int kChunk = L::kCols < 32 || L::kCols > 64 ? 16 : 32;
    constexpr int kChunks = L::kCols / kChunk;
    const int q = warp & 3, c0 = (warp - 4) / 4 * L::kCols;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)c0;
    int g = 0;
    bool ok = true;
    for (int it = 0; it < my_items && ok; ++it) {
      uint64_t acc[L::kCols / 2];  // FP32 pairs of neighbouring tokens
#pragma unroll
      for (int i = 0; i < L::kCols / 2; ++i) acc[i] = 0ull;
#pragma unroll 1
      for (int kb = 0; kb < nk; ++kb, ++g) {
        const int b = g % kBufs;
        const uint32_t parity = (g / kBufs) & 1;
        ok = mbar_wait(tmem_full(b), parity, abort, p.dev_status) &&
             mbar_wait(scale_full(b), parity, abort, p.dev_status);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(scale_buf + b * TN + c0);
        uint32_t v[2][kChunk];
        tmem_issue(tq + (uint32_t)(b * TN), v[0]);
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
          tmem_wait(v[ch & 1]);
          if (ch + 1 < kChunks) {
            tmem_issue(tq + (uint32_t)(b * TN + (ch + 1) * kChunk), v[(ch + 1) & 1]);
          }
#pragma unroll
          for (int i = 0; i < kChunk / 4; ++i) {
            const ulonglong2 s2 = sc[ch * (kChunk / 4) + i];
            const uint32_t* d = &v[ch & 1][4 * i];
            uint64_t* a = &acc[ch * (kChunk / 2) + 2 * i];
            fma_f32x2(a[0], pack2(d[0], d[1]), s2.x);
            fma_f32x2(a[1], pack2(d[2], d[3]), s2.y);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tmem_empty(b));
      }
      if (!ok) break;
      // lane = weight row: a warp's store covers 32 neighbouring outputs of a token
      const int item = first + it * step;
      if (L::kSplit && ranks > 1) {
        // the ring's memory: every load and MMA has left it (all D_b were waited for)
        float* part = reinterpret_cast<float*>(smem) + c0 * kRows + 32 * q + lane;
#pragma unroll
        for (int i = 0; i < L::kCols / 2; ++i)
          unpack2(acc[i], part[2 * i * kRows], part[(2 * i + 1) * kRows]);
      } else {
        const int64_t t0 = (int64_t)(item % p.mtiles) * TN + c0;
        const int64_t nn = (int64_t)(item / p.mtiles) * kRows + 32 * q + lane;
        const int left = nn < p.n ? (int)(p.m - t0 < L::kCols ? p.m - t0 : L::kCols) : 0;
        Out* dst = reinterpret_cast<Out*>(p.c) + t0 * p.ldc + nn;
#pragma unroll
        for (int i = 0; i < L::kCols / 2; ++i) {
          float x0, x1;
          unpack2(acc[i], x0, x1);
          if (2 * i < left) *dst = cast<Out>(x0);
          dst = next_token(dst, p.ldc);
          if (2 * i + 1 < left) *dst = cast<Out>(x1);
          dst = next_token(dst, p.ldc);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    // A wait ran out: the loads and MMAs already issued may still be in flight.
    // Wait for them (bounded) before TMEM is freed and shared memory released.
    if (warp == 0 && lane == 0)
      for (int g = issued > kStages ? issued - kStages : 0; g < issued; ++g)
        mbar_drain(full(g % kStages), (uint32_t)(g / kStages) & 1u, p.dev_status);
    if (warp == 1 && lane == 0) {
      mma_commit(drain_bar);
      mbar_drain(drain_bar, 0u, p.dev_status);
    }
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kTmemCols)
                 : "memory");
  }
  if (L::kSplit && ranks > 1) {
    // partial tiles [token][weight row]: each CTA adds and stores every ranks-th token
    cluster.sync();
    float* partial = reinterpret_cast<float*>(smem);
    const int64_t m0 = (int64_t)(first % p.mtiles) * TN;
    const int64_t n0 = (int64_t)(first / p.mtiles) * kRows;
    for (int i = threadIdx.x; i < TN / ranks * kRows; i += L::kThreads) {
      const int c = i / kRows * ranks + rank, row = i % kRows;
      if (m0 + c < p.m && n0 + row < p.n) {
        float x = 0.0f;
        for (int o = 0; o < ranks; ++o) x += cluster.map_shared_rank(partial, o)[c * kRows + row];
        reinterpret_cast<Out*>(p.c)[(m0 + c) * p.ldc + n0 + row] = cast<Out>(x);
      }
    }
    cluster.sync();  // no CTA leaves while another reads its partial tile
  }
}

template <int TN>
int launch(const CUtensorMap& tw, const CUtensorMap& ta, Params p, int split, bool f32,
           cudaStream_t stream) {
  const void* kern = f32 ? (const void*)fp8b_gemm_kernel<TN, float>
                         : (const void*)fp8b_gemm_kernel<TN, __nv_bfloat16>;
  if (nvfp4::occupancy(kern, Tile<TN>::kThreads, Tile<TN>::kSmemBytes) < 1) return NVFP4_ERR_CUDA;
  const int sms = nvfp4::sm_count();
  const int64_t grid = split > 1 ? (int64_t)p.items * split : (p.items < sms ? p.items : sms);
  if (grid > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(Tile<TN>::kThreads);
  cfg.dynamicSmemBytes = Tile<TN>::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<CUtensorMap*>(&tw), const_cast<CUtensorMap*>(&ta), &p};
  return cudaLaunchKernelExC(&cfg, kern, args) == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace

int launch_fp8b_gemm(const fp8b_act* a, const fp8b_weight* w, void* c, int c_dtype, int64_t ldc,
                     int32_t* dev_status, cudaStream_t stream) {
  const int64_t m = a->m, n = w->n, k = w->k;
  const int64_t ntiles = nvfp4::cdiv(n, kRows), kblocks = nvfp4::cdiv(k, kK);
  // Token tile: the smallest that holds all tokens, 256 beyond that.
  const int tn = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : m <= 128 ? 128 : 256;
  const int64_t mtiles = nvfp4::cdiv(m, tn), items = ntiles * mtiles;
  if (items > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  // K is split while that still finds idle SMs and leaves four blocks to each CTA.
  int split = 1;
  while (tn <= 64 && split < 8 && items * split * 2 <= nvfp4::sm_count() && kblocks / (split * 2) >= 4)
    split *= 2;
  CUtensorMap tw, ta;
  const cuuint32_t estr[2] = {1, 1};
  {
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)n};
    const cuuint64_t strides[1] = {(cuuint64_t)k};
    const cuuint32_t box[2] = {kK, kRows};
    if (!nvfp4::encode_tiled(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(w->codes), dims,
                             strides, box, estr, CU_TENSOR_MAP_SWIZZLE_128B))
      return NVFP4_ERR_CUDA;
  }
  {
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)m};
    const cuuint64_t strides[1] = {(cuuint64_t)a->ld};
    const cuuint32_t box[2] = {kK, (cuuint32_t)tn};
    if (!nvfp4::encode_tiled(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a->codes, dims, strides, box, estr,
                             CU_TENSOR_MAP_SWIZZLE_128B))
      return NVFP4_ERR_CUDA;
  }
  Params p;
  p.sa = a->scales;
  p.lds = a->ld_scales;
  p.sw = w->scales;
  p.c = c;
  p.ldc = ldc;
  p.m = m;
  p.n = n;
  p.kblocks = (int)kblocks;
  p.mtiles = (int)mtiles;
  p.items = (int)items;
  p.dev_status = dev_status;
  const bool f32 = c_dtype == NVFP4_DTYPE_F32;
  switch (tn) {
    case 16: return launch<16>(tw, ta, p, split, f32, stream);
    case 32: return launch<32>(tw, ta, p, split, f32, stream);
    case 64: return launch<64>(tw, ta, p, split, f32, stream);
    case 128: return launch<128>(tw, ta, p, split, f32, stream);
    default: return launch<256>(tw, ta, p, split, f32, stream);
  }
}
