// fp8_gemm.cu -- block-scaled FP8 (W8A8) product on the 5th-generation tensor
// cores (sm_103a), from one token to prefill sizes.
//
//   C[m, n] = sum_b sa[b][m] sw[n/128][b] D_b[m, n],  D_b = sum_{i in block b} a[m, i] w[n, i]
//
// D_b is formed by four kind::f8f6f4 MMAs (K = 32 each) into one of a ring of TMEM
// buffers; the epilogue warps take every D_b out of TMEM and add it, times its
// scales, to FP32 accumulators in registers (one packed FMA per two elements) while
// the tensor core forms the next.  Two forms of one kernel:
//   FEW   the 128 rows of the MMA are weights (one scale block), its N columns
//         tokens, N = 16, 32 or 64: no tensor work is spent on absent tokens, and the
//         weight stream, which bounds these sizes, is the same for all;
//   MANY  the 128 rows are tokens, the N = 128 or 256 columns weights: a thread's
//         accumulators share one token and one weight block, so one scale per K block.
//   warp 0   TMA producer: per K block 128 rows of one operand and N of the other,
//            128 codes each (128-byte swizzle; past n, m and k read as 0);
//   warp 1   allocates TMEM and issues the MMAs, committing each stage to its "empty"
//            barrier and each D_b to its "full" barrier (N = 64, 128: warps 1 and 3, K
//            blocks in turn);
//   warp 2   forms the products sa sw of each K block in shared memory, loads four K
//            blocks ahead in registers;
//   warps 4..  epilogue, a TMEM lane per thread and up to 128 columns.
// Few output tiles: a cluster of S CTAs splits K, each CTA leaves its partial tile in
// shared memory and adds and stores a share of it over the S partials in rank order
// (distributed shared memory), so results do not depend on timing.
// Every wait is bounded (2 s of globaltimer): one that runs out records
// NVFP4_ERR_TIMEOUT in the caller's status word and the CTA unwinds.
//
// What bounds it, and what it measured (BF16 out unless stated):
//   few tokens     HBM, the weight stream: 10 x 151936 x 5120 (FP32 out) 114 to 117 us, 6.7 to 6.85
//                  TB/s, 0.99 to 1.0 of the measured copy; 1 x 5120 x 10240 11.6 us, 4.5 TB/s (0.67), of which about
//                  5 us are launch, pipeline fill and the exchange of partial tiles.
//   77 rows        18.2 us for 77 x 17408 x 5120 (0.74 of HBM): 136 tiles on 152 SMs, each K block's
//                  32 KB from L2.
//   prefill        2048 x 17408 x 5120 133.7 us in a short graph of calls, 2730 TFLOP/s, 0.71 of
//                  twice the measured BF16 rate; 148 to 155 us in long runs of calls, under the
//                  power limit (0.61 to 0.64).  FP32 out 150 us.  A K block's MMAs take 512 cycles,
//                  the tile's period is 750.  Above the floor of 95 us are, by trials of the same
//                  kernel: about 13 us of the last wave (1088 tiles on 152 SMs are 7.16 waves, run
//                  as eight; SMs are active 87 % of the time), about 16 us of operand loads
//                  (without epilogue 122 us, without loads either 106), and 12 us of the epilogue,
//                  which takes every D_b out of TMEM for its scales, with TMEM full at two buffers
//                  of 256 columns.  No unit is busy throughout (tensor pipe 66 %, shared memory's
//                  data pipe 57 % while SMs are active).  Measured and not kept: CTA pairs (145 us,
//                  the handovers cross SMs), weights as MMA rows at 256 tokens (182 us, a scale
//                  per column from shared memory), two MMA warps (137 us).
//   129 to 1024 rows against narrow outputs   tiles do not fill the SMs: 256 x 5120 x 5120 14.3
//                  to 14.8 us, 512 x 5120 x 5120 18.8 to 19.7 us (floors 4.4 and 7.0): 80 tiles on
//                  152 SMs, unsplit.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "tc.cuh"

namespace {

using namespace nvfp4::tc;
namespace cg = cooperative_groups;

constexpr int kM = 128;                // MMA rows
constexpr int kK = 128;                // K block: one swizzled 128-byte row of codes
constexpr int kRing = 196 * 1024;      // bytes of the rings of an SM's CTAs, at most
constexpr int kScalePrefetch = 4;      // K blocks of scales in flight

template <bool FEW, int N>
struct Tile {
  static constexpr int kEpiWarps = N >= 64 ? 8 : 4;
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kCols = N / (kEpiWarps / 4);  // columns of one epilogue warp
  static constexpr int kTokens = FEW ? N : kM, kOut = FEW ? kM : N;  // of an output tile
  static constexpr int kABytes = kM * kK, kStageBytes = kABytes + N * kK;
  // Two CTAs an SM where registers allow: a K block of few tokens takes less time than
  // its handovers between producer, MMAs and epilogue, and two such chains overlap.
  static constexpr int kCtas = N <= 32 ? 2 : 1;
  // Issuing a K block's MMAs takes a warp about 500 cycles: where that is what a tile
  // waits for, two warps take K blocks in turn (128 x 5120 x 5120: 17.0 -> 14.6 us; with
  // two CTAs an SM, 11.5 -> 12.7 for one token, or N = 256, 132 -> 137 for prefill, not).
  static constexpr int kIssuers = N == 64 || N == 128 ? 2 : 1;
  static constexpr int kStages = kRing / kCtas / kStageBytes / kIssuers * kIssuers;
  static constexpr int kBufs = N >= 256 ? 2 : N >= 64 ? 4 : 8;  // TMEM ring
  static constexpr int kTmemCols = N * kBufs;
  static constexpr bool kSplit = N <= 128;  // K may be split over a cluster
  static constexpr int kWBlocks = FEW || N < 128 ? 1 : N / 128;  // weight blocks of an output tile
  static constexpr int kScales = kTokens * kWBlocks, kScaleBytes = kBufs * kScales * 4;
  static constexpr int kBars = 2 * kStages + 3 * kBufs + 1;
  static constexpr int kStoreBytes = FEW ? 0 : kEpiWarps * 2048;
  static constexpr size_t kSmemBytes =
      1024 + (size_t)kStages * kStageBytes + kScaleBytes + kStoreBytes + 8 * kBars + 16;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM");
  static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1 KB");
  // With rings that are multiples of the issuers a stage and a buffer always serve the same
  // warp, which so waits for every phase of their barriers.  (A warp that skipped one would
  // take the parity of the phase before for the one it waits for.)
  static_assert(kStages % kIssuers == 0 && kBufs % kIssuers == 0, "rings");
  static_assert(!kSplit || kM * N * 4 <= kStages * kStageBytes, "the partial tile reuses the ring");
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
  static_assert(kCtas * kTmemCols <= 512, "TMEM");
};

struct Params {
  const float* sa;
  int64_t lds;
  const float* sw;
  void* c;
  int64_t ldc;
  int64_t m, n;
  int kblocks, wblocks, mtiles, items;
  bool vector_store;  // C is 16-byte aligned, and so are its rows
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

// FEW: a thread's accumulators are one output column of `left` tokens; a warp's store
// covers 32 neighbouring outputs of a token.
template <int N, typename Out>
__device__ __forceinline__ void store_tokens(const uint64_t (&acc)[N / 2], Out* dst, int64_t ldc, int left) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float x0, x1;
    unpack2(acc[i], x0, x1);
    if (2 * i < left) *dst = cast<Out>(x0);
    dst = next_token(dst, ldc);
    if (2 * i + 1 < left) *dst = cast<Out>(x1);
    dst = next_token(dst, ldc);
  }
}

// MANY: a thread's accumulators are C consecutive outputs of one token (a lane's row).
// 64 bytes of each row at a time go through 2 KB of the warp's own shared memory, so
// that a store covers eight rows x 64 contiguous bytes rather than 32 rows x 16.  The
// 16-byte pieces of row r lie at piece ^ (r / 2 % 4): neither side meets bank conflicts.
// Rows that are not 16-byte aligned are stored by elements, neighbouring lanes
// neighbouring outputs.
template <int C, typename Out>
__device__ __forceinline__ void store_row(const uint64_t (&acc)[C / 2], const Params& p, int64_t row0, int64_t n0,
                                          int lane, uint4* stage) {
  constexpr int kPiece = 16 / sizeof(Out);  // outputs of a piece
#pragma unroll
  for (int g = 0; g < C / (4 * kPiece); ++g) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = (g * 4 + i) * kPiece / 2;  // first pair of the piece
        if constexpr (sizeof(Out) == 4) {
          float x[2];
          unpack2(acc[at + e / 2], x[0], x[1]);
          w[e] = __float_as_uint(x[e & 1]);
        } else {
          float x0, x1;
          unpack2(acc[at + e], x0, x1);
          const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
          w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      stage[lane * 4 + (i ^ (lane / 2 % 4))] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    const int64_t g0 = n0 + g * 4 * kPiece;
    if (p.vector_store && g0 + 4 * kPiece <= p.n) {
      const int64_t col = g0 + lane % 4 * kPiece;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + lane / 4;
        const uint4 v = stage[r * 4 + (lane % 4 ^ (r / 2 % 4))];
        const int64_t row = row0 + r;
        if (row < p.m) *reinterpret_cast<uint4*>(reinterpret_cast<Out*>(p.c) + row * p.ldc + col) = v;
      }
    } else {
      constexpr int kRow = 4 * kPiece;  // outputs of a row: 16 or 32 lanes
      const int e = lane % kRow;
#pragma unroll 4
      for (int r0 = 0; r0 < 32; r0 += 32 / kRow) {
        const int r = r0 + lane / kRow;
        const Out* src = reinterpret_cast<const Out*>(stage + r * 4 + (e / kPiece ^ (r / 2 % 4))) + e % kPiece;
        const int64_t row = row0 + r, col = g0 + e;
        if (row < p.m && col < p.n) reinterpret_cast<Out*>(p.c)[row * p.ldc + col] = *src;
      }
    }
    __syncwarp();
  }
}

template <bool FEW, int N, typename Out>
__global__ void __launch_bounds__(Tile<FEW, N>::kThreads, Tile<FEW, N>::kCtas)
fp8b_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                 const __grid_constant__ Params p) {
  using L = Tile<FEW, N>;
  constexpr int kStages = L::kStages, kBufs = L::kBufs, kCols = L::kCols;
  constexpr uint32_t kIdesc = idesc_e4m3(kM, N);
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  unsigned char* const smem = smem_raw + (ring - raw);
  float* const scale_buf = reinterpret_cast<float*>(smem + kStages * L::kStageBytes);
  uint4* const store_buf = reinterpret_cast<uint4*>(smem + kStages * L::kStageBytes + L::kScaleBytes);
  constexpr int kBarsAt = kStages * L::kStageBytes + L::kScaleBytes + L::kStoreBytes;
  const uint32_t bars = ring + kBarsAt;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto tmem_full = [&](int b) { return bars + 8u * (2 * kStages + b); };
  auto tmem_empty = [&](int b) { return bars + 8u * (2 * kStages + kBufs + b); };
  auto scale_full = [&](int b) { return bars + 8u * (2 * kStages + 2 * kBufs + b); };
  const uint32_t drain_bar = bars + 8u * (L::kBars - 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kBarsAt + 8 * L::kBars);
  volatile uint32_t* abort = tmem_slot + 1;

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = L::kSplit ? (int)cluster.block_rank() : 0;
  const int ranks = L::kSplit ? (int)cluster.num_blocks() : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // output tiles of this cluster: first, first + step, ... (one only where K is split);
  // neighbours share their weights
  const int first = (int)blockIdx.x / ranks, step = (int)gridDim.x / ranks;
  const int my_items = first < p.items ? (p.items - 1 - first) / step + 1 : 0;
  auto token0 = [&](int it) { return (first + it * step) % p.mtiles * L::kTokens; };
  auto out0 = [&](int it) { return (first + it * step) / p.mtiles * L::kOut; };
  const int kb0 = (int)((int64_t)p.kblocks * rank / ranks);
  const int nk = (int)((int64_t)p.kblocks * (rank + 1) / ranks) - kb0;
  const int total = my_items * nk;  // K blocks streamed through the ring

  if (threadIdx.x == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_b)) : "memory");
  }
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
    mbar_init(drain_bar, L::kIssuers);
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
  nvfp4::wait_for_previous_kernel();
  int issued = 0;  // stages filled (TMA producer)

  if (warp < 4) {
    // N = 256: the epilogue's two warpgroups take registers that the first has no
    // use for (128 x 88 + 256 x 208 = 384 x 168, what the block was launched with).
    if constexpr (N == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // -------------------------------------------------------- TMA producer
      if (lane == 0) {
        int g = 0;
        bool ok = true;
        for (int it = 0; it < my_items && ok; ++it) {
          const int a0 = FEW ? out0(it) : token0(it), b0 = FEW ? token0(it) : out0(it);
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
            tma_load_2d(dst, &tmap_a, (kb0 + kb) * kK, a0, full(s));
            tma_load_2d(dst + L::kABytes, &tmap_b, (kb0 + kb) * kK, b0, full(s));
          }
        }
      }
    } else if (warp == 1 || (warp == 3 && L::kIssuers == 2)) {
      // --------------------------------------------------------- MMA issuers
      // Each warp stays together and one elected lane issues: descriptors and addresses
      // are then uniform values (a lone thread's instructions cost 600 cycles a K block).
      // Every D_b has a buffer of its own, so issuers need not wait for one another.
      bool ok = true;
      for (int g = warp >> 1; g < total && ok; g += L::kIssuers) {
        const int s = g % kStages, b = g % kBufs;
        ok = g < kBufs ? mbar_wait(full(s), (g / kStages) & 1, abort, p.dev_status)
                       : mbar_wait_both(tmem_empty(b), (g / kBufs - 1) & 1, full(s), (g / kStages) & 1, abort,
                                        p.dev_status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok) {
          tc_fence_after();
          const uint32_t src = ring + (uint32_t)(s * L::kStageBytes);
          const uint64_t ad = smem_desc(src), bd = smem_desc(src + L::kABytes);
          const uint32_t d = tmem + (uint32_t)(b * N);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kK / 32; ++kk)
              mma_f8(d, ad + 2 * kk, bd + 2 * kk, kIdesc, kk > 0 ? 1u : 0u);
            mma_commit(empty(s));
            mma_commit(tmem_full(b));
          }
          __syncwarp();
        }
      }
    } else if (warp == 2) {
      // -------------------------------------------------------------- scales
      // the products sa sw of each K block: FEW of N tokens and one weight block, MANY of
      // 128 tokens and N / 128 weight blocks
      constexpr int kTok = L::kTokens >= 32 ? L::kTokens / 32 : 1, kW = L::kWBlocks;
      float sa[kScalePrefetch][kTok], sw[kScalePrefetch][kW];
      int lit = 0, lkb = 0, left = 0;  // load cursor, tokens of its tile from this lane on
      const float *pa = nullptr, *pw[kW];
      auto load = [&](int i) {
        if (lkb == 0) {
          const int m0 = token0(lit), wb = out0(lit) / kK;
          left = (int)(p.m - m0 < L::kTokens ? p.m - m0 : L::kTokens) - lane;
          pa = p.sa + kb0 * p.lds + m0 + lane;
#pragma unroll
          for (int j = 0; j < kW; ++j)  // (past n: values that nothing stores)
            pw[j] = p.sw + (int64_t)(wb + j < p.wblocks ? wb + j : wb) * p.kblocks + kb0;
        }
#pragma unroll
        for (int j = 0; j < kW; ++j) sw[i][j] = nvfp4::ld_ro(pw[j]++);
#pragma unroll
        for (int j = 0; j < kTok; ++j) sa[i][j] = 32 * j < left ? nvfp4::ld_ro(pa + 32 * j) : 0.0f;
        pa += p.lds;
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
            float v[kW][kTok];
#pragma unroll
            for (int w = 0; w < kW; ++w)
#pragma unroll
              for (int j = 0; j < kTok; ++j) v[w][j] = sa[i][j] * sw[i][w];
            if (g + kScalePrefetch < total) load(i);
            ok = g < kBufs || mbar_wait(tmem_empty(b), (g / kBufs - 1) & 1, abort, p.dev_status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) {
#pragma unroll
              for (int w = 0; w < kW; ++w)
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                  if (L::kTokens >= 32 || lane < L::kTokens)
                    scale_buf[b * L::kScales + w * L::kTokens + 32 * j + lane] = v[w][j];
              __syncwarp();
              if (lane == 0) mbar_arrive(scale_full(b));
            }
          }
        }
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    if constexpr (N == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    constexpr int kChunk = kCols < 32 || kCols > 64 ? 16 : 32;
    constexpr int kChunks = kCols / kChunk;
    const int q = warp & 3, c0 = (warp - 4) / 4 * kCols;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)c0;
    int g = 0;
    bool ok = true;
    for (int it = 0; it < my_items && ok; ++it) {
      uint64_t acc[kCols / 2];  // FP32 pairs of neighbouring columns
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = 0ull;
#pragma unroll 1
      for (int kb = 0; kb < nk; ++kb, ++g) {
        const int b = g % kBufs;
        const uint32_t parity = (g / kBufs) & 1;
        ok = mbar_wait_both(tmem_full(b), parity, scale_full(b), parity, abort, p.dev_status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        const float* scales = scale_buf + b * L::kScales;
        const float s = FEW ? 0.0f : scales[c0 / kK * kM + 32 * q + lane];
        const uint64_t s1 = pack2(__float_as_uint(s), __float_as_uint(s));
        uint32_t v[kChunk];
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
          tmem_issue(tq + (uint32_t)(b * N + ch * kChunk), v);
          ulonglong2 s2[kChunk / 4];
#pragma unroll
          for (int i = 0; i < kChunk / 4; ++i) {
            s2[i] = make_ulonglong2(s1, s1);
            if constexpr (FEW) s2[i] = reinterpret_cast<const ulonglong2*>(scales + c0)[ch * (kChunk / 4) + i];
          }
          tmem_wait(v);
          if (ch + 1 == kChunks) {  // D_b and its scales are in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tmem_empty(b));
          }
#pragma unroll
          for (int i = 0; i < kChunk / 4; ++i) {
            const uint32_t* d = &v[4 * i];
            uint64_t* a = &acc[ch * (kChunk / 2) + 2 * i];
            fma_f32x2(a[0], pack2(d[0], d[1]), s2[i].x);
            fma_f32x2(a[1], pack2(d[2], d[3]), s2[i].y);
          }
        }
      }
      if (!ok) break;
      // What is not finite is reported, such as a product of scales that overflowed: 0 times
      // it is NaN.  (Here, once a tile, that costs at most 1 %; by warp 2, whose products each
      // K block waits for, it took 77 x 17408 x 5120 from 18.1 to 23.2 us.)
      uint64_t zero = 0ull;
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) fma_f32x2(zero, acc[i], 0ull);
      float z0, z1;
      unpack2(zero, z0, z1);
      if (z0 + z1 != 0.0f) nvfp4::report(p.dev_status, NVFP4_ERR_NONFINITE);
      if (L::kSplit && ranks > 1) {
        // the ring's memory: every load and MMA has left it (all D_b were waited for);
        // [column][MMA row], so that neighbouring lanes write neighbouring words
        float* part = reinterpret_cast<float*>(smem) + c0 * kM + 32 * q + lane;
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) unpack2(acc[i], part[2 * i * kM], part[(2 * i + 1) * kM]);
      } else if constexpr (FEW) {
        const int64_t t0 = token0(it) + c0, nn = (int64_t)out0(it) + 32 * q + lane;
        const int left = nn < p.n ? (int)(p.m - t0 < kCols ? p.m - t0 : kCols) : 0;
        store_tokens<kCols>(acc, reinterpret_cast<Out*>(p.c) + t0 * p.ldc + nn, p.ldc, left);
      } else {
        store_row<kCols, Out>(acc, p, (int64_t)token0(it) + 32 * q, (int64_t)out0(it) + c0, lane,
                              store_buf + (warp - 4) * 128);
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
    if (warp == 1 || (warp == 3 && L::kIssuers == 2)) {  // (by the lane that issued them: elect picks the same one)
      if (elect_one()) {
        mma_commit(drain_bar);
        mbar_drain(drain_bar, 0u, p.dev_status);
      }
    }
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kTmemCols)
                 : "memory");
  }
  if (L::kSplit && ranks > 1) {
    // each CTA adds and stores a share of the partial tiles: FEW every ranks-th token,
    // 32 outputs of it a warp; MANY every ranks-th group of tokens likewise
    cluster.sync();
    const float* partial = reinterpret_cast<const float*>(smem);
    const int64_t m0 = token0(0), n0 = out0(0);
    for (int i = rank * L::kThreads + threadIdx.x; i < N * kM; i += ranks * L::kThreads) {
      // FEW: neighbouring threads take neighbouring MMA rows, which are outputs.  MANY:
      // the columns are the outputs; eight tokens x four columns a warp share the words
      // of a column and the bytes of a row between them.
      int row, col;
      if constexpr (FEW) {
        row = i % kM;
        col = i / kM;
      } else {
        const int t = i / 32, l = i % 32;
        row = t % (kM / 8) * 8 + l % 8;
        col = t / (kM / 8) * 4 + l / 8;
      }
      const int64_t token = m0 + (FEW ? col : row), out = n0 + (FEW ? row : col);
      if (token < p.m && out < p.n) {
        float x = 0.0f;
        for (int o = 0; o < ranks; ++o)
          x += *cluster.map_shared_rank(const_cast<float*>(partial) + col * kM + row, o);
        reinterpret_cast<Out*>(p.c)[token * p.ldc + out] = cast<Out>(x);
      }
    }
    cluster.sync();  // no CTA leaves while another reads its partial tile
  }
}

template <bool FEW, int N>
int launch(const CUtensorMap& ta, const CUtensorMap& tb, const Params& p, int split, bool f32,
           cudaStream_t stream) {
  using L = Tile<FEW, N>;
  const void* kern = f32 ? (const void*)fp8b_gemm_kernel<FEW, N, float>
                         : (const void*)fp8b_gemm_kernel<FEW, N, __nv_bfloat16>;
  if (nvfp4::occupancy(kern, L::kThreads, L::kSmemBytes) < 1) return NVFP4_ERR_CUDA;
  const int sms = nvfp4::sm_count();
  const int64_t slots = (int64_t)sms * L::kCtas;
  const int64_t grid = split > 1 ? (int64_t)p.items * split : (p.items < slots ? p.items : slots);
  if (grid > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  void* args[] = {const_cast<CUtensorMap*>(&ta), const_cast<CUtensorMap*>(&tb), const_cast<Params*>(&p)};
  return nvfp4::launch_dependent(kern, dim3((unsigned)grid), dim3(L::kThreads), L::kSmemBytes, stream,
                                 (unsigned)split, args) == cudaSuccess
             ? NVFP4_OK
             : NVFP4_ERR_CUDA;
}

bool encode(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t k, int64_t ld, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {kK, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return nvfp4::encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides,
                             box, estr, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

int launch_fp8b_gemm(const fp8b_act* a, const fp8b_weight* w, void* c, int c_dtype, int64_t ldc,
                     int32_t* dev_status, cudaStream_t stream) {
  const int64_t m = a->m, n = w->n, k = w->k;
  const int64_t kblocks = nvfp4::cdiv(k, kK);
  const int sms = nvfp4::sm_count();
  // Form and tile: FEW with the smallest that holds all tokens, MANY beyond 64 with the
  // tile whose whole waves take less time (a K block of 128 columns takes about 600
  // cycles, of 256 about 750: the handovers weigh on the smaller).  77 x 17408 x 5120: 128
  // columns 18.2 us, 256 columns 22.5; 2048 x 17408 x 5120: 193 and 134.
  const bool few = m <= 64;
  int tile = m <= 16 ? 16 : m <= 32 ? 32 : 64;
  if (!few) {
    const int64_t mt = nvfp4::cdiv(m, kM);
    const int64_t w128 = nvfp4::cdiv(mt * nvfp4::cdiv(n, 128), sms), w256 = nvfp4::cdiv(mt * nvfp4::cdiv(n, 256), sms);
    tile = w128 * 600 <= w256 * 750 ? 128 : 256;
  }
  const int64_t mtiles = nvfp4::cdiv(m, few ? tile : kM), ntiles = nvfp4::cdiv(n, few ? kM : tile);
  const int64_t items = mtiles * ntiles;
  if (items > 0x7FFFFFFF - 1024) return NVFP4_ERR_SHAPE;
  // K is split while that finds idle SMs and leaves eight blocks to each CTA.  Where two
  // CTAs share an SM, clusters (which stay within a group of SMs) fill about 8/5 of the
  // SMs' number: 5120 x 10240, one token: 6 parts 12.4 us, 7 parts 17.4, 3 parts 13.0, 1
  // part 21.9.  (Six parts at most for every shape, of the eight that a cluster may hold:
  // measured at this one.)
  const int64_t slots = tile <= 32 ? (int64_t)sms * 8 / 5 : sms;
  int split = 1;
  while (tile <= 128 && split < 6 && items * (split + 1) <= slots && kblocks / (split + 1) >= 8) ++split;
  CUtensorMap tw, ta;
  if (!encode(&tw, w->codes, n, k, k, few ? kM : tile) || !encode(&ta, a->codes, m, k, a->ld, few ? tile : kM))
    return NVFP4_ERR_CUDA;
  Params p;
  p.sa = a->scales;
  p.lds = a->ld_scales;
  p.sw = w->scales;
  p.c = c;
  p.ldc = ldc;
  p.m = m;
  p.n = n;
  p.kblocks = (int)kblocks;
  p.wblocks = (int)nvfp4::cdiv(n, kK);
  p.mtiles = (int)mtiles;
  p.items = (int)items;
  const bool f32 = c_dtype == NVFP4_DTYPE_F32;
  p.vector_store = nvfp4::aligned16(c) && ldc % (f32 ? 4 : 8) == 0;
  p.dev_status = dev_status;
  switch (tile) {
    case 16: return launch<true, 16>(tw, ta, p, split, f32, stream);
    case 32: return launch<true, 32>(tw, ta, p, split, f32, stream);
    case 64: return launch<true, 64>(tw, ta, p, split, f32, stream);
    case 128: return launch<false, 128>(ta, tw, p, split, f32, stream);
    default: return launch<false, 256>(ta, tw, p, split, f32, stream);
  }
}
