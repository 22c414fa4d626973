// attention.cu -- causal attention with grouped heads over packed prompts and over the
// paged cache, on the 5th-generation tensor cores (sm_103a).
//
//   out_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j
//
// The query heads that share a key head are rows of one tile: row r of 128 is token
// r / group, head r % group of it, so one token of many heads and many tokens of one
// head take the same path.  An item is one key head's NQ such tiles of a sequence
// against the keys that they see, 128 keys at a time:
//   S = Q K^T        tcgen05.mma, both operands in shared memory, FP32 into TMEM
//   P = exp2(S c - m)  registers; BF16 back into TMEM over S
//   O += P V         tcgen05.mma, P from TMEM, V from shared memory (rows of keys as
//                    they are in memory: the transposed operand form)
// with the softmax's running maximum m and sum carried along.  m is raised, and O and
// the sum rescaled, only when a tile's maximum exceeds it by 2^8: P is then at most 256
// and loses nothing (FP32 and BF16 keep their relative precision), and O, which lies in
// TMEM, is rarely touched.
//   NQ = 2 (heads of 64 and 128): two tiles of rows share each tile of keys; a
//          warpgroup of softmax threads, a row each, for either, so that one's
//          exponentials run while the tensor core works on the other's products;
//   NQ = 1 (few rows, and heads of 256, whose O takes 256 of TMEM's 512 columns): both
//          warpgroups work on the same tile, half of its keys each, and exchange the
//          rows' maxima through shared memory; S is double buffered.
//   warps 0..7  softmax; they rescale and finish O as well
//   warp 8      allocates TMEM, issues the MMAs: S two steps ahead of the P V it waits for
//   warp 9      schedules the items and loads K and V (TMA) into a ring
//   warp 10     loads Q
//
// Schedule: the items of all sequences and heads are laid end to end on a line, a tile of
// keys 128 units long and an item's start kItemCost, and every CTA takes an equal share of
// it, whatever the lengths: each finds its share from the lengths on the device.  An item
// that a share's border cuts leaves the parts' (maximum, sum, O) in the workspace, FP32, and
// a second kernel joins them in the order of the keys.  The borders depend on the lengths
// alone, so results do not depend on timing.
//
// Keys that a row does not see get weight 0 by selection, and P V stops at the last one that
// some row of the item sees (rounded up to 16, values behind it zeroed): what lies there, in
// other sequences or unused slots, does not matter.
#include <cuda_bf16.h>

#include "tc.cuh"

namespace {

using namespace nvfp4::tc;
using nvfp4::ld_ro;

constexpr int kRows = 128;                    // MMA rows of a tile of queries
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kSoftmaxWarps = 8;
constexpr int kWarps = kSoftmaxWarps + 4;     // (three of the last four work)
constexpr int kThreads = 32 * kWarps;
constexpr int kDescs = 4;                     // item descriptors in flight
constexpr int kItemCost = kKeys;              // an item's fixed cost, in keys
constexpr int kMinShare = 2 * kKeys + kItemCost;  // of a CTA, where there are that few
constexpr float kRescale = 8.0f;              // log2 of what the maximum may lag behind
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int NQ>
struct Tile {
  static constexpr int kUnitDims = D < 128 ? D : 128;  // of a unit of the ring: 128 keys of as many dims
  static constexpr int kUnits = D / kUnitDims;         // of a tile of K, and of V
  static constexpr int kBlocks = kUnitDims / 64;       // swizzled columns of 128 bytes
  static constexpr int kUnitBytes = kKeys * kUnitDims * 2;
  static constexpr int kQTile = kRows * D * 2;
  static constexpr int kQBytes = NQ * kQTile;
  static constexpr int kXchBytes = NQ == 1 ? 2 * 2 * kRows * 4 : 0;
  static constexpr int kDescBytes = kDescs * 64;
  static constexpr int kRest = kXchBytes + kDescBytes + 512;
  static constexpr int kFit = (227 * 1024 - kQBytes - kRest) / kUnitBytes;
  static constexpr int kStages = kFit < 10 ? kFit : 10;
  static constexpr size_t kSmemBytes = (size_t)kQBytes + (size_t)kStages * kUnitBytes + kRest;
  static constexpr int kCols = NQ == 2 ? kKeys : kKeys / 2;  // of S, a softmax thread's
  static constexpr int kOut = NQ == 2 ? D : D / 2;           // of O, a softmax thread's
  static_assert(kStages >= 5 && kStages > kUnits, "ring");
  static_assert(2 * kKeys + NQ * D <= 512, "TMEM");
};

struct Params {
  const int32_t* cu;
  const int32_t* kv_lens;  // nullptr: prompts
  const int32_t* table;
  int64_t ld_table, capacity;  // tokens of a table row
  int tokens, batch, kv_heads, group;
  int page_size, page_shift;   // tokens of a page; log2 of it, or -1
  int box;                     // tokens of a TMA box
  int pages;
  float scale;                 // |scale| log2 e, never 0
  int negative;
  __nv_bfloat16* out;
  int64_t ld_token, ld_head;
  unsigned char* ws;
  int32_t* dev_status;
};

struct Sequence {
  int begin, n;  // rows of q
  int len;       // keys
  int off;       // position of the first query (may be negative)
};

// What the roles need of an item, in shared memory.
struct __align__(16) Item {
  int row0, rows;   // tokens: first row of q, number (0: no more items)
  int pos0, end;    // position of the first; keys that some row sees
  int head, first;  // key head; first tile of this part
  int last, slot;   // past its last tile; -1: the whole item, else the part's place
};

// An item cut by a share's border, for the kernel that joins its parts.
struct Record {
  int parts, row0, rows, head;
};

__host__ __device__ constexpr int64_t slot_floats(int d, int nq) { return (int64_t)nq * kRows * (d + 2); }
constexpr size_t kRecordBytes = (size_t)ATTENTION_MAX_CTAS * 64;

__device__ __forceinline__ Sequence sequence(const Params& p, int s, bool* consistent = nullptr) {
  const int a = ld_ro(p.cu + s), b = ld_ro(p.cu + s + 1);
  const int64_t cached = p.kv_lens != nullptr ? ld_ro(p.kv_lens + s) : 0;
  Sequence q;
  q.begin = min(max(a, 0), p.tokens);
  q.n = max(min(max(b, 0), p.tokens) - q.begin, 0);
  q.len = p.kv_lens != nullptr ? (int)min(max(cached, (int64_t)0), p.capacity) : q.n;
  q.off = q.len - q.n;
  if (consistent != nullptr) *consistent = a >= 0 && b <= p.tokens && a <= b && cached <= p.capacity;
  return q;
}
// (64-bit division takes several times a 32-bit one's time)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line: item t of a (sequence, head) starts `before(t)` behind its head's start.
template <int NQ>
struct Line {
  int per;       // tokens of an item
  int64_t base;  // length of item 0
  int items;
  int64_t length;
  __device__ __forceinline__ Line(const Sequence& q, int group) {
    per = NQ * (kRows / group);
    items = (q.n + per - 1) / per;
    const int64_t cached = max(q.off, 0);
    base = cached + per + kItemCost;
    length = items > 0 ? before(items - 1) + cached + q.n + kItemCost : 0;
  }
  __device__ __forceinline__ int64_t before(int64_t t) const { return t * base + per * (t * (t - 1) / 2); }
};

// TMA and MMA instructions are issued by one lane of a converged warp, by predicate and not
// by a branch: their operands are then uniform values, which these instructions take as they
// are (issued behind a branch, or by a lane each, one takes 80 to 110 cycles).
__device__ __forceinline__ void tma_load_4d(uint32_t lead, uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            int c3, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred l;\n setp.ne.b32 l, %7, 0;\n"
      " @l cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred l;\n setp.ne.b32 l, %1, 0;\n"
      " @l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar), "r"(lead)
      : "memory");
}
// kind::f16 with BF16 operands, D = F32; bit 16: B is N-major in shared memory.
constexpr uint32_t idesc_bf16(int n, bool b_transposed) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_transposed ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kRows >> 4) << 24);
}
// Shared-memory operands, lower word of the descriptor: start address >> 4, leading offset
// (V as B: 64-element columns of 128 keys, 16 KB apart); upper word: 8-row groups 1 KB apart,
// version 1, 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_low_v(uint32_t addr) {
  return ((addr >> 4) & 0x3FFFu) | ((uint32_t)(kKeys * 128 >> 4) << 16);
}
// Four MMAs along a swizzled column: 64 elements of K, 32 bytes each apart.
__device__ __forceinline__ void mma_ss4(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred l, p, q;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
      " setp.ne.b32 l, %0, 0;\n setp.ne.b32 p, %5, 0;\n setp.eq.b32 q, 0, 0;\n"
      " mov.b64 a, {%2, %6};\n mov.b64 b, {%3, %6};\n"
      " @l tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, p;\n"
      " add.u32 x, %2, 2;\n add.u32 y, %3, 2;\n mov.b64 a, {x, %6};\n mov.b64 b, {y, %6};\n"
      " @l tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, q;\n"
      " add.u32 x, %2, 4;\n add.u32 y, %3, 4;\n mov.b64 a, {x, %6};\n mov.b64 b, {y, %6};\n"
      " @l tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, q;\n"
      " add.u32 x, %2, 6;\n add.u32 y, %3, 6;\n mov.b64 a, {x, %6};\n mov.b64 b, {y, %6};\n"
      " @l tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, q;\n}" ::"r"(lead),
      "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}
// Four MMAs along 64 keys: P in TMEM, 16 keys in 8 columns; V 16 rows of 128 bytes apart.  Of
// them the first `steps`.
__device__ __forceinline__ void mma_ts4(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate, int steps) {
  asm volatile(
      "{\n .reg .pred l, m, p, q;\n .reg .b32 x, y;\n .reg .b64 b;\n"
      " setp.ne.b32 l, %0, 0;\n setp.ne.b32 p, %5, 0;\n setp.eq.b32 q, 0, 0;\n"
      " setp.gt.and.s32 m, %7, 0, l;\n mov.b64 b, {%3, %6};\n"
      " @m tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %4, p;\n"
      " setp.gt.and.s32 m, %7, 1, l;\n add.u32 x, %2, 8;\n add.u32 y, %3, 128;\n mov.b64 b, {y, %6};\n"
      " @m tcgen05.mma.cta_group::1.kind::f16 [%1], [x], b, %4, q;\n"
      " setp.gt.and.s32 m, %7, 2, l;\n add.u32 x, %2, 16;\n add.u32 y, %3, 256;\n mov.b64 b, {y, %6};\n"
      " @m tcgen05.mma.cta_group::1.kind::f16 [%1], [x], b, %4, q;\n"
      " setp.gt.and.s32 m, %7, 3, l;\n add.u32 x, %2, 24;\n add.u32 y, %3, 384;\n mov.b64 b, {y, %6};\n"
      " @m tcgen05.mma.cta_group::1.kind::f16 [%1], [x], b, %4, q;\n}" ::"r"(lead),
      "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh), "r"(steps)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float exp2_approx(float x) {  // 2^-22 relative; 0 for -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
// A value that all lanes hold, so that the compiler knows: what is computed from it goes to
// the tensor core without a detour through each lane's registers.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }
// All softmax threads: true if `ok` holds for all of them (so they leave together).
__device__ __forceinline__ bool softmax_agree(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(32 * kSoftmaxWarps)
      : "memory");
  return r != 0;
}

// ----------------------------------------------------------------- kernel

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Params p) {
  using L = Tile<D, NQ>;
  constexpr int kStages = L::kStages, kUnits = L::kUnits, kBlocks = L::kBlocks;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* const ring_ptr = smem + L::kQBytes;
  float* const xch = reinterpret_cast<float*>(ring_ptr + kStages * L::kUnitBytes);
  Item* const items = reinterpret_cast<Item*>(reinterpret_cast<unsigned char*>(xch) + L::kXchBytes);
  const uint32_t q_smem = smem_u32(smem), ring = q_smem + L::kQBytes;
  const uint32_t bars = smem_u32(items) + L::kDescBytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto item_full = [&](int i) { return bars + 8u * (2 * kStages + i); };
  auto item_empty = [&](int i) { return bars + 8u * (2 * kStages + kDescs + i); };
  constexpr int kFixed = 2 * kStages + 2 * kDescs;
  const uint32_t q_full = bars + 8u * kFixed, q_empty = bars + 8u * (kFixed + 1);
  auto s_full = [&](int b) { return bars + 8u * (kFixed + 2 + b); };
  auto p_full = [&](int b) { return bars + 8u * (kFixed + 4 + b); };
  auto pv_done = [&](int t) { return bars + 8u * (kFixed + 6 + t); };
  const uint32_t drain_bar = bars + 8u * (kFixed + 8);
  static_assert(8 * (kFixed + 9 + kWarps + 1) + 12 <= 512, "shared memory behind the items");
  int64_t* const sums = reinterpret_cast<int64_t*>(reinterpret_cast<unsigned char*>(items) + L::kDescBytes + 8 * (kFixed + 9));
  int64_t& start_at = sums[kWarps];
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sums + kWarps + 1);
  volatile uint32_t* abort = tmem_slot + 1;
  int& start_seq = reinterpret_cast<int*>(tmem_slot)[2];
  // (uniform: a role's code is then known not to diverge, and its instructions' addresses and
  // descriptors stay in uniform registers)
  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (q_smem & 1023u) {  // (the swizzled tiles need it; the declaration asks for it)
    nvfp4::report(p.dev_status, NVFP4_ERR_ALIGN);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(item_full(i), 1);
      mbar_init(item_empty(i), kSoftmaxWarps + 2);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(p_full(b), NQ == 2 ? kSoftmaxWarps / 2 : kSoftmaxWarps);
      mbar_init(pv_done(b), 1);
    }
    mbar_init(drain_bar, 1);
    *abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x >= 288 && threadIdx.x < 291) {
    const CUtensorMap* m = threadIdx.x == 288 ? &map_q : threadIdx.x == 289 ? &map_k : &map_v;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  nvfp4::wait_for_previous_kernel();

  // This CTA's share [x0, x1) of the line, and the sequence that x0 lies in.
  const int run = (p.batch + kThreads - 1) / kThreads;
  const int s0 = min(p.batch, (int)threadIdx.x * run), s1 = min(p.batch, s0 + run);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    bool consistent;
    mine += p.kv_heads * Line<NQ>(sequence(p, s, &consistent), p.group).length;
    if (blockIdx.x == 0 && !consistent) nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
  }
  int64_t upto = mine;
  if (p.batch > 1) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += o;
    }
  }
  if (lane == (p.batch > 1 ? 31 : 0)) sums[warp] = upto;
  if (threadIdx.x == 0) start_seq = p.batch;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all of the SM's columns: they start at 0 (a constant for the MMAs' addresses)
  constexpr uint32_t tmem = 0;
  if (*tmem_slot != tmem) nvfp4::report(p.dev_status, NVFP4_ERR_CUDA);
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) upto += total;
    total += sums[w];
  }
  // total = shares * each + rest: the first `rest` shares are one longer
  const int64_t wanted = total / kMinShare;
  const int shares = (int)(wanted < 1 ? 1 : wanted < gridDim.x ? wanted : gridDim.x);
  const int64_t each = quotient(total, shares), rest = total - each * shares;
  auto border = [&](int c) -> int64_t { return c < shares ? c * each + min((int64_t)c, rest) : total; };
  const int64_t x0 = border((int)blockIdx.x), x1 = border((int)blockIdx.x + 1);
  if (x0 < x1 && upto > x0 && upto - mine <= x0) {
    int64_t at = upto - mine;
    int s = s0;
    for (; s + 1 < s1; ++s) {
      const int64_t len = p.kv_heads * Line<NQ>(sequence(p, s), p.group).length;
      if (at + len > x0) break;
      at += len;
    }
    start_seq = s;
    start_at = at;
  }
  __syncthreads();

  const int per_tile = kRows / p.group;  // tokens of a tile of rows
  int issued = 0, q_issued = 0;          // units and Q loads issued (TMA warps)
  const uint32_t lead = elect_one();     // the lane that issues for a warp

  // NQ = 2: the softmax's threads take registers that the others have no use for
  // (256 x 208 + 128 x 88 = 384 x 168, what the block was launched with).
  if (NQ == 2 && warp >= kSoftmaxWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 9) {
    // ------------------------------------------------- schedule, K and V loads
    // (all lanes together; lane i knows the page of a tile's box i)
    const int boxes = kKeys / p.box;
    bool ok = true;
    int seq = start_seq, head = 0, t = 0;
    Sequence q{}, next_q{};
    int64_t head_at = 0;
    if (seq < p.batch) {
      q = sequence(p, seq);
      const Line<NQ> line(q, p.group);
      head = (int)quotient(x0 - start_at, line.length);
      head_at = start_at + head * line.length;
      int lo = 0, hi = line.items;  // the item that x0 lies in
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (head_at + line.before(mid) <= x0)
          lo = mid;
        else
          hi = mid;
      }
      t = lo;
      if (seq + 1 < p.batch) next_q = sequence(p, seq + 1);
    }
    // The next part of this CTA's share, or rows = 0.  `row` is its table row, `begin` its
    // first token in packed prompts.
    struct Part {
      Item it;
      int64_t row;
      int begin;
      int record;  // parts of the whole item, where this is the first of several
    };
    auto advance = [&]() -> Part {
      Part r{};
      r.it.rows = 0;
      while (seq < p.batch) {
        const Line<NQ> line(q, p.group);
        if (t >= line.items) {
          t = 0;
          head_at += line.length;
          if (q.n == 0 || ++head >= p.kv_heads) {
            head = 0;
            ++seq;
            q = next_q;
            if (seq + 1 < p.batch) next_q = sequence(p, seq + 1);
          }
          continue;
        }
        const int64_t at = head_at + line.before(t) + kItemCost;  // of tile 0
        if (at - kItemCost >= x1) break;
        const int row = t * line.per, rows = min(line.per, q.n - row);
        const int end = max(q.off + row + rows, 0);
        const int tiles = max((end + kKeys - 1) / kKeys, 1);
        const int64_t a = at >= x0 ? 0 : (x0 - at + kKeys - 1) / kKeys;
        const int64_t b = at >= x1 ? 0 : (x1 - at + kKeys - 1) / kKeys;
        ++t;
        if (a >= tiles || b <= a) continue;
        r.it.row0 = q.begin + row;
        r.it.rows = rows;
        r.it.pos0 = q.off + row;
        r.it.end = end;
        r.it.head = head;
        r.it.first = (int)a;
        r.it.last = (int)min(b, (int64_t)tiles);
        r.it.slot = a > 0 ? 0 : b < tiles ? 1 : -1;
        r.row = seq * p.ld_table;
        r.begin = q.begin;
        if (a == 0 && b < tiles) {
          const int64_t last_tile = at + (int64_t)(tiles - 1) * kKeys, longer = rest * (each + 1);
          const int owner = (int)(last_tile < longer ? quotient(last_tile, each + 1) : rest + quotient(last_tile - longer, each));
          r.record = owner - (int)blockIdx.x + 1;
        }
        break;
      }
      return r;
    };
    // Where this lane's box of a tile lies: its page, and its first token there; how many boxes
    // some row sees.  The others are not loaded: their scores are masked whatever they are, and
    // P V stops before them.  (Boxes outside the cache, read as zeros, take the TMA unit about 1 us
    // each.)
    struct Place {
      int page, token, count;
    };
    auto place_of = [&](const Part& r, int tile) -> Place {
      const int j = tile * kKeys + lane * p.box;
      const int count = min(max((r.it.end - tile * kKeys + p.box - 1) / p.box, 0), boxes);
      if (lane >= count) return Place{0, 0, count};
      if (p.table == nullptr) return Place{0, r.begin + j, count};
      const int entry = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
      const int id = ld_ro(p.table + r.row + entry);
      return Place{id, j - entry * p.page_size, count};
    };
    int unit = 0;
    auto load_tile = [&](const CUtensorMap* map, const Part& r, const Place& at) {
      int page = at.page;
      if (page < 0 || page >= p.pages) {
        nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
        page = p.pages;
      }
      const int head = uniform(r.it.head), count = uniform(at.count);
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int s = unit % kStages;
        if (unit >= kStages) ok = ok && mbar_wait(empty(s), (unit / kStages - 1) & 1, abort, p.dev_status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return;
        issued = unit + 1;
        const bool withheld = nvfp4::kWithhold && blockIdx.x == 0 && unit == 0;  // test build: never issued
        ++unit;
        if (withheld) continue;
        if (lead) mbar_arrive_expect_tx(full(s), (uint32_t)(count * p.box * 128 * kBlocks));
        __syncwarp();
        const uint32_t dst = ring + (uint32_t)(s * L::kUnitBytes);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= count) break;
          const int pg = __shfl_sync(0xFFFFFFFFu, page, i), tk = __shfl_sync(0xFFFFFFFFu, at.token, i);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
            tma_load_4d(lead, dst + (uint32_t)(b * (kKeys * 128) + i * p.box * 128), map, u * L::kUnitDims + b * 64, head, tk,
                        pg, full(s));
        }
      }
    };
    Part cur = advance(), prev{};
    Place at{}, prev_at{};
    if (cur.it.rows) at = place_of(cur, cur.it.first);
    bool behind = false;  // a V is still to come
    int count = 0, record = 0;
    Part recorded{};
    while (ok) {
      const int i = count % kDescs;
      if (count >= kDescs) ok = mbar_wait(item_empty(i), (count / kDescs - 1) & 1, abort, p.dev_status);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      if (lane == 0) {
        items[i] = cur.it;
        mbar_arrive(item_full(i));
      }
      __syncwarp();
      ++count;
      if (cur.it.rows == 0) break;
      if (cur.record) {
        record = cur.record;
        recorded = cur;
      }
      Part next{};
      for (int tile = cur.it.first; tile < cur.it.last && ok; ++tile) {
        load_tile(&map_k, cur, at);
        // the next tile's pages are on their way while this one's are loaded
        Place next_at{};
        if (tile + 1 < cur.it.last) {
          next_at = place_of(cur, tile + 1);
        } else {
          next = advance();
          if (next.it.rows) next_at = place_of(next, next.it.first);
        }
        if constexpr (NQ == 2) {
          if (ok) load_tile(&map_v, cur, at);
        } else {
          // V one tile behind K, as the MMAs take them
          if (ok && behind) load_tile(&map_v, prev, prev_at);
          behind = true;
          prev = cur;
          prev_at = at;
        }
        at = next_at;
      }
      cur = next;
    }
    if (NQ == 1 && ok && behind) {
      unit += kUnits;  // the place of a K that does not come: V's is the same for every tile
      load_tile(&map_v, prev, prev_at);
    }
    if (lane == 0) {
      Record* rec = reinterpret_cast<Record*>(p.ws + (size_t)blockIdx.x * 64);
      *rec = Record{record, recorded.it.row0, recorded.it.rows, recorded.it.head};
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------------ Q loads
    for (int count = 0;; ++count) {
      const int i = count % kDescs;
      bool ok = mbar_wait(item_full(i), (count / kDescs) & 1, abort, p.dev_status);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      const int rows = uniform(items[i].rows), row0 = uniform(items[i].row0), head = uniform(items[i].head);
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty(i));
      if (rows == 0) break;
      ok = count == 0 || mbar_wait(q_empty, (count - 1) & 1, abort, p.dev_status);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      q_issued = count + 1;
      if (lead) mbar_arrive_expect_tx(q_full, (uint32_t)(NQ * (D / 64) * per_tile * p.group * 128));
      __syncwarp();
#pragma unroll
      for (int t = 0; t < NQ; ++t)
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          tma_load_4d(lead, q_smem + (uint32_t)(t * L::kQTile + b * (kRows * 128)), &map_q, b * 64, 0, head,
                      row0 + t * per_tile, q_full);
    }
  } else if (warp == 8) {
    // --------------------------------------------------------------------- MMAs
    // Steps g = 0, 1, ... over all items: NQ = 2: tile of keys g / 2, rows g % 2; NQ = 1: tile
    // g.  S of step g into buffer g % 2.  Two cursors, S's two steps ahead.
    constexpr uint32_t kIdescS = idesc_bf16(kKeys, false), kIdescO = idesc_bf16(L::kUnitDims, true);
    bool ok = true;
    struct Cursor {
      int count, tile, first, last, end, rows, x;  // item, tile of it; tiles of the CTA before
      int row_tile;
    };
    Cursor cs{}, cp{};
    auto fetch = [&](Cursor& c, bool release) {  // the cursor's next item
      const int i = c.count % kDescs;
      ok = mbar_wait(item_full(i), (c.count / kDescs) & 1, abort, p.dev_status);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) return;
      const Item& it = items[i];
      c.rows = uniform(it.rows);
      c.tile = c.first = uniform(it.first);
      c.last = uniform(it.last);
      c.end = uniform(it.end);
      c.row_tile = 0;
      ++c.count;
      __syncwarp();
      if (release && lane == 0) mbar_arrive(item_empty(i));
    };
    auto step = [&](Cursor& c, bool release) {
      if (NQ == 2 && c.row_tile == 0) {
        c.row_tile = 1;
        return;
      }
      c.row_tile = 0;
      ++c.x;
      if (++c.tile == c.last) fetch(c, release);
    };
    auto wait_unit = [&](int unit) {
      ok = ok && mbar_wait(full(unit % kStages), (unit / kStages) & 1, abort, p.dev_status);
      ok = __all_sync(0xFFFFFFFFu, ok);
    };
    int gs = 0;
    auto issue_s = [&]() {
      if (cs.tile == cs.first && cs.row_tile == 0) {
        ok = mbar_wait(q_full, (cs.count - 1) & 1, abort, p.dev_status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return;
      }
      const int u0 = NQ == 2 ? 2 * cs.x * kUnits : cs.x == 0 ? 0 : (2 * cs.x - 1) * kUnits;
      const uint32_t d = tmem + (uint32_t)(gs & 1) * kKeys;
      const bool last_use = NQ == 1 || cs.row_tile == 1;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        if (NQ == 1 || cs.row_tile == 0) wait_unit(u0 + u);
        if (!ok) return;
        tc_fence_after();
        const uint32_t a = desc_low(q_smem + (uint32_t)(cs.row_tile * L::kQTile + u * kBlocks * (kRows * 128)));
        const uint32_t b = desc_low(ring + (uint32_t)((u0 + u) % kStages * L::kUnitBytes));
#pragma unroll
        for (int c = 0; c < kBlocks; ++c)
          mma_ss4(lead, d, a + c * (kRows * 128 >> 4), b + c * (kKeys * 128 >> 4), kIdescS, (u > 0 || c > 0) ? 1u : 0u);
        if (u == kUnits - 1) commit(lead, s_full(gs & 1));
        if (last_use) commit(lead, empty((u0 + u) % kStages));
      }
      if (last_use && cs.tile + 1 == cs.last) commit(lead, q_empty);
      ++gs;
      step(cs, false);
    };
    int gp = 0;
    auto issue_pv = [&]() {
      ok = mbar_wait(p_full(gp & 1), (gp >> 1) & 1, abort, p.dev_status);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) return;
      const int u0 = NQ == 2 ? (2 * cp.x + 1) * kUnits : (2 * cp.x + 2) * kUnits;
      const int seen = min(max(cp.end - cp.tile * kKeys, 1), kKeys);
      const int steps = (seen + 15) / 16;  // of 16 keys
      const uint32_t a = tmem + (uint32_t)(gp & 1) * kKeys;
      const uint32_t o = tmem + 2 * kKeys + (uint32_t)(cp.row_tile * D);
      const bool last_use = NQ == 1 || cp.row_tile == 1;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        if (NQ == 1 || cp.row_tile == 0) wait_unit(u0 + u);
        if (!ok) return;
        tc_fence_after();
        const uint32_t b = desc_low_v(ring + (uint32_t)((u0 + u) % kStages * L::kUnitBytes));
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mma_ts4(lead, o + (uint32_t)(u * L::kUnitDims), a + 32 * h, b + 512 * h, kIdescO,
                  (cp.tile > cp.first || h > 0) ? 1u : 0u, steps - 4 * h);
        if (u == kUnits - 1) commit(lead, pv_done(gp & 1));
        if (last_use) commit(lead, empty((u0 + u) % kStages));
      }
      ++gp;
      step(cp, true);
    };
    fetch(cs, false);
    if (ok) fetch(cp, true);
    for (int i = 0; i < 2 && ok && cs.rows; ++i) issue_s();
    while (ok && cp.rows) {
      issue_pv();
      if (ok && cs.rows) issue_s();
    }
  } else if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------------ softmax
    if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    constexpr int kCols = L::kCols, kOut = L::kOut;
    const int group_of = warp >> 2;                                  // warpgroup
    const int r = (warp & 3) * 32 + lane;                            // row of the tile
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int t = NQ == 2 ? group_of : 0;
    const int c0 = NQ == 2 ? 0 : group_of * kCols;
    const int token = r / p.group, g = r - token * p.group;
    const uint32_t o_addr = lanes + 2 * kKeys + (uint32_t)(t * D + (NQ == 1 ? group_of * kOut : 0));
    const float scale = p.scale;
    const uint64_t scale2 = pack2(__float_as_uint(scale), __float_as_uint(scale));
    // P V of the CTA's tile i is complete.  A barrier per buffer of S: the wait before last on
    // one, two steps ago, is known to be over from S of this tile, so parities suffice.
    auto wait_pv = [&](int i) {
      return mbar_wait(pv_done(NQ == 2 ? t : i & 1), (NQ == 2 ? i : i >> 1) & 1, abort, p.dev_status);
    };
    bool ok = true;
    int x = 0, exchanges = 0;
    for (int count = 0;; ++count) {  // (NQ = 1: the warps leave together, at an exchange)
      const int di = count % kDescs;
      ok = ok && mbar_wait(item_full(di), (count / kDescs) & 1, abort, p.dev_status);
      ok = NQ == 1 ? softmax_agree(ok) : (bool)__all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      const Item it = items[di];
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty(di));
      if (it.rows == 0) break;
      const bool valid = token < per_tile && t * per_tile + token < it.rows;
      const bool busy = __any_sync(0xFFFFFFFFu, valid);  // this warp has rows
      const int limit = valid ? it.pos0 + t * per_tile + token + 1 : 0x7FFFFFFF;  // keys that the row sees
      float m = -INFINITY, l = 0.0f;
      for (int tile = it.first; tile < it.last; ++tile, ++x) {
        const int b = NQ == 2 ? t : x & 1;
        ok = ok && mbar_wait(s_full(b), (NQ == 2 ? x : x >> 1) & 1, abort, p.dev_status);
        if (NQ == 2) {
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t s_addr = lanes + (uint32_t)(b * kKeys + c0);
        uint32_t s[kCols / 32][32];
        float top = -INFINITY;
        if (busy) {
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) tmem_issue(s_addr + 32 * c, s[c]);
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) tmem_wait(s[c]);
          if (p.negative) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) s[i / 32][i % 32] ^= 0x80000000u;
          }
          const int seen = limit - tile * kKeys - c0;
          if (__any_sync(0xFFFFFFFFu, seen < kCols)) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if (i >= seen) s[i / 32][i % 32] = 0xFF800000u;
          }
          float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kCols; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top4[e] = max3(top4[e], __uint_as_float(s[(i + 2 * e) / 32][(i + 2 * e) % 32]),
                             __uint_as_float(s[(i + 2 * e + 1) / 32][(i + 2 * e + 1) % 32]));
          top = max3(fmaxf(top4[0], top4[1]), top4[2], top4[3]);
          if (!valid) top = 0.0f;  // (no row: whatever S holds there, O is not rescaled for it)
        }
        if constexpr (NQ == 1) {
          float* at = xch + (exchanges & 1) * 2 * kRows + r;
          ++exchanges;
          at[group_of * kRows] = top;
          ok = softmax_agree(ok);
          if (!ok) break;
          top = fmaxf(top, at[(group_of ^ 1) * kRows]);
        }
        if (busy) {
          // the reference maximum: raised for the whole warp once a row needs it
          const float raised = fmaxf(m, top);
          const bool grow = (raised - m) * scale > kRescale;  // (no key seen yet, neither before: not a number)
          if (__any_sync(0xFFFFFFFFu, grow)) {
            const float keep = m == -INFINITY ? 0.0f : exp2_approx((m - raised) * scale);
            l *= keep;
            m = raised;
            if (tile > it.first) {
              ok = ok && wait_pv(x - 1);
              ok = __all_sync(0xFFFFFFFFu, ok);
              tc_fence_after();
              const uint64_t keep2 = pack2(__float_as_uint(keep), __float_as_uint(keep));
#pragma unroll 1
              for (int c = 0; c < kOut; c += 16) {
                uint32_t o[16];
                tmem_issue(o_addr + c, o);
                tmem_wait(o);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  float lo, hi;
                  unpack2(fma2(pack2(o[i], o[i + 1]), keep2, 0ull), lo, hi);
                  o[i] = __float_as_uint(lo);
                  o[i + 1] = __float_as_uint(hi);
                }
                tmem_store(o_addr + c, o);
              }
            }
          }
          const float shift = m == -INFINITY ? 0.0f : -m * scale;
          const uint64_t shift2 = pack2(__float_as_uint(shift), __float_as_uint(shift));
          uint64_t sum[2] = {0ull, 0ull};
          const uint32_t p_addr = lanes + (uint32_t)(b * kKeys + c0 / 2);
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float lo, hi;
              unpack2(fma2(pack2(s[c][2 * i], s[c][2 * i + 1]), scale2, shift2), lo, hi);
              lo = exp2_approx(lo);
              hi = exp2_approx(hi);
              sum[i & 1] = add2(sum[i & 1], pack2(__float_as_uint(lo), __float_as_uint(hi)));
              w[i] = to_bf16x2(lo, hi);
            }
            tmem_store(p_addr + 16 * c, w);
          }
          float s0f, s1f;
          unpack2(add2(sum[0], sum[1]), s0f, s1f);
          l += s0f + s1f;
          tmem_store_wait();
        }
        // Values behind the last key that any row sees may be anything: zeros for those of
        // them that the last 16 keys of P V take in.
        if (tile * kKeys + kKeys > it.end && (NQ == 1 || t == 0)) {
          const int from = max(it.end - tile * kKeys, 0), to = (max(from, 1) + 15) / 16 * 16;
          const int u0 = NQ == 2 ? (2 * x + 1) * kUnits : (2 * x + 2) * kUnits;
          const int threads = NQ == 2 ? 128 : 256, me = threadIdx.x % threads;
          // A stage's barrier tells this load from the one before only once that one is complete:
          // it is S's or an earlier tile's, but with two units a tile and five stages V's of the
          // tile before.
          static_assert(kUnits == 1 || NQ == 1, "stages");
          if (kUnits == 2 && x > 0) ok = ok && wait_pv(x - 1);
          for (int u = 0; u < kUnits; ++u) {
            ok = ok && mbar_wait(full((u0 + u) % kStages), ((u0 + u) / kStages) & 1, abort, p.dev_status);
            unsigned char* v = ring_ptr + (u0 + u) % kStages * L::kUnitBytes;
            if (ok)
              for (int i = from * 8 * kBlocks + me; i < to * 8 * kBlocks; i += threads) {
                const int key = i / (8 * kBlocks), piece = i % (8 * kBlocks);
                *reinterpret_cast<uint4*>(v + piece / 8 * (kKeys * 128) + key * 128 + piece % 8 * 16) = make_uint4(0, 0, 0, 0);
              }
          }
          fence_proxy_async();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(b));
      }
      if (NQ == 2 && !ok) break;
      // the part's end: O / l to the output, or (m, l, O) to the workspace
      if constexpr (NQ == 1) {
        float* at = xch + (exchanges & 1) * 2 * kRows + r;
        ++exchanges;
        at[group_of * kRows] = l;
        ok = softmax_agree(ok);
        if (!ok) break;
        l += at[(group_of ^ 1) * kRows];
      }
      ok = wait_pv(x - 1);
      ok = __all_sync(0xFFFFFFFFu, ok);
      tc_fence_after();
      if (busy && ok) {
        float* part = nullptr;
        __nv_bfloat16* out = nullptr;
        float norm = 1.0f;
        if (it.slot < 0) {
          norm = 1.0f / l;
          out = p.out + (int64_t)(it.row0 + t * per_tile + token) * p.ld_token + (it.head * p.group + g) * p.ld_head +
                (NQ == 1 ? group_of * kOut : 0);
        } else {
          float* slot = reinterpret_cast<float*>(p.ws + kRecordBytes) + (2 * (int64_t)blockIdx.x + it.slot) * slot_floats(D, NQ);
          const int row = t * kRows + r;
          if (valid && (NQ == 2 || group_of == 0)) *reinterpret_cast<float2*>(slot + 2 * row) = make_float2(m, l);
          part = slot + 2 * NQ * kRows + (int64_t)row * D + (NQ == 1 ? group_of * kOut : 0);
        }
#pragma unroll 1
        for (int c = 0; c < kOut; c += 32) {
          uint32_t o[32];
          tmem_issue(o_addr + c, o);
          tmem_wait(o);
          if (!valid) continue;
          if (part != nullptr) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(part + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // (a row that sees nothing: 0, whatever O holds)
                const float lo = l != 0.0f ? __uint_as_float(o[i + 2 * e]) * norm : 0.0f;
                const float hi = l != 0.0f ? __uint_as_float(o[i + 2 * e + 1]) * norm : 0.0f;
                w[e] = to_bf16x2(lo, hi);
              }
              *reinterpret_cast<uint4*>(out + c + i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    // A wait ran out: what is in flight lands (bounded) before TMEM and shared memory go.
    if (warp == 9 && lane == 0)
      for (int u = issued > kStages ? issued - kStages : 0; u < issued; ++u)
        mbar_drain(full(u % kStages), (uint32_t)(u / kStages) & 1u, p.dev_status);
    if (warp == 10 && lane == 0 && q_issued > 0) mbar_drain(q_full, (uint32_t)(q_issued - 1) & 1u, p.dev_status);
    if (warp == 8 && lead) {
      mma_commit(drain_bar);
      mbar_drain(drain_bar, 0u, p.dev_status);
    }
    __syncthreads();
  }
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ------------------------------------------------------------------- join
//
// For each CTA whose share begins an item that others finish: out = sum_k w_k O_k / sum_k w_k l_k,
// w_k = exp2(m_k - max m), over the parts k in the order of the keys.  Few parts: a warp a row;
// many (few rows over a long axis): a block a row, a slice of the parts each warp, the slices
// added in order.  The weights come first, so that the sums' loads wait for nothing.

constexpr int kJoinWarps = 8;
constexpr int kJoinFew = 8;  // parts that one warp takes

template <int D, int NQ>
__global__ void __launch_bounds__(32 * kJoinWarps) attention_join_kernel(const __grid_constant__ Params p) {
  constexpr int E = D / 64;  // float2 of a lane
  __shared__ float2 acc[kJoinWarps][D / 2];
  __shared__ float weights[ATTENTION_MAX_CTAS];
  nvfp4::wait_for_previous_kernel();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Record rec = *reinterpret_cast<const Record*>(p.ws + (size_t)c * 64);
  const int parts = rec.parts, rows = rec.rows * p.group;
  if (parts <= 0) return;
  const int per_tile = kRows / p.group;
  const bool few = parts <= kJoinFew;
  const float* slots = reinterpret_cast<const float*>(p.ws + kRecordBytes) + 2 * (int64_t)c * slot_floats(D, NQ);
  // part 0 is the first CTA's second place, the others are the next CTAs' first
  auto slot_of = [&](int k) { return slots + (k == 0 ? 1 : 2 * k) * slot_floats(D, NQ); };
  const int first = few ? 0 : parts * warp / kJoinWarps, last = few ? parts : parts * (warp + 1) / kJoinWarps;
  const int row0 = few ? (int)blockIdx.y * kJoinWarps + warp : (int)blockIdx.y;
  const int step = few ? (int)gridDim.y * kJoinWarps : (int)gridDim.y;
  for (int i = row0; i < rows; i += step) {
    const int token = i / p.group, g = i - token * p.group;
    const int row = token / per_tile * kRows + token % per_tile * p.group + g;
    // (every warp forms all weights: lane k those of parts k, k + 32, ...)
    constexpr int kMost = (ATTENTION_MAX_CTAS + 31) / 32;
    float2 ml[kMost];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      ml[j] = make_float2(-INFINITY, 0.0f);
      if (lane + 32 * j < parts) ml[j] = *reinterpret_cast<const float2*>(slot_of(lane + 32 * j) + 2 * row);
      top = fmaxf(top, ml[j].x);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    float total = 0.0f, w0 = 0.0f;
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      // (a part of which the row sees no key has l = 0, and O that may be anything)
      const float w = ml[j].y == 0.0f ? 0.0f : exp2_approx((ml[j].x - top) * p.scale);
      if (j == 0) w0 = w;
      if (!few && warp == 0 && lane + 32 * j < parts) weights[lane + 32 * j] = w;
      total += ml[j].y * w;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    if (!few) __syncthreads();
    float2 o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int k = first; k < last; ++k) {
      const float w = few ? __shfl_sync(0xFFFFFFFFu, w0, k) : weights[k];
      const float2* src = reinterpret_cast<const float2*>(slot_of(k) + 2 * NQ * kRows + (int64_t)row * D) + lane;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float2 v = src[32 * e];
        o[e].x += w != 0.0f ? v.x * w : 0.0f;
        o[e].y += w != 0.0f ? v.y * w : 0.0f;
      }
    }
    const float norm = 1.0f / total;
    uint32_t* out = reinterpret_cast<uint32_t*>(p.out + (int64_t)(rec.row0 + token) * p.ld_token +
                                                (rec.head * p.group + g) * p.ld_head);
    if (few) {
#pragma unroll
      for (int e = 0; e < E; ++e) out[lane + 32 * e] = total != 0.0f ? to_bf16x2(o[e].x * norm, o[e].y * norm) : 0u;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) acc[warp][lane + 32 * e] = o[e];
      __syncthreads();
      if (threadIdx.x < D / 2) {
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
          sum.x += acc[w][threadIdx.x].x;
          sum.y += acc[w][threadIdx.x].y;
        }
        out[threadIdx.x] = total != 0.0f ? to_bf16x2(sum.x * norm, sum.y * norm) : 0u;
      }
      __syncthreads();
    }
  }
}

// One map for the caches and for packed keys (one page of all tokens).
bool encode_kv(CUtensorMap* map, const kv_pages& x, const paged_attention_input& in, int box) {
  const cuuint64_t dims[4] = {(cuuint64_t)in.dim, (cuuint64_t)in.kv_heads, (cuuint64_t)in.page_size, (cuuint64_t)in.pages};
  const cuuint64_t strides[3] = {(cuuint64_t)x.ld_head * 2, (cuuint64_t)x.ld_token * 2,
                                 in.pages > 1 ? (cuuint64_t)x.ld_page * 2 : 16};
  const cuuint32_t boxes[4] = {64, 1, (cuuint32_t)box, 1};
  const cuuint32_t each[4] = {1, 1, 1, 1};
  return nvfp4::encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, x.data, dims, strides, boxes, each,
                             CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, int NQ>
int launch(const paged_attention_input& in, const attn_rows& out, void* workspace, int32_t* dev_status,
           cudaStream_t stream) {
  using L = Tile<D, NQ>;
  Params p;
  p.cu = in.cu;
  p.kv_lens = in.block_table != nullptr ? in.kv_lens : nullptr;
  p.table = in.block_table;
  p.ld_table = in.ld_table;
  const int64_t capacity = in.max_pages * in.page_size;
  p.capacity = capacity < 0x7FFFFFFF ? capacity : 0x7FFFFFFF;
  p.tokens = (int)in.tokens;
  p.batch = (int)in.batch;
  p.kv_heads = (int)in.kv_heads;
  p.group = (int)(in.heads / in.kv_heads);
  p.page_size = (int)in.page_size;
  p.page_shift = -1;
  for (int i = 4; i < 17; ++i)
    if (in.page_size == (int64_t)1 << i) p.page_shift = i;
  p.pages = (int)in.pages;
  p.box = kKeys;
  if (in.block_table != nullptr)
    while (in.page_size % p.box != 0) p.box /= 2;
  p.negative = in.scale < 0.0f;
  p.scale = (in.scale < 0.0f ? -in.scale : in.scale) * kLog2e;
  if (!(p.scale >= 1e-37f)) p.scale = 1e-37f;  // (a score that is masked stays so: 0 times -inf is not a number)
  p.out = static_cast<__nv_bfloat16*>(out.data);
  p.ld_token = out.ld_token;
  p.ld_head = out.ld_head;
  p.ws = static_cast<unsigned char*>(workspace);
  p.dev_status = dev_status;

  CUtensorMap mq, mk, mv;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)p.group, (cuuint64_t)p.kv_heads, (cuuint64_t)in.tokens};
  const cuuint64_t strides[3] = {(cuuint64_t)in.q.ld_head * 2, (cuuint64_t)in.q.ld_head * p.group * 2,
                                 (cuuint64_t)in.q.ld_token * 2};
  const cuuint32_t boxes[4] = {64, (cuuint32_t)p.group, 1, (cuuint32_t)(kRows / p.group)};
  const cuuint32_t each[4] = {1, 1, 1, 1};
  if (!nvfp4::encode_tiled(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, in.q.data, dims, strides, boxes, each,
                           CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_kv(&mk, in.k, in, p.box) || !encode_kv(&mv, in.v, in, p.box))
    return NVFP4_ERR_CUDA;
  const void* kern = (const void*)attention_kernel<D, NQ>;
  if (nvfp4::occupancy(kern, kThreads, L::kSmemBytes) < 1) return NVFP4_ERR_CUDA;
  const int sms = nvfp4::sm_count();
  const unsigned grid = (unsigned)(sms < ATTENTION_MAX_CTAS ? sms : ATTENTION_MAX_CTAS);
  void* args[] = {&mq, &mk, &mv, &p};
  if (nvfp4::launch_dependent(kern, dim3(grid), dim3(kThreads), L::kSmemBytes, stream, 1, args) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  void* join_args[] = {&p};
  if (nvfp4::launch_dependent((const void*)attention_join_kernel<D, NQ>, dim3(grid, 8 * NQ), dim3(32 * kJoinWarps), 0, stream, 1,
                              join_args) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return NVFP4_OK;
}

}  // namespace

int launch_attention(const paged_attention_input* in, const attn_rows* out, void* workspace, int32_t* dev_status,
                     cudaStream_t stream) {
  // Two tiles of rows an item where sequences bring more than one tile's on average.
  const int64_t rows = in->tokens * (in->heads / in->kv_heads);
  const bool two = in->dim <= 128 && rows > kRows * in->batch;
  switch (in->dim) {
    case 64: return two ? launch<64, 2>(*in, *out, workspace, dev_status, stream)
                        : launch<64, 1>(*in, *out, workspace, dev_status, stream);
    case 128: return two ? launch<128, 2>(*in, *out, workspace, dev_status, stream)
                         : launch<128, 1>(*in, *out, workspace, dev_status, stream);
    default: return launch<256, 1>(*in, *out, workspace, dev_status, stream);
  }
}
