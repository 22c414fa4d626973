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
//   warp 8      allocates TMEM, issues the MMAs
//   warp 9      finds the items and loads K (TMA)
//   warp 10     loads Q and V
//
// Schedule: the items of all sequences and heads are laid end to end on a line, item_cost units
// for an item's start and end, then 128 for a tile of keys, and every CTA takes an equal share of
// it, whatever the lengths: each finds its share from the lengths on the device.  A longer item
// that a share's border cuts leaves the parts' (maximum, sum, O) in the workspace, FP32, and
// a second kernel joins them in the order of the keys.  The borders depend on the lengths
// alone, so results do not depend on timing.
//
// Keys that a row does not see get weight 0 by selection, and P V stops at the last one that
// some row of the item sees (rounded up to 16, values behind it zeroed): what lies there, in
// other sequences or unused slots, does not matter.
//
// What bounds it, and what it measured (fractions of a cuBLAS product's burst rate and of a
// copy's):
//   long prompts   the chain S -> softmax -> P V of each tile of rows: 3000 cycles a tile of keys
//                  for 2048 of MMAs, as S of the next tile waits for P V of this one, whose P lies
//                  over S (heads of 128: O and S of two tiles fill TMEM; heads of 64 would leave P
//                  a place of its own).  16384 tokens, 32 / 8 heads of 128: 1.42 ms, 1550 TFLOP/s
//                  (0.81), 1.53 (0.75) in long runs, where power limits it; 8192 tokens 383 us
//                  (0.75), heads of 64 331 us.  Heads of 256, S twice in TMEM: 8192 tokens, 32 / 4
//                  heads, 650 us, 1690 TFLOP/s (0.88).
//   short prompts  an item's start and end, about 4500 cycles: its first loads, the last P V, O's
//                  way through registers.  11 prompts of up to 1900 tokens, 28 / 4 heads: 74 us
//                  (0.38); one of 77 tokens: 7.5 us.
//   the cache      HBM: 64 sequences of up to 16000 keys, up to 5 queries each: 159 us, 6.1 TB/s
//                  (0.90); one token over 4000 keys, 32 / 4 heads of 256: 13.4 us, of which finding
//                  the share and the join are 3 us each.
#include <cuda_bf16.h>

#include <type_traits>

#include "tc.cuh"

namespace {

using namespace nvfp4::tc;
using nvfp4::ld_ro;

constexpr int kRows = 128;                    // MMA rows of a tile of queries
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);  // (three of the last four work)
constexpr int kDescs = 4;                     // item descriptors in flight
// An item's start and end, in the keys that its products would take meanwhile.  With full tiles of
// rows what was measured (us):              64    128    192    256    320    384    512    640
//   heads of 128, 11 packed prompts        93     76     72     71     72     75     77     81
//   heads of 256, 8192 tokens             864    825    772    722    690    650    639    641
// and with few rows, where keys arrive no faster, no difference up to 256 and 1 % more at 512.
constexpr int kItemCostFew = 128, kItemCost = 224, kItemCostWide = 512;
// Items of full tiles of rows are not cut up to so many tiles of keys: parts of 256 rows cost more
// than shares that differ, and where no item is longer there is nothing to join.  Prompts of 32 / 8
// heads of 128, cut and whole: 512 tokens 20 and 13 us, 1024 30 and 20, eight of 1024 (28 / 4 heads)
// 81 and 73, 11 of up to 1900 71 and 73; up to 12 tiles 2048 tokens 47 and 52.
// With few rows parts are small: cut always (whole up to 4 tiles: one token over 300 keys 9.0, 10.3).
constexpr int kWhole = 8;
constexpr int kMinShare = kKeys;              // of a CTA, where there is that little
constexpr float kRescale = 8.0f;              // log2 of what the maximum may lag behind
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int NQ>
struct Tile {
  // Units of the rings: 128 keys of as many dims.
  static constexpr int kDims = D < 128 ? D : 128, kUnits = D / kDims;  // (units of a tile)
  static constexpr int kBytes = kKeys * kDims * 2;
  static constexpr int kQTile = kRows * D * 2;
  static constexpr int kQBytes = NQ * kQTile;
  static constexpr int kXchBytes = NQ == 1 ? 2 * 2 * kRows * 4 : 0;
  static constexpr int kCols = NQ == 2 ? kKeys : kKeys / 2;  // of S, a softmax thread's
  static constexpr int kOut = NQ == 2 ? D : D / 2;           // of O, a softmax thread's
  static constexpr int kDescBytes = kDescs * 64;
  static constexpr int kRest = kXchBytes + kDescBytes + 512;
  static constexpr int kFit = 227 * 1024 - kQBytes - kRest;
  static constexpr int kStagesV = D == 64 ? 5 : 3;
  static constexpr int kLeft = kFit / kBytes - kStagesV;
  static constexpr int kStagesK = kLeft < 5 ? kLeft : 5;
  static constexpr int kStages = kStagesK + kStagesV, kRing = kStages * kBytes;
  static constexpr size_t kSmemBytes = (size_t)kQBytes + kRing + kRest;
  static_assert(kStagesK >= 2 && kStagesK >= kUnits && kStagesV > kUnits, "rings");
  static_assert(kBytes % 1024 == 0, "swizzled tiles start on 1 KB");
  static_assert(2 * kKeys + NQ * D <= 512, "TMEM");
};

struct Params {
  const int32_t* cu;
  const int32_t* kv_lens;  // nullptr: prompts
  const int32_t* table;
  int64_t ld_table, capacity;  // tokens of a table row
  int tokens, batch, kv_heads, group;
  int per_tile, per_item;      // tokens of a tile of rows, and of an item
  int page_size, page_shift;   // tokens of a page; log2 of it, or -1
  int box;                     // tokens of a TMA box
  bool full_tiles;             // most tiles of rows are full
  int pages;
  float scale;                 // |scale| log2 e, never 0
  int negative;
  __nv_bfloat16* out;
  int64_t ld_token, ld_head;
  bool wide;                   // rows of the output start on 32 bytes
  unsigned char* ws;
  int32_t* dev_status;
};

struct Sequence {
  int begin, n;  // rows of q
  int off;       // position of the first query (may be negative)
};

// What the roles need of an item, in shared memory.
struct __align__(16) Item {
  int row0, rows;   // tokens: first row of q, number (0: no more items)
  int pos0, end;    // position of the first; keys that some row sees
  int head, first;  // key head; first tile of this part
  int last, slot;   // past its last tile; -1: the whole item, else the part's place
  int64_t table;    // of its sequence: the block table's row,
  int begin;        // the first token of packed prompts
};

// An item cut by a share's border, for the kernel that joins its parts.
struct Record {
  int parts, row0, rows, head;
};

__host__ __device__ constexpr int64_t slot_floats(int d, int nq) { return (int64_t)nq * kRows * (d + 2); }
constexpr size_t kRecordBytes = (size_t)ATTENTION_MAX_CTAS * 64;

// Offsets and length as they are in memory, and what they come to within the tensors.
struct Raw {
  int a, b, cached;
};
__device__ __forceinline__ Raw load_raw(const Params& p, int s) {
  return Raw{ld_ro(p.cu + s), ld_ro(p.cu + s + 1), p.kv_lens != nullptr ? ld_ro(p.kv_lens + s) : 0};
}
__device__ __forceinline__ bool consistent(const Params& p, const Raw& r) {
  return r.a >= 0 && r.b <= p.tokens && r.a <= r.b && r.cached <= p.capacity;
}
__device__ __forceinline__ Sequence sequence(const Params& p, const Raw& r) {
  Sequence q;
  q.begin = min(max(r.a, 0), p.tokens);
  q.n = max(min(max(r.b, 0), p.tokens) - q.begin, 0);
  q.off = (p.kv_lens != nullptr ? (int)min((int64_t)max(r.cached, 0), p.capacity) : q.n) - q.n;
  return q;
}
// (64-bit division takes several times a 32-bit one's time; out of line for the instruction cache)
__device__ __noinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line: item t of a (sequence, head) starts `before(t)` behind its head's start.
struct Line {
  int per;       // tokens of an item
  int items;
  int64_t base;  // length of item 0
  int64_t length;
  __device__ __forceinline__ Line(const Sequence& q, int per_item, int item_cost) {
    per = per_item;
    items = q.n <= per ? (q.n > 0) : (q.n + per - 1) / per;
    const int cached = max(q.off, 0);
    base = (int64_t)cached + per + item_cost;
    length = items > 0 ? before(items - 1) + cached + q.n + item_cost : 0;
  }
  __device__ __forceinline__ int64_t before(int t) const {
    return t * base + (int64_t)per * ((int64_t)t * (t - 1) / 2);
  }
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
// Four MMAs along 64 keys (a half of P): 16 keys in 8 columns; V 16 rows of 128 bytes apart.  Of
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
// 32 bytes to one address: whole sectors.  Past the L1, where a warp's store of 32 rows would
// take a line each: 8192 tokens 32/8/128 407 -> 389 us, 32/4/256 875 -> 839 us, packed prompts
// 88 -> 80 us.
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
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

// The roles' code has to fit the SM's instruction cache together (32 KB; beyond it a warp gets an
// instruction every 2.6 cycles), so each part stands once, K and V are loaded by the same code, and
// loops are rolled where a trip takes longer than fetching its instructions (30 packed prompts of
// 300 tokens: 77 us with 23 % of the instruction requests missing, 65 us with 10 %).
template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Params p) {
  using L = Tile<D, NQ>;
  constexpr int kStages = L::kStages, kUnits = L::kUnits;
  constexpr int kMmaWarp = kSoftmaxWarps, kWarpK = kMmaWarp + 1, kWarpV = kMmaWarp + 2;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* const ring_ptr = smem + L::kQBytes;
  float* const xch = reinterpret_cast<float*>(ring_ptr + L::kRing);
  Item* const items = reinterpret_cast<Item*>(reinterpret_cast<unsigned char*>(xch) + L::kXchBytes);
  const uint32_t q_smem = smem_u32(smem), ring = q_smem + L::kQBytes;  // K's, then V's
  const uint32_t bars = smem_u32(items) + L::kDescBytes;
  // stages of the two rings: K's, then V's
  constexpr int kK = L::kStagesK, kV = L::kStagesV;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto stage_k = [&](int unit) { return unit % kK; };
  auto stage_v = [&](int unit) { return kK + unit % kV; };
  auto offset = [&](int s) { return (uint32_t)(s * L::kBytes); };
  auto item_full = [&](int i) { return bars + 8u * (2 * kStages + i); };
  auto item_empty = [&](int i) { return bars + 8u * (2 * kStages + kDescs + i); };
  constexpr int kFixed = 2 * kStages + 2 * kDescs;
  const uint32_t q_full = bars + 8u * kFixed, q_empty = bars + 8u * (kFixed + 1);
  auto s_full = [&](int b) { return bars + 8u * (kFixed + 2 + b); };
  auto p_full = [&](int b) { return bars + 8u * (kFixed + 4 + b); };
  auto pv_done = [&](int t) { return bars + 8u * (kFixed + 6 + t); };
  const uint32_t drain_bar = bars + 8u * (kFixed + 8);
  static_assert(8 * (kFixed + 9) + 8 <= 512, "shared memory behind the items");
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(reinterpret_cast<unsigned char*>(items) + L::kDescBytes + 8 * (kFixed + 9));
  volatile uint32_t* abort = tmem_slot + 1;
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
      mbar_init(p_full(b), kSoftmaxWarps / NQ);
      mbar_init(pv_done(b), 1);
    }
    mbar_init(drain_bar, 1);
    *abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == kWarpK && lane < 3) {
    const CUtensorMap* m = lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all of the SM's columns: they start at 0 (a constant for the MMAs' addresses)
  constexpr uint32_t tmem = 0;
  if (*tmem_slot != tmem) nvfp4::report(p.dev_status, NVFP4_ERR_CUDA);
  const int per_tile = p.per_tile;
  int issued = 0, q_issued = 0;          // units and Q loads issued (the loading warps)
  const uint32_t lead = elect_one();     // the lane that issues for a warp
  nvfp4::wait_for_previous_kernel();

  // Where this lane's box of a tile lies: its page, and its first token there; how many boxes
  // some row sees (the others are not loaded: their scores are masked whatever they are, and P V
  // stops before them).
  struct Place {
    int page, token, count;
  };
  auto place_of = [&](const Item& it, int tile) -> Place {
    const int count = (min(it.end - tile * kKeys, kKeys) + p.box - 1) / p.box;
    if (lane >= count) return Place{0, 0, count};
    const int j = tile * kKeys + lane * p.box;
    if (p.table == nullptr) return Place{0, it.begin + j, count};
    const int entry = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
    const int id = ld_ro(p.table + it.table + entry);
    return Place{id, j - entry * p.page_size, count};
  };
  if (warp == kWarpK || warp == kWarpV) {
    // ----------------------------------------- K and V loads, a warp each, all lanes together;
    // that of K finds the items, that of V loads their Q
    const bool keys = warp == kWarpK;
    const CUtensorMap* const map = keys ? &map_k : &map_v;
    const int ring0 = keys ? 0 : kK, stages = keys ? kK : kV;
    int slot = 0, phase = 1;  // of the warp's ring
    bool ok = true;
    auto load_tile = [&](int key_head, const Place& at) {
      int page = at.page;
      if (page < 0 || page >= p.pages) {
        nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
        page = p.pages;  // (read as zeros)
      }
      const int head = uniform(key_head), count = uniform(at.count);
      constexpr int kBlocks = L::kDims / 64;  // swizzled columns of 128 bytes
#pragma unroll 1
      for (int u = 0; u < kUnits; ++u) {
        const int s = uniform(ring0 + slot);
        ok = mbar_wait(empty(s), phase, abort, p.dev_status);  // (the first round passes: phase 1 is before 0)
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return;
        if (++slot == stages) {
          slot = 0;
          phase ^= 1;
        }
        const bool withheld = nvfp4::kWithhold && keys && issued == 0;  // (test build: by each CTA)
        ++issued;
        if (withheld) continue;
        if (lead) mbar_arrive_expect_tx(full(s), (uint32_t)(count * p.box * 128 * kBlocks));
        __syncwarp();
        const uint32_t dst = ring + offset(s);
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
          const int pg = __shfl_sync(0xFFFFFFFFu, page, i), tk = __shfl_sync(0xFFFFFFFFu, at.token, i);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
            tma_load_4d(lead, dst + (uint32_t)(b * (kKeys * 128) + i * p.box * 128), map, u * L::kDims + b * 64, head, tk,
                        pg, full(s));
        }
      }
    };
    // This CTA's share [x0, x1) of the line: a lane a run of neighbouring sequences, whose offsets
    // it finds in the L1 but for the first of a cache line (every 32nd sequence to a lane, a miss
    // each: 1000 sequences of 50 keys 142 us instead of 122).  (By this warp alone: the others get
    // their items from it, and up to some hundreds of sequences take less than the block's barriers.)
    const int item_cost = NQ == 2 ? kItemCost : D == 256 && p.full_tiles ? kItemCostWide : kItemCostFew;
    const int whole = NQ == 2 || (D == 256 && p.full_tiles) ? kWhole : 0;
    const int run = (p.batch + 31) >> 5;
    int64_t chunk = 0;  // of the lane's sequences
    Sequence q{};       // the last of them
    bool sound = true;
    if (keys) {
      const int end = min(p.batch, (lane + 1) * run);
      for (int s = lane * run; s < end; ++s) {
        const Raw raw = load_raw(p, s);
        q = sequence(p, raw);
        chunk += p.kv_heads * Line(q, p.per_item, item_cost).length;
        sound = sound && consistent(p, raw);
      }
    }
    if (blockIdx.x == 0 && !sound) nvfp4::report(p.dev_status, NVFP4_ERR_INDEX);
    auto scan = [&](int64_t v) -> int64_t {  // inclusive prefix sums over the lanes
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += o;
      }
      return v;
    };
    int64_t upto = p.batch > 1 ? scan(chunk) : chunk;
    const int64_t total = __shfl_sync(0xFFFFFFFFu, upto, p.batch > 1 ? 31 : 0);
    // total = shares * each + rest: the first `rest` shares are one longer
    const int shares = total >= (int64_t)kMinShare * gridDim.x ? (int)gridDim.x : max((int)((uint32_t)total / kMinShare), 1);
    const int64_t each = quotient(total, shares), rest = total - each * shares;
    auto border = [&](int c) -> int64_t { return c < shares ? c * each + min((int64_t)c, rest) : total; };
    const int64_t x0 = border((int)blockIdx.x), x1 = border((int)blockIdx.x + 1);
    int seq = p.batch, head = 0, t = 0;
    int64_t head_at = 0;
    if (keys && x0 < x1) {  // the sequence, head and item that x0 lies in
      int who = __ffs((int)__ballot_sync(0xFFFFFFFFu, upto > x0)) - 1;
      int64_t at = __shfl_sync(0xFFFFFFFFu, upto - chunk, who);
      seq = who * run;
      if (run > 1) {  // within the run, 32 sequences at a time
        const int end = min(p.batch, seq + run);
        for (int base = seq; base < end; base += 32) {
          q = base + lane < end ? sequence(p, load_raw(p, base + lane)) : Sequence{};
          chunk = p.kv_heads * Line(q, p.per_item, item_cost).length;
          upto = scan(chunk);
          const unsigned past = __ballot_sync(0xFFFFFFFFu, at + upto > x0);
          if (past != 0u) {
            who = __ffs((int)past) - 1;
            seq = base + who;
            at += __shfl_sync(0xFFFFFFFFu, upto - chunk, who);
            break;
          }
          at += __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
      }
      q.begin = __shfl_sync(0xFFFFFFFFu, q.begin, who);
      q.n = __shfl_sync(0xFFFFFFFFu, q.n, who);
      q.off = __shfl_sync(0xFFFFFFFFu, q.off, who);
      const Line line(q, p.per_item, item_cost);
      head = (int)quotient(x0 - at, line.length);
      head_at = at + head * line.length;
      int lo = 0, hi = line.items;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (head_at + line.before(mid) <= x0)
          lo = mid;
        else
          hi = mid;
      }
      t = lo;
    }
    Raw next_raw{};  // of sequence seq + 1, once `fetched`: on its way while seq's items are loaded
    bool fetched = false;
    // The next part of this CTA's share, or rows = 0.
    struct Part {
      Item it;
      int record;  // parts of the whole item, where this is the first of several
    };
    auto advance = [&]() -> Part {
      Part r{};
      r.it.rows = 0;
      while (seq < p.batch) {
        const Line line(q, p.per_item, item_cost);
        if (t >= line.items) {
          t = 0;
          head_at += line.length;
          if (q.n == 0 || ++head >= p.kv_heads) {
            head = 0;
            if (++seq < p.batch) {
              if (!fetched) next_raw = load_raw(p, seq);
              q = sequence(p, next_raw);
              fetched = seq + 1 < p.batch;
              if (fetched) next_raw = load_raw(p, seq + 1);
            }
          }
          continue;
        }
        const int64_t at = head_at + line.before(t) + item_cost;  // of tile 0
        if (at - item_cost >= x1) break;
        const int row = t * line.per, rows = min(line.per, q.n - row);
        const int end = max(q.off + row + rows, 0);
        const int tiles = max((int)(((uint32_t)end + kKeys - 1) / kKeys), 1);
        int64_t a = at >= x0 ? 0 : (x0 - at + kKeys - 1) >> 7;
        int64_t b = at >= x1 ? 0 : (x1 - at + kKeys - 1) >> 7;
        static_assert(kKeys == 1 << 7, "shift");
        if (tiles <= whole) {  // all of it to the share that its middle lies in
          const int64_t middle = at + (tiles * kKeys - item_cost) / 2;
          if (middle >= x1) break;
          a = middle < x0 ? tiles : 0;
          b = tiles;
        }
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
        r.it.table = seq * p.ld_table;
        r.it.begin = q.begin;
        if (a == 0 && b < tiles) {
          const int64_t last_tile = at + (int64_t)(tiles - 1) * kKeys, longer = rest * (each + 1);
          const int owner = (int)(last_tile < longer ? quotient(last_tile, each + 1) : rest + quotient(last_tile - longer, each));
          r.record = owner - (int)blockIdx.x + 1;
        }
        break;
      }
      return r;
    };
    Part cur{}, recorded{};
    int record = 0, count = 0, tile = 0;  // items; tile whose place comes next
    Place at{};                           // of the tile before it, once there is one
    bool have = false;
    for (;;) {
      const bool more = tile < cur.it.last;
      Place next{};  // (on its way while the tile before is loaded)
      if (more) next = place_of(cur.it, tile++);
      if (have) {
        load_tile(cur.it.head, at);
        if (!ok) break;
      } else if (!keys && more) {
        if (count > 1) ok = mbar_wait(q_empty, count & 1, abort, p.dev_status);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        q_issued = count;
        if (lead) mbar_arrive_expect_tx(q_full, (uint32_t)(NQ * (D / 64) * per_tile * p.group * 128));
        __syncwarp();
        const int head = uniform(cur.it.head), row0 = uniform(cur.it.row0);
#pragma unroll
        for (int t = 0; t < NQ; ++t)
#pragma unroll
          for (int b = 0; b < D / 64; ++b)
            tma_load_4d(lead, q_smem + (uint32_t)(t * L::kQTile + b * (kRows * 128)), &map_q, b * 64, 0, head,
                        row0 + t * per_tile, q_full);
      }
      at = next;
      have = more;
      if (more) continue;
      const int i = count % kDescs;  // the next item
      if (keys) {
        cur = advance();
        if (count >= kDescs) ok = mbar_wait(item_empty(i), (count / kDescs - 1) & 1, abort, p.dev_status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if (lane == 0) {
          items[i] = cur.it;
          mbar_arrive(item_full(i));
        }
        __syncwarp();
        if (cur.record) {
          record = cur.record;
          recorded = cur;
        }
      } else {
        ok = mbar_wait(item_full(i), (count / kDescs) & 1, abort, p.dev_status);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        cur.it = items[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty(i));
      }
      ++count;
      if (uniform(cur.it.rows) == 0) break;
      tile = uniform(cur.it.first);
    }
    if (keys && lane == 0) {
      Record* rec = reinterpret_cast<Record*>(p.ws + (size_t)blockIdx.x * 64);
      *rec = Record{record, recorded.it.row0, recorded.it.rows, recorded.it.head};
    }
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------------------- MMAs
    // Steps g = 0, 1, ... over all items: NQ = 2: tile of keys g / 2, rows g % 2; NQ = 1: tile
    // g.  S of step g into buffer g % 2.  Two cursors, S's two steps ahead: S of step g + 2 is
    // issued behind P V of step g, which reads the same buffer.  (One warp for both tiles of rows:
    // two fell into step, both softmaxes at once, then both products; 1.5 -> 2.2 ms.)
    const uint32_t idesc_s = idesc_bf16(kKeys, false) | (p.negative ? 1u << 13 : 0u);  // (-Q: a negative scale)
    constexpr uint32_t kIdescO = idesc_bf16(L::kDims, true);
    bool ok = true;
    struct Cursor {
      int count, tile, first, last, end, rows;  // items fetched; of the last of them
      int x, row, g;                            // tiles before; tile of rows; step
    };
    Cursor cs{}, cp{};  // of S, of P V
    auto fetch = [&](Cursor& c, bool release) {
      const int i = c.count % kDescs;
      ok = mbar_wait(item_full(i), (c.count / kDescs) & 1, abort, p.dev_status);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) return;
      const Item& it = items[i];
      c.rows = uniform(it.rows);
      c.tile = c.first = uniform(it.first);
      c.last = uniform(it.last);
      c.end = uniform(it.end);
      ++c.count;
      __syncwarp();
      if (release && lane == 0) mbar_arrive(item_empty(i));
    };
    auto wait = [&](uint32_t bar, uint32_t phase) {
      ok = ok && mbar_wait(bar, phase, abort, p.dev_status);
      ok = __all_sync(0xFFFFFFFFu, ok);
    };
    auto step = [&](Cursor& c, bool release) {
      ++c.g;
      if (NQ == 2 && c.row == 0) {
        c.row = 1;
        return;
      }
      c.row = 0;
      ++c.x;
      if (++c.tile == c.last) fetch(c, release);
    };
    auto issue_s = [&]() {
      if (cs.tile == cs.first && cs.row == 0) wait(q_full, (cs.count - 1) & 1);
      const uint32_t d = tmem + (uint32_t)(cs.g & 1) * kKeys;
      const bool last_use = cs.row == NQ - 1;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int unit = cs.x * kUnits + u, s = stage_k(unit);
        if (cs.row == 0) wait(full(s), (unit / kK) & 1);
        if (!ok) return;
        tc_fence_after();
        constexpr int kBlocks = L::kDims / 64;
        const uint32_t a = desc_low(q_smem + (uint32_t)(cs.row * L::kQTile + u * kBlocks * (kRows * 128)));
        const uint32_t b = desc_low(ring + offset(s));
#pragma unroll
        for (int c = 0; c < kBlocks; ++c)
          mma_ss4(lead, d, a + c * (kRows * 128 >> 4), b + c * (kKeys * 128 >> 4), idesc_s, (u > 0 || c > 0) ? 1u : 0u);
        if (u == kUnits - 1) commit(lead, s_full(cs.g & 1));
        if (last_use) commit(lead, empty(s));
      }
      if (last_use && cs.tile + 1 == cs.last) commit(lead, q_empty);
      step(cs, false);
    };
    auto issue_pv = [&]() {
      const int steps = (min(max(cp.end - cp.tile * kKeys, 1), kKeys) + 15) / 16;  // of 16 keys
      const uint32_t a = tmem + (uint32_t)(cp.g & 1) * kKeys, o = tmem + 2 * kKeys + (uint32_t)(cp.row * D);
      const bool last_use = cp.row == NQ - 1;
      wait(p_full(cp.g & 1), (cp.g >> 1) & 1);
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int unit = cp.x * kUnits + u, s = stage_v(unit);
        if (cp.row == 0) wait(full(s), (unit / kV) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t b = desc_low_v(ring + offset(s));
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mma_ts4(lead, o + (uint32_t)(u * L::kDims), a + (NQ == 2 ? kKeys / 4 : kKeys / 2) * h, b + 512 * h, kIdescO,
                  (cp.tile > cp.first || h > 0) ? 1u : 0u, steps - 4 * h);
        if (u == kUnits - 1) commit(lead, pv_done(cp.g & 1));
        if (last_use) commit(lead, empty(s));
      }
      step(cp, true);
    };
    fetch(cs, false);
    if (ok) fetch(cp, true);
    while (ok && cp.rows) {
      if (cs.rows && cs.g < cp.g + 2)
        issue_s();
      else
        issue_pv();
    }
  } else if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------------ softmax
    // NQ = 2: a row of one tile a thread.  NQ = 1: a row and half of the keys, and of O's columns.
    constexpr int kCols = L::kCols, kOut = L::kOut, kChunks = kCols / 32;
    const int half = warp >> 2;                                      // warpgroup
    const int t = NQ == 2 ? half : 0;                                // tile of rows
    const int r = (warp & 3) * 32 + lane;                            // row of the tile
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int key0 = NQ == 2 ? 0 : half * kCols;  // first key of the thread's
    const int token = r / p.group, g = r - token * p.group;
    const uint32_t o_addr = lanes + 2 * kKeys + (uint32_t)(NQ == 2 ? t * D : half * kOut);
    const float scale = p.scale;
    const uint64_t scale2 = pack2(__float_as_uint(scale), __float_as_uint(scale));
    // P V of the CTA's tile i is complete.  A barrier per buffer of S: the wait before last on
    // one, two steps ago, is known to be over from S of this tile, so parities suffice.
    auto wait_pv = [&](int i) {
      return mbar_wait(pv_done(NQ == 2 ? t : i & 1), (NQ == 2 ? i : i >> 1) & 1, abort, p.dev_status);
    };
    bool ok = true;
    int x = 0, exchanges = 0;
    // Whether to go on: NQ = 1: all warps alike, so that they leave together, at a barrier.
    auto agree = [&]() {
      if constexpr (NQ == 1)
        ok = softmax_agree(ok);
      else
        ok = __all_sync(0xFFFFFFFFu, ok);
    };
    // NQ = 1: the other half's value of the row (two places in turn)
    auto exchange = [&](float own) -> float {
      float* at = xch + (exchanges & 1) * 2 * kRows + r;
      ++exchanges;
      at[half * kRows] = own;
      agree();
      return at[(half ^ 1) * kRows];
    };
    for (int count = 0;; ++count) {
      const int di = count % kDescs;
      ok = ok && mbar_wait(item_full(di), (count / kDescs) & 1, abort, p.dev_status);
      agree();
      if (!ok) break;
      const Item it = items[di];
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty(di));
      if (it.rows == 0) break;
      const bool valid = token < per_tile && t * per_tile + token < it.rows;
      const bool busy = __any_sync(0xFFFFFFFFu, valid);  // this warp has rows
      const int limit = valid ? it.pos0 + t * per_tile + token + 1 : 0x7FFFFFFF;  // keys that the row sees
      float m = -INFINITY, l = 0.0f, top = -INFINITY;
      for (int tile = it.first; tile < it.last; ++tile, ++x) {
        const int b = NQ == 2 ? t : x & 1;
        ok = ok && mbar_wait(s_full(b), (NQ == 2 ? x : x >> 1) & 1, abort, p.dev_status);
        if (NQ == 2) {
          agree();
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t s_addr = lanes + (uint32_t)(b * kKeys + key0);  // (P goes over it, packed)
        const int seen = limit - tile * kKeys - key0;
        uint32_t s[kChunks][32];
        top = -INFINITY;
        if (busy) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) tmem_issue(s_addr + 32 * c, s[c]);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) tmem_wait(s[c]);
          if (__any_sync(0xFFFFFFFFu, seen < kCols)) {
            // (a bit a key, and only the 32s that some row does not see all of)
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const int n = seen - 32 * c;
              if (__any_sync(0xFFFFFFFFu, n < 32)) {
                const uint32_t keep = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!(keep >> i & 1u)) s[c][i] = 0xFF800000u;
              }
            }
          }
          float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kCols; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              most[e] = max3(most[e], __uint_as_float(s[(i + 2 * e) / 32][(i + 2 * e) % 32]),
                             __uint_as_float(s[(i + 2 * e + 1) / 32][(i + 2 * e + 1) % 32]));
          // (no row: whatever S holds there, O is not rescaled for it)
          top = valid ? max3(fmaxf(most[0], most[1]), most[2], most[3]) : 0.0f;
        }
        if constexpr (NQ == 1) {
          top = fmaxf(top, exchange(top));
          if (!ok) break;
        }
        if (busy) {
          // the reference maximum: raised for the whole warp once a row needs it
          const float raised = fmaxf(m, top);
          const bool raise = __any_sync(0xFFFFFFFFu, (raised - m) * scale > kRescale);  // (no key seen: not a number)
          float keep = 1.0f;
          if (raise) {
            keep = m == -INFINITY ? 0.0f : exp2_approx((m - raised) * scale);
            l *= keep;
            m = raised;
          }
          const float shift = m == -INFINITY ? 0.0f : -m * scale;
          const uint64_t shift2 = pack2(__float_as_uint(shift), __float_as_uint(shift));
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
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
            tmem_store(s_addr + 16 * c, w);
          }
          float s0f, s1f;
          unpack2(add2(sum[0], sum[1]), s0f, s1f);
          l += s0f + s1f;
          if (raise && tile > it.first) {
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
          tmem_store_wait();
        }
        // Values behind the last key that any row sees may be anything: zeros for those of
        // them that the last 16 keys of P V take in.  (NQ = 2: by the first tile of rows' threads:
        // the second's P V is issued behind theirs.)
        if (it.end - tile * kKeys < kKeys && t == 0) {
          const int from = max(it.end - tile * kKeys, 0), to = (max(from, 1) + 15) / 16 * 16;
          constexpr int threads = 32 * kSoftmaxWarps / NQ;
          // A stage's barrier tells this load from the one before only once that one is complete:
          // V's of three tiles before is, from S of this tile; with two units a tile and three
          // stages it may be the tile's before.
          if (kUnits == 2 && x > 0) ok = ok && wait_pv(x - 1);
          constexpr int kBlocks = L::kDims / 64;
#pragma unroll 1
          for (int u = 0; u < kUnits; ++u) {
            const int unit = x * kUnits + u, sv = stage_v(unit);
            ok = ok && mbar_wait(full(sv), (unit / kV) & 1, abort, p.dev_status);
            unsigned char* v = ring_ptr + offset(sv);
            if (ok)
#pragma unroll 1
              for (int i = from * 8 * kBlocks + (int)threadIdx.x; i < to * 8 * kBlocks; i += threads) {
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
      ok = ok && wait_pv(x - 1);
      if constexpr (NQ == 1) {
        l += exchange(l);
        if (!ok) break;
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
      tc_fence_after();
      if (busy && ok) {
        float* part = nullptr;
        __nv_bfloat16* out = nullptr;
        if (it.slot < 0) {
          out = p.out + (int64_t)(it.row0 + t * per_tile + token) * p.ld_token + (it.head * p.group + g) * p.ld_head +
                (NQ == 1 ? half * kOut : 0);
        } else {
          float* slot = reinterpret_cast<float*>(p.ws + kRecordBytes) + (2 * (int64_t)blockIdx.x + it.slot) * slot_floats(D, NQ);
          const int row = t * kRows + r;
          if (valid && (NQ == 2 || half == 0)) *reinterpret_cast<float2*>(slot + 2 * row) = make_float2(m, l);
          // eight columns of all rows, then the next eight: a warp's store is contiguous
          part = slot + 2 * NQ * kRows + ((NQ == 1 ? half * (kOut / 8) * NQ * kRows : 0) + row) * 8;
        }
        // (a row that sees nothing: 0, whatever O holds)
        const float norm = it.slot < 0 ? 1.0f / l : 1.0f;
        const bool nothing = it.slot < 0 && l == 0.0f;
#pragma unroll 1
        for (int c = 0; c < kOut; c += 32) {
          uint32_t o[32];
          tmem_issue(o_addr + c, o);
          tmem_wait(o);
          if (!valid) continue;
          if (part != nullptr) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) store32(part + (c + i) * NQ * kRows, o + i);
          } else {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = nothing ? 0u : to_bf16x2(__uint_as_float(o[2 * i]) * norm, __uint_as_float(o[2 * i + 1]) * norm);
            if (p.wide) {
              store32(out + c, w);
              store32(out + c + 16, w + 8);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                reinterpret_cast<uint4*>(out + c)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
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
    if ((warp == kWarpK || warp == kWarpV) && lane == 0) {
      const int ring0 = warp == kWarpK ? 0 : kK, stages = warp == kWarpK ? kK : kV;
      for (int u = issued > stages ? issued - stages : 0; u < issued; ++u)
        mbar_drain(full(ring0 + u % stages), (uint32_t)(u / stages) & 1u, p.dev_status);
      if (q_issued > 0) mbar_drain(q_full, (uint32_t)(q_issued - 1) & 1u, p.dev_status);
    }
    if (warp == kMmaWarp && lead) {
      mma_commit(drain_bar);
      mbar_drain(drain_bar, 0u, p.dev_status);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) {
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
// Parts that one warp takes: where each row has a block of its own (one token over 1000 keys 9.4 us,
// up to 8 parts by a warp 11.7), and where rows are more (20 rows 11.9 us, up to 4 parts 12.3).
constexpr int kJoinFewRows = 2, kJoinFew = 8;

template <int D, int NQ>
__global__ void __launch_bounds__(32 * kJoinWarps) attention_join_kernel(const __grid_constant__ Params p) {
  constexpr int kQuads = D / 4, E = (kQuads + 31) / 32;  // float4 of a row, of a lane
  __shared__ float4 acc[kJoinWarps][kQuads];
  __shared__ float weights[ATTENTION_MAX_CTAS];
  nvfp4::wait_for_previous_kernel();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Record rec = *reinterpret_cast<const Record*>(p.ws + (size_t)c * 64);
  const int parts = rec.parts, rows = rec.rows * p.group;
  if (parts <= 0) return;
  const int per_tile = p.per_tile;
  const bool few = parts <= (rows <= (int)gridDim.y ? kJoinFewRows : kJoinFew);
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
    float4 o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [](float4& a, const float4& v, float w) {
      a.x += v.x * w;
      a.y += v.y * w;
      a.z += v.z * w;
      a.w += v.w * w;
    };
#pragma unroll 4
    for (int k = first; k < last; ++k) {
      const float w = few ? __shfl_sync(0xFFFFFFFFu, w0, k) : weights[k];
      const float* src = slot_of(k) + 2 * NQ * kRows + row * 8;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int quad = lane + 32 * e;  // (half of eight columns)
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (quad < kQuads && w != 0.0f)
          v = *reinterpret_cast<const float4*>(src + (int64_t)(quad / 2) * (NQ * kRows * 8) + quad % 2 * 4);
        add(o[e], v, w);
      }
    }
    const float norm = 1.0f / total;
    uint2* out = reinterpret_cast<uint2*>(p.out + (int64_t)(rec.row0 + token) * p.ld_token + (rec.head * p.group + g) * p.ld_head);
    auto finish = [&](const float4& v) {
      return total != 0.0f ? make_uint2(to_bf16x2(v.x * norm, v.y * norm), to_bf16x2(v.z * norm, v.w * norm)) : make_uint2(0u, 0u);
    };
    if (few) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (lane + 32 * e < kQuads) out[lane + 32 * e] = finish(o[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (lane + 32 * e < kQuads) acc[warp][lane + 32 * e] = o[e];
      __syncthreads();
      if (threadIdx.x < kQuads) {
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) add(sum, acc[w][threadIdx.x], 1.0f);
        out[threadIdx.x] = finish(sum);
      }
      __syncthreads();
    }
  }
}

// Blocks that join an item's parts (a column of them for each of the launch's `ctas` records).  One a
// row up to 24 rows of an item, where items have more parts than one warp takes (they share the CTAs):
// 5 tokens of 32 / 8 heads over 4000 keys, 8 blocks and 20: one sequence 15.4 and 13.5 us, two 16.9 and
// 15.6, eight 31.1 and 33.1.  Blocks past an item's rows only cost their launch (one token, 4 rows, of
// four to six sequences over 4000 keys: 16 to 24 blocks 20.1 to 26.7 us, 8 blocks 19.1 to 25.3).
unsigned join_blocks(int nq, int64_t tokens, int64_t batch, int kv_heads, int group, int per_item, int ctas) {
  const int64_t each = nvfp4::cdiv(tokens, batch), rows = (each < per_item ? each : per_item) * group;  // (on average)
  return nq == 1 && rows > 8 && rows <= 24 && batch * kv_heads * kJoinFew < ctas ? (unsigned)rows : 8 * (unsigned)nq;
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
int launch(const paged_attention_input& in, bool many, const attn_rows& out, void* workspace, int32_t* dev_status,
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
  p.per_tile = kRows / p.group;
  p.per_item = NQ * p.per_tile;
  p.full_tiles = many;
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
  p.wide = reinterpret_cast<uintptr_t>(out.data) % 32 == 0 && out.ld_token % 16 == 0 && out.ld_head % 16 == 0;
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
  // (no item can be cut)
  const int64_t uncut = NQ == 2 || (D == 256 && many) ? kWhole * kKeys : kKeys;
  if ((in.block_table != nullptr ? capacity : in.tokens) <= uncut) return NVFP4_OK;
  const unsigned blocks = join_blocks(NQ, in.tokens, in.batch, p.kv_heads, p.group, p.per_item, (int)grid);
  void* join_args[] = {&p};
  if (nvfp4::launch_dependent((const void*)attention_join_kernel<D, NQ>, dim3(grid, blocks), dim3(32 * kJoinWarps), 0, stream, 1,
                              join_args) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return NVFP4_OK;
}

}  // namespace

int launch_attention(const paged_attention_input* in, const attn_rows* out, void* workspace, int32_t* dev_status,
                     cudaStream_t stream) {
  // Two tiles of rows an item where sequences bring more than one tile's on average (32 / 8 heads
  // of 128 over 2000 keys, 16 sequences: 24 tokens each 37 us, with two tiles 40; 48 tokens 48, with
  // one tile 58).
  const bool many = in->tokens * (in->heads / in->kv_heads) > kRows * in->batch;
  switch (in->dim) {
    case 64: return many ? launch<64, 2>(*in, many, *out, workspace, dev_status, stream)
                         : launch<64, 1>(*in, many, *out, workspace, dev_status, stream);
    case 128: return many ? launch<128, 2>(*in, many, *out, workspace, dev_status, stream)
                          : launch<128, 1>(*in, many, *out, workspace, dev_status, stream);
    default: return launch<256, 1>(*in, many, *out, workspace, dev_status, stream);
  }
}

#ifdef NVFP4_TEST_WITHHOLD
// Test build: the rule for the joining kernel's blocks.
extern "C" int nvfp4_test_join_blocks(int nq, int64_t tokens, int64_t batch, int kv_heads, int group, int per_item, int ctas) {
  return (int)join_blocks(nq, tokens, batch, kv_heads, group, per_item, ctas);
}
#endif
