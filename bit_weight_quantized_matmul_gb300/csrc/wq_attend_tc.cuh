// wq_attend_tc.cuh -- attention over the 4-bit KV cache, many query rows per cached head (prompts, chunks
// of prompts, long drafts).
//
// A block owns one cached head of one sequence and GROUPS * 128 query rows (row r = token * group + head of
// the group), and walks the tokens they see in tiles of 128.  Per tile the codes become fp16 operands in
// shared memory once, for all rows, and tcgen05.mma computes
//   S [128 rows x 128 tokens] = Q [128 x D] . K^T          (operands K-major, fp32 in tensor memory)
//   O [128 rows x D]         += P [128 x 128 tokens] . V    (P from tensor memory, V with D contiguous)
// with P = 2^(S f - m + 11) as fp16, written over S's columns.  One thread owns a query row: its maximum, sum
// and mask need no exchange.  m moves only when a score passes it by more than 4 (P stays below 2^15), and
// only then O is read back and scaled.
//
// Roles: 4 GROUPS softmax warps (thread = row), four decode warps (thread = token: 16-byte code loads a tile
// ahead, fp16 rows in the 128-byte swizzle), one thread that issues the MMAs.  While one group's softmax
// runs, the tensor cores work for the other; K and V are double-buffered.
//
// q4_0 rows hold (c - 8) d, elements of an octet in the order 0 4 1 5 2 6 3 7 in which masking a word of codes
// leaves them; Q's rows and O's columns follow it.  Where |d| >= 8192 in some block could overflow fp16, the token's
// whole row holds an eighth and is marked: the softmax takes its scores, or its weight in the product, eightfold.
// NVFP4 rows hold E2M1(c) E4M3(s), exact, and g enters with the softmax scale and the output.  Rounding K, V and P
// to fp16's 11 bits is what this path costs in precision (2^-12 each, independent; beside a block with |d| >= 8192,
// 2^-22 in the values of the token's other blocks).
//
// A V scale that is no finite number cannot be left to the product (0 * NaN spoils rows that do not see
// the token): the block is stored as zeros and the rows that do see the token are made NaN.
//
// Measured on GB300 (19 sequences of 16384 tokens, 8 cached heads of 128, 256 rows each, one block an SM): 1082
// TFLOP/s (q4_0), 1169 (NVFP4), 0.56 and 0.61 of the measured bf16 rate.  Bound by a chain: a tile of 128 tokens
// takes 4500 cycles, of which a row's softmax takes 2300 and its group's two products 1100, and the other group
// has the tensor cores meanwhile.  Tried and slower, against 1114 (q4_0) before scales of 8192 and more were told
// apart: half tiles of 64 tokens with scores ahead of the products (more, smaller MMAs: 815 TFLOP/s), one pass over S
// with P kept in registers (915), two threads a row (970), a row's 128 scores in registers (spills), the codes of two
// tiles in registers (1118 / 1150).
//
// Every wait is bounded; after one ran out the roles stop, and the MMAs issued are waited for before
// tensor memory is released.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "wq_kv.cuh"

namespace wq {
namespace {

using kv::ex2;
using kv::large;
using kv::max3;
using kv::mul2;
using kv::pack_f16x2;

constexpr int kTile = 128;      // tokens of a tile
constexpr int kSms = 152;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 4.0f;  // how far (base 2) a score may pass m before m moves
constexpr float kUp = 11.0f;    // P = 2^(score - m + kUp): at most 2^15, and exact to 11 bits down to 2^-25 of the largest

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31},"
      "[%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's loads from tensor memory; r's values are theirs only from here on.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// One lane of the warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void mma_ss_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  if (elect_one())
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts_one(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  if (elect_one()) mma_bf16_ts(d_tmem, a_tmem, b_desc, idesc, accumulate);   // the types are the descriptor's
}
__device__ __forceinline__ void commit_one(uint64_t* bar) {
  if (elect_one()) tc_commit(bar);
}
// Instruction descriptor, kind::f16: fp32 accumulator, fp16 A (K-major) and B (K-major, or with its N
// dimension contiguous).
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Bounded wait after an abort: neither looks at the flag nor records a status.
__device__ __forceinline__ void wait_quiet(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kSpinLimit && !mbar_try_wait(bar, parity); ++i) {
  }
}
// A whole warp's bounded wait: all lanes go on, or none.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort));
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Pairs of fp32 in one register pair, and operations on both, each rounded as by itself.
__device__ __forceinline__ uint64_t two(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2f(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2f(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Element of an octet that position e of an operand row holds.
template <int FMT>
__device__ __forceinline__ constexpr int octet(int e) { return FMT == WQ_Q4_0 ? (e & 1) * 4 + (e >> 1) : e; }

// Eight codes -> eight fp16 values in operand order (eighth, q4_0: an eighth of them).  s: the block's scale in both halves.
template <int FMT>
__device__ __forceinline__ uint4 operand8(uint32_t w, uint32_t s, bool eighth) {
  uint32_t r[4];
  if (FMT == WQ_Q4_0) {
    // c - 8 = (1024 + c) - 1032 and (1024 + 16 c) / 16 - 72, or (1024 + c) / 8 - 129 and (1024 + 16 c) / 128 - 9, exact
    // (scaled here and not in s, which may have no bits to spare); times s one rounding
    const uint32_t m0 = eighth ? 0x30003000u : 0x3C003C00u, c0 = eighth ? 0xD808D808u : 0xE408E408u;
    const uint32_t m1 = eighth ? 0x20002000u : 0x2C002C00u, c1 = eighth ? 0xC880C880u : 0xD480D480u;
    r[0] = fma2((w & 0x000F000Fu) | 0x64006400u, m0, c0);
    r[1] = fma2((w & 0x00F000F0u) | 0x64006400u, m1, c1);
    w >>= 8;
    r[2] = fma2((w & 0x000F000Fu) | 0x64006400u, m0, c0);
    r[3] = fma2((w & 0x00F000F0u) | 0x64006400u, m1, c1);
  } else {
    kv::e2m1_pairs(w, r);
  }
  return make_uint4(mul2(r[0], s), mul2(r[1], s), mul2(r[2], s), mul2(r[3], s));
}

// What the softmax has to know of 32 tokens, a bit each (uint4): .x the page is missing, .y a scale of V is no finite
// number (stored as zero), .z the row of K, .w that of V holds an eighth.

struct Params {
  AttendArgs a;
  int group;        // query heads per cached head
  int row_tiles;    // blocks of GROUPS * 128 query rows per cached head
  int parts;        // blocks that share the tokens of one of them
  bool sorted;      // SEL: the sequences that see most first
  float* part_o;    // [row tile][part][GROUPS * 128][D] unnormalised outputs
  float* part_ml;   // [row tile][part][GROUPS * 128][2] their m (base 2) and l
};

// The token of a row, by a 32-bit division where that does.
__device__ __forceinline__ int64_t row_token(int64_t r, int group) {
  return r >> 32 ? r / group : (int64_t)((uint32_t)r / (uint32_t)group);
}

template <int D, int GROUPS, bool SEL>
struct Lay {
  static constexpr int NB = SEL && D == 128 && GROUPS == 1 ? 1 : 2;   // buffers for tiles of K, and of V
  static constexpr int CH = D / 64;                       // 128-byte chunks of an operand row
  static constexpr int Q_OFF = 0;                         // [GROUPS][CH][128 rows][128 bytes]
  static constexpr int TB = CH * 128 * 128;               // bytes of a K or V tile [CH][128 tokens][128 bytes]
  static constexpr int K_OFF = GROUPS * TB;               // NB of them
  static constexpr int V_OFF = K_OFF + NB * TB;
  static constexpr int MASK_OFF = V_OFF + NB * TB;         // [4 tiles][4 warps] uint4 of marks
  static constexpr int SUM_OFF = MASK_OFF + 4 * 4 * 16;   // [4 tiles][4 warps] bit 0: .x or .y, 1: .z, 2: .w has a mark
  static constexpr int BAR_OFF = SUM_OFF + 4 * 4 * 4;
  static constexpr int NBAR = 8 + 3 * GROUPS + 3;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int TOTAL = MISC_OFF + 16 + 1024;
  static constexpr int SOFT = 4 * GROUPS, DEC = SOFT, MMA = SOFT + 4;   // first warps of the roles
  static constexpr int THREADS = (SOFT + 5) * 32;
  static constexpr int COLS = GROUPS * (128 + D) <= 256 ? 256 : 512;    // tensor memory columns
  // two blocks an SM where shared memory and tensor memory hold them: at 96 registers heads of 64 spill 36 to 52 bytes, and
  // 4 x 224 tokens over 1500 of 20 heads take 38 us (q4_0), with one block an SM 53; 1 x 224, whose blocks all fit, 16 and 14
  static constexpr int BLOCKS = TOTAL <= 113 * 1024 && COLS <= 256 ? 2 : 1;
};

// SEL: the rows may see the first tokens besides their window, or nodes of a tree (kv::sight).
template <int FMT, int D, int GROUPS, bool SEL>
__global__ void __launch_bounds__((Lay<D, GROUPS, SEL>::THREADS), (Lay<D, GROUPS, SEL>::BLOCKS))
    attend_tc_kernel(const __grid_constant__ Params p) {
  using L = Lay<D, GROUPS, SEL>;
  const AttendArgs& a = p.a;
  if (SEL) griddep_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t* kfull = bars;               // [2] K tile decoded
  uint64_t* kempty = bars + 2;          // [2] the MMAs reading it finished
  uint64_t* vfull = bars + 4;
  uint64_t* vempty = bars + 6;
  uint64_t* sfull = bars + 8;           // [GROUPS] scores complete
  uint64_t* pfull = sfull + GROUPS;     // [GROUPS] P written
  uint64_t* ofull = pfull + GROUPS;     // [GROUPS] O complete up to a tile
  uint64_t* qfull = ofull + GROUPS;     // Q in shared memory
  uint64_t* done = qfull + 1;           // every warp has finished
  uint64_t* drain = done + 1;           // the MMA issuer's last commit, after an abort
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)warp_id(), 0), lane = (int)lane_id();   // known to be one for the warp

  // Which rows: the last row tiles of a sequence, which see most, first.
  uint32_t x = blockIdx.x;
  const int part = x % p.parts;
  x /= p.parts;
  const int rt = p.row_tiles - 1 - (int)(x % p.row_tiles);
  x /= p.row_tiles;
  const int h = x % a.kv.heads;
  int64_t b = x / a.kv.heads;
  if (SEL && p.sorted) b = kv::by_length<L::THREADS>(a, (int)b, reinterpret_cast<int*>(smem));

  // Q's rows as they are to their places, D / 8 lanes a row, while the lengths are still on their way; the softmax threads scale
  // their own rows there.  (Read from global memory by its thread, a row took 5 us of a block's beginning: 32 lines a load.)
  if (warp < L::SOFT) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int e = lane % kLanes;
    const int64_t r_w = (int64_t)rt * GROUPS * 128 + warp * 32, i_w = row_token(r_w, p.group);
    const uint32_t rest = (uint32_t)(r_w - i_w * p.group);
    const uint16_t* q0 = reinterpret_cast<const uint16_t*>(a.q.p) + b * a.q.batch + (int64_t)h * p.group * a.q.head + 8 * e;
    const uint32_t to = smem_u32(smem + L::Q_OFF + (warp >> 2) * L::TB + (warp & 3) * 32 * 128 + (e >> 3) * 16384);
#pragma unroll 4
    for (int x = lane / kLanes; x < 32; x += kRows) {
      const uint32_t up = (rest + x) / (uint32_t)p.group;
      const bool in = i_w + up < a.tokens;
      const uint16_t* src = q0 + (in ? (i_w + up) * a.q.token + (int64_t)(rest + x - up * (uint32_t)p.group) * a.q.head : 0);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + x * 128 + (((e & 7) ^ (x & 7)) << 4)), "l"(src),
                   "r"(in ? 16 : 0) : "memory");
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], 4);
      mbar_init(&kempty[i], 1);
      mbar_init(&vfull[i], 4);
      mbar_init(&vempty[i], 1);
    }
    for (int i = 0; i < GROUPS; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
      mbar_init(&ofull[i], 1);
    }
    mbar_init(qfull, L::SOFT);
    mbar_init(done, L::THREADS / 32);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == L::MMA) tmem_alloc(tmem_slot, L::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Only now: a successor that allocates tensor memory before it waits for this kernel may take an SM's from a block that has none
  // yet, and the two would wait for each other.
  if (SEL) griddep_launch_dependents();

  const int n = kv::count_of(a.counts, b, a.tokens);
  const int len = max(a.lens[b], 0);                          // positions are counted from here
  const int held = (int)min((int64_t)len, a.kv.capacity);     // what can be seen of them
  if (held < len && threadIdx.x == 0) set_status(WQ_STATUS_ARG);
  const int64_t r0 = (int64_t)rt * GROUPS * 128, rows = (int64_t)n * p.group;
  // A tree's node i sees the context up to len - n, from its depth's window on, and nodes by their bits.
  const bool tree = SEL && a.tree_mask;
  const int base = len - n;
  auto hi_of = [&](int64_t i) {
    return !a.causal ? held : (int)max((int64_t)0, min((int64_t)held, (int64_t)len - n + (tree ? 0 : i + 1)));
  };
  auto lo_at = [&](int64_t i) { return a.window ? (int)max((int64_t)0, (int64_t)len - n + i - a.window + 1) : 0; };
  auto lo_of = [&](int64_t i) {
    return lo_at(SEL && tree && a.tree_depth && a.window ? min(max(a.tree_depth[b * a.depth_batch + i], 0), n - 1) : i);
  };
  const bool any = r0 < rows;
  const int lo_min = any ? lo_at(tree ? 0 : r0 / p.group) : 0;
  const int hi_max = any ? (tree ? held : hi_of(min(rows - 1, r0 + GROUPS * 128 - 1) / p.group)) : 0;
  // The tiles of the block's tokens; SEL: those of the first tokens stand before them, and a tile's place is looked up.
  const int ends = (hi_max + kTile - 1) / kTile, near = SEL ? min(lo_min / kTile, ends) : lo_min / kTile;
  const int firsts = SEL && a.window ? min(near, (min(a.sinks, hi_max) + kTile - 1) / kTile) : 0;
  const int all = SEL ? firsts + ends - near : hi_max > lo_min ? ends - near : 0, each = (all + p.parts - 1) / p.parts;
  const int tile0 = (SEL ? 0 : near) + min(all, part * each), tiles = min(all, (part + 1) * each) - min(all, part * each);
  auto place = [&](int j) { return SEL && tile0 + j >= firsts ? tile0 + j + (near - firsts) : tile0 + j; };
  const int groups = GROUPS == 2 && r0 + 128 < rows ? 2 : 1;      // groups of rows that are there

  if (warp < L::SOFT) {
    // ---------------------------------------------------------------- softmax: thread = query row
    const int grp = warp >> 2;
    const int64_t r = r0 + threadIdx.x, i = row_token(r, p.group);            // softmax warps come first: threadIdx.x < 128 GROUPS
    const int hq = h * p.group + (int)(r - i * p.group);
    const bool mine = r < rows;
    const int lo = mine ? lo_of(i) : 0, hi = mine ? hi_of(i) : 0x7FFFFFFF;   // what is no row need not be masked
    const int sinks = SEL && a.window ? a.sinks : 0;
    const uint32_t* nodes = tree && mine ? a.tree_mask + b * a.mask_batch + i * a.tree_words : nullptr;
    const uint32_t s_at = tmem + ((uint32_t)(warp & 3) << 21) + grp * 128;
    const uint32_t o_at = tmem + ((uint32_t)(warp & 3) << 21) + GROUPS * 128 + grp * D;
    float fac = 0.0f, m = -INFINITY, l = 0.0f;
    bool ok = true;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();                             // the warp's rows of Q have come in as they are
    if (tiles > 0 && grp < groups) {
      // Q: the row times 2^e with its largest element in 2^12 .. 2^13, fp16, and with the signs of the scale and of g: the
      // largest score has to be the largest product
      uint8_t* row = smem + L::Q_OFF + grp * L::TB + (threadIdx.x & 127) * 128;
      auto chunk = [&](int e) { return reinterpret_cast<uint4*>(row + (e >> 3) * 16384 + (((e & 7) ^ (threadIdx.x & 7)) << 4)); };
      float amax = 0.0f;
#pragma unroll 4
      for (int e = 0; e < D / 8; ++e) {
        const uint4 w = mine ? *chunk(e) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(bf16_bits_to_f32((u[k >> 1] >> (16 * (k & 1))) & 0xFFFFu)));
      }
      int e2 = 12 + 127 - (int)(__float_as_uint(amax) >> 23);
      e2 = amax == 0.0f || amax == INFINITY ? 0 : min(e2, 112);
      const float kg = FMT == WQ_NVFP4 && a.kv.g[0] ? *a.kv.g[0] : 1.0f;
      const float up = copysignf(__uint_as_float((uint32_t)(127 + e2) << 23), a.scale) * copysignf(1.0f, kg);
      fac = fabsf(a.scale) * kLog2e * fabsf(kg) * __uint_as_float((uint32_t)(127 - e2) << 23);
#pragma unroll 4
      for (int e = 0; e < D / 8; ++e) {
        const uint4 w = mine ? *chunk(e) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int el = octet<FMT>(k);
          v[k] = bf16_bits_to_f32((u[el >> 1] >> (16 * (el & 1))) & 0xFFFFu) * up;
        }
        *chunk(e) = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(qfull);

    if (grp < groups) {
      for (int j = 0; j < tiles && ok; ++j) {
        if (!wait_all(&sfull[grp], j & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const int t0 = place(j) * kTile;
        const uint4* marks = reinterpret_cast<const uint4*>(smem + L::MASK_OFF) + (j & 3) * 4;
        const uint4 sum = *reinterpret_cast<const uint4*>(smem + L::SUM_OFF + (j & 3) * 16);
        const uint32_t odd = sum.x | sum.y | sum.z | sum.w;
        if (FMT == WQ_Q4_0 && (odd & 2u)) {
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t v[32];
            tmem_ld32(s_at + c, v);
            wait_ld(v);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if ((marks[c >> 5].z >> k) & 1u) v[k] = __float_as_uint(__uint_as_float(v[k]) * 8.0f);
            tmem_st32(s_at + c, v);
          }
          tc_wait_st();
        }
        const bool masked = __any_sync(0xFFFFFFFFu, (t0 < lo && !(SEL && t0 + kTile <= sinks)) || t0 + kTile > hi || (odd & 1u));
        // what this row sees of the 32 tokens from c on, as bits
        // SEL: looked up once for both passes where two blocks share the registers, which then hold fewer addresses (26 nodes
        // over 60001 63 -> 59 us; with one block an SM, 20 to 64 nodes, 271 -> 277).
        constexpr bool kOnce = SEL && L::BLOCKS == 2;
        auto bits = [&](int c) { return kv::sight<!kOnce>(t0 + c, lo, hi, sinks, nodes, a.tree_words, base, held) & ~marks[c >> 5].x; };
        const uint4 seen = kOnce && masked ? make_uint4(bits(0), bits(32), bits(64), bits(96)) : make_uint4(0, 0, 0, 0);
        auto sees = [&](int c) -> uint32_t {
          if (kOnce) return c < 64 ? (c < 32 ? seen.x : seen.y) : c < 96 ? seen.z : seen.w;
          if (SEL) return bits(c);
          const int first = lo - (t0 + c), past = hi - (t0 + c);
          uint32_t bits = past >= 32 ? 0xFFFFFFFFu : past <= 0 ? 0u : (1u << past) - 1u;
          if (first > 0) bits = first >= 32 ? 0u : bits & ~((1u << first) - 1u);
          return bits & ~marks[c >> 5].x;
        };
        // Loops are kept short (the roles share the instruction caches) and chains apart (four maxima, four sums).
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          uint32_t v[2][32];
          tmem_ld32(s_at + c, v[0]);
          tmem_ld32(s_at + c + 32, v[1]);
          wait_ld(v[0]);
          wait_ld(v[1]);
          if (masked) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t see = sees(c + 32 * u);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[u][k] = (see >> k) & 1u ? v[u][k] : 0xFF800000u;
            }
          }
#pragma unroll
          for (int k = 0; k < 64; k += 2)
            tops[(k >> 1) & 3] = max3(tops[(k >> 1) & 3], __uint_as_float(v[k >> 5][k & 31]), __uint_as_float(v[k >> 5][(k & 31) + 1]));
        }
        float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        top = top == -INFINITY ? top : top * fac;
        if (FMT == WQ_Q4_0 && (odd & 4u)) top += 3.0f;   // a weight taken eightfold has to fit too
        const bool move = top > m + kSlack || (m == -INFINITY && top > m);
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float f = move ? ex2(m - top) : 1.0f;
          if (move) m = top;
          l *= f;
          if (j > 0) {
            if (!wait_all(&ofull[grp], (j - 1) & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t v[32];
              tmem_ld32(o_at + c, v);
              wait_ld(v);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
              tmem_st32(o_at + c, v);
            }
            tc_wait_st();
          }
        }
        const float base = m == -INFINITY ? 0.0f : kUp - m;
        const uint64_t fac2 = two(fac, fac), base2 = two(base, base);
        uint64_t sums[2] = {0, 0};      // two pairs of fp32 zeros
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t v[32], pk[16];
          tmem_ld32(s_at + c, v);
          wait_ld(v);
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float e0, e1;
            split(fma2f(two(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), fac2, base2), e0, e1);
            v[k] = __float_as_uint(ex2(e0));
            v[k + 1] = __float_as_uint(ex2(e1));
          }
          if (masked) {                 // not by the score alone: -inf times a scale of zero is no number
            const uint32_t see = sees(c);
            if (see & marks[c >> 5].y) l = __uint_as_float(0x7FC00000u);   // a value that is no number
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = (see >> k) & 1u ? v[k] : 0u;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float e0 = __uint_as_float(v[2 * k]), e1 = __uint_as_float(v[2 * k + 1]);
            sums[k & 1] = add2f(sums[k & 1], two(e0, e1));
            pk[k] = pack_f16x2(e0, e1);
          }
          tmem_st16(s_at + (c >> 1), pk);
        }
        float even, odd_sum;
        split(add2f(sums[0], sums[1]), even, odd_sum);
        l += even + odd_sum;
        tc_wait_st();
        if (FMT == WQ_Q4_0 && (odd & 4u)) {      // a column of P holds two tokens
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            uint32_t v[32];
            tmem_ld32(s_at + c, v);
            wait_ld(v);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t bits = marks[(c >> 4) + (k >> 4)].w >> (2 * (k & 15));
              v[k] = mul2(v[k], 0x3C003C00u + (bits & 1u) * 0x0C00u + (bits & 2u) * 0x06000000u);
            }
            tmem_st32(s_at + c, v);
          }
          tc_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[grp]);
      }
      if (ok && tiles > 0 && !wait_all(&ofull[grp], (tiles - 1) & 1, abort_flag)) ok = false;
      tc_fence_after();
    }
    // O / l to the output, or O, m and l as they are to this part's place
    const bool some = mine && tiles > 0 && l != 0.0f;
    const float vg = FMT == WQ_NVFP4 && a.kv.g[1] ? *a.kv.g[1] : 1.0f;
    const float mul = p.parts > 1 ? vg : some ? vg / l : 0.0f;
    const bool row_there = ok && i < a.tokens;
    const int64_t at = p.parts > 1 ? ((b * a.kv.heads + h) * p.row_tiles + rt) * p.parts * (GROUPS * 128) +
                                         (int64_t)part * (GROUPS * 128) + threadIdx.x
                                   : b * a.out.batch + i * a.out.token + hq * a.out.head;
    if (row_there && p.parts > 1) {
      *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(some ? m - kUp : -INFINITY, some ? l : 0.0f);
    } else if (row_there && a.lse) {
      a.lse[(b * a.tokens + i) * a.q_heads + hq] = some ? (m - kUp + log2f(l)) * kLn2 : -INFINITY;
    }
    const bool f32 = p.parts > 1 || a.f32;
    float* o32 = p.parts > 1 ? p.part_o + at * D : reinterpret_cast<float*>(a.out.p) + at;
    uint16_t* o16 = reinterpret_cast<uint16_t*>(a.out.p) + at;
    const bool computed = ok && tiles > 0 && grp < groups;            // the same for the whole warp
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t u[32];
      if (computed) {
        tmem_ld32(o_at + c, u);
        wait_ld(u);
      }
      if (!row_there) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[octet<FMT>(k)] = computed && some ? __uint_as_float(u[8 * e + k]) * mul : 0.0f;
        if (f32) {
          float4* dst = reinterpret_cast<float4*>(o32 + c + 8 * e);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
          *reinterpret_cast<uint4*>(o16 + c + 8 * e) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
      }
    }
  } else if (warp < L::MMA) {
    // ---------------------------------------------------------------- decode: thread = token of the tile
    constexpr int SB = kv::scale_bytes(D);
    const int r = threadIdx.x - L::DEC * 32, dw = warp - L::DEC;
    struct Raw {
      uint4 k[D / 32], v[D / 32];
      uint32_t ks[SB / 4], vs[SB / 4];
    };
    // Row of this thread's token in tile j; -1: past the end, -2: no such page.
    auto locate = [&](int j) -> int64_t {
      if (j >= tiles) return -1;               // whose position may pass 32 bits
      const int t = place(j) * kTile + r;
      if (t >= hi_max) return -1;
      int64_t page = b;
      int off = t;
      if (a.kv.table) {
        const int pg = kv::page_of(a.kv, t);
        off = t - pg * a.kv.page_size;
        page = a.kv.table[b * a.kv.table_ld + pg];
      }
      if (page < 0 || page >= a.kv.pages) {
        set_status(WQ_STATUS_ARG);
        return -2;
      }
      return (page * a.kv.heads + h) * (int64_t)a.kv.page_size + off;
    };
    auto fetch = [&](int64_t row, Raw& w) {
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        w.k[e] = row >= 0 ? *reinterpret_cast<const uint4*>(a.kv.codes[0] + row * (D / 2) + 16 * e) : make_uint4(0, 0, 0, 0);
        w.v[e] = row >= 0 ? *reinterpret_cast<const uint4*>(a.kv.codes[1] + row * (D / 2) + 16 * e) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int e = 0; e < SB / 4; ++e) {       // zero scales: a row that is not there holds zeros
        w.ks[e] = row >= 0 ? *reinterpret_cast<const uint32_t*>(a.kv.scales[0] + row * SB + 4 * e) : 0u;
        w.vs[e] = row >= 0 ? *reinterpret_cast<const uint32_t*>(a.kv.scales[1] + row * SB + 4 * e) : 0u;
      }
    };
    // A row of codes to its place in an operand tile.
    auto store = [&](uint8_t* tile, const uint4 (&codes)[D / 32], const uint32_t (&scales)[SB / 4], bool eighth) {
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const uint32_t w[4] = {codes[e].x, codes[e].y, codes[e].z, codes[e].w};
        uint32_t s0, s1;                       // scales of the block's first and second half
        if (FMT == WQ_Q4_0) {
          s0 = s1 = __byte_perm(scales[e >> 1], 0, (e & 1) ? 0x3232u : 0x1010u);
        } else {
          const uint32_t two = __byte_perm(scales[e >> 1], 0, (e & 1) ? 0x3322u : 0x1100u);
          kv::e4m3_pairs(two, s0, s1);
        }
#pragma unroll
        for (int o = 0; o < 4; ++o) {
          const int oct = 4 * e + o;
          *reinterpret_cast<uint4*>(tile + (oct >> 3) * 16384 + r * 128 + (((oct & 7) ^ (r & 7)) << 4)) =
              operand8<FMT>(w[o], o < 2 ? s0 : s1, eighth);
        }
      }
    };
    Raw raw;
    int64_t row = locate(0), row_next = locate(1);
    fetch(row, raw);
    bool ok = true;
    for (int j = 0; j < tiles && ok; ++j) {
      const int buf = j % L::NB;
      // V scales that are no finite numbers become zeros, the token is marked
      bool bad = false;
#pragma unroll
      for (int e = 0; e < SB / 4; ++e)
#pragma unroll
        for (int k = 0; k < (FMT == WQ_Q4_0 ? 2 : 4); ++k) {
          const uint32_t bits = FMT == WQ_Q4_0 ? 0x7C00u << (16 * k) : 0x7Fu << (8 * k);
          const uint32_t all = FMT == WQ_Q4_0 ? 0xFFFFu << (16 * k) : 0xFFu << (8 * k);
          if ((raw.vs[e] & bits) == bits) {
            raw.vs[e] &= ~all;
            bad = true;
          }
        }
      uint4 marks = make_uint4(__ballot_sync(0xFFFFFFFFu, row == -2), __ballot_sync(0xFFFFFFFFu, bad), 0u, 0u);
      uint32_t kl = 0, vl = 0;
      if (FMT == WQ_Q4_0) {
#pragma unroll
        for (int e = 0; e < SB / 4; ++e) {
          kl |= large(raw.ks[e]);
          vl |= large(raw.vs[e]);
        }
        marks.z = __ballot_sync(0xFFFFFFFFu, kl != 0);
        marks.w = __ballot_sync(0xFFFFFFFFu, vl != 0);
      }
      if (j >= L::NB && !wait_all(&kempty[buf], ((j / L::NB) & 1) ^ 1, abort_flag)) { ok = false; break; }
      if (lane == 0) {
        reinterpret_cast<uint4*>(smem + L::MASK_OFF)[(j & 3) * 4 + dw] = marks;
        reinterpret_cast<uint32_t*>(smem + L::SUM_OFF)[(j & 3) * 4 + dw] =
            ((marks.x | marks.y) != 0 ? 1u : 0u) | (marks.z != 0 ? 2u : 0u) | (marks.w != 0 ? 4u : 0u);
      }
      store(smem + L::K_OFF + buf * L::TB, raw.k, raw.ks, kl != 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kfull[buf]);
      if (j >= L::NB && !wait_all(&vempty[buf], ((j / L::NB) & 1) ^ 1, abort_flag)) { ok = false; break; }
      store(smem + L::V_OFF + buf * L::TB, raw.v, raw.vs, vl != 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&vfull[buf]);
      row = row_next;
      fetch(row, raw);
      row_next = locate(j + 2);
    }
  } else if (tiles > 0) {
    // ---------------------------------------------------------------- MMA issuer
    // The whole warp runs this, and one lane is elected at each instruction: addresses and descriptors then stay in
    // uniform registers (moved there one by one from a single thread's, they cost more than the MMAs).
    constexpr uint32_t kS = idesc_f16(128, 128, false), kO = idesc_f16(128, D, true);
    const uint64_t qd = smem_desc(smem_u32(smem + L::Q_OFF), 16, 1024, 2);
    const uint64_t kd = smem_desc(smem_u32(smem + L::K_OFF), 16, 1024, 2);
    const uint64_t vd = smem_desc(smem_u32(smem + L::V_OFF), 16384, 1024, 2);   // D contiguous: 64 elements, then 16 KB on
    auto scores = [&](int g, int j) {
      const uint64_t ad = qd + (uint64_t)(g * L::TB >> 4), bd = kd + (uint64_t)((j % L::NB) * L::TB >> 4);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t at = (uint64_t)((k >> 2) * 1024 + (k & 3) * 2);
        mma_ss_one(tmem + g * 128, ad + at, bd + at, kS, k != 0 ? 1u : 0u);
      }
      commit_one(&sfull[g]);
    };
    bool ok = wait_all(qfull, 0, abort_flag) && wait_all(&kfull[0], 0, abort_flag);
    if (ok) {
      tc_fence_after();
      for (int g = 0; g < groups; ++g) scores(g, 0);
      commit_one(&kempty[0]);
    }
    for (int j = 0; j < tiles && ok; ++j) {
      const int buf = j % L::NB, next = (j + 1) % L::NB;
      for (int g = 0; g < groups && ok; ++g) {
        if (g == 0 && !wait_all(&vfull[buf], (j / L::NB) & 1, abort_flag)) { ok = false; break; }
        if (!wait_all(&pfull[g], j & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint64_t bd = vd + (uint64_t)(buf * L::TB >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k)               // 16 tokens: 8 columns of P, 2 KB of V
          mma_ts_one(tmem + GROUPS * 128 + g * D, tmem + g * 128 + 8 * k, bd + 128 * k, kO, (j | k) != 0 ? 1u : 0u);
        commit_one(&ofull[g]);
        if (g == groups - 1) commit_one(&vempty[buf]);
        if (j + 1 < tiles) {
          if (g == 0 && !wait_all(&kfull[next], ((j + 1) / L::NB) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          scores(g, j + 1);
          if (g == groups - 1) commit_one(&kempty[next]);
        }
      }
    }
    if (!ok || *abort_flag) commit_one(drain);
  }

  // Teardown: every warp arrives, then the MMA warp releases tensor memory.  The softmax warps have seen
  // every MMA's results but the last commits' arrivals on kempty / vempty, which touch shared memory only.
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(done);
  if (warp == L::MMA) {
    wait_quiet(done, 0);
    if (tiles > 0) {
      if (*abort_flag) wait_quiet(drain, 0);
      else wait_quiet(&vempty[(tiles - 1) % L::NB], ((tiles - 1) / L::NB) & 1);
    }
    tc_fence_after();
    tmem_dealloc(tmem, L::COLS);
  }
}

template <int FMT, int D, int GROUPS, bool SEL>
int launch(const Params& p, cudaStream_t s) {
  using L = Lay<D, GROUPS, SEL>;
  static std::atomic<uint64_t> allowed{0};
  if (!allow_smem(allowed, attend_tc_kernel<FMT, D, GROUPS, SEL>, L::TOTAL)) return WQ_ERR_CUDA;
  const int64_t grid = p.a.batch * p.a.kv.heads * p.row_tiles * p.parts;
  if (grid > 0x7FFFFFFF) return WQ_ERR_SHAPE;
  if (SEL) {
    if (launch_early(attend_tc_kernel<FMT, D, GROUPS, SEL>, dim3((unsigned)grid), dim3(L::THREADS), L::TOTAL, s, 1u, p) != cudaSuccess)
      return WQ_ERR_CUDA;
  } else {
    attend_tc_kernel<FMT, D, GROUPS, SEL><<<(unsigned)grid, L::THREADS, L::TOTAL, s>>>(p);
  }
  count_launch();
  return cudaGetLastError() == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}
template <int FMT, int D, bool SEL>
int launch_g(const Params& p, int groups, cudaStream_t s) {
  return groups == 2 ? launch<FMT, D, 2, SEL>(p, s) : launch<FMT, D, 1, SEL>(p, s);
}
template <bool SEL>
int launch_tc(const AttendArgs& a, const AttendTcPlan& pl, cudaStream_t s) {
  Params p{};
  p.a = a;
  p.group = (int)(a.q_heads / a.kv.heads);
  p.row_tiles = pl.row_tiles;
  p.parts = pl.parts;
  p.sorted = SEL && a.batch > 1 && a.batch <= kv::kSorted &&
             a.batch * a.kv.heads * pl.row_tiles * pl.parts > kSms * (pl.groups == 1 ? 2 : 1);
  p.part_o = reinterpret_cast<float*>(a.workspace);
  p.part_ml = p.part_o + pl.slots * a.kv.dim;
  if (a.kv.fmt == WQ_Q4_0) return a.kv.dim == 64 ? launch_g<WQ_Q4_0, 64, SEL>(p, pl.groups, s) : launch_g<WQ_Q4_0, 128, SEL>(p, pl.groups, s);
  return a.kv.dim == 64 ? launch_g<WQ_NVFP4, 64, SEL>(p, pl.groups, s) : launch_g<WQ_NVFP4, 128, SEL>(p, pl.groups, s);
}

}  // namespace
}  // namespace wq
