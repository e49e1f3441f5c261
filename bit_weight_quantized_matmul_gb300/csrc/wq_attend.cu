// wq_attend.cu -- attention over the 4-bit KV cache, few query rows per cached head (decode).
//
// With x_t the codes of token t, S = scale * Q K^T and O = softmax(S) V are computed from the codes
// as they lie in the cache.  A block owns one cached head of one sequence, its up to 8 * NT query rows
// (row r = token * group + head of the group) and a range of tokens; each of its
// four warps streams 32-token tiles of that range through a ring of its own in shared memory
// (cp.async: no wait of one warp on another) and keeps its own running maximum m, sum l and O,
// joined at the end.  The transposed products put tokens (then head elements) on the 16-row side of
// mma.m16n8k16, so that one to eight query rows fill its 8-column side:
//   S^T [16 tokens x 8 rows] = K [16 x D] . Q^T [D x 8],    O^T [D x 8 rows] += V^T [D x 16] . P^T [16 x 8].
// ldmatrix on the packed bytes deals them out as the two A operands need them: plain, a lane gets
// eight codes of one token; transposed, four codes of each of two tokens, side by side in a register.
//
// q4_0, K: a nibble in place is an fp16 subnormal (c * 2^-24, or c * 2^-20 in bits 4 .. 7), exact in the
// MMA, so unpacking is one AND per two codes; the 2^-4 between the two is folded into Q, the offset of 8 is
// the accumulator's initial value, -8 * sum(Q) over the block, and d multiplies the block's partial score in
// fp32.  V: a nibble under the exponent of 1024 less 1032 is c - 8 (the sum over tokens runs over weights
// that differ by many orders of magnitude, so an offset taken off afterwards would leave its rounding in
// elements that are small), times d, rounded to fp16: 2^-12 of a value of any size.  (d on the weight's side takes
// six instructions less per 16 tokens and block, 0 to 2 % of the time, but p d leaves fp16's range for small d and
// small p alike.)  NVFP4: E2M1(c) * E4M3(s) is exact in fp16 (6 significant bits), g enters with the softmax scale
// and the output.  The weights p are rounded to fp16 as 2^kUp p: to 11 bits down to 2^-26 (q4_0) or 2^-29 (NVFP4)
// of a row's largest.  Q is scaled per row by a power of two, so that its bf16 values are exact in fp16.
//
// A d that (c - 8) d may overflow with (|d| >= 8192) and scales of V that are no finite numbers are not looked for at
// each tile, which took 3 %.  Either leaves O not finite; a warp that finds its O so goes through its tiles a second time,
// with d / 8 and 8 p where d is large, and with such scales out of the product.
//
// Must read 0.5625 bytes an element of the visible K and V once.  Measured on GB300: one sequence of 2^20 tokens, 8 heads
// of 128, 226 us with the join, 5.3 TB/s of 6.8 for a copy (2^21 439 us, 5.5 TB/s); 57 x 8 heads x 4500 tokens (one
// block for every place on the device) 65 us from a cold cache, 4.5 TB/s; 64 sequences of 1000 to 8000 89 us, 3.7 TB/s,
// for the blocks past the first 456 run when most places are empty; one sequence of 131071 34 us and 5 for the join.
// Bound by the instruction chain of a warp: 19 (NVFP4) to 21 (q4_0) instructions per token and head of 128, 12 warps
// an SM for their registers, one issued every fourth cycle or so, DRAM at 45 to 75 % of its peak.  Short sequences are
// bound by what a block does before its first tile and after its last (about 4 us for each block that follows another
// in a place).  Heads of 128 with 17 to 32 rows do not fit the registers (q4_0 spills 588 bytes a thread, NVFP4 208).
#include <cuda_runtime.h>

#include <type_traits>

#include "wq_kv.cuh"

namespace wq {
namespace {

using kv::ex2;
using kv::large;
using kv::max3;
using kv::mul2;
using kv::pack_f16x2;

constexpr int kWarps = 4;
constexpr int kStages = 3;   // tiles in a warp's ring
constexpr int kSms = 152;
// More query rows than this per cached head go to the tensor-memory kernel, whose tile holds 128.  It takes the same time for
// 8 rows as for 64; this one, with its rows in tiles of 32 past 32 for the comparison, by number of rows (8 sequences of 4096
// tokens with 8 heads of 128, the join included):
//   rows              8    16    24    32    40    64
//   q4_0   this    17.4  22.4  42.9  43.6  65.4  66.2 us     the other  44.2  43.5  43.9  43.9  44.5  45.4
//   NVFP4  this    18.4  22.4  34.1  34.8  51.8  52.3        the other  39.2  39.3  40.3  40.6  41.1  42.3
constexpr int kFewRows = 32;
// More registers a thread beat more warps: 4, 3 and 2 blocks of NT = 1 an SM read one sequence of 2^20 tokens at
// 4.6, 5.6 and 5.3 TB/s.
constexpr int blocks_per_sm(int NT) { return NT == 1 ? 3 : 2; }
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Tokens of a tile: 2 KB of codes for K and for V (32 query rows keep half of it, for their registers).
constexpr int tile_tokens(int D, int NT) { return NT > 2 ? 32 : 4096 / D; }
// Bytes of a stage: room for K and V codes, then K and V scales, of a 2 KB tile.
constexpr int kStageBytes = 2 * 2048 + 2 * 256;
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int q_bytes(int D, int NT) { return NT > 2 ? NT * (D / 32) * 32 * 16 : 0; }
// Joining the warps: O [warp][row][D], then m and l [warp][row].
constexpr int join_bytes(int D, int NT) { return kWarps * 8 * NT * (D * 4 + 8); }
constexpr int smem_bytes(int D, int NT) {
  return (kRingBytes > join_bytes(D, NT) ? kRingBytes : join_bytes(D, NT)) + q_bytes(D, NT);
}

struct Params {
  AttendArgs a;
  int group;        // query heads per cached head
  int cluster;      // blocks of a cluster, which share the tokens of a cached head (or 1)
  int parts;        // or blocks that do, joined by the join kernel (or 1)
  int row_tiles;    // join kernel: row tiles of a cached head
  float* part_o;    // [row tile][part][row][D] unnormalised outputs
  float* part_ml;   // [row tile][part][row][2] their m (base 2) and l
};

// Byte offset of 16-byte chunk `col` (a block of 32 codes) of token `row` in a tile: the chunks of
// eight neighbouring rows fall into different banks for ldmatrix.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int row, int col) {
  return (uint32_t)(row * (D / 2) + ((col ^ ((D == 128 ? row >> 1 : row >> 2) & (D / 32 - 1))) << 4));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A B + C with C kept.
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// Two fp32 operations in one instruction, each rounded as by itself.
__device__ __forceinline__ void mul_pair(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\t"
      "mul.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}" : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
__device__ __forceinline__ void add_pair(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\t"
      "add.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}" : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
// The top bit of each scale in a word that is infinite or NaN.
template <int FMT>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return FMT == WQ_Q4_0 ? ((x & 0x7C007C00u) + 0x04000400u) & 0x80008000u : ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
// For each half 1/8 (8) where it is large, else 1.
__device__ __forceinline__ uint32_t eighth(uint32_t x) { return 0x3C003C00u - (large(x) >> 15) * 0x0C00u; }
__device__ __forceinline__ uint32_t eightfold(uint32_t x) { return 0x3C003C00u + (large(x) >> 15) * 0x0C00u; }
// Which of a lane's eight elements of a block pair p of a K operand holds (see the K unpacking).
template <int FMT>
__device__ __forceinline__ constexpr int pair_lo(int p) { return FMT == WQ_Q4_0 ? p : 2 * p; }
template <int FMT>
__device__ __forceinline__ constexpr int pair_hi(int p) { return FMT == WQ_Q4_0 ? p + 4 : 2 * p + 1; }

// Write four output elements.
__device__ __forceinline__ void put4(const AttendArgs& a, int64_t at, float4 v) {
  if (a.f32) *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out.p) + at) = v;
  else *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out.p) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void ld_shared_cluster_f32x4(uint32_t addr, float (&v)[4]) {
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(addr) : "memory");
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, blocks_per_sm(NT)) attend_kernel(const __grid_constant__ Params p) {
  constexpr int NB = D / 32;            // 32-element blocks of a row
  constexpr int kTile = tile_tokens(D, NT), kGroups = kTile / 16;   // 16 tokens lie in one page
  constexpr int kCodes = kTile * (D / 2), kScales = kTile * kv::scale_bytes(D);
  // p = 2^(score - m + kUp): the weights use fp16's upper range too (q4_0's may still be multiplied by 8)
  constexpr float kUp = FMT == WQ_NVFP4 ? 15.0f : 12.0f;
  constexpr bool kQSmem = NT > 2;       // Q fragments live in shared memory instead of registers
  extern __shared__ __align__(128) uint8_t smem[];
  const AttendArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;

  uint32_t x = blockIdx.x;
  const int splits = p.cluster * p.parts;   // one of them is 1
  const int split = x % splits;         // the blocks of a cluster are neighbours
  x /= splits;
  const int64_t item = x;               // (sequence, cached head)
  const int h = x % a.kv.heads;
  const int64_t b = x / a.kv.heads;

  // Q is asked for first: its addresses need nothing that is still on its way.  Lane (g, q) holds row
  // 8 j + g's elements 32 blk + 8 q .. + 7 (rows past counts[b] too: they are there, and their columns unused).
  uint4 qw[NT][NB];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const uint32_t r = 8 * j + g, i = r / (uint32_t)p.group;
    const bool in = i < a.tokens;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q.p) + b * a.q.batch + i * a.q.token +
                          ((int64_t)h * p.group + (r - i * (uint32_t)p.group)) * a.q.head + 8 * q;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
      qw[j][blk] = in ? *reinterpret_cast<const uint4*>(src + 32 * blk) : make_uint4(0, 0, 0, 0);
  }

  // The rows' tokens and what they see.
  const int n = kv::count_of(a.counts, b, a.tokens);
  const int len = max(a.lens[b], 0);                          // positions are counted from here
  const int held = (int)min((int64_t)len, a.kv.capacity);     // what can be seen of them
  if (held < len && threadIdx.x == 0) set_status(WQ_STATUS_ARG);
  const int rows = n * p.group;                               // rows of this sequence, 8 * NT at most
  auto hi_of = [&](int64_t i) { return a.causal ? (int)max((int64_t)0, min((int64_t)held, (int64_t)len - n + i + 1)) : held; };
  auto lo_of = [&](int64_t i) { return a.window ? (int)max((int64_t)0, (int64_t)len - n + i - a.window + 1) : 0; };
  const int lo_min = n > 0 ? lo_of(0) : 0, hi_max = n > 0 ? hi_of(n - 1) : 0;
  const int lo_max = n > 0 ? lo_of(n - 1) : 0, hi_min = n > 0 ? hi_of(0) : 0;
  const int tile0 = lo_min / kTile;
  const int ntiles = hi_max > lo_min ? (hi_max + kTile - 1) / kTile - tile0 : 0;
  const int per = (ntiles + splits - 1) / splits;
  const int t_end = tile0 + min(ntiles, (split + 1) * per);
  const int t_begin = tile0 + min(ntiles, split * per) + warp;

  const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes;
  uint8_t* qs = smem + (kRingBytes > join_bytes(D, NT) ? kRingBytes : join_bytes(D, NT));

  // ---------------------------------------------------------------- streaming tiles
  // A lane looks up one 16-token group of the warp's next kSpan tiles at a time: row / 16 (a cache of 2^35
  // rows would not fit the GPU), -1: past the end, -2: no such page.
  constexpr int kSpan = 32 / kGroups;
  auto locate = [&](int first) -> int {
    const int tile = first + lane / kGroups * kWarps;
    if (tile >= t_end) return -1;             // whose position may pass 32 bits
    const int t = tile * kTile + 16 * (lane % kGroups);
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
    return (int)(page * a.kv.heads + h) * (a.kv.page_size >> 4) + (off >> 4);
  };
  // Lane l copies bytes 16 l .. 16 l + 15 of every 512 of the codes, and 8 l .. 8 l + 7 of the scales.
  uint32_t missing = 0;                 // per stage and group: the page is not there
  const uint32_t to = tile_at<D>(lane / NB, lane % NB);
  auto issue = [&](int tile, int stage, int mine, int from) {   // from: the lane that holds the first group
    constexpr int SB = kv::scale_bytes(D), kTokens = 8 / SB;   // tokens whose scales are 8 bytes
    const uint32_t dst = ring + stage * kStageBytes;
    int row16[kGroups], least = 0;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      row16[u] = __shfl_sync(0xFFFFFFFFu, mine, from + u);
      least = min(least, row16[u]);
    }
    constexpr int kPer = D / 64;        // 512-byte pieces of a group
    if (least >= 0 && (tile + 1) * kTile <= hi_max) {
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        const uint8_t* k = a.kv.codes[0] + lane * 16 + (uint64_t)(uint32_t)row16[u] * (8 * D);
        const uint8_t* v = a.kv.codes[1] + lane * 16 + (uint64_t)(uint32_t)row16[u] * (8 * D);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          cp16(dst + to + 512 * (u * kPer + j), k + 512 * j, 16);
          cp16(dst + to + kCodes + 512 * (u * kPer + j), v + 512 * j, 16);
        }
      }
      const int mine16 = __shfl_sync(0xFFFFFFFFu, mine, from + lane * kTokens / 16 % kGroups);
      if (kScales == 256 || lane < kScales / 8) {
        const uint64_t at = (uint64_t)(uint32_t)mine16 * (16 * SB) + (lane * kTokens & 15) * SB;
        cp_small<8>(dst + 2 * kCodes + 8 * lane, a.kv.scales[0] + at, 8);
        cp_small<8>(dst + 2 * kCodes + kScales + 8 * lane, a.kv.scales[1] + at, 8);
      }
      missing &= ~(15u << (4 * stage));
      return;
    }
    uint32_t gone = 0;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      const int64_t row = row16[u] < 0 ? -1 : (int64_t)row16[u] * 16;
      gone |= (row16[u] == -2 ? 1u : 0u) << u;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int r = (512 * j + 16 * lane) / (D / 2);
        const bool in = row >= 0 && tile * kTile + 16 * u + r < hi_max;
        const int64_t at = in ? row * (D / 2) + 512 * j + 16 * lane : 0;
        cp16(dst + to + (u * kPer + j) * 512, a.kv.codes[0] + at, in ? 16 : 0);
        cp16(dst + to + kCodes + (u * kPer + j) * 512, a.kv.codes[1] + at, in ? 16 : 0);
      }
      if (lane * kTokens / 16 == u) {
        const int left = hi_max - (tile * kTile + lane * kTokens);   // tokens from this lane's first one on
        const int bytes = row >= 0 ? min(max(left, 0), kTokens) * SB : 0;
        const int64_t at = bytes ? (row + (lane * kTokens & 15)) * SB : 0;
        cp_small<8>(dst + 2 * kCodes + 8 * lane, a.kv.scales[0] + at, bytes);
        cp_small<8>(dst + 2 * kCodes + kScales + 8 * lane, a.kv.scales[1] + at, bytes);
      }
    }
    missing = (missing & ~(15u << (4 * stage))) | gone << (4 * stage);
  };
  int rows_now = locate(t_begin), rows_next = locate(t_begin + kSpan * kWarps);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (t_begin + s * kWarps < t_end) issue(t_begin + s * kWarps, s, rows_now, s * kGroups);
    cp_commit();
  }

  // ---------------------------------------------------------------- Q
  // A row is multiplied by 2^e, which brings its largest element to 2^12 .. 2^13.
  uint32_t qf[kQSmem ? 1 : NT][NB][4];
  // q4_0: -8 sum(Q) of a block, columns 2q and 2q + 1, twice: an accumulator's four registers, kept as such
  // (two of them would be copied for every MMA)
  float init[NT][FMT == WQ_Q4_0 ? NB : 1][4];
  float fac[NT][2];                             // accumulated score -> score in base 2
  const float kg = FMT == WQ_NVFP4 && a.kv.g[0] ? *a.kv.g[0] : 1.0f;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    uint32_t u[NB][4];
    float amax = 0.0f;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      u[blk][0] = qw[j][blk].x; u[blk][1] = qw[j][blk].y; u[blk][2] = qw[j][blk].z; u[blk][3] = qw[j][blk].w;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(bf16_bits_to_f32((u[blk][e >> 1] >> (16 * (e & 1))) & 0xFFFFu)));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    int e2 = 12 + 127 - (int)(__float_as_uint(amax) >> 23);
    e2 = amax == 0.0f || amax == INFINITY ? 0 : min(e2, 112);
    const float up = __uint_as_float((uint32_t)(127 + e2) << 23), down = __uint_as_float((uint32_t)(127 - e2) << 23);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      float v[8], sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = bf16_bits_to_f32((u[blk][e >> 1] >> (16 * (e & 1))) & 0xFFFFu) * up;
        sum += v[e];
      }
      uint32_t f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float k = FMT == WQ_Q4_0 && (e & 1) ? 0.0625f : 1.0f;
        f[e] = pack_f16x2(v[pair_lo<FMT>(e)] * k, v[pair_hi<FMT>(e)] * k);
      }
      if (kQSmem) {
        if (warp == 0) reinterpret_cast<uint4*>(qs)[(j * NB + blk) * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[kQSmem ? 0 : j][blk][e] = f[e];
      }
      if (FMT == WQ_Q4_0) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
        sum *= -8.0f * 5.9604644775390625e-8f;   // -8 * 2^-24
        init[j][FMT == WQ_Q4_0 ? blk : 0][0] = __shfl_sync(0xFFFFFFFFu, sum, 8 * q);
        init[j][FMT == WQ_Q4_0 ? blk : 0][1] = __shfl_sync(0xFFFFFFFFu, sum, 8 * q + 4);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          asm volatile("mov.f32 %0, %1;" : "=f"(init[j][FMT == WQ_Q4_0 ? blk : 0][2 + c]) : "f"(init[j][FMT == WQ_Q4_0 ? blk : 0][c]));
      }
    }
    const float f = a.scale * kLog2e * (FMT == WQ_Q4_0 ? 16777216.0f : kg) * down;
    fac[j][0] = __shfl_sync(0xFFFFFFFFu, f, 8 * q);
    fac[j][1] = __shfl_sync(0xFFFFFFFFu, f, 8 * q + 4);
  }
  if (kQSmem) __syncthreads();

  // Columns' visible ranges (8 j + 2q and + 1); columns that are no rows count as seeing all.
  int c_lo[NT][2], c_hi[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * j + 2 * q + c, i = r / p.group;
      c_lo[j][c] = r < rows ? lo_of(i) : 0;
      c_hi[j][c] = r < rows ? hi_of(i) : hi_max;
    }

  float o[NT][2 * NB][4], m[NT][2], l[NT][2];
  auto reset = [&] {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      m[j][0] = m[j][1] = -INFINITY;
      l[j][0] = l[j][1] = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int d = 0; d < 2 * NB; ++d) o[j][d][k] = 0.0f;
    }
  };
  reset();

  // ---------------------------------------------------------------- tiles
  // This lane's row address for ldmatrix: four blocks of eight tokens (D = 128), or two of sixteen.
  const uint32_t lane_at = D == 128 ? tile_at<D>(lane & 7, lane >> 3) : tile_at<D>(8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1);
  // A weight of zero takes nothing from a finite scale of V only.  Where some row does not see all of a tile, scales that
  // are no finite numbers become zero, and their elements of the rows that do see the token become NaN.  sp: V's scales.
  auto clean = [&](int tile, uint8_t* sp) {
    uint2 w = make_uint2(0u, 0u);
    if (kScales == 256 || lane < kScales / 8) w = *reinterpret_cast<const uint2*>(sp + 8 * lane);
    const uint32_t bad0 = not_finite<FMT>(w.x), bad1 = not_finite<FMT>(w.y);
    if (!__any_sync(0xFFFFFFFFu, (bad0 | bad1) != 0)) return;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      bool hit[NT][2] = {};
#pragma unroll 1
      for (int r = 0; r < kTile; ++r) {       // the scale of this lane's elements 4g .. 4g + 3 of the block
        const uint8_t* at = sp + r * kv::scale_bytes(D) + 2 * blk;
        const uint32_t sc = FMT == WQ_Q4_0 ? *reinterpret_cast<const uint16_t*>(at) : at[g >> 2];
        const int t = tile * kTile + r;
        if (not_finite<FMT>(sc) == 0) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) hit[j][c] |= t >= c_lo[j][c] && t < c_hi[j][c];
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (hit[j][i & 1]) o[j][2 * blk + (i >> 2)][i & 3] = __uint_as_float(0x7FC00000u);
    }
    __syncwarp();
    constexpr int kTop = FMT == WQ_Q4_0 ? 15 : 7;
    constexpr uint32_t kAll = FMT == WQ_Q4_0 ? 0xFFFFu : 0xFFu;
    if (bad0 | bad1) *reinterpret_cast<uint2*>(sp + 8 * lane) = make_uint2(w.x & ~((bad0 >> kTop) * kAll), w.y & ~((bad1 >> kTop) * kAll));
    __syncwarp();
  };
  // One tile.  masked: some row does not see all of it, or (careful) V's scales are looked at.
  auto work = [&](auto masked_c, bool careful, int tile, int stage, uint32_t gone) {
    constexpr bool masked = decltype(masked_c)::value;
    const uint32_t base = ring + stage * kStageBytes;
    uint8_t* gen = smem + (base - smem_u32(smem));
    if (masked && careful) clean(tile, gen + 2 * kCodes + kScales);
    // ---- scores, two groups at a time
    float s[kGroups][NT][4];
#pragma unroll
    for (int u = 0; u < kGroups; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[u][j][k] = 0.0f;
#pragma unroll
    for (int u0 = 0; u0 < kGroups; u0 += 2) {
      uint32_t kw[2][2][4];               // [group][token g or g + 8][block]
      float kd[2][2][FMT == WQ_Q4_0 ? NB : 1];
      uint32_t ks[2][2][FMT == WQ_NVFP4 ? NB : 1];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (NB == 4) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) ldsm(kw[u][hf], base + lane_at + (16 * (u0 + u) + 8 * hf) * (D / 2));
        } else {
          uint32_t r[4];
          ldsm(r, base + lane_at + 16 * (u0 + u) * (D / 2));
          kw[u][0][0] = r[0]; kw[u][0][1] = r[1]; kw[u][1][0] = r[2]; kw[u][1][1] = r[3];
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint8_t* sp = gen + 2 * kCodes + (16 * (u0 + u) + 8 * hf + g) * kv::scale_bytes(D);
          uint32_t w[2];
          if (NB == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(sp);
            w[0] = v.x; w[1] = v.y;
          } else {
            w[0] = w[1] = *reinterpret_cast<const uint32_t*>(sp);
          }
          if (FMT == WQ_Q4_0) {
#pragma unroll
            for (int blk = 0; blk < NB; ++blk)
              kd[u][hf][FMT == WQ_Q4_0 ? blk : 0] = f16_bits_to_f32((w[blk >> 1] >> (16 * (blk & 1))) & 0xFFFFu);
          } else {
            // the word of lane q lies in the 16-block q >> 1 of its 32 elements
            const uint32_t sel = (q >> 1) ? 0x3311u : 0x2200u;
#pragma unroll
            for (int pr = 0; pr < NB / 2; ++pr)
              kv::e4m3_pairs(__byte_perm(w[pr], 0, sel), ks[u][hf][FMT == WQ_NVFP4 ? 2 * pr : 0], ks[u][hf][FMT == WQ_NVFP4 ? 2 * pr + 1 : 0]);
          }
        }
      }
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        uint32_t av[2][2][4];             // [group][token g or g + 8][pair]
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t w = kw[u][hf][blk];
            if (FMT == WQ_Q4_0) {
              av[u][hf][0] = w & 0x000F000Fu;
              av[u][hf][1] = w & 0x00F000F0u;
              av[u][hf][2] = (w >> 8) & 0x000F000Fu;
              av[u][hf][3] = (w >> 8) & 0x00F000F0u;
            } else {
              kv::e2m1_pairs(w, av[u][hf]);
#pragma unroll
              for (int e = 0; e < 4; ++e) av[u][hf][e] = mul2(av[u][hf][e], ks[u][hf][FMT == WQ_NVFP4 ? blk : 0]);
            }
          }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t f[4];
          if (kQSmem) {
            const uint4 v = reinterpret_cast<const uint4*>(qs)[(j * NB + blk) * 32 + lane];
            f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = qf[kQSmem ? 0 : j][blk][e];
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (FMT == WQ_Q4_0) {
              const int ib = FMT == WQ_Q4_0 ? blk : 0;
              float c[4];
              mma_from(c, av[u][0][0], av[u][1][0], av[u][0][1], av[u][1][1], f[0], f[1], init[j][ib]);
              mma(c, av[u][0][2], av[u][1][2], av[u][0][3], av[u][1][3], f[2], f[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) s[u0 + u][j][k] = fmaf(kd[u][k >> 1][ib], c[k], s[u0 + u][j][k]);
            } else {
              mma(s[u0 + u][j], av[u][0][0], av[u][1][0], av[u][0][1], av[u][1][1], f[0], f[1]);
              mma(s[u0 + u][j], av[u][0][2], av[u][1][2], av[u][0][3], av[u][1][3], f[2], f[3]);
            }
          }
        }
      }
    }

    // ---- online softmax: c[0], c[1] are token g's columns 2q, 2q + 1, c[2], c[3] token g + 8's
    uint32_t pf[kGroups][NT][2];              // p as fp16 pairs of columns: tokens g, g + 8
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        float (&v)[4] = s[u][j];
        mul_pair(v[0], v[1], fac[j][0], fac[j][1]);
        mul_pair(v[2], v[3], fac[j][0], fac[j][1]);
        if (masked) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int t = tile * kTile + 16 * u + 8 * (k >> 1) + g;
            if (t < c_lo[j][k & 1] || t >= c_hi[j][k & 1] || ((gone >> u) & 1u)) v[k] = -INFINITY;
          }
        }
        top[0] = max3(top[0], v[0], v[2]);
        top[1] = max3(top[1], v[1], v[3]);
      }
      // most tiles of a long sequence move no maximum: then nothing is exchanged or rescaled
      if (__any_sync(0xFFFFFFFFu, top[0] > m[j][0] || top[1] > m[j][1])) {
        float f[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], d));
          top[c] = fmaxf(top[c], m[j][c]);
          f[c] = ex2(m[j][c] + (top[c] == -INFINITY ? 0.0f : -top[c]));
          m[j][c] = top[c];
          l[j][c] *= f[c];
        }
#pragma unroll
        for (int d = 0; d < 2 * NB; ++d) {
          mul_pair(o[j][d][0], o[j][d][1], f[0], f[1]);
          mul_pair(o[j][d][2], o[j][d][3], f[0], f[1]);
        }
      }
      const float base0 = m[j][0] == -INFINITY ? 0.0f : kUp - m[j][0], base1 = m[j][1] == -INFINITY ? 0.0f : kUp - m[j][1];
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        float (&v)[4] = s[u][j];
        add_pair(v[0], v[1], base0, base1);
        add_pair(v[2], v[3], base0, base1);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = ex2(v[k]);
        add_pair(l[j][0], l[j][1], v[0], v[1]);
        add_pair(l[j][0], l[j][1], v[2], v[3]);
        pf[u][j][0] = pack_f16x2(v[0], v[1]);
        pf[u][j][1] = pack_f16x2(v[2], v[3]);
      }
    }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      uint32_t pb[NT][2];               // B operand: row g's tokens 2q, 2q + 1 and 2q + 8, 2q + 9
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        pb[j][0] = movm_t(pf[u][j][0]);
        pb[j][1] = movm_t(pf[u][j][1]);
      }
      uint32_t vw[2][4];                // [tokens 0 .. 7 or 8 .. 15][block]
      if (NB == 4) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) ldsm_t(vw[hf], base + kCodes + lane_at + (16 * u + 8 * hf) * (D / 2));
      } else {
        uint32_t r[4];
        ldsm_t(r, base + kCodes + lane_at + 16 * u * (D / 2));
        vw[0][0] = r[0]; vw[0][1] = r[1]; vw[1][0] = r[2]; vw[1][1] = r[3];
      }
      uint32_t vs[2][4];                // scales of tokens (2q, 2q + 1) + 8 hf as fp16 pairs, per 32-block
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint8_t* sp = gen + 2 * kCodes + kScales + (16 * u + 8 * hf + 2 * q) * kv::scale_bytes(D);
        uint32_t t0[2], t1[2];
        if (NB == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(sp);
          t0[0] = v.x; t0[1] = v.y; t1[0] = v.z; t1[1] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(sp);
          t0[0] = t0[1] = v.x;
          t1[0] = t1[1] = v.y;
        }
#pragma unroll
        for (int pr = 0; pr < NB / 2; ++pr) {
          if (FMT == WQ_Q4_0) {
            vs[hf][2 * pr] = __byte_perm(t0[pr], t1[pr], 0x5410u);
            vs[hf][2 * pr + 1] = __byte_perm(t0[pr], t1[pr], 0x7632u);
          } else {
            // four codes of lane g lie in the 16-block g >> 2 of the 32 elements
            kv::e4m3_pairs(__byte_perm(t0[pr], t1[pr], (g >> 2) ? 0x7351u : 0x6240u), vs[hf][2 * pr], vs[hf][2 * pr + 1]);
          }
        }
      }
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        uint32_t av[2][4];              // [tokens][element 4g + e of the block]
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t w = vw[hf][blk];
          if (FMT == WQ_Q4_0) {
            kv::signed_pairs(w, av[hf][0], av[hf][1]);
            kv::signed_pairs(w >> 8, av[hf][2], av[hf][3]);
            const uint32_t d = masked && careful ? mul2(vs[hf][blk], eighth(vs[hf][blk])) : vs[hf][blk];
#pragma unroll
            for (int e = 0; e < 4; ++e) av[hf][e] = mul2(av[hf][e], d);
          } else {
            // pairs of elements 0, 1 and 2, 3 of token 2q, then of token 2q + 1
            uint32_t r[4];
            kv::e2m1_pairs(w, r);
            av[hf][0] = mul2(__byte_perm(r[0], r[2], 0x5410u), vs[hf][blk]);
            av[hf][1] = mul2(__byte_perm(r[0], r[2], 0x7632u), vs[hf][blk]);
            av[hf][2] = mul2(__byte_perm(r[1], r[3], 0x5410u), vs[hf][blk]);
            av[hf][3] = mul2(__byte_perm(r[1], r[3], 0x7632u), vs[hf][blk]);
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t b0 = pb[j][0], b1 = pb[j][1];
          if (FMT == WQ_Q4_0 && masked && careful) {
            b0 = mul2(b0, eightfold(vs[0][blk]));
            b1 = mul2(b1, eightfold(vs[1][blk]));
          }
          mma(o[j][2 * blk], av[0][0], av[0][1], av[1][0], av[1][1], b0, b1);
          mma(o[j][2 * blk + 1], av[0][2], av[0][3], av[1][2], av[1][3], b0, b1);
        }
      }
    }
  };
  // Once a weight's product was not finite its sum in O stays so: then the warp goes through its tiles once more, carefully.
  int from = (kStages - 1) * kGroups, start = t_begin;
  for (bool careful = false;; careful = true) {
    int stage = 0;
    for (int tile = start; tile < t_end; tile += kWarps) {
      {
        const int ahead = tile + (kStages - 1) * kWarps;
        int s = stage + kStages - 1;
        if (s >= kStages) s -= kStages;
        if (from == 32) {               // the next kSpan tiles' rows; those after them come in meanwhile
          from = 0;
          rows_now = rows_next;
          rows_next = locate(ahead + kSpan * kWarps);
        }
        if (ahead < t_end) issue(ahead, s, rows_now, from);
        from += kGroups;
        cp_commit();
      }
      cp_wait<kStages - 1>();
      __syncwarp();
      const uint32_t gone = (missing >> (4 * stage)) & 15u;
      if (careful || gone != 0 || tile * kTile < lo_max || (tile + 1) * kTile > hi_min) {
        if (tile >= t_begin) work(std::true_type{}, careful, tile, stage, gone);
      } else {
        work(std::false_type{}, false, tile, stage, 0u);
      }
      if (++stage == kStages) stage = 0;
      __syncwarp();                     // every lane has read the stage before it is filled again
    }
    if (careful) break;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float z = 0.0f;                 // 0 times O, all added up
#pragma unroll
        for (int d = 0; d < 2 * NB; ++d) z = fmaf(o[j][d][c], 0.0f, fmaf(o[j][d][c + 2], 0.0f, z));
        odd |= z != 0.0f && 8 * j + 2 * q + c < rows;
      }
    if (!__any_sync(0xFFFFFFFFu, odd)) break;
    reset();
    cp_wait<0>();                       // the ring is empty; two rounds fill it again
    __syncwarp();
    rows_now = locate(t_begin);
    rows_next = locate(t_begin + kSpan * kWarps);
    from = 0;
    start = t_begin - (kStages - 1) * kWarps;
  }
  cp_wait<0>();

  // ---------------------------------------------------------------- joining the warps
  // o[j][2 blk + e2]: c[0], c[1]: element 32 blk + 4 g + 2 e2 of rows 2q, 2q + 1; c[2], c[3]: the next one
  const float vg = FMT == WQ_NVFP4 && a.kv.g[1] ? *a.kv.g[1] : 1.0f;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], d);
  __syncthreads();                      // the rings are free
  float* so = reinterpret_cast<float*>(smem);
  float2* sml = reinterpret_cast<float2*>(smem + kWarps * 8 * NT * D * 4);
  if (g == 0) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) sml[warp * 8 * NT + 8 * j + 2 * q + c] = make_float2(m[j][c] - kUp, l[j][c]);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = FMT == WQ_NVFP4 ? o[j][2 * blk + e2][k] * vg : o[j][2 * blk + e2][k];
        float* dst = so + (warp * 8 * NT + 8 * j + 2 * q) * D + 32 * blk + 4 * g + 2 * e2;
        *reinterpret_cast<float2*>(dst) = make_float2(v[0], v[2]);
        *reinterpret_cast<float2*>(dst + D) = make_float2(v[1], v[3]);
      }
  __syncthreads();
  // Thread t of a row's kPerRow takes its elements 4 t, 4 t + 4 kPerRow, ...
  constexpr int kRows = 8 * NT, kPerRow = 32 * kWarps / kRows < D / 4 ? 32 * kWarps / kRows : D / 4;
  const bool joins = threadIdx.x < kRows * kPerRow;
  const int row = joins ? threadIdx.x / kPerRow : 0, part = joins ? threadIdx.x % kPerRow : 0;
  float top = -INFINITY, sum = 0.0f, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[w * kRows + row].x);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float2 v = sml[w * kRows + row];
    f[w] = v.y == 0.0f ? 0.0f : ex2(v.x - top);
    sum = fmaf(v.y, f[w], sum);
  }
  float4 acc[D / (4 * kPerRow)];
#pragma unroll
  for (int k = 0; k < D / (4 * kPerRow); ++k) {
    acc[k] = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(so + (w * kRows + row) * D + 4 * (part + k * kPerRow));
      acc[k].x = fmaf(f[w], v.x, acc[k].x);
      acc[k].y = fmaf(f[w], v.y, acc[k].y);
      acc[k].z = fmaf(f[w], v.z, acc[k].z);
      acc[k].w = fmaf(f[w], v.w, acc[k].w);
    }
  }

  // ---------------------------------------------------------------- joining the blocks of a cluster
  // Each leaves its O, m and l in its own shared memory (warp 0's part), and writes every cluster'th
  // vector of the joined rows.
  int first = 0, step = 1;
  if (p.cluster > 1) {
    first = (int)cluster_ctarank();
    step = p.cluster;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < D / (4 * kPerRow); ++k)
      if (joins) *reinterpret_cast<float4*>(so + row * D + 4 * (part + k * kPerRow)) = acc[k];
    if (joins && part == 0) sml[row] = make_float2(top, sum);
    cluster_sync();
    float2 ml[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ml[c] = make_float2(-INFINITY, 0.0f);
      if (c < p.cluster) {
        const uint32_t at = map_shared_rank(smem_u32(sml + row), c);
        ml[c] = make_float2(ld_shared_cluster_f32(at), ld_shared_cluster_f32(at + 4));
      }
    }
    top = -INFINITY;
    sum = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) top = fmaxf(top, ml[c].x);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ml[c].x = ml[c].y == 0.0f ? 0.0f : ex2(ml[c].x - top);
      sum = fmaf(ml[c].y, ml[c].x, sum);
    }
#pragma unroll
    for (int k = 0; k < D / (4 * kPerRow); ++k) {
      const int vec = part + k * kPerRow;
      if (vec % step != first) continue;
      acc[k] = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c < p.cluster) {
          float v[4];
          ld_shared_cluster_f32x4(map_shared_rank(smem_u32(so + row * D + 4 * vec), c), v);
          acc[k].x = fmaf(ml[c].x, v[0], acc[k].x);
          acc[k].y = fmaf(ml[c].x, v[1], acc[k].y);
          acc[k].z = fmaf(ml[c].x, v[2], acc[k].z);
          acc[k].w = fmaf(ml[c].x, v[3], acc[k].w);
        }
      }
    }
  }

  const int i = row / p.group;
  if (!joins) {
  } else if (p.parts > 1) {
    const int64_t slot = (item * p.parts + split) * kRows + row;
    if (part == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * slot) = make_float2(top, sum);
#pragma unroll
    for (int k = 0; k < D / (4 * kPerRow); ++k)
      *reinterpret_cast<float4*>(p.part_o + slot * D + 4 * (part + k * kPerRow)) = acc[k];
  } else if (i < a.tokens) {
    const int hq = h * p.group + row - i * p.group;
    const bool some = row < rows && sum != 0.0f;
    const float inv = some ? 1.0f / sum : 0.0f;
    const int64_t at = b * a.out.batch + i * a.out.token + hq * a.out.head;
#pragma unroll
    for (int k = 0; k < D / (4 * kPerRow); ++k) {
      const int vec = part + k * kPerRow;
      if (vec % step != first) continue;
      if (some) acc[k] = make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
      else acc[k] = make_float4(0, 0, 0, 0);
      put4(a, at + 4 * vec, acc[k]);
    }
    if (a.lse && part == 0 && first == 0)
      a.lse[(b * a.tokens + i) * a.q_heads + hq] = some ? (top + log2f(sum)) * kLn2 : -INFINITY;
  }
  griddep_launch_dependents();
  if (p.cluster > 1) cluster_sync();    // the others may still read this block's shared memory
}

// Joins the parts of a query row and head.  Few parts: a warp per row.  More than kFewParts: a block per row,
// its warps over the parts, then the warps in order.  Lanes are over the elements.  Launched while the attention
// kernel runs; it waits for it.
constexpr int kJoinWarps = 8, kFewParts = 8;
template <int D, bool FEW>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Params p, int tile_rows) {
  constexpr int E = D / 32, kStep = FEW ? 1 : kJoinWarps;
  const AttendArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t id = FEW ? (int64_t)blockIdx.x * kJoinWarps + warp : blockIdx.x;   // (sequence, token, head)
  const bool there = id < a.batch * a.tokens * a.q_heads;
  const int64_t bi = id / a.q_heads, b = bi / a.tokens, i = bi - b * a.tokens;
  const int hq = (int)(id - bi * a.q_heads), h = hq / p.group;
  const int64_t r = i * p.group + (hq - h * p.group);
  const int parts = there && i < kv::count_of(a.counts, b, a.tokens) ? p.parts : 0;
  const int64_t slot = ((b * a.kv.heads + h) * p.row_tiles + r / tile_rows) * p.parts * tile_rows + r % tile_rows;
  griddep_wait();
  float top = -INFINITY, sum = 0.0f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int s = lane; s < parts; s += 32) top = fmaxf(top, p.part_ml[2 * (slot + (int64_t)s * tile_rows)]);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
#pragma unroll 4
  for (int s = FEW ? 0 : warp; s < parts; s += kStep) {
    const int64_t at = slot + (int64_t)s * tile_rows;
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
    const float f = ml.y == 0.0f ? 0.0f : ex2(ml.x - top);
    sum = fmaf(ml.y, f, sum);
    float v[E];
    if (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p.part_o + at * D + E * lane);
    else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(p.part_o + at * D + E * lane);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(f, v[e], o[e]);
  }
  if (!FEW) {
    __shared__ float so[kJoinWarps][D], sl[kJoinWarps];
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][E * lane + e] = o[e];
    if (lane == 0) sl[warp] = sum;
    __syncthreads();
    if (warp != 0) return;
    sum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      sum += sl[w];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += so[w][E * lane + e];
    }
  }
  if (!there) return;
  const bool some = sum != 0.0f;
  const float inv = some ? 1.0f / sum : 0.0f;
  const int64_t at = b * a.out.batch + i * a.out.token + hq * a.out.head + E * lane;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = some ? o[e] * inv : 0.0f;
  if (E == 4) {
    put4(a, at, make_float4(o[0], o[1], o[2 % E], o[3 % E]));
  } else if (a.f32) {
    *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out.p) + at) = make_float2(o[0], o[1]);
  } else {
    *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out.p) + at) = pack_bf16x2(o[0], o[1]);
  }
  if (a.lse && lane == 0) a.lse[id] = some ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

struct Plan {
  bool tc;           // the tensor-memory kernel
  int nt;              // 8 rows each
  int cluster, parts;  // blocks that share the tokens of a cached head, in a cluster or joined: one of the two is 1
  AttendTcPlan tcp;
  size_t slots;      // partial rows in the workspace
};

Plan plan(const KvArgs& kv, int64_t batch, int64_t tokens, int64_t q_heads, int64_t max_len, int64_t window) {
  Plan pl{};
  const int64_t group = q_heads / kv.heads, rows = tokens * group;
  // The window only ever lowers the number of parts, so that the workspace without it suffices (parts of 2048 tokens
  // are more tiles than `most` asks for, so a window that lowers `want` below 8 leaves clusters).
  const int64_t held = max_len > 0 && max_len < kv.capacity ? max_len : kv.capacity;
  const int64_t seen = window > 0 && window + tokens < held ? window + tokens : held;
  pl.tc = rows > kFewRows;
  if (pl.tc) {
    // Two groups of rows a block where that leaves a block for every SM, or where there is work for long (one group, two:
    // 1024 tokens of 32/8 heads of 128 over 4096 137 and 84 us, 512 of 20/20 of 64 over 8192 68 and 60; below the bound
    // 1024 of 16/16 of 128 over 1100 28 and 37, but 2 x 128 of 32/8 of 128 over 9000 88 and 63).  Tokens are shared where
    // SMs are left, four tiles of 128 to a part at least.
    const int64_t heads = batch * kv.heads, half = (rows + 127) / 128;
    pl.tcp.groups = heads * ((half + 1) / 2) >= kSms || half * heads * held >= (int64_t)kSms * 4096 ? 2 : 1;
    if (half == 1) pl.tcp.groups = 1;
    pl.tcp.row_tiles = (int)((half + pl.tcp.groups - 1) / pl.tcp.groups);
    const int64_t tiles = (seen + 127) / 128, most = (tiles + 3) / 4, room = kSms * (kv.dim == 64 && pl.tcp.groups == 1 ? 2 : 1);
    int64_t want = room / (heads * pl.tcp.row_tiles);
    if (want > most) want = most;
    pl.tcp.parts = (int)(want > 1 ? want : 1);
    pl.tcp.slots = pl.tcp.parts > 1 ? (size_t)(heads * pl.tcp.row_tiles * pl.tcp.parts * pl.tcp.groups * 128) : 0;
    pl.parts = pl.tcp.parts;
    pl.slots = pl.tcp.slots;
    return pl;
  }
  pl.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  const int64_t blocks = batch * kv.heads;
  const int tile = tile_tokens(kv.dim, pl.nt);
  const int64_t tiles = (seen + tile - 1) / tile, most = (tiles + 2 * kWarps - 1) / (2 * kWarps);
  int64_t want = (int64_t)kSms * blocks_per_sm(pl.nt) / (blocks > 0 ? blocks : 1);
  if (want > most) want = most;
  // Clusters come in powers of two.  Where that leaves blocks unused, parts of at least 2048 tokens are worth the
  // join kernel: five parts of 16000 tokens of 80 heads of 128 take 48 us and clusters of four 54, of 2000 tokens
  // 14.6 and 13.3.  (More blocks than fit at once never paid: 128 heads x 16000 in clusters of two, parts of
  // three, clusters of four: 74, 72, 75; 152 heads x 2000: 15, 18, 21.)
  const bool uneven = want > 2 && (want & (want - 1)) != 0 && tiles * tile >= 2048 * want;
  pl.cluster = want > 8 || uneven ? 1 : want >= 8 ? 8 : want >= 4 ? 4 : want >= 2 ? 2 : 1;
  pl.parts = want > 8 || uneven ? (int)want : 1;
  pl.slots = pl.parts > 1 ? (size_t)(blocks * pl.parts * 8 * pl.nt) : 0;
  return pl;
}

template <int D>
int launch_join(const Params& p, int tile_rows, cudaStream_t s) {
  const bool few = p.parts <= kFewParts;
  const int64_t rows = p.a.batch * p.a.tokens * p.a.q_heads, blocks = few ? (rows + kJoinWarps - 1) / kJoinWarps : rows;
  if (blocks > 0x7FFFFFFF) return WQ_ERR_SHAPE;
  cudaLaunchConfig_t jc{};
  jc.gridDim = dim3((unsigned)blocks);
  jc.blockDim = dim3(32 * kJoinWarps);
  jc.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  jc.attrs = at;
  jc.numAttrs = 1;
  if (cudaLaunchKernelEx(&jc, few ? join_kernel<D, true> : join_kernel<D, false>, p, tile_rows) != cudaSuccess)
    return WQ_ERR_CUDA;
  count_launch();
  return WQ_OK;
}

template <int FMT, int D, int NT>
int launch(const Params& p, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  if (!allow_smem(allowed, attend_kernel<FMT, D, NT>, smem_bytes(D, NT))) return WQ_ERR_CUDA;
  const int64_t grid = p.a.batch * p.a.kv.heads * p.cluster * p.parts;
  if (grid > 0x7FFFFFFF) return WQ_ERR_SHAPE;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = smem_bytes(D, NT);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, attend_kernel<FMT, D, NT>, p) != cudaSuccess) return WQ_ERR_CUDA;
  count_launch();
  if (p.parts > 1) {
    const int rc = launch_join<D>(p, 8 * NT, s);
    if (rc != WQ_OK) return rc;
  }
  return cudaGetLastError() == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}
template <int FMT, int D>
int launch_nt(const Params& p, int nt, cudaStream_t s) {
  return nt == 1 ? launch<FMT, D, 1>(p, s) : nt == 2 ? launch<FMT, D, 2>(p, s) : launch<FMT, D, 4>(p, s);
}

}  // namespace

size_t attend_workspace(const KvArgs& kv, int64_t batch, int64_t tokens, int64_t q_heads, int64_t max_len) {
  return plan(kv, batch, tokens, q_heads, max_len, 0).slots * ((size_t)kv.dim + 2) * sizeof(float);
}

int attend(const AttendArgs& a, cudaStream_t s) {
  const Plan pl = plan(a.kv, a.batch, a.tokens, a.q_heads, a.max_len, a.window);
  Params p{};
  p.a = a;
  p.group = (int)(a.q_heads / a.kv.heads);
  p.row_tiles = pl.tc ? pl.tcp.row_tiles : 1;
  p.cluster = pl.cluster;
  p.parts = pl.parts;
  p.part_o = reinterpret_cast<float*>(a.workspace);
  p.part_ml = p.part_o + pl.slots * a.kv.dim;
  if (pl.tc) {
    const int rc = attend_tc(a, pl.tcp, s);
    if (rc != WQ_OK || pl.parts == 1) return rc;
    return a.kv.dim == 64 ? launch_join<64>(p, 128 * pl.tcp.groups, s) : launch_join<128>(p, 128 * pl.tcp.groups, s);
  }
  if (a.kv.fmt == WQ_Q4_0) return a.kv.dim == 64 ? launch_nt<WQ_Q4_0, 64>(p, pl.nt, s) : launch_nt<WQ_Q4_0, 128>(p, pl.nt, s);
  return a.kv.dim == 64 ? launch_nt<WQ_NVFP4, 64>(p, pl.nt, s) : launch_nt<WQ_NVFP4, 128>(p, pl.nt, s);
}

int take_status_attend() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
