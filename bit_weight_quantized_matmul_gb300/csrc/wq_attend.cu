// wq_attend.cu -- attention over the 4-bit KV cache: which kernel, how the tokens are shared out, and the join of shared ones.
#include <algorithm>

#include "wq_attend_few.cuh"

namespace wq {
namespace {

struct JoinParams {
  AttendArgs a;
  int group, parts, row_tiles;   // query heads and row tiles per cached head; parts of a row tile
  const float* part_o;           // as the kernels left them
  const float* part_ml;
};

// Joins the parts of a query row and head.  Few parts: a warp per row.  More than kFewParts: a block per row,
// its warps over the parts, then the warps in order.  Lanes are over the elements.  Launched while the attention
// kernel runs; it waits for it.
constexpr int kJoinWarps = 8, kFewParts = 8;
template <int D, bool FEW>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ JoinParams p, int tile_rows) {
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
  bool tc;             // the tensor-memory kernel
  AttendFewPlan few;   // cluster, parts: one of the two is 1
  AttendTcPlan tcp;
  int parts;           // of the one that is taken
  size_t slots;        // partial rows in the workspace
};

Plan plan(const KvArgs& kv, int64_t batch, int64_t tokens, int64_t q_heads, int64_t max_len, int64_t window, int64_t sinks, bool sel) {
  Plan pl{};
  const int64_t group = q_heads / kv.heads, rows = tokens * group;
  // The window only ever lowers the number of parts, so that the workspace without it suffices (parts of 2048 tokens
  // are more tiles than `most` asks for, so a window that lowers `want` below 8 leaves clusters).
  const int64_t held = max_len > 0 && max_len < kv.capacity ? max_len : kv.capacity;
  const int64_t seen = window > 0 && window + tokens + sinks < held ? window + tokens + sinks : held;
  pl.tc = rows > few_rows(kv.fmt, kv.dim, sel);
  if (pl.tc) {
    // Two groups of rows a block where that leaves a block for every SM, or where there is work for long (one group, two:
    // 1024 tokens of 32/8 heads of 128 over 4096 137 and 84 us, 512 of 20/20 of 64 over 8192 68 and 60; below the bound
    // 1024 of 16/16 of 128 over 1100 28 and 37, but 2 x 128 of 32/8 of 128 over 9000 88 and 63).  Tokens are shared where
    // SMs are left, four tiles of 128 to a part at least (sinks and trees: below).
    const int64_t heads = batch * kv.heads, half = (rows + 127) / 128;
    pl.tcp.groups = heads * ((half + 1) / 2) >= kSms || half * heads * held >= (int64_t)kSms * 4096 ? 2 : 1;
    // Sinks and trees of heads of 64: one group where that is more than a block an SM, of which two fit (4 x 301 tokens behind a
    // window of 292 of 20 heads two groups 43 us, one 26; 2 x 1024 behind 2048 109 and 100; 32 x 20 .. 64 nodes over 1000 ..
    // 6000 250 and 176; below the bound 3 x 200 behind 4000 48 and 52).
    if (half == 1 || (sel && kv.dim == 64 && heads * half > kSms)) pl.tcp.groups = 1;
    pl.tcp.row_tiles = (int)((half + pl.tcp.groups - 1) / pl.tcp.groups);
    // Behind a window a row tile sees what one of its tokens does and as many tokens more as it has, and a tile more for
    // where they begin (512 tokens behind 100 of 32/8 heads of 128 21 us, two parts 27; 130 behind 400 of 32/4 24,
    // three parts 18).
    const int64_t wide = pl.tcp.groups * 128 / group + 1;
    const int64_t mine = sel && window > 0 && window + sinks + wide + 128 < seen ? window + sinks + wide + 128 : seen;
    const int64_t tiles = (mine + 127) / 128, most = (tiles + 3) / 4, room = kSms * ((kv.dim == 64 || sel) && pl.tcp.groups == 1 ? 2 : 1);
    int64_t want = room / (heads * pl.tcp.row_tiles);
    if (!sel) {
      if (want > most) want = most;
    } else {
      // Sinks and trees: two tiles to a part, four past the eight parts that a warp joins, and no few parts past those (two,
      // three, four tiles: 20 nodes over 2000 of 32/8 heads of 128 17.1, 18.4, 20.2 us, 3 x 40 over 800 .. 1500 of 8/1 of 64
      // 15.0, 16.3, 17.9; 4 x 24 over 1000 .. 3000 of 32/8 of 128 in nine parts 31.7, in eight 25.7; 2 x 64 over 4000 .. 6000
      // of 16/16 35 and 32).  Four tiles stay whole where the join has many rows (512 tokens behind 300 of 32/8 of 128 whole
      // 26.7, halved 31.3, 8 x 40 over 400 .. 500 of 16/16 18.3 and 21.6; 2 x 200 behind 300 of 6/6 of 64 19.2 and 16.1).
      want = std::min(want, (tiles + 1) / 2);
      if (tiles <= 4 && 2 * heads * pl.tcp.row_tiles * pl.tcp.groups > kSms) want = 1;
      if (want > kFewParts) want = std::max<int64_t>(kFewParts, std::min(want, most));
      if (want < kFewParts + 4) want = std::min<int64_t>(want, kFewParts);
    }
    pl.tcp.parts = (int)(want > 1 ? want : 1);
    pl.tcp.slots = pl.tcp.parts > 1 ? (size_t)(heads * pl.tcp.row_tiles * pl.tcp.parts * pl.tcp.groups * 128) : 0;
    pl.parts = pl.tcp.parts;
    pl.slots = pl.tcp.slots;
    return pl;
  }
  pl.few.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  const int64_t blocks = batch * kv.heads;
  const int tile = tile_tokens(kv.dim, pl.few.nt);
  const int64_t tiles = (seen + tile - 1) / tile, most = (tiles + 2 * kWarps - 1) / (2 * kWarps);
  int64_t want = (int64_t)kSms * blocks_per_sm(pl.few.nt) / (blocks > 0 ? blocks : 1);
  if (want > most) want = most;
  // More items than half of the places: each of long sequences in two parts, in the order of by_length, so that what runs last
  // is short (a block alone on its SM does not go faster than one of three): 64 x 1 over 1000 .. 32000 behind a window of
  // 4096 of 32/8 heads of 128 in one part 84 us, in two 80, in three 83; 40 x 2 nodes over 1000 .. 9000 90, 68, 67; 64 x 2 nodes
  // behind a window of 1000, whose blocks are short, 56, 68, 78; 32 x 3 over 500 .. 8000 of 20 heads of 64 58, 66, 72; 64 x 5
  // (20 rows) over 1000 .. 16000 274, 308, 314.
  if (sel && want < 2 && kv.dim == 128 && pl.few.nt <= 2 && seen >= 4096) {
    pl.few.cluster = 1;
    pl.few.parts = pl.parts = 2;
    pl.few.slots = pl.slots = (size_t)(blocks * 2 * 8 * pl.few.nt);
    return pl;
  }
  // Clusters come in powers of two.  Where that leaves blocks unused, parts of at least 2048 tokens are worth the
  // join kernel: five parts of 16000 tokens of 80 heads of 128 take 48 us and clusters of four 54, of 2000 tokens
  // 14.6 and 13.3.  (More blocks than fit at once never paid: 128 heads x 16000 in clusters of two, parts of
  // three, clusters of four: 74, 72, 75; 152 heads x 2000: 15, 18, 21.)
  const bool uneven = want > 2 && (want & (want - 1)) != 0 && tiles * tile >= 2048 * want;
  pl.few.cluster = want > 8 || uneven ? 1 : want >= 8 ? 8 : want >= 4 ? 4 : want >= 2 ? 2 : 1;
  pl.few.parts = pl.parts = want > 8 || uneven ? (int)want : 1;
  pl.few.slots = pl.slots = pl.parts > 1 ? (size_t)(blocks * pl.parts * 8 * pl.few.nt) : 0;
  return pl;
}

template <int D>
int launch_join(const JoinParams& p, int tile_rows, cudaStream_t s) {
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

}  // namespace

size_t attend_workspace(const KvArgs& kv, int64_t batch, int64_t tokens, int64_t q_heads, int64_t max_len, bool sel) {
  return plan(kv, batch, tokens, q_heads, max_len, 0, 0, sel).slots * ((size_t)kv.dim + 2) * sizeof(float);
}

int attend(const AttendArgs& a, cudaStream_t s) {
  const bool sel = a.tree_mask || (a.window > 0 && a.sinks > 0);
  const Plan pl = plan(a.kv, a.batch, a.tokens, a.q_heads, a.max_len, a.window, sel ? a.sinks : 0, sel);
  const int rc = pl.tc ? (sel ? attend_tc_sel : attend_tc)(a, pl.tcp, s) : (sel ? attend_few_sel : attend_few)(a, pl.few, s);
  if (rc != WQ_OK || pl.parts == 1) return rc;
  JoinParams p{};
  p.a = a;
  p.group = (int)(a.q_heads / a.kv.heads);
  p.parts = pl.parts;
  p.row_tiles = pl.tc ? pl.tcp.row_tiles : 1;
  p.part_o = reinterpret_cast<const float*>(a.workspace);
  p.part_ml = p.part_o + pl.slots * a.kv.dim;
  const int tile_rows = pl.tc ? 128 * pl.tcp.groups : 8 * pl.few.nt;
  return a.kv.dim == 64 ? launch_join<64>(p, tile_rows, s) : launch_join<128>(p, tile_rows, s);
}

int attend_few(const AttendArgs& a, const AttendFewPlan& pl, cudaStream_t s) { return launch_few<false>(a, pl, s); }

int take_status_attend() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
