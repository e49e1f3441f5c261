// wq_internal.h -- host-side interfaces between the library's translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/wq.h"
#include "wq_once.h"

namespace wq {

// Layout of a packed weight's `scales` blob (see include/wq.h).
struct ScalesLayout {
  size_t absmax_bytes = 0;  // NF4: int8 absmax codes
  size_t s2_off = 0;        // NF4: byte offset of the fp32 s2 array
  int64_t n_groups = 0;     // NF4: number of s2 values
  size_t offset_off = 0;    // NF4: byte offset of the fp32 offset
  size_t sf_bytes = 0;      // NVFP4: E4M3 block scales
  size_t g_off = 0;         // NVFP4: byte offset of the fp32 g
  size_t total = 0;
};
// Packed bytes of one weight row (K elements) of a format.
inline int64_t packed_row_bytes(int fmt, int64_t K) {
  switch (fmt) {
    case WQ_Q8_0:
    case WQ_FP8: return K;
    case WQ_Q5_0:
    case WQ_Q4_1: return K / 128 * 80;
    default: return K / 2;
  }
}
ScalesLayout scales_layout(int fmt, int64_t N, int64_t K);

inline size_t align16(size_t n) { return (n + 15) / 16 * 16; }

// Host-side launch counter (all translation units).
void count_launch(int n = 1);

// Lets a kernel have `bytes` of dynamic shared memory on the current device.  done: one per kernel, static.
template <class Kernel>
inline bool allow_smem(std::atomic<uint64_t>& done, Kernel* kern, int bytes) {
  int device = -1;
  return cudaGetDevice(&device) == cudaSuccess && once_per_device(done, device, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  });
}

// Launches `kernel` so that it may begin while the kernel before it on the stream ends: the launch is then not waited for,
// which is a microsecond of a call of few tokens.  The kernel calls griddep_wait() before it touches memory, and lets the next one
// begin (griddep_launch_dependents()) only behind that: then what came before it is complete for the next one too.  One that uses
// tensor memory allocates it before it lets the next one begin.
template <class... Params, class... Args>
inline cudaError_t launch_early(void (*kernel)(Params...), dim3 blocks, dim3 threads, size_t smem, cudaStream_t s, unsigned cluster,
                                const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = blocks;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// ---- pack / dequant / activation quantiser (wq_pack.cu)
int pack_nf4(const float* W, int64_t N, int64_t K, uint8_t* packed, uint8_t* scales, cudaStream_t s);
int pack_nvfp4(const float* W, int64_t N, int64_t K, uint8_t* packed, uint8_t* scales, cudaStream_t s);
int pack_q4_0(const float* W, int64_t N, int64_t K, uint8_t* packed, uint8_t* scales, cudaStream_t s);
int pack_q8_0(const float* W, int64_t N, int64_t K, uint8_t* packed, uint8_t* scales, cudaStream_t s);
int pack_q4_1(const float* W, int64_t N, int64_t K, uint8_t* packed, uint8_t* scales, cudaStream_t s);
int pack_q5_0(const float* W, int64_t N, int64_t K, uint8_t* packed, uint8_t* scales, cudaStream_t s);
int pack_fp8(const float* W, int64_t N, int64_t K, uint8_t* packed, uint8_t* scales, cudaStream_t s);
int dequant(const uint8_t* packed, const uint8_t* scales, int fmt, int64_t N, int64_t K, float* out,
            cudaStream_t s);
int quant_act_nvfp4(const uint16_t* x, int64_t M, int64_t K, const float* g_in, uint8_t* codes,
                    uint8_t* scales, float* g_out, cudaStream_t s);
int take_status_pack();
int selftest_timeout(uint32_t polls, cudaStream_t s);  // bounded wait on a barrier nobody arrives on
int selftest_encoders(const float* in, int64_t n, uint8_t* out, cudaStream_t s);

// ---- linear: CUDA-core path (wq_simt.cu)
struct LinearArgs {
  const void* x;               // bf16 [M, K] (W4A16) -- unused for W4A4
  const uint8_t* act_codes;    // W4A4 activations
  const uint8_t* act_scales;
  const float* act_g;
  const uint8_t* packed;
  const uint8_t* scales;
  int fmt;
  int64_t M, N, K;
  const uint16_t* bias;
  void* y;                     // single output [M, N] (nout == 1, ld == N)
  bool out_f32;
  bool weights_static;         // may launch with programmatic dependent launch
  // Output destinations: columns [col_end[d-1], col_end[d]) of row m go to
  // ys[d] + m * ld[d] + (n - col_end[d-1]) (elements).  set_single_out() fills one destination.
  int nout;
  void* ys[WQ_OUT_MAX];
  int64_t ld[WQ_OUT_MAX];
  int64_t col_end[WQ_OUT_MAX];
};
inline void set_single_out(LinearArgs& a) {
  a.nout = 1;
  a.ys[0] = a.y;
  a.ld[0] = a.N;
  a.col_end[0] = a.N;
  for (int d = 1; d < WQ_OUT_MAX; ++d) { a.ys[d] = a.y; a.ld[d] = a.N; a.col_end[d] = a.N; }
}
// One Linear of any shape and output layout: the tensor-core paths where their rules hold,
// else the CUDA-core kernel.
int linear_one(const LinearArgs& a, cudaStream_t s);
int linear_simt(const LinearArgs& a, cudaStream_t s);
int take_status_simt();

// ---- linear: decode-sized single Linear on the CUDA cores (wq_gemv.cu)
constexpr int kGemvMaxM = 4;  // single Linears with up to this many activation rows take the GEMV
constexpr int kTcpDecodeMaxK = 2048;  // longer single decode Linears split K over a cluster instead
bool gemv_eligible(const LinearArgs& a);
int linear_gemv(const LinearArgs& a, cudaStream_t s);

// ---- linear: tensor-core paths (wq_tc.cu: decode split-K; wq_tcp.cu: persistent work list;
//      wq_w4a4.cu: block-scaled FP4)
constexpr int kGroupMax = WQ_GROUP_MAX;
bool tcp_eligible(const LinearArgs& a);
int linear_tcp(const LinearArgs* probs, int count, cudaStream_t s);
int take_status_tcp();
// return 1 = handled (status in *rc), 0 = shape not eligible for this path
int linear_tc(const LinearArgs& a, cudaStream_t s, int* rc);
int take_status_tc();
int linear_w4a4_tc(const LinearArgs& a, cudaStream_t s, int* rc);
int take_status_w4a4();
// NVFP4 W4A16 GEMM with 512-row activation tiles (wq_w4a16.cu); 0 = shape not taken
int linear_w4a16_tc(const LinearArgs& a, cudaStream_t s, int* rc);
int take_status_w4a16();

// ---- 4-bit KV cache (wq_kv.cu) and attention over it (wq_attend.cu)
struct KvArgs {
  uint8_t* codes[2];    // K, V
  uint8_t* scales[2];
  const float* g[2];    // NVFP4 global scales, NULL = 1
  const int32_t* table; // NULL: sequence b owns page b
  int64_t table_ld;
  int64_t pages;
  int64_t capacity;     // tokens per sequence
  int32_t page_size, fmt, heads, dim;
  uint32_t page_mul, page_shift;  // t / page_size = umulhi(t, page_mul) >> page_shift for 0 <= t < 2^31
};
struct HeadsArg {
  void* p;
  int64_t batch, token, head;  // element strides
};
struct KvMoveArgs {
  KvArgs kv;
  HeadsArg x[2];        // K, V rows (x[i].p == NULL: not wanted)
  int64_t batch, tokens;
  const int32_t* start;
  const int32_t* counts;
  bool f32;
};
int kv_append(const KvMoveArgs& a, cudaStream_t s);
int kv_read(const KvMoveArgs& a, cudaStream_t s);
// Tokens laid end to end (x[..].batch unused), each to its slot.
struct KvSlotArgs {
  KvArgs kv;
  HeadsArg x[2];
  int64_t tokens;
  const int64_t* slots;
};
int kv_append_slots(const KvSlotArgs& a, cudaStream_t s);
int take_status_kv();

// ---- pages, slots and trees (wq_pages.cu)
struct KvReserveArgs {
  KvArgs kv;
  const int32_t* free_pages;   // release writes it
  int64_t free_size;
  const int32_t* top;
  int32_t* top_out;            // may be top
  int64_t batch;
  const int32_t* lens;
  const int32_t* counts;       // reserve: new tokens; release: tokens that stay (NULL: none)
  int32_t* granted;
  int64_t tokens;              // of the slot map
  int64_t* slots;
  int32_t* positions;
  int32_t* starts;
};
struct KvKeepArgs {
  KvArgs kv;
  int64_t batch;
  const int32_t* start;
  const int32_t* path;         // [batch, path_ld]
  int64_t path_ld;
  const int32_t* counts;
};
int kv_reserve(const KvReserveArgs& a, cudaStream_t s);
int kv_release(const KvReserveArgs& a, cudaStream_t s);
int kv_keep(const KvKeepArgs& a, cudaStream_t s);
struct TreeMaskArgs {
  const int32_t* parents;      // [batch, tokens]
  const int32_t* counts;
  const int32_t* lens;         // read where there are a window and sinks
  int64_t batch, tokens, window, sinks;
  uint32_t* mask;
  int32_t* depth;
};
int tree_mask(const TreeMaskArgs& a, cudaStream_t s);
int take_status_pages();

struct AttendArgs {
  KvArgs kv;
  HeadsArg q, out;
  float* lse;
  int64_t batch, tokens, q_heads;
  const int32_t* lens;
  const int32_t* counts;
  int64_t max_len;
  float scale;
  int64_t window;       // 0: none
  bool causal, f32;
  void* workspace;
  size_t workspace_bytes;
  // Rows that see more than one run of tokens (the SEL kernels): the first `sinks` behind a window, drafted nodes by bits.
  int32_t sinks;
  int32_t tree_words;           // of a node's bits
  const uint32_t* tree_mask;    // NULL: no tree
  const int32_t* tree_depth;    // NULL: node i is at depth i
  int64_t mask_batch, depth_batch;
};
size_t attend_workspace(const KvArgs& kv, int64_t batch, int64_t tokens, int64_t q_heads, int64_t max_len, bool sel);
int attend(const AttendArgs& a, cudaStream_t s);
int take_status_attend();
// Few query rows per cached head (wq_attend_few.cuh; 8 * nt of them): blocks of a cluster, or parts joined afterwards, share
// the tokens.  Many (wq_attend_tc.cuh): groups of 128 rows a block, parts that share the tokens of a row tile.  The _sel forms,
// in translation units of their own, are for sinks and trees.
struct AttendFewPlan {
  int nt, cluster, parts;
  size_t slots;
};
struct AttendTcPlan {
  int groups, row_tiles, parts;
  size_t slots;
};
int attend_few(const AttendArgs& a, const AttendFewPlan& pl, cudaStream_t s);
int attend_few_sel(const AttendArgs& a, const AttendFewPlan& pl, cudaStream_t s);
int attend_tc(const AttendArgs& a, const AttendTcPlan& pl, cudaStream_t s);
int attend_tc_sel(const AttendArgs& a, const AttendTcPlan& pl, cudaStream_t s);
int take_status_attend_tc();
int take_status_attend_few_sel();
int take_status_attend_tc_sel();

// driver entry point for tensor-map encoding (resolved once through the runtime)
bool encode_tmap_2d(void* tmap, CUtensorMapDataType dtype, const void* base, uint64_t inner, uint64_t outer,
                    uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz);

}  // namespace wq
