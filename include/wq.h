/*
 * wq.h -- C ABI of libwq: fused dequantise-and-multiply of a block-quantised
 * Linear layer on GB300 (sm_103a),
 *
 *     y[M, N] = x[M, K] . dequant(W)[N, K]^T  (+ bias[N]).
 *
 * Source of the operation
 *   - PR "asr: add a 4-bit nf4 option for the Whisper engine", summary and
 *     "Why NF4 and not the NVFP4 snapshot": the weights are stored in 4 bits,
 *     activations stay bf16, and the dequantisation is fused into the matmul
 *     instead of unpacking W to bf16 and calling an ordinary GEMM.
 *   - model card "whisper-large-v3-turbo -- NVFP4", "What is quantized" and
 *     "Honest summary": NVFP4 weights (E2M1, E4M3 scale per 16, FP32 global
 *     scale) run as W4A16, and on Blackwell as W4A4 with activations
 *     quantised per 16 values at runtime.
 *   - PR "Run quantized Whisper on the fused Metal decode path", "Summary":
 *     GGUF q8_0 / q4_0 blocks of 32 with an fp16 scale.
 *
 * Conventions (all entry points)
 *   - W is PyTorch-Linear shaped, W[N, K] row-major, K contiguous; every
 *     quantisation block runs along K.  x is [M, K] row-major, y is [M, N]
 *     row-major.  bf16 / fp16 values are passed as their 16-bit patterns.
 *   - Every pointer argument is a DEVICE pointer unless stated otherwise.  The
 *     caller allocates and owns every buffer; the library never allocates,
 *     frees or synchronises (except wq_last_device_status).
 *   - Every call is asynchronous on `stream` (a cudaStream_t, NULL = legacy
 *     default stream) and returns a wq_status.  Arguments are checked before
 *     any launch; a failed check launches nothing.  No C++ exception crosses
 *     the ABI.
 *   - Device pointers must be 16-byte aligned (WQ_ERR_ALIGN otherwise).
 *   - Calls that share output buffers race if they overlap on the GPU; order
 *     them on one stream.
 */
#ifndef WQ_H_
#define WQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum wq_fmt {
  WQ_NF4 = 1,        /* NF4 codes, block 64, absmax double-quantised (int8 per 256, fp32 scale) */
  WQ_NVFP4 = 2,      /* E2M1 codes, block 16, E4M3 block scale, fp32 global; bf16 activations   */
  WQ_NVFP4_W4A4 = 3, /* NVFP4 weights AND NVFP4 activations (see wq_act_nvfp4)                   */
  WQ_Q4_0 = 4,       /* 4-bit codes, block 32, fp16 d, value (q - 8) * d                        */
  WQ_Q8_0 = 5,       /* int8 codes, block 32, fp16 d, value q * d                               */
  WQ_Q4_1 = 6,       /* 4-bit codes, block 32, fp16 d and fp16 minimum m, value q * d + m       */
  WQ_Q5_0 = 7,       /* 5-bit codes, block 32, fp16 d, value (q - 16) * d                       */
  WQ_FP8 = 8         /* FP8 E4M3 codes, one fp32 scale s per weight row, value E4M3(q) * s      */
} wq_fmt;

typedef enum wq_status {
  WQ_OK = 0,
  WQ_ERR_ARG = -1,     /* NULL pointer, unknown flag, negative size                    */
  WQ_ERR_SHAPE = -2,   /* K not a multiple of the format's block (or other size rule) */
  WQ_ERR_ALIGN = -3,   /* a device pointer is not 16-byte aligned                     */
  WQ_ERR_FMT = -4,     /* unknown format, or a format the entry point does not take   */
  WQ_ERR_CUDA = -5,    /* a CUDA launch / driver call failed                           */
  WQ_ERR_TIMEOUT = -6  /* a kernel gave up on a bounded wait (see wq_last_device_status) */
} wq_status;

/* Activations of WQ_NVFP4_W4A4, as written by wq_quant_act_nvfp4.  The struct
 * itself lives in HOST memory; its members are device pointers:
 *   codes  [M, K/2] bytes, two E2M1 codes per byte, element 2j in the low nibble
 *   scales [M, K/16] E4M3 bytes, row-major
 *   g      one fp32: the per-tensor decode multiplier                             */
typedef struct wq_act_nvfp4 {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* g;
} wq_act_nvfp4;

/* ---------------------------------------------------------------- sizes
 * Bytes of the two buffers a packed weight occupies (0 for an invalid
 * format / shape).  Storage layout:
 *   packed  NF4, NVFP4, q4_0, q4_1: N*K/2 bytes, two codes per byte, element
 *           2j of the row-major flattening in the low nibble of byte j.
 *           q8_0: N*K int8.  FP8: N*K E4M3 bytes.
 *           q5_0, q4_1: N*K*5/8 bytes in 80-byte units, one per 128
 *           consecutive elements of a row: 64 bytes of (low) nibbles, element 2j
 *           in the low nibble of byte j, then 16 bytes of side data -- q5_0: the
 *           fifth bits (bit j of byte i = element 8i + j); q4_1: the unit's four
 *           (fp16 d, fp16 m) pairs, one per 32-block.
 *   scales  NF4:   int8 absmax codes [N*K/64] | zero pad to 16 B |
 *                  fp32 second-level scale s2 [ceil(N*K/64 / 256)] | fp32 offset
 *           NVFP4: E4M3 block scales [N, K/16] row-major | zero pad to 16 B | fp32 g
 *           q4_0, q8_0, q5_0: fp16 d [N*K/32] | zero pad to 16 B
 *           q4_1:  16 zero bytes (its scales are inside the packed units)
 *           FP8:   fp32 s [N] | zero pad to 16 B
 * Size rules: NF4 K % 64 == 0; NVFP4 K % 32 == 0; q4_0 / q8_0 / FP8
 * K % 32 == 0; q5_0 / q4_1 K % 128 == 0.                                      */
size_t wq_packed_bytes(int fmt, int64_t N, int64_t K);
size_t wq_scales_bytes(int fmt, int64_t N, int64_t K);

/* ---------------------------------------------------------------- packers
 * Quantise fp32 weights W [N, K] (device) into `packed` and `scales` (device,
 * sizes above).  Deterministic and bit-identical for a given W.  The packers
 * use `packed` as working space before writing it, so W must not alias either
 * output.  WQ_NVFP4_W4A4 weights are packed with wq_pack_nvfp4.
 *
 * wq_pack_nf4   (PR "asr: add a 4-bit nf4 option ...", "What's here"):
 *   per 64-block absmax a; code = number of NF4 codebook midpoints below w / a
 *   (ties to the lower code); the absmax values are centred on their exact
 *   mean (fp32 offset) and quantised to int8 per group of 256 with an fp32
 *   scale s2 = max|a - offset| / 127.
 * wq_pack_nvfp4 (model card "whisper-large-v3-turbo -- NVFP4",
 *   "What is quantized"): g = amax(W) / 2688; per 16-block
 *   s = E4M3((amax_b / 6) / g), code = E2M1(w / (E4M3(s) * g)); round to
 *   nearest even, saturating.
 * wq_pack_q4_0  (PR "Run quantized Whisper on the fused Metal decode path",
 *   "Summary"): d = fp16(extreme / -8), q = clamp(rint(w / d) + 8, 0, 15).
 * wq_pack_q8_0  (same passage): d = fp16(amax / 127), q = clamp(rint(w / d), +-127).
 * wq_pack_q4_1, wq_pack_q5_0 (same PR, "Why the policy": the other GGUF block
 *   types): q4_1 m = fp16(min), d = fp16((max - min) / 15),
 *   q = clamp(rint((w - m) / d), 0, 15); q5_0 d = fp16(extreme / -16),
 *   q = clamp(rint(w / d) + 16, 0, 31).
 * wq_pack_fp8   (model card "whisper-large-v3-turbo -- NVFP4", "Honest
 *   summary": the FP8 build): s = amax(row) / 448, q = E4M3(w / s), round to
 *   nearest even, saturating (q = 0 for an all-zero row).
 * Every rint / E4M3 rounding is half to even, against the stored fp16 / fp32
 * scale values.
 */
int wq_pack_nf4(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream);
int wq_pack_nvfp4(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream);
int wq_pack_q4_0(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream);
int wq_pack_q8_0(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream);
int wq_pack_q4_1(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream);
int wq_pack_q5_0(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream);
int wq_pack_fp8(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream);

/* ---------------------------------------------------------------- dequant
 * Decode a packed weight to fp32 W_out [N, K] (device): the exact fp32 value
 * each code stands for (NF4: codebook * (q*s2 + offset); NVFP4:
 * (E2M1 * E4M3) * g; q4_0: (q-8)*d; q8_0: q*d; q4_1: q*d + m; q5_0:
 * (q-16)*d; FP8: E4M3(q)*s).  A verification export: the
 * fused paths below never materialise W.                                       */
int wq_dequant(const void* packed, const void* scales, int fmt, int64_t N, int64_t K,
               float* W_out, void* stream);

/* ---------------------------------------------------------------- activations
 * NVFP4 runtime activation quantiser (model card "whisper-large-v3-turbo --
 * NVFP4", "What is quantized": activations quantised per 16-value group at
 * runtime).  x: bf16 [M, K] (K % 32 == 0).  g_in: NULL for a dynamic
 * per-tensor global g = amax(x) / 2688 (1 if x is all zero), or a device
 * pointer to a static fp32 g.  Writes codes [M, K/2], scales [M, K/16] and
 * g_out (one fp32, the g that was used).  Bit-identical to the block encoder
 * of wq_pack_nvfp4.                                                            */
int wq_quant_act_nvfp4(const uint16_t* x, int64_t M, int64_t K, const float* g_in,
                       uint8_t* codes, uint8_t* scales, float* g_out, void* stream);

/* ---------------------------------------------------------------- linear
 * y = x . dequant(W)^T (+ bias), fp32 accumulation, bf16 output.
 *   x      bf16 [M, K]; for WQ_NVFP4_W4A4 a HOST pointer to a wq_act_nvfp4
 *   bias   bf16 [N] or NULL
 *   y      bf16 [M, N]
 * M == 0 is a no-op.  Dispatch: M <= 16 runs the decode path (tensor-core
 * GEMV, split-K over a thread-block cluster); larger M runs the persistent
 * tensor-core GEMM; K not a multiple of 64 runs a CUDA-core kernel with the
 * same per-weight decode.  WQ_NVFP4_W4A4 with M > 16 and K a multiple of 256
 * runs the block-scaled FP4 tensor-core GEMM (both operands packed); other
 * W4A4 shapes run the CUDA-core kernel.                                         */
int wq_linear(const void* x, const void* packed, const void* scales, int fmt,
              int64_t M, int64_t N, int64_t K, const uint16_t* bias, void* y, void* stream);

/* Flags of wq_linear_ex. */
enum {
  /* y is fp32 [M, N] instead of bf16 (same kernels; the final bf16 rounding is skipped). */
  WQ_FLAG_OUT_F32 = 1u << 0,
  /* The caller promises that `packed`, `scales` and `bias` are not written by
   * work still running on `stream`.  The kernel is then launched with
   * programmatic dependent launch and starts streaming its weights before the
   * preceding kernel on the stream has finished; it waits for that kernel
   * only before it reads x or writes y.                                        */
  WQ_FLAG_WEIGHTS_STATIC = 1u << 1,
  /* Force the CUDA-core path (verification aid). */
  WQ_FLAG_FORCE_SIMT = 1u << 2
};

int wq_linear_ex(const void* x, const void* packed, const void* scales, int fmt,
                 int64_t M, int64_t N, int64_t K, const uint16_t* bias, void* y,
                 unsigned flags, void* stream);

/* ---------------------------------------------------------------- grouped
 * Several independent Linears of ONE format in one launch (the fused Q/K/V
 * projection of PR "Run quantized Whisper on the fused Metal decode path",
 * "Summary", generalised to any set of Linears whose inputs are ready).  Each
 * problem has the meaning of one wq_linear call (same layouts and rules);
 * outputs must not overlap.  `problems` is a HOST array of `count` entries,
 * 1 <= count <= WQ_GROUP_MAX; WQ_NVFP4_W4A4 is not accepted (WQ_ERR_FMT).
 * flags: WQ_FLAG_OUT_F32 / WQ_FLAG_WEIGHTS_STATIC apply to every problem.     */
#define WQ_GROUP_MAX 48
typedef struct wq_problem {
  const void* x;          /* bf16 [M, K]          */
  const void* packed;     /* packed weight        */
  const void* scales;     /* its scales blob      */
  const uint16_t* bias;   /* bf16 [N] or NULL     */
  void* y;                /* bf16 (or fp32) [M, N] */
  int64_t M, N, K;
} wq_problem;

int wq_linear_grouped(const wq_problem* problems, int count, int fmt, unsigned flags, void* stream);

/* ---------------------------------------------------------------- grouped, strided outputs
 * wq_linear_grouped_ex: as wq_linear_grouped, but each problem's output columns
 * go to up to WQ_OUT_MAX row-strided destinations instead of one dense y.  This
 * is the fused Q/K/V projection of PR "Run quantized Whisper on the fused Metal
 * decode path", "Summary" and "Test plan": the projections of a token are
 * computed in one launch, the bias added on the device, and K and V written
 * straight into their rows of a KV-cache slab, with no copy afterwards.  It
 * also serves a merged weight: the cross-attention K and V weights stacked as
 * one [2N, K] matrix (packed once), whose first N output columns go to the K
 * slab and the last N to the V slab.
 *
 * Destination d of a problem receives the output columns
 * [c_d, c_d + out[d].ncols), c_d = out[0].ncols + ... + out[d-1].ncols: element
 * (m, n) is written to out[d].y + m * out[d].ld + (n - c_d) (elements of bf16, or
 * fp32 with WQ_FLAG_OUT_F32).  Rules (WQ_ERR_ARG / WQ_ERR_ALIGN otherwise):
 * 1 <= nout <= WQ_OUT_MAX; the ncols sum to N; every ncols but the last is a
 * multiple of 16; ld >= ncols and ld * element size is a multiple of 16 bytes;
 * every y is 16-byte aligned.  Destinations must not overlap each other or any
 * other problem's.  Nothing outside the addressed elements is written: rows of
 * a slab other than the M addressed ones, and the columns of a row beyond
 * ncols, keep their contents.                                                  */
#define WQ_OUT_MAX 4
typedef struct wq_out {
  void* y;         /* first element of the destination (device)   */
  int64_t ld;      /* row stride in elements                       */
  int64_t ncols;   /* output columns this destination receives     */
} wq_out;

typedef struct wq_problem_ex {
  const void* x;          /* bf16 [M, K]                              */
  const void* packed;     /* packed weight [N, K]                     */
  const void* scales;     /* its scales blob                          */
  const uint16_t* bias;   /* bf16 [N] or NULL                         */
  int64_t M, N, K;
  int nout;               /* destinations used, 1 .. WQ_OUT_MAX        */
  wq_out out[WQ_OUT_MAX];
} wq_problem_ex;

int wq_linear_grouped_ex(const wq_problem_ex* problems, int count, int fmt, unsigned flags, void* stream);

/* ---------------------------------------------------------------- 4-bit KV cache
 * A cache of K and V rows in one of the 4-bit formats whose scales are local to
 * a token, so that tokens can be appended one by one: WQ_Q4_0 (fp16 d per 32
 * elements, value (c - 8) * d) or WQ_NVFP4 (E4M3 scale per 16 elements and one
 * static fp32 g for K and one for V, value (E2M1(c) * s) * g).  Blocks run along
 * the head's `dim` elements.  9/16 byte per element in either format.
 *
 * Storage.  `pages` pages of `page_size` tokens:
 *   codes   [pages, heads, page_size, dim / 2] bytes, element 2j of a row in the
 *           low nibble of byte j
 *   scales  WQ_Q4_0:  fp16 d      [pages, heads, page_size, dim / 32]
 *           WQ_NVFP4: E4M3 bytes  [pages, heads, page_size, dim / 16]
 * (a page is bit for bit the packed codes and scales of a weight [heads *
 * page_size, dim] of that format).  Position t of sequence b lies in page
 * table[b * table_ld + t / page_size] at t % page_size; with table == NULL the
 * sequence owns page b whole (a contiguous slab per sequence).  The capacity of a
 * sequence is table_ld * page_size, or page_size without a table (and 2^31 - 256 at most).
 *
 * Rules: dim is 64 or 128; page_size is a multiple of 16, at most 2^30; heads >= 1;
 * pages * heads * page_size < 2^35 (WQ_ERR_SHAPE otherwise); codes and
 * scales 16-byte aligned, k_g / v_g / table 4-byte aligned.  k_g / v_g are used by
 * WQ_NVFP4 only; NULL stands for 1.  The struct lives in HOST memory; its pointers
 * are device pointers.
 *
 * Positions and lengths come from device memory, so the host cannot check them:
 * the kernels do.  A position outside a sequence's capacity, or a table entry
 * outside [0, pages), is neither read nor written (kv_append drops the token,
 * kv_read gives zeros, attend treats the token as not there), and
 * wq_last_device_status reports WQ_ERR_ARG.                                       */
typedef struct wq_kv_cache {
  void* k_codes;
  void* k_scales;
  void* v_codes;
  void* v_scales;
  const float* k_g;        /* WQ_NVFP4: one fp32 each, or NULL for 1            */
  const float* v_g;
  const int32_t* table;    /* [batch, table_ld] page numbers, or NULL           */
  int64_t table_ld;
  int64_t pages;
  int64_t page_size;       /* tokens per page                                   */
  int32_t fmt;             /* WQ_Q4_0 or WQ_NVFP4                               */
  int32_t heads;           /* K/V heads                                         */
  int32_t dim;             /* elements per head: 64 or 128                      */
} wq_kv_cache;

/* A [batch, token, head, dim] array by its strides in elements (dim is
 * contiguous): a column range of a fused projection's output is one.  p and
 * every stride times the element size are multiples of 16 bytes; strides are not
 * negative.  Lives in HOST memory; p is a device pointer.                         */
typedef struct wq_heads {
  void* p;
  int64_t batch, token, head;
} wq_heads;

/* wq_kv_append: quantise k and v (bf16) into the cache: token i of sequence b,
 * 0 <= i < counts[b], goes to position start[b] + i.  start NULL: 0; counts NULL:
 * `tokens` for every sequence (values outside [0, tokens] are clamped).  Codes and
 * scales equal those of wq_pack_q4_0 / wq_quant_act_nvfp4 (static g) on the same
 * values.  A NaN in a q4_0 block makes the block read back as NaN; an NVFP4
 * block cannot hold one.  Tokens of one call must not share a position.
 *
 * wq_kv_read: decode positions start[b] + i, 0 <= i < counts[b], to k and v
 * [batch, tokens, heads, dim] (bf16 rounded to nearest even, or fp32 with
 * WQ_FLAG_OUT_F32); rows from counts[b] on are zero.  k or v may be NULL.
 *
 * batch * tokens < 2^31.                                                         */
int wq_kv_append(const wq_kv_cache* cache, const wq_heads* k, const wq_heads* v, int64_t batch, int64_t tokens,
                 const int32_t* start, const int32_t* counts, void* stream);
int wq_kv_read(const wq_kv_cache* cache, const wq_heads* k, const wq_heads* v, int64_t batch, int64_t tokens,
               const int32_t* start, const int32_t* counts, unsigned flags, void* stream);

/* wq_kv_append_slots: quantise the rows of `tokens` tokens laid end to end (a batch of unequal requests without
 * padding; k->batch and v->batch are not used) into the cache, token i to slots[i] = page * page_size + offset, the
 * form in which wq_kv_reserve gives them.  A token whose slot is negative is skipped; one past the cache's pages is
 * too, and wq_last_device_status reports WQ_ERR_ARG.  The cache's table is not read.  Tokens of one call must not share
 * a slot.  slots: 8-byte aligned.                                                */
int wq_kv_append_slots(const wq_kv_cache* cache, const wq_heads* k, const wq_heads* v, int64_t tokens,
                       const int64_t* slots, void* stream);

/* ---------------------------------------------------------------- pages and slots of a changing batch
 * The table of a cache, which all its layers may share, is kept on the device: free_pages[0 .. top) is a stack of page
 * numbers that no sequence holds (room for free_size).  Sequence b holds ceil(lens[b] / page_size) pages; what its row
 * of the table has behind them is not looked at.
 *
 * wq_kv_reserve: pages for counts[b] tokens behind the lens[b] of each sequence, in the order of the sequences, the
 * stack's last page first, written to the table (which has to be writable).  A sequence whose pages the stack does not
 * hold any more gets none, and so does one whose tokens would pass its capacity; behind the first that the stack fails,
 * only those get their tokens that need no new page.  Outputs (each may be NULL, but top_out):
 *   granted    [batch] counts[b], or 0 where the sequence got nothing: the counts of the following calls
 *   starts     [batch + 1] where each sequence's tokens begin when all counts[b] are laid end to end (those that got
 *              nothing too), and their sum
 *   slots      [tokens] the slot of each of these tokens, -1 without one; -1 behind the last token
 *   positions  [tokens] its position, lens[b] + i; 0 behind the last token
 *   top_out    the pages that are left; may be `top` itself
 * More tokens than `tokens`, be it 0, are not written, and wq_last_device_status reports WQ_ERR_ARG (with slots and positions
 * both NULL there is no map that could be too short, and nothing to report); so it does for a page number outside the
 * cache (slot -1).  Negative lens and counts are taken for 0.  No output may overlap an input
 * but top_out, which may be top.
 *
 * wq_kv_release: of each sequence's pages those behind its first keep[b] tokens (NULL: all of them) go back on the stack,
 * in the order of the sequences and of their pages; those past its capacity are not there.  The table is not written.
 * Pages that find no room on the stack are dropped, and wq_last_device_status reports WQ_ERR_ARG.  So it does where a
 * number that goes back is none of the cache's pages, as when lens[b] is more than was granted; it goes on the stack all
 * the same, and whoever is given it gets slots of -1.  A page goes back once for every sequence that holds it: of several
 * that share pages (a common prefix) all but the last one have to keep them, or the stack holds them twice.
 *
 * batch <= WQ_TURN_MAX; slots 8-byte aligned, the others 4-byte.                 */
#define WQ_TURN_MAX 65536
int wq_kv_reserve(const wq_kv_cache* cache, const int32_t* free_pages, int64_t free_size, const int32_t* top,
                  int32_t* top_out, int64_t batch, const int32_t* lens, const int32_t* counts, int32_t* granted,
                  int64_t tokens, int64_t* slots, int32_t* positions, int32_t* starts, void* stream);
int wq_kv_release(const wq_kv_cache* cache, int32_t* free_pages, int64_t free_size, const int32_t* top, int32_t* top_out,
                  int64_t batch, const int32_t* lens, const int32_t* keep, void* stream);

/* ---------------------------------------------------------------- trees of drafted tokens
 * A draft is a tree of up to `tokens` nodes behind what a sequence holds, parents before their children: parents[b][i]
 * is the number of node i's parent, or -1.  Its K and V are appended in the nodes' order.
 *
 * wq_tree_mask: mask [batch, tokens, ceil(tokens / 32)]: bit j of node i's words (bit j % 32 of word j / 32) is set where
 * j is i or an ancestor of it; with window > 0 at most window - 1 levels up.  depth [batch, tokens] (or NULL): the number of
 * its ancestors.  Both are 0 for nodes from counts[b] on (NULL: none).  A parent that does not come before its
 * child is taken for -1, and wq_last_device_status reports WQ_ERR_ARG.  tokens <= WQ_TREE_MAX.
 *
 * wq_tree_mask_ex: the same for attention behind a window with sinks.  An ancestor j whose position is below `sinks`,
 * lens[b] - counts[b] + depth[j] < sinks, keeps its bit however many levels up it is: a draft behind a context shorter
 * than the sinks sees of itself what decoding it token by token would.  lens [batch]: what each sequence holds, its
 * draft among it, as wq_attend_ex takes it; needed with both a window and sinks (each alone changes nothing here).
 * Nothing ties a mask to the window and the sinks that it is used with: give both calls the same.
 *
 * wq_kv_keep: the rows of the nodes on an accepted path move up behind the context: position start[b] + path[b][i] to
 * start[b] + i for i < counts[b] (NULL: path_ld; values outside [0, path_ld] are clamped), codes and scales bit for bit,
 * all read before any is written.  path is [batch, path_ld], path_ld <= WQ_PATH_MAX.  A row whose node is negative, or whose
 * position or place lies outside the cache, stays, and wq_last_device_status reports WQ_ERR_ARG.  Sequences must not share the pages
 * that are written.                                                               */
#define WQ_TREE_MAX 1024
#define WQ_PATH_MAX 512
typedef struct wq_tree {
  const uint32_t* mask;    /* as above; any bits may be set                                  */
  const int32_t* depth;    /* NULL: node i is at depth i.  Only a window looks at it          */
  int64_t mask_batch;      /* elements from one sequence's to the next: 0 for one tree for all */
  int64_t depth_batch;
} wq_tree;
int wq_tree_mask(const int32_t* parents, int64_t batch, int64_t tokens, const int32_t* counts, int64_t window,
                 uint32_t* mask, int32_t* depth, void* stream);
int wq_tree_mask_ex(const int32_t* parents, int64_t batch, int64_t tokens, const int32_t* counts, int64_t window,
                    int64_t sinks, const int32_t* lens, uint32_t* mask, int32_t* depth, void* stream);
int wq_kv_keep(const wq_kv_cache* cache, const int32_t* start, int64_t batch, const int32_t* path, int64_t path_ld,
               const int32_t* counts, void* stream);

/* ---------------------------------------------------------------- attention over the cache
 * wq_attend: out = softmax(scale * q . K^T) . V over the cached tokens, per
 * sequence and query head.  q is bf16 [batch, tokens, q_heads, dim]; q_heads is a
 * multiple of the cache's heads, and query head h reads cache head
 * h / (q_heads / heads).  lens[b] is the number of tokens that sequence b holds
 * (those of this call included: append first).  counts as above: the last
 * counts[b] positions are this call's query tokens; query i sits at position
 * p = lens[b] - counts[b] + i (also where lens[b] is past the capacity).
 *   visible tokens   0 <= t < lens[b]; with WQ_FLAG_CAUSAL also t <= p, and with
 *                    window > 0 (WQ_FLAG_CAUSAL only) also t > p - window
 *   out              bf16, or fp32 with WQ_FLAG_OUT_F32, [batch, tokens, q_heads, dim]
 *   lse              fp32 [batch, tokens, q_heads] dense, or NULL: the natural log
 *                    of the sum of exp(scale * q . k) over the visible tokens
 * A row that sees no token, and a row from counts[b] on, gets out = 0 and
 * lse = -inf.  Cache contents past lens[b] are never used, whatever they hold.
 * max_len: what the caller knows on the host of lens (an upper bound, used to
 * plan the split of long sequences only; 0 stands for the capacity).
 * scale: finite.  Softmax statistics and sums are fp32; K, V and the weights enter
 * the products with 11 significant bits, whatever the size of the scales (the weights
 * down to 2^-25 of a row's largest, absolutely below; with more than 32 query rows per
 * cached head, where the |d| of a q4_0 block of V is 8192 or more, the weights of the 128
 * tokens around it down to 2^-22 of the largest, and the values beside it to 2^-22).
 * A NaN query, key or key scale makes the rows that see it NaN.  A V block whose scale
 * is not finite makes its own elements of the rows that see the token non-finite, or,
 * with more than 32 query rows per cached head (tokens * q_heads / heads), the
 * whole of those rows NaN.  No other row is touched by either.
 *
 * workspace: wq_attend_workspace_bytes(...) bytes (16-byte aligned, no
 * initialisation; may be NULL where that is 0) that no other call in flight uses. */
enum { WQ_FLAG_CAUSAL = 1u << 3 };
size_t wq_attend_workspace_bytes(const wq_kv_cache* cache, int64_t batch, int64_t tokens, int64_t q_heads,
                                 int64_t max_len);
int wq_attend(const wq_kv_cache* cache, const wq_heads* q, const wq_heads* out, float* lse, int64_t batch,
              int64_t tokens, int64_t q_heads, const int32_t* lens, const int32_t* counts, int64_t max_len,
              float scale, int64_t window, unsigned flags, void* workspace, size_t workspace_bytes, void* stream);

/* wq_attend_ex: wq_attend, and (WQ_FLAG_CAUSAL only)
 *   sinks > 0     the first `sinks` tokens stay visible behind the window: 0 <= t <= p and (t > p - window or t < sinks).
 *                 Without a window they change nothing.  What lies between them and the window is not read.
 *   tree          (NULL: none; in HOST memory) the counts[b] query tokens are nodes of a draft.  Node i sees the context,
 *                 t < lens[b] - counts[b], with a window and sinks as a token at lens[b] - counts[b] + depth[i]
 *                 (clamped to 0 .. counts[b] - 1) does, and node j, at t = lens[b] - counts[b] + j, where bit j of its
 *                 mask is set: itself too only then.  tokens <= WQ_TREE_MAX.
 * What wq_attend says of more than 32 query rows per cached head holds from 17 on here for WQ_Q4_0 heads of 128.
 * workspace: wq_attend_ex_workspace_bytes(...) bytes, enough with and without sinks and trees; as above.   */
size_t wq_attend_ex_workspace_bytes(const wq_kv_cache* cache, int64_t batch, int64_t tokens, int64_t q_heads,
                                    int64_t max_len);
int wq_attend_ex(const wq_kv_cache* cache, const wq_heads* q, const wq_heads* out, float* lse, int64_t batch,
                 int64_t tokens, int64_t q_heads, const int32_t* lens, const int32_t* counts, int64_t max_len,
                 float scale, int64_t window, int64_t sinks, const wq_tree* tree, unsigned flags, void* workspace,
                 size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- status
 * wq_last_device_status: synchronises the current device, returns and clears
 * the device-side status word (WQ_OK; WQ_ERR_TIMEOUT if a kernel abandoned a
 * bounded wait since the last call; WQ_ERR_ARG if a KV cache kernel met a
 * position or page outside the cache).  Not for hot loops.
 * wq_status_string: a static description of a status code.
 * wq_kernel_launches: number of kernels this library has launched in this
 * process (host-side counter).                                                 */
int wq_last_device_status(void);
const char* wq_status_string(int status);
uint64_t wq_kernel_launches(void);

/* ---------------------------------------------------------------- failure detection
 * wq_selftest_timeout: launches one small kernel that waits, with the same
 * bounded mbarrier poll every kernel of this library uses, on a barrier that
 * nothing ever arrives on, giving up after `polls` polls (1 <= polls <= 2^20).
 * The kernel then records WQ_ERR_TIMEOUT in the device status word and
 * returns normally: no trap, the context stays usable.  A following
 * wq_last_device_status() returns WQ_ERR_TIMEOUT (and clears it).  Exercises
 * the path a real stall takes (a TMA transaction or a peer that never
 * arrives) without faulting the GPU.  WQ_ERR_ARG for polls out of range.    */
int wq_selftest_timeout(uint32_t polls, void* stream);

/* ---------------------------------------------------------------- encoder check
 * wq_selftest_encoders: a verification export.  For each of the n fp32 values
 * in[i] (device), writes four bytes out[4i .. 4i+3] (device):
 *   [0] the E2M1 code the library's packers / activation quantiser assign
 *   [1] the E2M1 code of the hardware conversion cvt.rn.satfinite.e2m1x2.f32
 *   [2] the E4M3 byte the library's block-scale encoder assigns
 *   [3] the E4M3 byte of cvt.rn.satfinite.e4m3x2.f32
 * so that tests can pin both the library's encoders (model card
 * "whisper-large-v3-turbo -- NVFP4", "What is quantized": E2M1 codes, E4M3
 * block scales) and the hardware's rounding of ties and signed zeros.
 * WQ_ERR_ARG for n < 0 or n > 2^30, WQ_ERR_ALIGN for unaligned pointers.     */
int wq_selftest_encoders(const float* in, int64_t n, uint8_t* out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* WQ_H_ */
