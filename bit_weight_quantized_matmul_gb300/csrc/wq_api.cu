// wq_api.cu -- the C ABI of include/wq.h: argument checks, storage layout,
// dispatch between the tensor-core and CUDA-core paths.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <mutex>

#include "wq_internal.h"

namespace wq {

static std::atomic<uint64_t> g_launches{0};
void count_launch(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

ScalesLayout scales_layout(int fmt, int64_t N, int64_t K) {
  ScalesLayout L;
  const int64_t n = N * K;
  switch (fmt) {
    case WQ_NF4: {
      const int64_t nb = n / 64;
      L.absmax_bytes = (size_t)nb;
      L.n_groups = (nb + 255) / 256;
      L.s2_off = align16((size_t)nb);
      L.offset_off = L.s2_off + 4 * (size_t)L.n_groups;
      L.total = L.offset_off + 4;
      break;
    }
    case WQ_NVFP4:
    case WQ_NVFP4_W4A4:
      L.sf_bytes = (size_t)(n / 16);
      L.g_off = align16(L.sf_bytes);
      L.total = L.g_off + 4;
      break;
    case WQ_Q4_0:
    case WQ_Q8_0:
    case WQ_Q5_0:
      L.total = align16((size_t)(n / 32) * 2);
      break;
    case WQ_Q4_1:
      L.total = 16;  // the (d, m) pairs live in the packed units; 16 zero bytes
      break;
    case WQ_FP8:
      L.total = align16((size_t)N * 4);
      break;
    default:
      break;
  }
  return L;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link-time libcuda dependency)
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bool encode_tmap_2d(void* tmap, CUtensorMapDataType dtype, const void* base, uint64_t inner, uint64_t outer,
                    uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {row_stride_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(reinterpret_cast<CUtensorMap*>(tmap), dtype, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

int linear_one(const LinearArgs& a, cudaStream_t s) {
  int rc = WQ_OK;
  const bool dense = a.nout == 1 && a.ld[0] == a.N;
  if (a.fmt == WQ_NVFP4_W4A4) {
    if (dense && linear_w4a4_tc(a, s, &rc)) return rc;
  } else if (a.M <= 16) {
    // Measured on GB300 (back-to-back launches, NF4): one activation row runs fastest on the CUDA
    // cores (1280 x 1280: 3.5 us; 5120 x 1280: 5.0 us), as do up to 4 rows of a narrow or long-K
    // weight; the persistent tensor-core kernel (whole-K 128-row tiles) takes short-K Linears from
    // there on (5120 x 1280 at 4 rows: 6.1 against 9.9 us; 1280 x 1280 at 16 rows: 5.6 against
    // 8.3 us for the cluster split-K kernel, which keeps the long-K ones).
    const bool tcp_short = a.K <= kTcpDecodeMaxK && tcp_eligible(a);
    if (gemv_eligible(a) && (a.M == 1 || (a.M <= kGemvMaxM && !(tcp_short && a.N >= 4096))))
      return linear_gemv(a, s);
    if (tcp_short) return linear_tcp(&a, 1, s);
    if (dense && linear_tc(a, s, &rc)) return rc;
    if (gemv_eligible(a)) return linear_gemv(a, s);
  }
  if (a.fmt != WQ_NVFP4_W4A4 && dense && linear_w4a16_tc(a, s, &rc)) return rc;
  if (a.fmt != WQ_NVFP4_W4A4 && tcp_eligible(a)) return linear_tcp(&a, 1, s);
  return linear_simt(a, s);
}

}  // namespace wq

using namespace wq;

namespace {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int block_of(int fmt) {
  switch (fmt) {
    case WQ_NF4: return 64;
    case WQ_NVFP4:
    case WQ_NVFP4_W4A4: return 32;  // 16-blocks; rows of packed codes must stay 16-byte aligned
    case WQ_Q4_0:
    case WQ_Q8_0:
    case WQ_FP8: return 32;
    case WQ_Q4_1:
    case WQ_Q5_0: return 128;  // whole 128-element storage units per row
    default: return 0;
  }
}

int check_weight(int fmt, int64_t N, int64_t K) {
  if (block_of(fmt) == 0) return WQ_ERR_FMT;
  if (N < 0 || K < 0) return WQ_ERR_ARG;
  if (K % block_of(fmt) != 0) return WQ_ERR_SHAPE;
  if (N > (int64_t(1) << 31) || K > (int64_t(1) << 31) || N * K > (int64_t(1) << 40)) return WQ_ERR_SHAPE;
  return WQ_OK;
}

int pack_common(int fmt, const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream,
                int (*fn)(const float*, int64_t, int64_t, uint8_t*, uint8_t*, cudaStream_t)) {
  int rc = check_weight(fmt, N, K);
  if (rc != WQ_OK) return rc;
  if (N * K == 0) return WQ_OK;
  if (!W || !packed || !scales) return WQ_ERR_ARG;
  if (!aligned16(W) || !aligned16(packed) || !aligned16(scales)) return WQ_ERR_ALIGN;
  return fn(W, N, K, reinterpret_cast<uint8_t*>(packed), reinterpret_cast<uint8_t*>(scales),
            reinterpret_cast<cudaStream_t>(stream));
}

int check_cache(const wq_kv_cache* c, KvArgs& a) {
  if (!c) return WQ_ERR_ARG;
  if (c->fmt != WQ_Q4_0 && c->fmt != WQ_NVFP4) return WQ_ERR_FMT;
  if (c->heads < 1 || c->pages < 0 || c->page_size < 0 || (c->table && c->table_ld < 0)) return WQ_ERR_ARG;
  if ((c->dim != 64 && c->dim != 128) || c->heads > 65535) return WQ_ERR_SHAPE;
  if (c->page_size == 0 || c->page_size % 16 != 0 || c->page_size > (1 << 30) || c->pages > (int64_t(1) << 31))
    return WQ_ERR_SHAPE;
  if (c->table && c->table_ld > (int64_t(1) << 30)) return WQ_ERR_SHAPE;
  if ((double)c->pages * c->heads * (double)(c->page_size / 16) >= 2147483648.0) return WQ_ERR_SHAPE;  // 2^35 rows: a terabyte
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return WQ_ERR_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales))
    return WQ_ERR_ALIGN;
  if (((uintptr_t)c->table & 3u) || ((uintptr_t)c->k_g & 3u) || ((uintptr_t)c->v_g & 3u)) return WQ_ERR_ALIGN;
  a.codes[0] = reinterpret_cast<uint8_t*>(c->k_codes);
  a.codes[1] = reinterpret_cast<uint8_t*>(c->v_codes);
  a.scales[0] = reinterpret_cast<uint8_t*>(c->k_scales);
  a.scales[1] = reinterpret_cast<uint8_t*>(c->v_scales);
  a.g[0] = c->fmt == WQ_NVFP4 ? c->k_g : nullptr;
  a.g[1] = c->fmt == WQ_NVFP4 ? c->v_g : nullptr;
  a.table = c->table;
  a.table_ld = c->table_ld;
  a.pages = c->pages;
  a.page_size = (int32_t)c->page_size;
  int log = 4;  // page_size <= 2^log; the rounded-up multiplier's error times t stays below 2^(31 + log)
  while ((int64_t(1) << log) < c->page_size) ++log;
  a.page_mul = (uint32_t)((uint64_t(1) << (31 + log)) / (uint64_t)c->page_size + (c->page_size == (int64_t(1) << log) ? 0 : 1));
  a.page_shift = (uint32_t)(log - 1);
  a.fmt = c->fmt;
  a.heads = c->heads;
  a.dim = c->dim;
  a.capacity = c->table ? c->table_ld * c->page_size : c->page_size;
  if (a.capacity > 0x7FFFFF00) a.capacity = 0x7FFFFF00;  // positions are int32, and whole tiles past them too
  return WQ_OK;
}

int check_heads(const wq_heads* h, size_t esz, HeadsArg& a) {
  if (!h || !h->p || h->batch < 0 || h->token < 0 || h->head < 0) return WQ_ERR_ARG;
  if (!aligned16(h->p) || ((uint64_t)h->batch * esz) % 16 || ((uint64_t)h->token * esz) % 16 ||
      ((uint64_t)h->head * esz) % 16)
    return WQ_ERR_ALIGN;
  a = HeadsArg{h->p, h->batch, h->token, h->head};
  return WQ_OK;
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool too_many(int64_t batch, int64_t tokens) {
  return batch > 0x7FFFFFFF || tokens > 0x7FFFFFFF || batch * tokens > 0x7FFFFFFF;
}

size_t workspace_bytes_of(const wq_kv_cache* cache, int64_t batch, int64_t tokens, int64_t q_heads, int64_t max_len, bool sel) {
  KvArgs kv{};
  if (check_cache(cache, kv) != WQ_OK || batch <= 0 || tokens <= 0 || too_many(batch, tokens) || max_len < 0 ||
      q_heads <= 0 || q_heads > 65535 || q_heads % kv.heads != 0)
    return 0;
  return attend_workspace(kv, batch, tokens, q_heads, max_len, sel);
}

// The part of a reserve or release call that the two share.
int check_turn(const wq_kv_cache* cache, const int32_t* free_pages, int64_t free_size, const int32_t* top, int32_t* top_out,
               int64_t batch, const int32_t* lens, KvReserveArgs& a) {
  const int rc = check_cache(cache, a.kv);
  if (rc != WQ_OK) return rc;
  if (!cache->table || !top || !top_out || free_size < 0 || (free_size > 0 && !free_pages) || batch < 0 || (batch > 0 && !lens))
    return WQ_ERR_ARG;
  if (batch > WQ_TURN_MAX || free_size > 0x7FFFFFFF) return WQ_ERR_SHAPE;
  if (!aligned(free_pages, 4) || !aligned(top, 4) || !aligned(top_out, 4) || !aligned(lens, 4)) return WQ_ERR_ALIGN;
  a.free_pages = free_pages;
  a.free_size = free_size;
  a.top = top;
  a.top_out = top_out;
  a.batch = batch;
  a.lens = lens;
  return WQ_OK;
}

// The part of an append or read call that the two share; *rows: whether there is anything to do.
int check_move(const wq_kv_cache* cache, int64_t batch, int64_t tokens, const int32_t* start, const int32_t* counts,
               KvMoveArgs& a, bool* rows) {
  int rc = check_cache(cache, a.kv);
  if (rc != WQ_OK) return rc;
  if (batch < 0 || tokens < 0) return WQ_ERR_ARG;
  if (too_many(batch, tokens) || (!cache->table && batch > cache->pages)) return WQ_ERR_SHAPE;
  if (((uintptr_t)start & 3u) || ((uintptr_t)counts & 3u)) return WQ_ERR_ALIGN;
  a.batch = batch;
  a.tokens = tokens;
  a.start = start;
  a.counts = counts;
  *rows = batch > 0 && tokens > 0;
  return WQ_OK;
}

}  // namespace

extern "C" {

size_t wq_packed_bytes(int fmt, int64_t N, int64_t K) {
  if (check_weight(fmt, N, K) != WQ_OK) return 0;
  return (size_t)(N * packed_row_bytes(fmt, K));
}

size_t wq_scales_bytes(int fmt, int64_t N, int64_t K) {
  if (check_weight(fmt, N, K) != WQ_OK) return 0;
  return scales_layout(fmt, N, K).total;
}

int wq_pack_nf4(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream) {
  return pack_common(WQ_NF4, W, N, K, packed, scales, stream, pack_nf4);
}
int wq_pack_nvfp4(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream) {
  return pack_common(WQ_NVFP4, W, N, K, packed, scales, stream, pack_nvfp4);
}
int wq_pack_q4_0(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream) {
  return pack_common(WQ_Q4_0, W, N, K, packed, scales, stream, pack_q4_0);
}
int wq_pack_q8_0(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream) {
  return pack_common(WQ_Q8_0, W, N, K, packed, scales, stream, pack_q8_0);
}

int wq_pack_q4_1(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream) {
  return pack_common(WQ_Q4_1, W, N, K, packed, scales, stream, pack_q4_1);
}
int wq_pack_q5_0(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream) {
  return pack_common(WQ_Q5_0, W, N, K, packed, scales, stream, pack_q5_0);
}
int wq_pack_fp8(const float* W, int64_t N, int64_t K, void* packed, void* scales, void* stream) {
  return pack_common(WQ_FP8, W, N, K, packed, scales, stream, pack_fp8);
}

int wq_dequant(const void* packed, const void* scales, int fmt, int64_t N, int64_t K, float* W_out, void* stream) {
  int rc = check_weight(fmt, N, K);
  if (rc != WQ_OK) return rc;
  if (N * K == 0) return WQ_OK;
  if (!packed || !scales || !W_out) return WQ_ERR_ARG;
  if (!aligned16(packed) || !aligned16(scales) || !aligned16(W_out)) return WQ_ERR_ALIGN;
  return dequant(reinterpret_cast<const uint8_t*>(packed), reinterpret_cast<const uint8_t*>(scales), fmt, N, K,
                 W_out, reinterpret_cast<cudaStream_t>(stream));
}

int wq_quant_act_nvfp4(const uint16_t* x, int64_t M, int64_t K, const float* g_in, uint8_t* codes, uint8_t* scales,
                       float* g_out, void* stream) {
  if (M < 0 || K < 0) return WQ_ERR_ARG;
  if (K % 32 != 0) return WQ_ERR_SHAPE;
  if (M * K == 0) return WQ_OK;
  if (!x || !codes || !scales || !g_out) return WQ_ERR_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || ((uintptr_t)g_out & 3u) ||
      (g_in && ((uintptr_t)g_in & 3u)))
    return WQ_ERR_ALIGN;
  return quant_act_nvfp4(x, M, K, g_in, codes, scales, g_out, reinterpret_cast<cudaStream_t>(stream));
}

int wq_linear_ex(const void* x, const void* packed, const void* scales, int fmt, int64_t M, int64_t N, int64_t K,
                 const uint16_t* bias, void* y, unsigned flags, void* stream) {
  if (flags & ~(unsigned)(WQ_FLAG_OUT_F32 | WQ_FLAG_WEIGHTS_STATIC | WQ_FLAG_FORCE_SIMT)) return WQ_ERR_ARG;
  int rc = check_weight(fmt, N, K);
  if (rc != WQ_OK) return rc;
  if (M < 0) return WQ_ERR_ARG;
  if (M == 0 || N == 0) return WQ_OK;
  if (!x || !packed || !scales || !y) return WQ_ERR_ARG;
  if (!aligned16(packed) || !aligned16(scales) || !aligned16(y) || (bias && !aligned16(bias)))
    return WQ_ERR_ALIGN;
  LinearArgs a{};
  if (fmt == WQ_NVFP4_W4A4) {
    const wq_act_nvfp4* act = reinterpret_cast<const wq_act_nvfp4*>(x);  // host struct of device pointers
    if (!act->codes || !act->scales || !act->g) return WQ_ERR_ARG;
    if (!aligned16(act->codes) || !aligned16(act->scales) || ((uintptr_t)act->g & 3u)) return WQ_ERR_ALIGN;
    a.act_codes = act->codes;
    a.act_scales = act->scales;
    a.act_g = act->g;
  } else {
    if (!aligned16(x)) return WQ_ERR_ALIGN;
    a.x = x;
  }
  a.packed = reinterpret_cast<const uint8_t*>(packed);
  a.scales = reinterpret_cast<const uint8_t*>(scales);
  a.fmt = fmt;
  a.M = M;
  a.N = N;
  a.K = K;
  a.bias = bias;
  a.y = y;
  set_single_out(a);
  a.out_f32 = (flags & WQ_FLAG_OUT_F32) != 0;
  a.weights_static = (flags & WQ_FLAG_WEIGHTS_STATIC) != 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (flags & WQ_FLAG_FORCE_SIMT) return linear_simt(a, s);
  return linear_one(a, s);
}

int wq_linear_grouped(const wq_problem* problems, int count, int fmt, unsigned flags, void* stream) {
  if (!problems || count < 1 || count > WQ_GROUP_MAX) return WQ_ERR_ARG;
  wq_problem_ex ex[WQ_GROUP_MAX];
  for (int i = 0; i < count; ++i) {
    const wq_problem& p = problems[i];
    ex[i] = wq_problem_ex{};
    ex[i].x = p.x;
    ex[i].packed = p.packed;
    ex[i].scales = p.scales;
    ex[i].bias = p.bias;
    ex[i].M = p.M;
    ex[i].N = p.N;
    ex[i].K = p.K;
    ex[i].nout = 1;
    ex[i].out[0] = wq_out{p.y, p.N, p.N};
  }
  return wq_linear_grouped_ex(ex, count, fmt, flags, stream);
}

int wq_linear_grouped_ex(const wq_problem_ex* problems, int count, int fmt, unsigned flags, void* stream) {
  if (!problems || count < 1 || count > WQ_GROUP_MAX) return WQ_ERR_ARG;
  if (flags & ~(unsigned)(WQ_FLAG_OUT_F32 | WQ_FLAG_WEIGHTS_STATIC)) return WQ_ERR_ARG;
  if (fmt == WQ_NVFP4_W4A4) return WQ_ERR_FMT;
  const size_t esz = (flags & WQ_FLAG_OUT_F32) ? 4 : 2;
  LinearArgs args[WQ_GROUP_MAX];
  int n = 0;
  bool all_tc = true;
  for (int i = 0; i < count; ++i) {
    const wq_problem_ex& p = problems[i];
    int rc = check_weight(fmt, p.N, p.K);
    if (rc != WQ_OK) return rc;
    if (p.M < 0) return WQ_ERR_ARG;
    if (p.nout < 1 || p.nout > WQ_OUT_MAX) return WQ_ERR_ARG;
    if (p.M == 0 || p.N == 0) continue;
    if (!p.x || !p.packed || !p.scales) return WQ_ERR_ARG;
    if (!aligned16(p.x) || !aligned16(p.packed) || !aligned16(p.scales) || (p.bias && !aligned16(p.bias)))
      return WQ_ERR_ALIGN;
    LinearArgs a{};
    int64_t c = 0;
    for (int d = 0; d < p.nout; ++d) {
      const wq_out& o = p.out[d];
      if (!o.y || o.ncols <= 0 || o.ld < o.ncols) return WQ_ERR_ARG;
      if (d + 1 < p.nout && o.ncols % 16 != 0) return WQ_ERR_ARG;
      if (!aligned16(o.y) || ((size_t)o.ld * esz) % 16 != 0) return WQ_ERR_ALIGN;
      if (o.ld > 0x7FFFFFFF) return WQ_ERR_SHAPE;
      c += o.ncols;
      a.ys[d] = o.y;
      a.ld[d] = o.ld;
      a.col_end[d] = c;
    }
    if (c != p.N) return WQ_ERR_ARG;
    a.nout = p.nout;
    for (int d = p.nout; d < WQ_OUT_MAX; ++d) { a.ys[d] = a.ys[p.nout - 1]; a.ld[d] = a.ld[p.nout - 1]; a.col_end[d] = c; }
    a.x = p.x;
    a.y = p.out[0].y;
    a.packed = reinterpret_cast<const uint8_t*>(p.packed);
    a.scales = reinterpret_cast<const uint8_t*>(p.scales);
    a.fmt = fmt;
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.bias = p.bias;
    a.out_f32 = (flags & WQ_FLAG_OUT_F32) != 0;
    a.weights_static = (flags & WQ_FLAG_WEIGHTS_STATIC) != 0;
    all_tc = all_tc && tcp_eligible(a);
    args[n++] = a;
  }
  if (n == 0) return WQ_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (all_tc) return linear_tcp(args, n, s);
  for (int i = 0; i < n; ++i) {  // some problem outside the tensor-core rules: one launch each
    const int rc = linear_one(args[i], s);
    if (rc != WQ_OK) return rc;
  }
  return WQ_OK;
}

int wq_linear(const void* x, const void* packed, const void* scales, int fmt, int64_t M, int64_t N, int64_t K,
              const uint16_t* bias, void* y, void* stream) {
  return wq_linear_ex(x, packed, scales, fmt, M, N, K, bias, y, 0u, stream);
}

int wq_kv_append(const wq_kv_cache* cache, const wq_heads* k, const wq_heads* v, int64_t batch, int64_t tokens,
                 const int32_t* start, const int32_t* counts, void* stream) {
  KvMoveArgs a{};
  bool rows = false;
  int rc = check_move(cache, batch, tokens, start, counts, a, &rows);
  if (rc != WQ_OK || !rows) return rc;
  if ((rc = check_heads(k, 2, a.x[0])) != WQ_OK || (rc = check_heads(v, 2, a.x[1])) != WQ_OK) return rc;
  return kv_append(a, reinterpret_cast<cudaStream_t>(stream));
}

int wq_kv_read(const wq_kv_cache* cache, const wq_heads* k, const wq_heads* v, int64_t batch, int64_t tokens,
               const int32_t* start, const int32_t* counts, unsigned flags, void* stream) {
  if (flags & ~(unsigned)WQ_FLAG_OUT_F32) return WQ_ERR_ARG;
  KvMoveArgs a{};
  bool rows = false;
  int rc = check_move(cache, batch, tokens, start, counts, a, &rows);
  if (rc != WQ_OK || !rows) return rc;
  a.f32 = (flags & WQ_FLAG_OUT_F32) != 0;
  if (!k && !v) return WQ_ERR_ARG;
  if (k && (rc = check_heads(k, a.f32 ? 4 : 2, a.x[0])) != WQ_OK) return rc;
  if (v && (rc = check_heads(v, a.f32 ? 4 : 2, a.x[1])) != WQ_OK) return rc;
  return kv_read(a, reinterpret_cast<cudaStream_t>(stream));
}

int wq_kv_append_slots(const wq_kv_cache* cache, const wq_heads* k, const wq_heads* v, int64_t tokens, const int64_t* slots,
                       void* stream) {
  KvSlotArgs a{};
  int rc = check_cache(cache, a.kv);
  if (rc != WQ_OK) return rc;
  if (tokens < 0) return WQ_ERR_ARG;
  if (tokens > 0x7FFFFFFF) return WQ_ERR_SHAPE;
  if (tokens == 0) return WQ_OK;
  if (!slots) return WQ_ERR_ARG;
  if (!aligned(slots, 8)) return WQ_ERR_ALIGN;
  if ((rc = check_heads(k, 2, a.x[0])) != WQ_OK || (rc = check_heads(v, 2, a.x[1])) != WQ_OK) return rc;
  a.tokens = tokens;
  a.slots = slots;
  return kv_append_slots(a, reinterpret_cast<cudaStream_t>(stream));
}

int wq_kv_reserve(const wq_kv_cache* cache, const int32_t* free_pages, int64_t free_size, const int32_t* top, int32_t* top_out,
                  int64_t batch, const int32_t* lens, const int32_t* counts, int32_t* granted, int64_t tokens, int64_t* slots,
                  int32_t* positions, int32_t* starts, void* stream) {
  KvReserveArgs a{};
  const int rc = check_turn(cache, free_pages, free_size, top, top_out, batch, lens, a);
  if (rc != WQ_OK) return rc;
  if (tokens < 0 || (batch > 0 && !counts) || (granted && (granted == counts || granted == lens))) return WQ_ERR_ARG;
  if (tokens > 0x7FFFFFFF) return WQ_ERR_SHAPE;
  if (!aligned(counts, 4) || !aligned(granted, 4) || !aligned(slots, 8) || !aligned(positions, 4) || !aligned(starts, 4))
    return WQ_ERR_ALIGN;
  a.counts = counts;
  a.granted = granted;
  a.tokens = slots || positions ? tokens : 0;
  a.slots = slots;
  a.positions = positions;
  a.starts = starts;
  return kv_reserve(a, reinterpret_cast<cudaStream_t>(stream));
}

int wq_kv_release(const wq_kv_cache* cache, int32_t* free_pages, int64_t free_size, const int32_t* top, int32_t* top_out,
                  int64_t batch, const int32_t* lens, const int32_t* keep, void* stream) {
  KvReserveArgs a{};
  const int rc = check_turn(cache, free_pages, free_size, top, top_out, batch, lens, a);
  if (rc != WQ_OK) return rc;
  if (!aligned(keep, 4)) return WQ_ERR_ALIGN;
  a.counts = keep;
  return kv_release(a, reinterpret_cast<cudaStream_t>(stream));
}

int wq_kv_keep(const wq_kv_cache* cache, const int32_t* start, int64_t batch, const int32_t* path, int64_t path_ld,
               const int32_t* counts, void* stream) {
  KvKeepArgs a{};
  const int rc = check_cache(cache, a.kv);
  if (rc != WQ_OK) return rc;
  if (batch < 0 || path_ld < 0) return WQ_ERR_ARG;
  if (path_ld > WQ_PATH_MAX || batch > 0x7FFFFFFF || (!cache->table && batch > cache->pages)) return WQ_ERR_SHAPE;
  if (batch == 0 || path_ld == 0) return WQ_OK;
  if (!start || !path) return WQ_ERR_ARG;
  if (!aligned(start, 4) || !aligned(path, 4) || !aligned(counts, 4)) return WQ_ERR_ALIGN;
  a.batch = batch;
  a.start = start;
  a.path = path;
  a.path_ld = path_ld;
  a.counts = counts;
  return kv_keep(a, reinterpret_cast<cudaStream_t>(stream));
}

int wq_tree_mask(const int32_t* parents, int64_t batch, int64_t tokens, const int32_t* counts, int64_t window, uint32_t* mask,
                 int32_t* depth, void* stream) {
  return wq_tree_mask_ex(parents, batch, tokens, counts, window, 0, nullptr, mask, depth, stream);
}

int wq_tree_mask_ex(const int32_t* parents, int64_t batch, int64_t tokens, const int32_t* counts, int64_t window, int64_t sinks,
                    const int32_t* lens, uint32_t* mask, int32_t* depth, void* stream) {
  if (batch < 0 || tokens < 0 || window < 0 || sinks < 0) return WQ_ERR_ARG;
  if (tokens > WQ_TREE_MAX || too_many(batch, tokens)) return WQ_ERR_SHAPE;
  if (batch == 0 || tokens == 0) return WQ_OK;
  if (!parents || !mask || (window > 0 && sinks > 0 && !lens)) return WQ_ERR_ARG;
  if (!aligned(parents, 4) || !aligned(counts, 4) || !aligned(lens, 4) || !aligned(mask, 4) || !aligned(depth, 4)) return WQ_ERR_ALIGN;
  TreeMaskArgs a{};
  a.parents = parents;
  a.counts = counts;
  a.lens = lens;
  a.batch = batch;
  a.tokens = tokens;
  a.window = window;
  a.sinks = sinks < (int64_t(1) << 32) ? sinks : int64_t(1) << 32;   // no more: positions are below 2^32
  a.mask = mask;
  a.depth = depth;
  return tree_mask(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t wq_attend_workspace_bytes(const wq_kv_cache* cache, int64_t batch, int64_t tokens, int64_t q_heads,
                                 int64_t max_len) {
  return workspace_bytes_of(cache, batch, tokens, q_heads, max_len, false);
}

size_t wq_attend_ex_workspace_bytes(const wq_kv_cache* cache, int64_t batch, int64_t tokens, int64_t q_heads,
                                    int64_t max_len) {
  const size_t plain = workspace_bytes_of(cache, batch, tokens, q_heads, max_len, false);
  const size_t sel = workspace_bytes_of(cache, batch, tokens, q_heads, max_len, true);
  return plain > sel ? plain : sel;
}

int wq_attend(const wq_kv_cache* cache, const wq_heads* q, const wq_heads* out, float* lse, int64_t batch,
              int64_t tokens, int64_t q_heads, const int32_t* lens, const int32_t* counts, int64_t max_len,
              float scale, int64_t window, unsigned flags, void* workspace, size_t workspace_bytes, void* stream) {
  return wq_attend_ex(cache, q, out, lse, batch, tokens, q_heads, lens, counts, max_len, scale, window, 0, nullptr, flags,
                      workspace, workspace_bytes, stream);
}

int wq_attend_ex(const wq_kv_cache* cache, const wq_heads* q, const wq_heads* out, float* lse, int64_t batch,
                 int64_t tokens, int64_t q_heads, const int32_t* lens, const int32_t* counts, int64_t max_len,
                 float scale, int64_t window, int64_t sinks, const wq_tree* tree, unsigned flags, void* workspace,
                 size_t workspace_bytes, void* stream) {
  if (flags & ~(unsigned)(WQ_FLAG_OUT_F32 | WQ_FLAG_CAUSAL)) return WQ_ERR_ARG;
  AttendArgs a{};
  int rc = check_cache(cache, a.kv);
  if (rc != WQ_OK) return rc;
  a.causal = (flags & WQ_FLAG_CAUSAL) != 0;
  a.f32 = (flags & WQ_FLAG_OUT_F32) != 0;
  if (batch < 0 || tokens < 0 || q_heads < 0 || max_len < 0 || window < 0 || (window > 0 && !a.causal)) return WQ_ERR_ARG;
  if (!(scale > -INFINITY && scale < INFINITY)) return WQ_ERR_ARG;
  if (sinks < 0 || (sinks > 0 && !a.causal)) return WQ_ERR_ARG;
  if (tree) {
    if (!a.causal || !tree->mask || tree->mask_batch < 0 || tree->depth_batch < 0) return WQ_ERR_ARG;
    if (tokens > WQ_TREE_MAX) return WQ_ERR_SHAPE;
    if (!aligned(tree->mask, 4) || !aligned(tree->depth, 4)) return WQ_ERR_ALIGN;
    a.tree_mask = tree->mask;
    a.tree_depth = tree->depth;
    a.mask_batch = tree->mask_batch;
    a.depth_batch = tree->depth_batch;
    a.tree_words = (int32_t)((tokens + 31) / 32);
  }
  a.sinks = (int32_t)(sinks < 0x7FFFFFFF ? sinks : 0x7FFFFFFF);
  if (too_many(batch, tokens) || (!cache->table && batch > cache->pages) || q_heads > 65535 || q_heads % a.kv.heads != 0) return WQ_ERR_SHAPE;
  if (batch == 0 || tokens == 0 || q_heads == 0) return WQ_OK;
  if (!lens) return WQ_ERR_ARG;
  if (((uintptr_t)lens & 3u) || ((uintptr_t)counts & 3u) || ((uintptr_t)lse & 3u)) return WQ_ERR_ALIGN;
  if ((rc = check_heads(q, 2, a.q)) != WQ_OK || (rc = check_heads(out, a.f32 ? 4 : 2, a.out)) != WQ_OK) return rc;
  const size_t need = attend_workspace(a.kv, batch, tokens, q_heads, max_len, tree || (window > 0 && sinks > 0));
  if (need > 0 && (!workspace || workspace_bytes < need)) return WQ_ERR_ARG;
  if (need > 0 && !aligned16(workspace)) return WQ_ERR_ALIGN;
  a.lse = lse;
  a.batch = batch;
  a.tokens = tokens;
  a.q_heads = q_heads;
  a.lens = lens;
  a.counts = counts;
  a.max_len = max_len;
  a.scale = scale;
  a.window = window < (int64_t(1) << 31) ? window : int64_t(1) << 31;  // no wider: positions are below 2^31, and nothing overflows
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  return attend(a, reinterpret_cast<cudaStream_t>(stream));
}

int wq_selftest_timeout(uint32_t polls, void* stream) {
  if (polls < 1 || polls > (1u << 20)) return WQ_ERR_ARG;
  return wq::selftest_timeout(polls, reinterpret_cast<cudaStream_t>(stream));
}

int wq_selftest_encoders(const float* in, int64_t n, uint8_t* out, void* stream) {
  if (n < 0 || n > (int64_t(1) << 30)) return WQ_ERR_ARG;
  if (n == 0) return WQ_OK;
  if (!in || !out) return WQ_ERR_ARG;
  if (!aligned16(in) || !aligned16(out)) return WQ_ERR_ALIGN;
  return wq::selftest_encoders(in, n, out, reinterpret_cast<cudaStream_t>(stream));
}

int wq_last_device_status(void) {
  if (cudaDeviceSynchronize() != cudaSuccess) return WQ_ERR_CUDA;
  int worst = WQ_OK;
  const int parts[12] = {take_status_pack(), take_status_simt(), take_status_tc(), take_status_tcp(),
                        take_status_w4a4(), take_status_w4a16(), take_status_kv(), take_status_attend(),
                        take_status_attend_tc(), take_status_attend_few_sel(), take_status_attend_tc_sel(),
                        take_status_pages()};
  for (int v : parts)
    if (v != WQ_OK) worst = v;
  return worst;
}

const char* wq_status_string(int status) {
  switch (status) {
    case WQ_OK: return "ok";
    case WQ_ERR_ARG: return "invalid argument (null pointer, negative size or unknown flag)";
    case WQ_ERR_SHAPE: return "unsupported shape (K not a multiple of the format's block, or too large)";
    case WQ_ERR_ALIGN: return "device pointer not 16-byte aligned";
    case WQ_ERR_FMT: return "unknown or unsupported format for this entry point";
    case WQ_ERR_CUDA: return "CUDA launch or runtime error";
    case WQ_ERR_TIMEOUT: return "a kernel abandoned a bounded wait";
    default: return "unknown status";
  }
}

uint64_t wq_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

}  // extern "C"
