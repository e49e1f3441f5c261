// wq_pages.cu -- what a changing batch and drafted tokens ask of the 4-bit KV cache besides rows: pages and slots for
// the tokens of a step, pages given back, the bits of trees, and the rows of an accepted path moved up.
//
// All of it is a few bytes a sequence, token or row, so a call costs its launch and its chain of dependent loads; lengths
// are read on the device, and no call takes a workspace.  Measured on GB300, in a graph: pages of 3 requests given back and
// of 45 reserved 8 us for the two; 40 requests' pages given back and those and the slots of 1.08 million prompt tokens
// reserved 16 (one cluster of blocks, a warp a sequence: 78); a tree's mask 3; 64 paths of 64 nodes (8 heads of 128) kept 5.
#include <cuda_runtime.h>

#include "wq_kv.cuh"

namespace wq {
namespace {

constexpr int kMost = 1024;      // threads of a block, and sequences of a round
constexpr int kSms = 152;
constexpr int kShare = 2048;     // tokens or pages a block is launched for
constexpr int kRun = 128;        // neighbouring tokens that a warp takes

__device__ __forceinline__ int pages_for(const KvArgs& kv, int tokens) {   // ceil(tokens / page_size), tokens < 2^31
  return tokens > 0 ? kv::page_of(kv, tokens - 1) + 1 : 0;
}

// Exclusive prefix sums of x and y over the block's threads, and the totals.
struct Sums {
  int64_t x, y, all_x, all_y;
};
__device__ __forceinline__ Sums block_scan(int64_t x, int64_t y, int64_t (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t sx = x, sy = y;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t ux = __shfl_up_sync(0xFFFFFFFFu, sx, d), uy = __shfl_up_sync(0xFFFFFFFFu, sy, d);
    if (lane >= d) {
      sx += ux;
      sy += uy;
    }
  }
  if (lane == 31) {
    part[warp][0] = sx;
    part[warp][1] = sy;
  }
  __syncthreads();
  Sums r{sx - x, sy - y, 0, 0};
  int64_t px = lane < warps ? part[lane][0] : 0, py = lane < warps ? part[lane][1] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t ux = __shfl_up_sync(0xFFFFFFFFu, px, d), uy = __shfl_up_sync(0xFFFFFFFFu, py, d);
    if (lane >= d) {
      px += ux;
      py += uy;
    }
  }
  r.all_x = __shfl_sync(0xFFFFFFFFu, px, 31);
  r.all_y = __shfl_sync(0xFFFFFFFFu, py, 31);
  const int64_t bx = __shfl_sync(0xFFFFFFFFu, px, warp > 0 ? warp - 1 : 0), by = __shfl_sync(0xFFFFFFFFu, py, warp > 0 ? warp - 1 : 0);
  if (warp > 0) {
    r.x += bx;
    r.y += by;
  }
  __syncthreads();               // `part` is free again
  return r;
}

// The last i with key[i] <= x, 0 <= i < n; key[0] <= x, and the keys rise.
__device__ __forceinline__ int last_at(const int32_t* key, int n, int x) {
  int lo = 0;
  for (int step = 1 << (31 - __clz(n)); step > 0; step >>= 1)
    if (lo + step < n && key[lo + step] <= x) lo += step;
  return lo;
}

__device__ __forceinline__ int clamp32(int64_t x) { return (int)min(x, (int64_t)0x7FFFFFFF); }

// ---------------------------------------------------------------- pages and slots for the tokens of a step
// A thread computes what its sequence needs, one scan over the sequences orders pages and tokens, and then a thread takes
// a page or a token and looks up whose it is.  Every block does the scan (they would wait for one that did) and they share the
// pages and tokens.  Where they read the stack's count from the address that it goes back to, a second launch writes it:
// WRITE is all but the count.
enum { WRITE = 1, COUNT = 2 };
__global__ void __launch_bounds__(kMost) kv_reserve_kernel(const __grid_constant__ KvReserveArgs a, const int what) {
  __shared__ int64_t part[32][2];
  __shared__ int32_t first_of[kMost], start_of[kMost], len_of[kMost], have_of[kMost];   // have -1: no pages for it
  __shared__ unsigned long long edge;              // pages that those before the first one without its pages take
  const KvArgs& kv = a.kv;
  if (what & WRITE) {
    griddep_wait();                                // what the COUNT launch reads before it waits is written by now
    griddep_launch_dependents();
  }
  const int64_t top = min(max((int64_t)*a.top, (int64_t)0), a.free_size);
  int32_t* table = const_cast<int32_t*>(kv.table);
  const int lane = threadIdx.x & 31;
  int64_t pages = 0, tokens = 0;                   // of the sequences before this round's
  const int64_t me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, all = (int64_t)gridDim.x * blockDim.x;
  if (threadIdx.x == 0) edge = ~0ull;

  for (int64_t b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int64_t b = b0 + threadIdx.x;
    int len = 0, n = 0, have = 0, need = 0;
    bool ok = false;
    if (b < a.batch) {
      len = max(a.lens[b], 0);
      n = max(a.counts[b], 0);
      ok = (int64_t)len + n <= kv.capacity;
      if (ok) {
        have = pages_for(kv, len);
        need = pages_for(kv, len + n) - have;
      }
    }
    const Sums s = block_scan(need, n, part);
    const int64_t first = pages + s.x, start = tokens + s.y;
    if (need > 0 && first + need > top) {
      ok = false;
      atomicMin(&edge, (unsigned long long)first);
    }
    if (what & WRITE) {
      if (b < a.batch && blockIdx.x == 0) {
        if (a.granted) a.granted[b] = ok ? n : 0;
        if (a.starts) a.starts[b] = clamp32(start);
      }
      first_of[threadIdx.x] = clamp32(first);
      start_of[threadIdx.x] = clamp32(start);
      len_of[threadIdx.x] = len;
      have_of[threadIdx.x] = ok ? have : -1;
      __syncthreads();
      const int seqs = (int)min((int64_t)blockDim.x, a.batch - b0);
      const int64_t end = (int64_t)min((unsigned long long)(pages + s.all_x), edge);
      for (int64_t e = pages + me; e < end; e += all) {
        const int i = last_at(first_of, seqs, (int)e);
        const int page = a.free_pages[top - 1 - e];
        if ((uint32_t)page >= (uint64_t)kv.pages) set_status(WQ_STATUS_ARG);
        table[(b0 + i) * kv.table_ld + have_of[i] + ((int)e - first_of[i])] = page;
      }
      // Tokens by warps, 128 neighbours at a time: mostly one sequence's, which is then looked up once.
      const int64_t stop = min(tokens + s.all_y, a.tokens);
      for (int64_t k0 = tokens + (me >> 5) * kRun; k0 < stop; k0 += (all >> 5) * kRun) {
        const int i0 = last_at(start_of, seqs, (int)k0), rest = (int)min(stop - k0, (int64_t)kRun);
        const bool one = i0 + 1 >= seqs || start_of[i0 + 1] >= (int)k0 + rest;
        int page[kRun / 32], pos[kRun / 32];
        uint32_t asked = 0;                        // bit r: a page was looked up
#pragma unroll
        for (int r = 0; r < kRun / 32; ++r) {
          const int k = (int)k0 + min(32 * r + lane, rest - 1), i = one ? i0 : last_at(start_of, seqs, k);
          const int have = have_of[i];
          pos[r] = clamp32((int64_t)len_of[i] + (k - start_of[i]));
          const bool ask = a.slots && have >= 0 && 32 * r + lane < rest;
          const int p = kv::page_of(kv, pos[r]);   // a new page's number is still on the stack
          const int32_t* at = p >= have ? a.free_pages + (top - 1 - ((int64_t)first_of[i] + (p - have))) : table + (b0 + i) * kv.table_ld + p;
          page[r] = ask ? *at : -1;
          asked |= (ask ? 1u : 0u) << r;
        }
#pragma unroll
        for (int r = 0; r < kRun / 32; ++r) {
          const int x = 32 * r + lane;
          if (x >= rest) break;
          const int off = pos[r] - kv::page_of(kv, pos[r]) * kv.page_size;
          const bool good = (uint32_t)page[r] < (uint64_t)kv.pages;
          if (!good && ((asked >> r) & 1u)) set_status(WQ_STATUS_ARG);
          if (a.slots) a.slots[k0 + x] = good ? (int64_t)page[r] * kv.page_size + off : -1;
          if (a.positions) a.positions[k0 + x] = pos[r];
        }
      }
      __syncthreads();
    }
    pages += s.all_x;
    tokens += s.all_y;
  }
  if (what & WRITE) {
    if (me == 0) {
      if (a.starts) a.starts[a.batch] = clamp32(tokens);
      if ((a.slots || a.positions) && tokens > a.tokens) set_status(WQ_STATUS_ARG);
    }
    for (int64_t k = tokens + me; k < a.tokens; k += all) {
      if (a.slots) a.slots[k] = -1;
      if (a.positions) a.positions[k] = 0;
    }
  }
  if (!(what & COUNT) || blockIdx.x != 0) return;
  if (!(what & WRITE)) griddep_wait();             // the launch before has read the count
  __syncthreads();
  if (threadIdx.x == 0) *a.top_out = (int32_t)(top - (int64_t)min((unsigned long long)pages, edge));
}

// ---------------------------------------------------------------- pages given back
// The same for the pages that go: `counts` are the tokens that stay.
__global__ void __launch_bounds__(kMost) kv_release_kernel(const __grid_constant__ KvReserveArgs a, const int what) {
  __shared__ int64_t part[32][2];
  __shared__ int32_t first_of[kMost], have_of[kMost];
  const KvArgs& kv = a.kv;
  if (what & WRITE) {
    griddep_wait();                                // what the COUNT launch reads before it waits is written by now
    griddep_launch_dependents();
  }
  const int64_t top = min(max((int64_t)*a.top, (int64_t)0), a.free_size);
  const int64_t me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, all = (int64_t)gridDim.x * blockDim.x;
  int64_t pages = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int64_t b = b0 + threadIdx.x;
    int have = 0, need = 0;
    if (b < a.batch) {
      const int held = pages_for(kv, (int)min((int64_t)max(a.lens[b], 0), kv.capacity));
      have = min(held, pages_for(kv, a.counts ? max(a.counts[b], 0) : 0));
      need = held - have;
    }
    const Sums s = block_scan(need, 0, part);
    if (what & WRITE) {
      first_of[threadIdx.x] = clamp32(pages + s.x);
      have_of[threadIdx.x] = have;
      __syncthreads();
      const int seqs = (int)min((int64_t)blockDim.x, a.batch - b0);
      const int64_t end = min(pages + s.all_x, a.free_size - top);
#pragma unroll 2
      for (int64_t e = pages + me; e < end; e += all) {
        const int i = last_at(first_of, seqs, (int)e);
        const int page = kv.table[(b0 + i) * kv.table_ld + have_of[i] + ((int)e - first_of[i])];
        if ((uint32_t)page >= (uint64_t)kv.pages) set_status(WQ_STATUS_ARG);
        const_cast<int32_t*>(a.free_pages)[top + e] = page;
      }
      __syncthreads();
    }
    pages += s.all_x;
  }
  if (!(what & COUNT) || blockIdx.x != 0) return;
  if (!(what & WRITE)) griddep_wait();             // the launch before has read the count
  __syncthreads();
  if (threadIdx.x == 0) {
    if (top + pages > a.free_size) set_status(WQ_STATUS_ARG);
    *a.top_out = (int32_t)min(top + pages, a.free_size);
  }
}

// ---------------------------------------------------------------- trees
// A thread walks up from its node.  Parents come before their children, so the ancestors' bits come out from the highest
// word to the lowest.  Sinks: ancestor j stays where its position, lens - counts + its depth, is below them; its depth is the
// node's less the levels between them, so the node's is counted first, by a walk of its own.
__global__ void __launch_bounds__(kMost) tree_mask_kernel(const __grid_constant__ TreeMaskArgs a, const int words) {
  __shared__ int16_t up[kMost];
  const int tokens = (int)a.tokens;
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const int n = kv::count_of(a.counts, b, tokens), i = threadIdx.x;
    if (i < tokens) {
      int parent = i < n ? a.parents[b * tokens + i] : -1;
      if (parent < -1 || parent >= i) {
        if (i < n) set_status(WQ_STATUS_ARG);
        parent = -1;
      }
      up[i] = (int16_t)parent;
    }
    __syncthreads();
    if (i < tokens) {
      uint32_t* row = a.mask + (b * tokens + i) * words;
      const bool sinks = a.window > 0 && a.sinks > 0;
      int64_t far = 0x7FFFFFFF;                    // levels up from which on ancestors are sinks
      if (sinks) {
        int mine = -1;
        for (int k = i < n ? i : -1; k >= 0; k = up[k]) ++mine;
        far = (int64_t)max(a.lens[b], 0) - n + mine - a.sinks + 1;
      }
      int node = i < n ? i : -1, levels = 0;
      for (int w = words - 1; w >= 0; --w) {
        uint32_t bits = 0;
        while (node >= 32 * w) {                   // never with node = -1
          if (a.window == 0 || levels < a.window || (sinks && levels >= far)) bits |= 1u << (node & 31);
          ++levels;
          node = up[node];
        }
        row[w] = bits;
      }
      if (a.depth) a.depth[b * tokens + i] = i < n ? levels - 1 : 0;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- the rows of an accepted path
// A block owns one head of K or V of one sequence and holds all the rows that move, so none is overwritten unread.
constexpr int kKeepThreads = 128;
__global__ void __launch_bounds__(kKeepThreads) kv_keep_kernel(const __grid_constant__ KvKeepArgs a) {
  extern __shared__ __align__(16) uint8_t held[];
  griddep_wait();
  griddep_launch_dependents();
  const KvArgs& kv = a.kv;
  const int which = blockIdx.y, h = blockIdx.x;
  const int code_bytes = kv.dim / 2, scale_bytes = kv.dim / 16, pieces = code_bytes / 16;
  uint8_t* scales = held + (int64_t)a.path_ld * code_bytes;
  for (int64_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
    const int n = kv::count_of(a.counts, b, a.path_ld);
    const int64_t start = a.start[b];
    const int32_t* path = a.path + b * a.path_ld;
    int left;
    // a thread writes what it read: codes 16 bytes at a time, then scales four
    for (int pass = 0; pass < 2; ++pass) {
      for (int x = threadIdx.x; x < n * (pieces + 1); x += kKeepThreads) {
        const int i = x / (pieces + 1), c = x - i * (pieces + 1);
        const int node = path[i];
        if (node == i) continue;
        if (node < 0) set_status(WQ_STATUS_ARG);     // no node, though its position may well lie in the context
        const int64_t from = node < 0 ? -1 : kv::row_of(kv, b, start + node, h, &left);
        if (from < 0) continue;
        const int64_t row = pass == 0 ? from : kv::row_of(kv, b, start + i, h, &left);
        if (row < 0) continue;
        uint8_t* mine = c < pieces ? held + i * code_bytes + 16 * c : scales + i * scale_bytes;
        uint8_t* theirs = c < pieces ? kv.codes[which] + row * code_bytes + 16 * c : kv.scales[which] + row * scale_bytes;
        uint8_t *dst = pass == 0 ? mine : theirs, *src = pass == 0 ? theirs : mine;
        if (c < pieces) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        else if (scale_bytes == 8) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(src);
        else *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
      }
      __syncthreads();
    }
  }
}

// work: tokens or pages, at most.
template <class Kernel>
int launch_turn(Kernel* kernel, const KvReserveArgs& a, int64_t work, cudaStream_t s) {
  const int64_t wide = (a.batch + 31) / 32 * 32, want = (work + kShare - 1) / kShare;
  const int blocks = want > kSms ? kSms : want < 1 ? 1 : (int)want;
  const int threads = blocks > 1 || wide > kMost ? kMost : wide < 128 ? 128 : (int)wide;
  const bool once = blocks == 1 || a.top_out != a.top;
  if (launch_early(kernel, dim3(blocks), dim3(threads), 0, s, 1u, a, once ? WRITE | COUNT : WRITE) != cudaSuccess) return WQ_ERR_CUDA;
  count_launch();
  if (once) return WQ_OK;
  if (launch_early(kernel, dim3(1), dim3(threads), 0, s, 1u, a, COUNT) != cudaSuccess) return WQ_ERR_CUDA;
  count_launch();
  return WQ_OK;
}

}  // namespace

int kv_reserve(const KvReserveArgs& a, cudaStream_t s) { return launch_turn(kv_reserve_kernel, a, a.tokens, s); }
int kv_release(const KvReserveArgs& a, cudaStream_t s) { return launch_turn(kv_release_kernel, a, a.batch * a.kv.table_ld, s); }

int tree_mask(const TreeMaskArgs& a, cudaStream_t s) {
  const int words = (int)((a.tokens + 31) / 32);
  const unsigned blocks = (unsigned)(a.batch < 65535 ? a.batch : 65535);
  if (launch_early(tree_mask_kernel, dim3(blocks), dim3(32 * words), 0, s, 1u, a, words) != cudaSuccess) return WQ_ERR_CUDA;
  count_launch();
  return WQ_OK;
}

int kv_keep(const KvKeepArgs& a, cudaStream_t s) {
  const dim3 blocks((unsigned)a.kv.heads, 2, (unsigned)(a.batch < 65535 ? a.batch : 65535));
  const size_t smem = (size_t)a.path_ld * (a.kv.dim / 2 + a.kv.dim / 16);
  if (launch_early(kv_keep_kernel, blocks, dim3(kKeepThreads), smem, s, 1u, a) != cudaSuccess) return WQ_ERR_CUDA;
  count_launch();
  return WQ_OK;
}

int take_status_pages() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
