// wq_pages.cu -- what a changing batch and drafted tokens ask of the 4-bit KV cache besides rows: pages and slots for
// the tokens of a step, pages given back, the bits of trees, and the rows of an accepted path moved up.
//
// All of it is a few bytes a sequence, token or row, so a call costs its launch and its chain of dependent loads; each is
// one launch, reads its lengths on the device and takes no workspace.
#include <cuda_runtime.h>

#include "wq_kv.cuh"

namespace wq {
namespace {

constexpr int kMost = 1024;      // threads of a block, and sequences of a round
constexpr int kOwn = 4;          // tokens or pages that the thread of a sequence handles by itself

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

// What the warps have to know of a sequence that its thread does not handle by itself.
struct Job {
  int32_t b, len, n, have, need, ok;
  int64_t first, start;          // its first page's place in the order of pages, its first token's
};

// ---------------------------------------------------------------- pages and slots for the tokens of a step
// A thread computes what its sequence needs, one scan over the sequences orders pages and tokens.  The blocks of the
// cluster all do that (they would wait for one that did), and share the writing.  The stack's count may be read and written
// at one address: every block has read it when the first one writes.
__global__ void __launch_bounds__(kMost) kv_reserve_kernel(const __grid_constant__ KvReserveArgs a) {
  __shared__ int64_t part[32][2];
  __shared__ Job jobs[kMost];
  __shared__ int count;
  const KvArgs& kv = a.kv;
  const int rank = (int)cluster_ctarank(), blocks = (int)(gridDim.x), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t pages = 0, tokens = 0;                   // of the sequences before this round's
  const int64_t top = min(max((int64_t)*a.top, (int64_t)0), a.free_size);
  int64_t taken = 0;

  // Page number of a sequence's page p, new ones from the stack.
  auto page_at = [&](const Job& j, int p) -> int {
    return p >= j.have ? a.free_pages[top - 1 - (j.first + (p - j.have))] : kv.table[j.b * kv.table_ld + p];
  };
  auto put_page = [&](const Job& j, int k) {
    const int page = page_at(j, j.have + k);
    if ((uint32_t)page >= (uint64_t)kv.pages) set_status(WQ_STATUS_ARG);
    const_cast<int32_t*>(kv.table)[j.b * kv.table_ld + j.have + k] = page;
  };
  auto put_token = [&](const Job& j, int i) {
    const int64_t k = j.start + i;
    if (k >= a.tokens) return;
    const int pos = (int)min((int64_t)j.len + i, (int64_t)0x7FFFFFFF);
    int64_t slot = -1;
    if (j.ok && a.slots) {
      const int p = kv::page_of(kv, pos), page = page_at(j, p);
      if ((uint32_t)page < (uint64_t)kv.pages) slot = (int64_t)page * kv.page_size + (pos - p * kv.page_size);
      else set_status(WQ_STATUS_ARG);
    }
    if (a.slots) a.slots[k] = slot;
    if (a.positions) a.positions[k] = pos;
  };

  for (int64_t b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    if (threadIdx.x == 0) count = 0;
    const int64_t b = b0 + threadIdx.x;
    Job j{};
    if (b < a.batch) {
      j.b = (int)b;
      j.len = max(a.lens[b], 0);
      j.n = max(a.counts[b], 0);
      const int64_t end = (int64_t)j.len + j.n;
      j.ok = end <= kv.capacity;
      if (j.ok) {
        j.have = pages_for(kv, j.len);
        j.need = pages_for(kv, (int)end) - j.have;
      }
    }
    const Sums s = block_scan(j.need, j.n, part);
    j.first = pages + s.x;
    j.start = tokens + s.y;
    if (j.need > 0 && j.first + j.need > top) j.ok = 0;
    if (j.ok && j.need > 0) taken = j.first + j.need;
    const int n = j.n;
    j.n = (int)min((int64_t)j.n, max(a.tokens - j.start, (int64_t)0));   // those that have a place in the map
    const int need = j.ok ? j.need : 0;
    if (b < a.batch) {
      if (rank == 0) {
        if (a.granted) a.granted[b] = j.ok ? n : 0;
        if (a.starts) a.starts[b] = (int32_t)min(j.start, (int64_t)0x7FFFFFFF);
      }
      if (need <= kOwn && j.n <= kOwn) {
        if (rank == 0) {
          for (int k = 0; k < need; ++k) put_page(j, k);
          for (int i = 0; i < j.n; ++i) put_token(j, i);
        }
      } else {
        j.need = need;
        jobs[atomicAdd(&count, 1)] = j;            // their order does not matter
      }
    }
    __syncthreads();
    // Warps of all blocks take pieces of 32 tokens in turn.
    const int wide = (int)(blockDim.x >> 5);
    for (int at = warp; at < count; at += wide) {
      const Job w = jobs[at];
      for (int k = rank * 32 + lane; k < w.need; k += 32 * blocks) put_page(w, k);
#pragma unroll 4
      for (int i = rank * 32 + lane; i < w.n; i += 32 * blocks) put_token(w, i);
    }
    __syncthreads();
    pages += s.all_x;
    tokens += s.all_y;
  }
  if (rank == 0 && threadIdx.x == 0) {
    if (a.starts) a.starts[a.batch] = (int32_t)min(tokens, (int64_t)0x7FFFFFFF);
    if (a.tokens > 0 && tokens > a.tokens) set_status(WQ_STATUS_ARG);
  }
  for (int64_t k = tokens + rank * (int)blockDim.x + threadIdx.x; k < a.tokens; k += (int64_t)blocks * blockDim.x) {
    if (a.slots) a.slots[k] = -1;
    if (a.positions) a.positions[k] = 0;
  }
  // The pages taken: the largest of the block's threads (those that got none are behind those that did).
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) taken = max(taken, __shfl_xor_sync(0xFFFFFFFFu, taken, d));
  if (lane == 0) part[warp][0] = taken;
  if (blocks > 1) cluster_sync();                  // every block has read the count
  else __syncthreads();
  if (rank == 0 && threadIdx.x == 0) {
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) taken = max(taken, part[w][0]);
    *a.top_out = (int32_t)(top - taken);
  }
}

// ---------------------------------------------------------------- pages given back
__global__ void __launch_bounds__(kMost) kv_release_kernel(const __grid_constant__ KvReserveArgs a) {
  __shared__ int64_t part[32][2];
  __shared__ Job jobs[kMost];
  __shared__ int count;
  const KvArgs& kv = a.kv;
  const int rank = (int)cluster_ctarank(), blocks = (int)gridDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t top = min(max((int64_t)*a.top, (int64_t)0), a.free_size);
  int64_t pages = 0;
  auto push = [&](const Job& j, int k) {
    const int64_t at = top + j.first + k;
    if (at < a.free_size) const_cast<int32_t*>(a.free_pages)[at] = kv.table[j.b * kv.table_ld + j.have + k];
  };
  for (int64_t b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    if (threadIdx.x == 0) count = 0;
    const int64_t b = b0 + threadIdx.x;
    Job j{};
    if (b < a.batch) {
      j.b = (int)b;
      j.len = (int)min((int64_t)max(a.lens[b], 0), kv.capacity);
      j.have = min(pages_for(kv, j.len), pages_for(kv, a.counts ? max(a.counts[b], 0) : 0));   // pages that stay
      j.need = pages_for(kv, j.len) - j.have;
    }
    const Sums s = block_scan(j.need, 0, part);
    j.first = pages + s.x;
    if (j.need > kOwn) jobs[atomicAdd(&count, 1)] = j;
    else if (rank == 0)
      for (int k = 0; k < j.need; ++k) push(j, k);
    __syncthreads();
    const int wide = (int)(blockDim.x >> 5);
    for (int at = warp; at < count; at += wide) {
      const Job w = jobs[at];
#pragma unroll 4
      for (int k = rank * 32 + lane; k < w.need; k += 32 * blocks) push(w, k);
    }
    __syncthreads();
    pages += s.all_x;
  }
  if (blocks > 1) cluster_sync();                  // every block has read the count
  if (rank == 0 && threadIdx.x == 0) {
    if (top + pages > a.free_size) set_status(WQ_STATUS_ARG);
    *a.top_out = (int32_t)min(top + pages, a.free_size);
  }
}

// ---------------------------------------------------------------- trees
// A thread walks up from its node.  Parents come before their children, so the ancestors' bits come out from the highest
// word to the lowest.
__global__ void __launch_bounds__(kMost) tree_mask_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ counts,
                                                          int64_t batch, int tokens, int words, int64_t window,
                                                          uint32_t* __restrict__ mask, int32_t* __restrict__ depth) {
  __shared__ int16_t up[kMost];
  for (int64_t b = blockIdx.x; b < batch; b += gridDim.x) {
    const int n = kv::count_of(counts, b, tokens), i = threadIdx.x;
    if (i < tokens) {
      int parent = i < n ? parents[b * tokens + i] : -1;
      if (parent < -1 || parent >= i) {
        if (i < n) set_status(WQ_STATUS_ARG);
        parent = -1;
      }
      up[i] = (int16_t)parent;
    }
    __syncthreads();
    if (i < tokens) {
      uint32_t* row = mask + (b * tokens + i) * words;
      int node = i < n ? i : -1, levels = 0;
      for (int w = words - 1; w >= 0; --w) {
        uint32_t bits = 0;
        while (node >= 32 * w) {                   // never with node = -1
          if (window == 0 || levels < window) bits |= 1u << (node & 31);
          ++levels;
          node = up[node];
        }
        row[w] = bits;
      }
      if (depth) depth[b * tokens + i] = i < n ? levels - 1 : 0;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- the rows of an accepted path
// A block owns one head of K or V of one sequence and holds all the rows that move, so none is overwritten unread.
constexpr int kKeepThreads = 128;
__global__ void __launch_bounds__(kKeepThreads) kv_keep_kernel(const __grid_constant__ KvKeepArgs a) {
  extern __shared__ __align__(16) uint8_t held[];
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
        const int64_t from = kv::row_of(kv, b, start + node, h, &left);
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

int launched() {
  count_launch();
  return cudaGetLastError() == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

template <class Kernel>
int launch_turn(Kernel* kernel, const KvReserveArgs& a, int64_t work, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  const int64_t wide = (a.batch + 31) / 32 * 32;
  const bool large = work > 4096;
  cfg.gridDim = dim3(large ? 8 : 1);
  cfg.blockDim = dim3((unsigned)(large || wide > kMost ? kMost : wide < 128 ? 128 : wide));
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = large ? 8 : 1;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return WQ_ERR_CUDA;
  return launched();
}

}  // namespace

int kv_reserve(const KvReserveArgs& a, cudaStream_t s) { return launch_turn(kv_reserve_kernel, a, a.tokens, s); }
int kv_release(const KvReserveArgs& a, cudaStream_t s) { return launch_turn(kv_release_kernel, a, a.batch * a.kv.table_ld, s); }

int tree_mask(const int32_t* parents, const int32_t* counts, int64_t batch, int64_t tokens, int64_t window, uint32_t* mask,
              int32_t* depth, cudaStream_t s) {
  const unsigned threads = (unsigned)((tokens + 31) / 32 * 32), blocks = (unsigned)(batch < 65535 ? batch : 65535);
  tree_mask_kernel<<<blocks, threads, 0, s>>>(parents, counts, batch, (int)tokens, (int)((tokens + 31) / 32), window, mask, depth);
  return launched();
}

int kv_keep(const KvKeepArgs& a, cudaStream_t s) {
  const dim3 blocks((unsigned)a.kv.heads, 2, (unsigned)(a.batch < 65535 ? a.batch : 65535));
  const size_t smem = (size_t)a.path_ld * (a.kv.dim / 2 + a.kv.dim / 16);
  kv_keep_kernel<<<blocks, kKeepThreads, smem, s>>>(a);
  return launched();
}

int take_status_pages() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
