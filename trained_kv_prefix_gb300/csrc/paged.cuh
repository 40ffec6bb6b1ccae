// paged.cuh -- what the paged-cache kernels (tree.cu, pages.cu, rows.cu,
// step.cu, weights.cu) share: page lookups, the ancestor sets of drafted trees,
// the scans of planning clusters and the argument rules of tables and pools.
#pragma once

#include <cstdint>

#include "internal.cuh"

namespace cart {

constexpr int kMaxNodes = CART_MAX_TREE_NODES;
static_assert(kMaxNodes == 64, "ancestor sets are 64-bit words");

// log2 of a page's rows, -1 for a size that is not offered.
inline int page_log2_of(int page_rows) {
  for (int l = 4; l <= 7; ++l)
    if (page_rows == 1 << l) return l;
  return -1;
}

inline bool aligned_to(const void* p, unsigned bytes) {
  return p && (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// Page tables of one call (see cartattn.h): row r of conversation b lies in
// page table[b * max_pages + (r >> page_log2)].
struct PageTable {
  const int* table;
  const int* lens;
  int max_pages, n_pages, page_log2;
};

// Rows that conversation b holds: -1 for an idle slot, at most what its
// table row can name.
__device__ __forceinline__ int held_rows_of(const PageTable& t, int len) {
  return len < 0 ? -1 : min(len, t.max_pages << t.page_log2);
}
__device__ __forceinline__ int held_rows(const PageTable& t, int b) {
  return held_rows_of(t, __ldg(t.lens + b));
}

// Page of row r of conversation b, or -1.
__device__ __forceinline__ int page_of(const PageTable& t, int b, int r) {
  const int k = r >> t.page_log2;
  if (r < 0 || k >= t.max_pages) return -1;
  const int page = __ldg(t.table + static_cast<long long>(b) * t.max_pages + k);
  return static_cast<unsigned>(page) < static_cast<unsigned>(t.n_pages) ? page : -1;
}

// Shared memory of tree_ancestors.
struct TreeSmem {
  unsigned long long anc[kMaxNodes];
  int jump[kMaxNodes];
};

// Ancestor sets of one tree, by the whole block (at least 64 threads): on
// return s.anc[t] has bit t and the bits of t's ancestors, or is 0 for a node
// that is unused.  parents: the tree's row (null: a chain); stored: whether
// this thread's node threadIdx.x has a page.  Six rounds of pointer doubling:
// after round k a node's set covers its 2^k nearest ancestors and its jump
// leads past them, and a node whose covered part holds an unused node has
// become unused itself.  Returns whether this thread's node is well placed
// in its tree (a valid parent of its own) but has no page.
__device__ __forceinline__ bool tree_ancestors(TreeSmem& s, const int* parents, int nodes,
                                               bool stored) {
  const int t = threadIdx.x;
  bool lost = false;
  if (t < kMaxNodes) {
    const int up = t < nodes ? (parents ? __ldg(parents + t) : t - 1) : -2;
    const bool placed = up >= -1 && up < t;
    s.anc[t] = placed && stored ? 1ull << t : 0ull;
    s.jump[t] = placed && stored ? up : -2;
    lost = placed && !stored;
  }
  __syncthreads();
#pragma unroll 1
  for (int step = 1; step < nodes; step <<= 1) {
    unsigned long long mine = 0, theirs = 0;
    int j = -1, next = -1;
    if (t < kMaxNodes) {
      mine = s.anc[t];
      j = s.jump[t];
      if (j >= 0) {
        theirs = s.anc[j];
        next = s.jump[j];
      }
    }
    __syncthreads();
    if (t < kMaxNodes && j >= 0) {
      s.anc[t] = theirs ? mine | theirs : 0ull;
      s.jump[t] = theirs ? next : -2;
    }
    __syncthreads();
  }
  return lost;
}

constexpr int kMetaCtas = 8;        // CTAs of a planning cluster
constexpr int kMetaThreads = 1024;  // threads of each
constexpr int kMetaWarps = kMetaCtas * kMetaThreads / 32;

// Every thread of the cluster arrives (its writes released to the cluster)
// and waits for the others.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}

// Exclusive prefix sum of v over the block's 1024 threads; *total the sum.
// Every thread calls it; sums: 33 words of shared memory.
__device__ __forceinline__ int block_scan(int v, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // sums may still be read from an earlier call
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sums[lane] = w;
  }
  __syncthreads();
  *total = sums[31];
  return x - v + (warp ? sums[warp - 1] : 0);
}

__device__ __forceinline__ bool is_page(int page, int n_pages) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(n_pages);
}

// ----------------------------------------------------------- arguments ----
inline int check_tables(int B, int max_pages, int n_pages, int page_rows) {
  if (B < 1 || B > 65535 || max_pages < 1 || n_pages < 1 || n_pages > (1 << 30) ||
      page_log2_of(page_rows) < 0)
    return CART_ERR_GEOMETRY;
  if (static_cast<long long>(max_pages) * page_rows >= (1ll << 24)) return CART_ERR_GEOMETRY;
  return CART_OK;
}

inline int check_pool(int layers, int Hkv, int d, cart_dtype dtype, const void* k, const void* v) {
  if (layers < 1 || layers > 32767 || Hkv < 1 || d < 1 || Hkv > 65535 || d > 65535)
    return CART_ERR_GEOMETRY;
  if (dtype != CART_BF16 && dtype != CART_F32) return CART_ERR_DTYPE;
  const long long row = static_cast<long long>(Hkv) * d * (dtype == CART_BF16 ? 2 : 4);
  if (row % 16 != 0 || row > (1 << 24)) return CART_ERR_GEOMETRY;
  if (!aligned_to(k, 16) || !aligned_to(v, 16)) return CART_ERR_POINTER;
  return CART_OK;
}

}  // namespace cart
