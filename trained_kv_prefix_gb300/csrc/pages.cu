// pages.cu -- operators on the pages of the private caches (cartattn.h,
// "Paged private caches"): fork, reserve, accept, compact.
//
// The tables are small (a conversation's table row, one count per page) and
// the data large (a page in every layer), so reserve and compact run as two
// launches: a plan by ONE thread-block cluster, whose phases are separated by
// cluster barriers and which leaves a list of page copies in the workspace,
// and the copies by the whole GPU as its programmatic dependent.  Everything
// is decided by prefix sums over conversation and page numbers, and counts
// are the only atomics (integer additions), so results do not depend on the
// order in which threads run.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cart {
namespace {

constexpr int kMaxForks = 8192;

// Workspace of reserve and compact (int32 words): the head, then the lists.
struct PagesWs {
  size_t count, base, ids, slots, copies, starts, total;  // byte offsets
};
enum { kHeadSeg = 0, kHeadCopies = 16, kHeadFirst = 17, kHeadInts = 64 };

PagesWs pages_ws(int B, int n_pages) {
  PagesWs w{};
  size_t off = kHeadInts * 4;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~static_cast<size_t>(255);
    return o;
  };
  w.count = take(static_cast<size_t>(B) * 4);
  w.base = take(static_cast<size_t>(B) * 4);
  w.ids = take(static_cast<size_t>(n_pages) * 4);
  w.slots = take(static_cast<size_t>(n_pages) * 4);
  w.copies = take(static_cast<size_t>(std::max(B, n_pages)) * 16);
  w.starts = take((static_cast<size_t>(B) + 1) * 8);
  w.total = off;
  return w;
}

// ---------------------------------------------------------------- fork ----
// One block per fork.  A conversation that is a destination is nobody's
// source and no other fork's destination (checked over the lists), so the
// block alone touches its table row, and no source row changes.  Bound by
// latency: 700 forks of up to 512 pages take 8.4 us.
__global__ void __launch_bounds__(256) fork_kernel(int B, int* table, int max_pages, int* lens,
                                                   int* refs, int n_pages, int page_log2,
                                                   const int* __restrict__ src,
                                                   const int* __restrict__ dst,
                                                   const int* __restrict__ rows, int forks,
                                                   int* done) {
  const int f = blockIdx.x, from = __ldg(src + f), to = __ldg(dst + f);
  bool bad = from < 0 || from >= B || to < 0 || to >= B;
  for (int g = threadIdx.x; g < forks; g += blockDim.x)
    bad |= __ldg(src + g) == to || (g != f && __ldg(dst + g) == to);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) done[f] = 0;
    return;
  }
  int n = min(lens[from], max_pages << page_log2);
  if (rows) n = min(n, __ldg(rows + f));
  n = max(n, 0);
  const int end = (n + (1 << page_log2) - 1) >> page_log2;
  const int* a = table + static_cast<long long>(from) * max_pages;
  int* z = table + static_cast<long long>(to) * max_pages;
  for (int k = threadIdx.x; k < max_pages; k += blockDim.x) {
    const int now = k < end ? a[k] : -1, old = z[k];
    if (now == old) continue;
    if (is_page(now, n_pages)) atomicAdd(refs + now, 1);
    if (is_page(old, n_pages)) atomicSub(refs + old, 1);
    z[k] = now;
  }
  if (threadIdx.x == 0) {
    lens[to] = n;
    done[f] = 1;
  }
}

// Copies go by chunks of 16 KB: 256 threads with four 16-byte loads each.
constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 4;
constexpr int kChunk = kCopyThreads * kCopyLoads * 16;
__host__ __device__ __forceinline__ int chunks_of(int rows, int row_bytes) {
  return static_cast<int>((static_cast<long long>(rows) * row_bytes + kChunk - 1) / kChunk);
}

// -------------------------------------------------------------- reserve ----
struct ReserveArgs {
  int B, max_pages, n_pages, page_log2;
  int *table, *lens, *refs, *done;
  const int* rows;
  int *head, *count, *base, *free;
  int4* copies;  // [B]: (from page, to page, rows); rows 0: none
  long long* starts;  // [B + 1]: chunks of one layer and pool before each copy
  int row_bytes;
};

// Conversation b's request: whether it asks, whether it is to append, the page
// of its next row and the end of its pages.
struct Request {
  bool asks, appends;
  int first, end, len;
};
__device__ __forceinline__ Request request(const ReserveArgs& a, int b) {
  const int n = __ldg(a.rows + b);
  Request r;
  r.asks = n >= 0 && n <= (a.max_pages << a.page_log2);
  r.len = min(max(__ldcg(a.lens + b), 0), n);
  r.appends = r.len < n;
  r.first = r.asks ? r.len >> a.page_log2 : 0;
  r.end = r.asks ? (n + (1 << a.page_log2) - 1) >> a.page_log2 : 0;
  return r;
}

// A table entry that is to be replaced by an own page, between the phases:
// its page is shared.
__device__ __forceinline__ int mark_shared(int page) { return -2 - page; }

// Bound by the latency of its four phases, each a chain of a few loads behind
// a cluster barrier; one launch of eight CTAs, since a launch per phase would
// cost 3 us of host time each.  13 us alone for 256 branches over 1600 pages.
__global__ void __cluster_dims__(kMetaCtas, 1, 1) __launch_bounds__(kMetaThreads)
    reserve_plan_kernel(const ReserveArgs a) {
  pdl_release();
  __shared__ int sums[33];
  const int rank = cluster_rank(), lane = threadIdx.x & 31;
  const int gw = rank * (kMetaThreads / 32) + (threadIdx.x >> 5);
  // ---- pages behind the last of rows[b] rows go back
  for (int b = gw; b < a.B; b += kMetaWarps) {
    const Request q = request(a, b);
    if (!q.asks) continue;
    int* row = a.table + static_cast<long long>(b) * a.max_pages;
    for (int k = q.end + lane; k < a.max_pages; k += 32) {
      const int page = row[k];
      if (is_page(page, a.n_pages)) atomicSub(a.refs + page, 1);
      if (page != -1) row[k] = -1;
    }
    if (lane == 0) a.lens[b] = q.len;
  }
  cluster_sync();
  // ---- pages that each conversation needs; shared ones are marked, since
  // the counts change again below.  And the free pages of this CTA's part.
  for (int b = gw; b < a.B; b += kMetaWarps) {
    const Request q = request(a, b);
    int* row = a.table + static_cast<long long>(b) * a.max_pages;
    int n = 0, part_rows = 0;
    for (int k0 = q.first; k0 < q.end; k0 += 32) {
      const int k = k0 + lane;
      bool need = false;
      if (k < q.end) {
        const int page = __ldcg(row + k);
        const bool held = is_page(page, a.n_pages);
        need = !held || __ldcg(a.refs + page) > 1;
        if (need) row[k] = held ? mark_shared(page) : -1;
        if (need && held && k == q.first) part_rows = q.len & ((1 << a.page_log2) - 1);
      }
      n += __popc(__ballot_sync(0xffffffffu, need));
    }
    if (lane == 0) {  // (page q.first is lane 0's)
      a.count[b] = n;
      a.copies[b].z = part_rows;
    }
  }
  const int part = (a.n_pages + kMetaCtas - 1) / kMetaCtas;
  const int lo = rank * part, hi = min(lo + part, a.n_pages);
  int mine = 0, n_part = 0;
  for (int i = lo + threadIdx.x; i < hi; i += kMetaThreads) mine += __ldcg(a.refs + i) <= 0;
  block_scan(mine, sums, &n_part);
  if (threadIdx.x == 0) a.head[kHeadSeg + rank] = n_part;
  cluster_sync();
  // ---- free pages in order (every CTA its part), and over conversations the
  // running need and the chunks to copy (CTA 0)
  int before = 0, n_free = 0;
  for (int r = 0; r < kMetaCtas; ++r) {
    const int n = __ldcg(a.head + kHeadSeg + r);
    before += r < rank ? n : 0;
    n_free += n;
  }
  for (int i0 = lo; i0 < hi; i0 += kMetaThreads) {
    const int i = i0 + threadIdx.x;
    const bool is_free = i < hi && __ldcg(a.refs + i) <= 0;
    int n;
    const int at = block_scan(is_free, sums, &n);
    if (is_free) a.free[before + at] = i;
    before += n;
  }
  if (rank == 0) {
    long long run = 0, chunks = 0;  // run saturates above any pool
    for (int b0 = 0; b0 < a.B; b0 += kMetaThreads) {
      const int b = b0 + threadIdx.x;
      const int need = b < a.B ? __ldcg(a.count + b) : 0;
      const int rows = b < a.B ? __ldcg(&a.copies[b].z) : 0;
      int n;
      const int base = static_cast<int>(min(run + block_scan(need, sums, &n), 0x40000000ll));
      run += n;
      // (a conversation that finds too few pages copies nothing)
      const int c = base + need <= n_free ? chunks_of(rows, a.row_bytes) : 0;
      const int at = block_scan(c, sums, &n);
      if (b < a.B) {
        a.base[b] = base;
        a.starts[b] = chunks + at;
      }
      chunks += n;
    }
    if (threadIdx.x == 0) a.starts[a.B] = chunks;
  }
  cluster_sync();
  // ---- hand the pages out
  for (int b = gw; b < a.B; b += kMetaWarps) {
    const Request q = request(a, b);
    const int n = __ldcg(a.count + b), base = __ldcg(a.base + b);
    const bool ok = n == 0 || base + n <= n_free;
    int* row = a.table + static_cast<long long>(b) * a.max_pages;
    int4 copy = make_int4(0, 0, 0, 0);
    int taken = 0;
    for (int k0 = q.first; k0 < q.end && n > 0; k0 += 32) {
      const int k = k0 + lane;
      const int e = k < q.end ? __ldcg(row + k) : 0;
      const unsigned need = __ballot_sync(0xffffffffu, e < 0);
      if (e < 0) {
        const int old = e == -1 ? -1 : mark_shared(e);  // (its own inverse)
        if (!ok) {
          row[k] = old;
        } else {
          const int page = __ldcg(a.free + base + taken + __popc(need & ((1u << lane) - 1)));
          row[k] = page;
          a.refs[page] = 1;
          if (old >= 0) {
            atomicSub(a.refs + old, 1);
            if (k == q.first) copy = make_int4(old, page, q.len & ((1 << a.page_log2) - 1), 0);
          }
        }
      }
      taken += __popc(need);
    }
    if (lane == 0) {
      a.copies[b] = copy;
      a.done[b] = q.asks && (ok || !q.appends);
    }
  }
}

// -------------------------------------------------------------- compact ----
struct CompactArgs {
  int n_pages;
  int *refs, *moved, *live;
  int *head, *holes, *from;
  int4* copies;
  int page_rows;
};

// With lp(i) the live pages below i and n = lp(n_pages): the free page i < n
// is the (i - lp(i))-th hole, and the live page j >= n the (lp(j) - lp(n))-th
// to move.  Bound by latency: 9 us alone for 1200 pages.
__global__ void __cluster_dims__(kMetaCtas, 1, 1) __launch_bounds__(kMetaThreads)
    compact_plan_kernel(const CompactArgs a) {
  pdl_release();
  __shared__ int sums[33];
  const int rank = cluster_rank();
  const int part = (a.n_pages + kMetaCtas - 1) / kMetaCtas;
  const int lo = rank * part, hi = min(lo + part, a.n_pages);
  int mine = 0, n_part = 0;
  for (int i = lo + threadIdx.x; i < hi; i += kMetaThreads) mine += __ldcg(a.refs + i) > 0;
  block_scan(mine, sums, &n_part);
  if (threadIdx.x == 0) a.head[kHeadSeg + rank] = n_part;
  cluster_sync();
  int before = 0, n = 0;
  for (int r = 0; r < kMetaCtas; ++r) {
    const int c = __ldcg(a.head + kHeadSeg + r);
    before += r < rank ? c : 0;
    n += c;
  }
  if (n == a.n_pages && rank == 0 && threadIdx.x == 0) a.head[kHeadFirst] = n;
  for (int i0 = lo; i0 < hi; i0 += kMetaThreads) {
    const int i = i0 + threadIdx.x;
    const int refs = i < hi ? __ldcg(a.refs + i) : 0;
    const bool live = refs > 0;
    int c;
    const int lp = before + block_scan(live, sums, &c);
    if (i < hi) {
      if (i == n) a.head[kHeadFirst] = lp;
      if (live && i >= n)
        a.from[lp] = i;
      else
        a.moved[i] = live ? i : -1;
      if (!live) {
        if (i < n) a.holes[i - lp] = i;
        if (refs) a.refs[i] = 0;
      }
    }
    before += c;
  }
  cluster_sync();
  const int first = __ldcg(a.head + kHeadFirst);
  const int moves = n - first;
  for (int r = rank * kMetaThreads + threadIdx.x; r < moves; r += kMetaCtas * kMetaThreads) {
    const int j = __ldcg(a.from + first + r), i = __ldcg(a.holes + r);
    a.moved[j] = i;
    a.refs[i] = __ldcg(a.refs + j);
    a.refs[j] = 0;
    a.copies[r] = make_int4(j, i, a.page_rows, 0);
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.head[kHeadCopies] = moves;
    *a.live = n;
  }
}

// --------------------------------------------------------------- copies ----
struct CopyArgs {
  const int4* copies;
  const int* n_copies;      // copies of whole pages: how many
  const long long* starts;  // or copies of some rows each: chunks before them
  int count;                // (of `count` copies)
  char *k, *v;
  long long layer_bytes, page_bytes;
  int row_bytes, layers;
  int* table;               // compact: entries renamed by `moved` (null: none)
  const int* moved;
  long long entries;
  int n_pages;
};

// A CTA takes every gridDim-th chunk of all layers and pools, all of its loads
// in flight before its stores.  Bound by HBM: compacting 16 layers moves 2.38
// GB of whole pages in 354 us, 6.7 TB/s, as fast as a plain copy.  Where copies
// have rows of their own number, the chunks are found through their starts, so
// that none is empty: 256 branches' part pages, 0.79 GB, take 122 us, 6.5 TB/s
// (with empty chunks left in 155 us).
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs a) {
  pdl_wait();
  if (a.table)
    for (long long e = blockIdx.x * static_cast<long long>(kCopyThreads) + threadIdx.x;
         e < a.entries; e += static_cast<long long>(gridDim.x) * kCopyThreads) {
      const int page = a.table[e];
      const int to = is_page(page, a.n_pages) ? __ldcg(a.moved + page) : -1;
      if (to != page) a.table[e] = to;
    }
  const int whole = static_cast<int>((a.page_bytes + kChunk - 1) / kChunk);  // chunks of a page
  const long long per_pool =
      a.starts ? __ldcg(a.starts + a.count) : static_cast<long long>(whole) * __ldcg(a.n_copies);
  const long long total = per_pool * 2 * a.layers;
  for (long long u = blockIdx.x; u < total; u += gridDim.x) {
    const int pool_of = static_cast<int>(u / per_pool);
    const long long x = u - pool_of * per_pool;
    int i;  // the copy
    long long off;
    if (a.starts) {  // the last copy that starts at or before chunk x
      int lo = 0, hi = a.count;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.starts + mid) <= x)
          lo = mid;
        else
          hi = mid;
      }
      i = lo;
      off = (x - __ldg(a.starts + lo)) * kChunk;
    } else {
      i = static_cast<int>(x / whole);
      off = (x - static_cast<long long>(i) * whole) * kChunk;
    }
    const int4 c = __ldg(a.copies + i);
    const long long bytes = static_cast<long long>(c.z) * a.row_bytes;
    char* pool = ((pool_of & 1) ? a.v : a.k) + (pool_of >> 1) * a.layer_bytes;
    const char* from = pool + c.x * a.page_bytes + off;
    char* to = pool + c.y * a.page_bytes + off;
    uint4 r[kCopyLoads];
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j) {
      const int at = (j * kCopyThreads + threadIdx.x) * 16;
      if (off + at < bytes) r[j] = __ldcs(reinterpret_cast<const uint4*>(from + at));
    }
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j) {
      const int at = (j * kCopyThreads + threadIdx.x) * 16;
      if (off + at < bytes) __stcs(reinterpret_cast<uint4*>(to + at), r[j]);
    }
  }
}

cudaError_t launch_copies(const CopyArgs& a, cudaStream_t st) {
  const int sms = sm_count();
  if (sms < 1) return cudaErrorInvalidValue;
  return launch_dependent(copy_kernel, dim3(8 * sms), dim3(kCopyThreads), 0, st, a);
}

// --------------------------------------------------------------- accept ----
struct AcceptArgs {
  PageTable pt;
  int nodes, row_bytes, page_rows;
  const int *parents, *node;
  int* new_lens;
  char *k, *v;
  long long layer_bytes, page_bytes;
};

// Block (layer and pool, conversation).  Thread i owns 16-byte columns of the
// rows and moves them along the path in order: node i of the path is never
// before slot i, so a slot is written only after the node that lay there has
// been read.  Bound by latency (the tree's ancestors, then eight rows at a
// time): paths in trees of 64 nodes, 64 conversations, 32 layers, of which 1.9
// rows a conversation change their place, take 11 us, 2.9 TB/s.
__global__ void __launch_bounds__(128) accept_kernel(const AcceptArgs a) {
  __shared__ TreeSmem tree;
  __shared__ long long from[kMaxNodes], to[kMaxNodes];
  const int b = blockIdx.y, t = threadIdx.x;
  const int len = held_rows(a.pt, b);
  const int page = len >= 0 && t < a.nodes ? page_of(a.pt, b, len + t) : -1;
  tree_ancestors(tree, a.parents ? a.parents + static_cast<long long>(b) * a.nodes : nullptr,
                 a.nodes, page >= 0);
  const int last = __ldg(a.node + b);
  const unsigned long long path = last >= 0 && last < a.nodes ? tree.anc[last] : 0ull;
  const int n = __popcll(path);
  if (blockIdx.x == 0 && t == 0) a.new_lens[b] = path ? len + n : __ldg(a.pt.lens + b);
  if (t < a.nodes && (path >> t & 1)) {
    // node t is the i-th of the path; its slot's row is a node's row too
    const int i = __popcll(path & ((1ull << t) - 1)), r = len + t, z = len + i;
    const int zp = page_of(a.pt, b, z);
    from[i] = page * a.page_bytes + static_cast<long long>(r & (a.page_rows - 1)) * a.row_bytes;
    to[i] = i == t || zp < 0 ? -1
                             : zp * a.page_bytes +
                                   static_cast<long long>(z & (a.page_rows - 1)) * a.row_bytes;
  }
  __syncthreads();
  char* pool = ((blockIdx.x & 1) ? a.v : a.k) + (blockIdx.x >> 1) * a.layer_bytes;
  for (int c = t * 16; c < a.row_bytes; c += 128 * 16)
    for (int i0 = 0; i0 < n; i0 += 8) {
      uint4 r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < n && to[i0 + i] >= 0)
          r[i] = *reinterpret_cast<const uint4*>(pool + from[i0 + i] + c);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < n && to[i0 + i] >= 0)
          *reinterpret_cast<uint4*>(pool + to[i0 + i] + c) = r[i];
    }
}

// ----------------------------------------------------------- arguments ----
int row_bytes_of(int Hkv, int d, cart_dtype dtype) {
  return Hkv * d * (dtype == CART_BF16 ? 2 : 4);
}

int to_status(cudaError_t e) { return e == cudaSuccess ? CART_OK : CART_ERR_CUDA; }

}  // namespace
}  // namespace cart

using namespace cart;

extern "C" {

int cart_pages_fork(int B, int* table, int max_pages, int* lens, int* refs, int n_pages,
                    int page_rows, const int* src, const int* dst, const int* rows, int forks,
                    int* done, void* stream) {
  int rc = check_tables(B, max_pages, n_pages, page_rows);
  if (rc) return rc;
  if (forks < 1 || forks > kMaxForks) return CART_ERR_GEOMETRY;
  if (!aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(refs, 4) ||
      !aligned_to(src, 4) || !aligned_to(dst, 4) || (rows && !aligned_to(rows, 4)) ||
      !aligned_to(done, 4))
    return CART_ERR_POINTER;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope tr("pages_fork", st);
  fork_kernel<<<forks, 256, 0, st>>>(B, table, max_pages, lens, refs, n_pages,
                                     page_log2_of(page_rows), src, dst, rows, forks, done);
  return to_status(cudaGetLastError());
}

size_t cart_pages_workspace_size(int B, int max_pages, int n_pages) {
  if (check_tables(B, max_pages, n_pages, 16)) return 0;
  return pages_ws(B, n_pages).total;
}

int cart_pages_reserve(int B, int layers, int Hkv, int d, cart_dtype dtype, void* k_pages,
                       void* v_pages, int n_pages, int page_rows, int* table, int max_pages,
                       int* lens, int* refs, const int* rows, int* done, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int rc = check_tables(B, max_pages, n_pages, page_rows);
  if (!rc) rc = check_pool(layers, Hkv, d, dtype, k_pages, v_pages);
  if (rc) return rc;
  if (!aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(refs, 4) ||
      !aligned_to(rows, 4) || !aligned_to(done, 4))
    return CART_ERR_POINTER;
  const PagesWs w = pages_ws(B, n_pages);
  if (!aligned_to(workspace, 16) || workspace_bytes < w.total) return CART_ERR_WORKSPACE;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  ReserveArgs a{};
  a.B = B;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.page_log2 = page_log2_of(page_rows);
  a.table = table;
  a.lens = lens;
  a.refs = refs;
  a.done = done;
  a.rows = rows;
  a.head = reinterpret_cast<int*>(ws);
  a.count = reinterpret_cast<int*>(ws + w.count);
  a.base = reinterpret_cast<int*>(ws + w.base);
  a.free = reinterpret_cast<int*>(ws + w.ids);
  a.copies = reinterpret_cast<int4*>(ws + w.copies);
  a.starts = reinterpret_cast<long long*>(ws + w.starts);
  a.row_bytes = row_bytes_of(Hkv, d, dtype);
  TraceScope tr("pages_reserve", st);
  reserve_plan_kernel<<<kMetaCtas, kMetaThreads, 0, st>>>(a);
  rc = to_status(cudaGetLastError());
  if (rc) return rc;
  CopyArgs c{};
  c.copies = a.copies;
  c.starts = a.starts;
  c.count = B;
  c.k = static_cast<char*>(k_pages);
  c.v = static_cast<char*>(v_pages);
  c.row_bytes = row_bytes_of(Hkv, d, dtype);
  c.page_bytes = static_cast<long long>(c.row_bytes) * page_rows;
  c.layer_bytes = c.page_bytes * n_pages;
  c.layers = layers;
  return to_status(launch_copies(c, st));
}

int cart_pages_accept(int B, int nodes, int layers, int Hkv, int d, cart_dtype dtype,
                      void* k_pages, void* v_pages, int n_pages, int page_rows, const int* table,
                      int max_pages, const int* lens, const int* parents, const int* node,
                      int* new_lens, void* stream) {
  int rc = check_tables(B, max_pages, n_pages, page_rows);
  if (!rc) rc = check_pool(layers, Hkv, d, dtype, k_pages, v_pages);
  if (rc) return rc;
  if (nodes < 1 || nodes > kMaxNodes) return CART_ERR_GEOMETRY;
  if (!aligned_to(table, 4) || !aligned_to(lens, 4) || (parents && !aligned_to(parents, 4)) ||
      !aligned_to(node, 4) || !aligned_to(new_lens, 4) || new_lens == lens)
    return CART_ERR_POINTER;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AcceptArgs a{};
  a.pt = PageTable{table, lens, max_pages, n_pages, page_log2_of(page_rows)};
  a.nodes = nodes;
  a.page_rows = page_rows;
  a.parents = parents;
  a.node = node;
  a.new_lens = new_lens;
  a.k = static_cast<char*>(k_pages);
  a.v = static_cast<char*>(v_pages);
  a.row_bytes = row_bytes_of(Hkv, d, dtype);
  a.page_bytes = static_cast<long long>(a.row_bytes) * page_rows;
  a.layer_bytes = a.page_bytes * n_pages;
  TraceScope tr("pages_accept", st);
  accept_kernel<<<dim3(2 * layers, B), 128, 0, st>>>(a);
  return to_status(cudaGetLastError());
}

int cart_pages_compact(int B, int layers, int Hkv, int d, cart_dtype dtype, void* k_pages,
                       void* v_pages, int n_pages, int page_rows, int* table, int max_pages,
                       int* refs, int* moved, int* live, void* workspace, size_t workspace_bytes,
                       void* stream) {
  int rc = check_tables(B, max_pages, n_pages, page_rows);
  if (!rc) rc = check_pool(layers, Hkv, d, dtype, k_pages, v_pages);
  if (rc) return rc;
  if (!aligned_to(table, 4) || !aligned_to(refs, 4) || !aligned_to(moved, 4) ||
      !aligned_to(live, 4))
    return CART_ERR_POINTER;
  const PagesWs w = pages_ws(B, n_pages);
  if (!aligned_to(workspace, 16) || workspace_bytes < w.total) return CART_ERR_WORKSPACE;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  CompactArgs a{};
  a.n_pages = n_pages;
  a.refs = refs;
  a.moved = moved;
  a.live = live;
  a.head = reinterpret_cast<int*>(ws);
  a.holes = reinterpret_cast<int*>(ws + w.ids);
  a.from = reinterpret_cast<int*>(ws + w.slots);
  a.copies = reinterpret_cast<int4*>(ws + w.copies);
  a.page_rows = page_rows;
  TraceScope tr("pages_compact", st);
  compact_plan_kernel<<<kMetaCtas, kMetaThreads, 0, st>>>(a);
  rc = to_status(cudaGetLastError());
  if (rc) return rc;
  CopyArgs c{};
  c.copies = a.copies;
  c.n_copies = a.head + kHeadCopies;
  c.k = static_cast<char*>(k_pages);
  c.v = static_cast<char*>(v_pages);
  c.row_bytes = row_bytes_of(Hkv, d, dtype);
  c.page_bytes = static_cast<long long>(c.row_bytes) * page_rows;
  c.layer_bytes = c.page_bytes * n_pages;
  c.layers = layers;
  c.table = table;
  c.moved = moved;
  c.entries = static_cast<long long>(B) * max_pages;
  c.n_pages = n_pages;
  return to_status(launch_copies(c, st));
}

}  // extern "C"
