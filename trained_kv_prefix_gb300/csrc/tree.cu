// tree.cu -- attention of a tree of drafted tokens per conversation over the
// shared cartridge, the conversation's paged rows and each token's ancestors
// (cart_attn_decode_tree).
//
// Three kernels, chained by programmatic dependent launch:
//   prep    up to eight nodes of a conversation per block: the tree's ancestor
//           sets, the nodes' queries rotated into the workspace, their rotated
//           keys and values written to their page rows, the output of unused
//           ones set to 0.  One more block writes which CTAs walk which segment.
//   attend  persistent, one or two CTAs per SM: tcgen05 products over 128-key
//           tiles.
//   merge   joins the parts of rows whose keys more than one CTA walked.
//
// Work.  The query rows of conversation b and kv head g are r = t*G + hh (t
// the node, hh the head of the group): R = nodes*G rows that see the same
// cached keys.  A segment is up to 128 of them, or 256 (two query tiles that
// share the staged keys) where R is above 128, with the key tiles they walk:
//   fused    cartridge tiles, then the conversation's own rows, cached and new:
//            one segment per (conversation, kv head, 128 or 256 rows).
//   stacked  (where that saves enough cartridge tiles, see tree_ws) the rows of
//            all conversations, stacked, against the cartridge, so that its
//            tiles meet full query tiles; and one segment per (conversation,
//            kv head) against its own rows.
// New rows lie behind the cached ones in the same pages, so they share the
// last tiles; a row's ancestor set masks them.
//
// The tiles of all segments, one after the other, are cut into equal runs,
// one per CTA (a segment counts some tiles more for its start and end), so
// every SM has the same work whatever the lengths are, which the host does
// not know.  A segment that one CTA walks whole, and whose rows no other
// segment holds, is written at once; else its piece leaves a normalised
// partial output and its log-sum-exp for the merge.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "internal.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cart {
namespace {

// What a staged V row needs before the products read it; else it has a value
// that is not finite (in any kv head), and this is its bit of Piece::bad.
constexpr int kVKeep = -1, kVZero = -2;

// A node's ancestors and itself (0: unused), those of them in its window, and
// what its V row needs; with a window also what cached row first_row() + i
// needs, where the node is the i-th.
struct NodeSet {
  unsigned long long anc, vis;
  int row, cached;
};

struct TreeArgs {
  PageTable pt;
  int B, nodes, Hq, Hkv, p, window;
  float scale_log2;
  const __nv_bfloat16 *q, *k_new, *v_new, *kc, *vc;
  __nv_bfloat16 *k_pages, *v_pages, *o;
  const int* parents;
  __nv_bfloat16* qr;        // [B, nodes, Hq, d] rotated queries
  NodeSet* set;             // [B, nodes]
  uint32_t* status;
  // ---- schedule: query rows of one (conversation, kv head), most rows of a
  // segment (128 or 256), segments of a (conversation, kv head)
  int R, rt, segs;
  int stacked, n_ctas;
  // the CTAs whose pieces hold tiles of each segment (see segment_span): the
  // stacked segments, then those of every (conversation, kv head)
  int2* spans;
  int* cut;  // the own segment that each CTA's run leaves unfinished, or -1
  // ---- partial outputs: rows of the stacked pieces, from row own0 on those of
  // the own ones
  float *part, *lse;
  int own0;
  // ---- merge: blocks by cut (else by own segment), rows of a block
  int by_cut, merge_rows;
};

struct Turns {
  float2 t[kMaxHeadDim / 2];
};

// First row in the window of a conversation's shallowest node (below 0: in the
// cartridge).  The node with D ancestors sees from D rows further on, so all
// nodes see the rows from nodes - 1 further on.
__device__ __forceinline__ int first_row(const TreeArgs& a, int len) { return len - a.window + 1; }

// ------------------------------------------------------------- schedule ----
// Key tiles of conversation b's own segments (n == 0: it is idle, or its table
// has no place for a new row; which nodes are used is not known here, so one
// whose every node is unused has its tiles all the same): cartridge tiles cart_lo .. n_ct - 1 (fused only), then tiles of 128 own rows
// from row_lo on.  first_cart: the first cartridge tile any of its nodes sees.
struct ConvTiles {
  int len, first_cart, n_cart, row_lo, n;
};
__device__ __forceinline__ ConvTiles conv_tiles_of(const TreeArgs& a, int len) {
  ConvTiles c;
  c.len = len;
  const int rows = a.pt.max_pages << a.pt.page_log2, n_ct = (a.p + kTile - 1) / kTile;
  // position of the first key that the shallowest node sees
  const int lo = a.window > 0 ? a.p + first_row(a, c.len) : 0;
  c.first_cart = lo > 0 ? min(lo / kTile, n_ct) : 0;
  c.n_cart = a.stacked ? 0 : n_ct - c.first_cart;
  c.row_lo = lo > a.p ? (lo - a.p) / kTile : 0;
  c.n = c.len < 0 || c.len >= rows
            ? 0
            : c.n_cart + (min(c.len + a.nodes, rows) + kTile - 1) / kTile - c.row_lo;
  return c;
}
__device__ __forceinline__ ConvTiles conv_tiles(const TreeArgs& a, int b) {
  return conv_tiles_of(a, held_rows(a.pt, b));
}
// A segment of n tiles is n + kStartUnits units of the schedule: its start and
// end cost about as much as that many tiles.
constexpr int kStartUnits = 3;
__device__ __forceinline__ long long conv_units(const TreeArgs& a, int n) {
  return n > 0 ? static_cast<long long>(n + kStartUnits) * a.Hkv * a.segs : 0;
}

// The schedule as every thread of a block needs it: the first unit of the
// thread's conversations b0 .. b1 - 1 and the units they have, the stacked
// segments' first cartridge tile and units, which come first, and the number
// of all units.
struct Starts {
  int b0, b1, cart_lo;
  long long start, mine, cart_units, total;
};
template <int kThreads>
struct StartsSmem {
  long long sum[kThreads / 32];
  int lo;
};
template <int kThreads>
__device__ __forceinline__ Starts scan_starts(const TreeArgs& a, StartsSmem<kThreads>& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_ct = (a.p + kTile - 1) / kTile;
  const int per = (a.B + kThreads - 1) / kThreads;
  Starts r;
  r.b0 = min(static_cast<int>(threadIdx.x) * per, a.B);
  r.b1 = min(r.b0 + per, a.B);
  r.mine = 0;
  int lo = n_ct;
  for (int b = r.b0; b < r.b1; ++b) {
    const ConvTiles c = conv_tiles(a, b);
    r.mine += conv_units(a, c.n);
    if (c.n > 0) lo = min(lo, c.first_cart);
  }
  if (threadIdx.x == 0) s.lo = n_ct;
  long long x = r.mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lane == 31) s.sum[warp] = x;
  __syncthreads();
  if (lane == 0) atomicMin(&s.lo, lo);
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    before += w < warp ? s.sum[w] : 0;
    all += s.sum[w];
  }
  __syncthreads();
  r.cart_lo = s.lo;
  const int n_c = n_ct - r.cart_lo;
  const int stacks = (a.B * a.R + a.rt - 1) / a.rt;
  r.cart_units =
      a.stacked && n_c > 0 ? static_cast<long long>(n_c + kStartUnits) * stacks * a.Hkv : 0;
  r.start = r.cart_units + before + x - r.mine;
  r.total = r.cart_units + all;
  return r;
}

// Tiles [t0, t0 + n) of a segment of `tiles` tiles, from unit `first` on, that
// lie in the run [lo, hi) of one CTA (n <= 0: its start alone).
struct Cut {
  int t0, n;
};
__device__ __forceinline__ Cut cut_segment(long long first, int tiles, long long lo, long long hi) {
  const long long u0 = max(lo - first, 0ll);
  const long long u1 = min(hi - first, static_cast<long long>(tiles + kStartUnits));
  Cut c;
  c.t0 = static_cast<int>(max(u0 - kStartUnits, 0ll));
  c.n = static_cast<int>(u1 - kStartUnits) - c.t0;
  return c;
}

// x / y for x >= 0, y > 0; the 64-bit division takes several times as long as
// the 32-bit one that nearly every schedule gets by with.
__device__ __forceinline__ long long div_units(long long x, long long y) {
  return ((x | y) >> 31) == 0 ? static_cast<unsigned>(x) / static_cast<unsigned>(y) : x / y;
}

// CTAs, with runs of `chunk` units, that hold tiles of a segment:
// twice the first of them, plus 1 if its piece does not begin with its run,
// and their number.
__device__ __forceinline__ int2 segment_span(long long first, int tiles, long long chunk) {
  if (tiles <= 0) return make_int2(0, 0);
  int lo = static_cast<int>(div_units(first, chunk));
  const int hi = static_cast<int>(div_units(first + tiles + kStartUnits - 1, chunk));
  // (runs may hold the segment's start alone, without a tile)
  while (cut_segment(first, tiles, lo * chunk, (lo + 1) * chunk).n <= 0) ++lo;
  return make_int2(2 * lo + (lo * chunk < first), hi - lo + 1);
}

// One block: the spans of all segments, for the merge.
__device__ __forceinline__ void write_spans(const TreeArgs& a) {
  __shared__ StartsSmem<256> s;
  for (int i = threadIdx.x; i < a.n_ctas; i += 256) a.cut[i] = -1;
  const Starts r = scan_starts<256>(a, s);  // (with barriers: the list is cleared)
  const long long chunk = div_units(r.total + a.n_ctas - 1, a.n_ctas);
  const int stacks = a.stacked ? (a.B * a.R + a.rt - 1) / a.rt * a.Hkv : 0;
  if (a.stacked) {
    const int n_c = (a.p + kTile - 1) / kTile - r.cart_lo;
    for (int i = threadIdx.x; i < stacks; i += 256)
      a.spans[i] = segment_span(static_cast<long long>(i) * (n_c + kStartUnits), n_c, chunk);
  }
  // own segments, by threads over all of them (their conversations' starts
  // through shared memory, 256 conversations at a time)
  __shared__ long long start[256];
  __shared__ int tiles[256];
  const int per = a.Hkv * a.segs;
  const int rounds = (a.B + 255) / 256;  // conversations per thread of the scan
  long long x = r.start;
  for (int k = 0; k < rounds; ++k) {
    const int b = r.b0 + k;
    if (b < r.b1) {
      tiles[threadIdx.x] = conv_tiles(a, b).n;
      start[threadIdx.x] = x;
      x += conv_units(a, tiles[threadIdx.x]);
    } else {
      tiles[threadIdx.x] = -1;  // no conversation
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 256 * per; i += 256) {
      const int t = i / per, n = tiles[t];
      if (n < 0) continue;
      const int seg = i % per, id = (t * rounds + k) * per + seg;
      const int2 span =
          segment_span(start[t] + static_cast<long long>(seg) * (n + kStartUnits), n, chunk);
      a.spans[stacks + id] = span;
      if (span.y > 1) a.cut[span.x >> 1] = id;
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------- prep ----
// Rows of a node: its query heads, new keys, new values.  D/16 lanes share a
// row: lane l of them holds the 8 values from 8l on and those D/2 further, so
// a warp has 512/D rows of 2 x 16 bytes per lane at a time.
template <int D>
struct PrepShape {
  static constexpr int kLanes = D / 16;      // lanes per row
  static constexpr int kRows = 32 / kLanes;  // rows per warp at a time
  static constexpr int kBatch = 2;           // of them in flight
};
constexpr int kPrepNodes = 8;  // most nodes per block
// blocks per conversation of note_cached_rows
__host__ __device__ __forceinline__ int cached_blocks(int nodes) { return (nodes - 1 + 7) / 8; }

// Whether one of two packed bf16 values is not finite.
__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ bool not_finite(uint4 v) {
  return not_finite(v.x) || not_finite(v.y) || not_finite(v.z) || not_finite(v.w);
}

// Rotates eight pairs: (x, y) element by element by the angles c[0], c[step],
// c[2 * step], ...
__device__ __forceinline__ void rotate8(uint4& x, uint4& y, const float2* c, int step) {
  uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 fa = bf16x2_to_float2(a[i]), fb = bf16x2_to_float2(b[i]);
    float2 ya, yb;
    rope_pair(fa.x, fb.x, c[2 * i * step], ya.x, yb.x);
    rope_pair(fa.y, fb.y, c[(2 * i + 1) * step], ya.y, yb.y);
    a[i] = pack_bf16x2(ya.x, ya.y);
    b[i] = pack_bf16x2(yb.x, yb.y);
  }
  x = make_uint4(a[0], a[1], a[2], a[3]);
  y = make_uint4(b[0], b[1], b[2], b[3]);
}

// Eight of the nodes - 1 cached rows of a conversation that some nodes see and
// others do not, a warp per row: whether a value of it is not finite.
template <int D>
__device__ __forceinline__ void note_cached_rows(const TreeArgs& a, int block) {
  const int blocks = cached_blocks(a.nodes), b = block / blocks;
  const int i = block % blocks * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= a.nodes - 1) return;
  const int len = held_rows(a.pt, b), r = first_row(a, len) + i;
  const int page = r < len ? page_of(a.pt, b, r) : -1;
  bool bad = false;
  if (page >= 0) {
    const uint4* v = reinterpret_cast<const uint4*>(
        a.v_pages + ((static_cast<long long>(page) << a.pt.page_log2) +
                     (r & ((1 << a.pt.page_log2) - 1))) * a.Hkv * D);
#pragma unroll 4
    for (int e = lane; e < a.Hkv * D / 8; e += 32) bad |= not_finite(__ldcg(v + e));
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) a.set[b * a.nodes + i].cached = bad ? kMaxNodes + i : kVKeep;
}

// Block 0 writes the spans; with a window, the next ones look through cached
// rows; each of the others prepares the nodes t0 .. t0 + per - 1 of one
// conversation.  Bound by latency for a few nodes (lengths, pages, parents
// and the rows are loaded side by side): 7 us alone for 64 conversations with
// one node; by the rows' traffic for many: 64 nodes, G = 4, 101 MB in and out,
// 22.6 us, 4.5 TB/s.  (More rows in flight, other launch bounds or other nodes
// per block move a call by 2 % either way.)
template <int D, bool kWindow>
__global__ void __launch_bounds__(256, 4) tree_prep_kernel(const __grid_constant__ TreeArgs a,
                                                        const __grid_constant__ Turns f, int per) {
  using S = PrepShape<D>;
  constexpr int HALF = D / 2;
  pdl_release();
  if (blockIdx.x == 0) {
    write_spans(a);
    return;
  }
  __shared__ TreeSmem tree;
  __shared__ float2 cs[kPrepNodes][HALF];
  __shared__ int page_s[kPrepNodes], bad_s[kPrepNodes];
  const int blocks = (a.nodes + per - 1) / per;  // per conversation
  int block = blockIdx.x - 1;
  if (kWindow) {
    const int cached = a.B * cached_blocks(a.nodes);
    if (block < cached) {
      note_cached_rows<D>(a, block);
      return;
    }
    block -= cached;
  }
  const int b = block / blocks, t0 = block % blocks * per;
  const int mine = min(per, a.nodes - t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long bt0 = static_cast<long long>(b) * a.nodes + t0;
  const int heads = a.Hq + 2 * a.Hkv, rows = mine * heads;
  const int sub = lane / S::kLanes, e0 = lane % S::kLanes * 8;
  auto row_in = [&](int i) {
    const int h = i % heads;
    const long long bt = bt0 + i / heads;
    return (h < a.Hq           ? a.q + (bt * a.Hq + h) * D
            : h < a.Hq + a.Hkv ? a.k_new + (bt * a.Hkv + h - a.Hq) * D
                               : a.v_new + (bt * a.Hkv + h - a.Hq - a.Hkv) * D) + e0;
  };
  uint4 lo[S::kBatch], hi[S::kBatch];
  auto load = [&](int i0, uint4 (&lo)[S::kBatch], uint4 (&hi)[S::kBatch]) {
#pragma unroll
    for (int k = 0; k < S::kBatch; ++k) {
      const int i = i0 + k * 8 * S::kRows;
      if (i >= rows) break;
      const __nv_bfloat16* x = row_in(i);
      lo[k] = __ldg(reinterpret_cast<const uint4*>(x));
      hi[k] = __ldg(reinterpret_cast<const uint4*>(x + HALF));
    }
  };
  load(warp * S::kRows + sub, lo, hi);  // before the tree is known
  const int len = held_rows(a.pt, b);
  const int node = threadIdx.x;
  const int page = len >= 0 && node < a.nodes ? page_of(a.pt, b, len + node) : -1;
  const bool lost = tree_ancestors(
      tree, a.parents ? a.parents + static_cast<long long>(b) * a.nodes : nullptr, a.nodes,
      page >= 0);
  if (node >= t0 && node < t0 + mine) {
    const unsigned long long anc = tree.anc[node];
    if (lost && len >= 0) atomicOr(a.status, kDevErrNoPage);
    // nearer ancestors have higher numbers: a window keeps the top ones
    unsigned long long vis = anc;
    if (kWindow)
      for (int n = __popcll(vis); n > a.window; --n) vis &= vis - 1;
    a.set[bt0 + node - t0].anc = anc;
    a.set[bt0 + node - t0].vis = vis;
    page_s[node - t0] = page;
    bad_s[node - t0] = 0;
  }
  for (int i = threadIdx.x; i < mine * HALF; i += 256) {
    const int n = i / HALF, j = i % HALF;
    // (the i-th angles of a row's lanes side by side: no bank conflicts)
    cs[n][j % 8 * S::kLanes + j / 8] =
        rope_cs_turns(f.t[j], a.p + len + __popcll(tree.anc[t0 + n]) - 1);
  }
  __syncthreads();
  for (int i0 = warp * S::kRows + sub; i0 - sub < rows; i0 += 8 * S::kRows * S::kBatch) {
    if (i0 >= 8 * S::kRows) load(i0, lo, hi);
#pragma unroll
    for (int k = 0; k < S::kBatch; ++k) {
      const int i = i0 + k * 8 * S::kRows;
      if (i >= rows) break;
      const int n = i / heads, h = i % heads;
      const long long bt = bt0 + n;
      const bool used = tree.anc[t0 + n] != 0;
      const long long row =
          ((static_cast<long long>(page_s[n]) << a.pt.page_log2) +
           ((len + t0 + n) & ((1 << a.pt.page_log2) - 1))) * a.Hkv * D;
      if (h < a.Hq + a.Hkv) rotate8(lo[k], hi[k], &cs[n][lane % S::kLanes], S::kLanes);
      __nv_bfloat16* to;
      if (h < a.Hq) {
        if (used) {
          to = a.qr + (bt * a.Hq + h) * D;
        } else {
          to = a.o + (bt * a.Hq + h) * D;
          lo[k] = hi[k] = make_uint4(0, 0, 0, 0);
        }
      } else {
        if (!used) continue;
        const int g = h < a.Hq + a.Hkv ? h - a.Hq : h - a.Hq - a.Hkv;
        to = (h < a.Hq + a.Hkv ? a.k_pages : a.v_pages) + row + g * D;
        if (h >= a.Hq + a.Hkv && (not_finite(lo[k]) || not_finite(hi[k]))) bad_s[n] = 1;
      }
      *reinterpret_cast<uint4*>(to + e0) = lo[k];
      *reinterpret_cast<uint4*>(to + e0 + HALF) = hi[k];
    }
  }
  __syncthreads();
  if (threadIdx.x < mine) {
    const int t = t0 + threadIdx.x;
    a.set[bt0 + threadIdx.x].row = !tree.anc[t] ? kVZero : bad_s[threadIdx.x] ? t : kVKeep;
  }
}

// --------------------------------------------------------------- attend ----
constexpr int kTreeMaxCtas = 320;  // bound of the workspace: two CTAs per SM
constexpr int kAbsentRing = 8;

// NT query tiles of 128 rows per CTA, each with a warpgroup of its own; they
// share the staged keys.  NT = 2 (one CTA per SM) loads keys once for 256
// rows; NT = 1 (two CTAs per SM) is for segments of at most 128 rows, where
// one CTA's start, end and softmax overlap the other's loads and products.
template <int D, int NT>
struct TreeLayout {
  static constexpr int kThreads = NT * 128 + 64;
  static constexpr int kTileBytes = kTile * D * 2;  // one 128-row Q, K or V tile
  static constexpr int kStages = NT == 1 && D == 128 ? 1 : 2;  // K and V rings
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + NT * kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kStage = kV + kStages * kTileBytes;  // 4 KB per softmax warp
  static constexpr int kSmall = kStage + NT * 4 * 4096;     // TreeSmall
  static constexpr int kBytes = kSmall + 1024;
  static_assert(kBytes <= (NT == 1 ? 115712 : 232448), "shared memory of one CTA");
};

// One piece of a segment, as the producer publishes it in a two-slot ring
// (n == 0: no more).
struct Piece {
  int n;           // key tiles
  int own;         // 0: stacked rows against the cartridge
  int b, g;        // conversation (own), kv head
  int row0, rows;  // first query row (over all conversations), rows of the segment
  int len;         // cached rows (own)
  int n_cart;      // tiles of the segment that are cartridge tiles
  int cart_lo, row_lo, t0;
  int ring;        // K/V ring position of its first tile
  int slot;        // partial output, -1: the final output
  // values that are not finite: of new rows (by node), and of the cached rows
  // that some nodes' windows hold and others' do not (see v_row_kind)
  unsigned bad[4];
};

enum TreeBar {
  kTQFull = 0,   // TMA: the piece's query tiles
  kTQEmpty,      // its last S product has read them
  kTPieceFull0,
  kTPieceFull1,
  kTPieceEmpty0, // MMA warp and softmax warps are done with the slot
  kTPieceEmpty1,
  kTKFull0,
  kTKFull1,
  kTKEmpty0,
  kTKEmpty1,
  kTVFull0,
  kTVFull1,
  kTVEmpty0,
  kTVEmpty1,
  kTSFull0,      // S of stream x is in TMEM
  kTSFull1,
  kTPFull0,      // P of stream x is in TMEM (128 arrivals)
  kTPFull1,
  kTODone0,      // the piece's last PV of stream x
  kTODone1,
  kTDrain,
  kTNumBars
};

// The shared memory next to the tiles.
template <int kThreads>
struct TreeSmall {
  uint64_t bars[kTNumBars];
  StartsSmem<kThreads> scan;
  long long begin_off;
  int begin_b, begin_len, abort_flag;
  uint32_t tmem;
  Piece pieces[2];
  unsigned absent[kAbsentRing];
};
static_assert(sizeof(TreeSmall<320>) <= 1024, "shared memory next to the tiles");

__device__ __forceinline__ unsigned low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// The pieces of one CTA's run, in order.
struct Walk {
  long long x, lo, hi, cart_units;
  int cta, cart_lo, n_cart_all, b;
  long long off;  // units of conversation b that lie before x
  int len_next;   // lens[b + 1], loaded ahead
  ConvTiles c;
};
__device__ __forceinline__ void load_next_len(const TreeArgs& a, Walk& w) {
  if (w.b + 1 < a.B) w.len_next = __ldg(a.pt.lens + w.b + 1);
}

// The next piece that has tiles; false at the run's end.
__device__ __forceinline__ bool next_piece(const TreeArgs& a, Walk& w, Piece& o) {
  while (w.x < w.hi) {
    if (w.x < w.cart_units) {
      const int v = w.n_cart_all + kStartUnits;
      const int seg = static_cast<int>(div_units(w.x, v));
      const long long first = static_cast<long long>(seg) * v;
      const Cut k = cut_segment(first, w.n_cart_all, w.x, w.hi);
      w.x = min(first + v, w.hi);
      if (k.n <= 0) continue;
      o.own = 0;
      o.b = 0;
      o.g = seg % a.Hkv;
      o.row0 = seg / a.Hkv * a.rt;
      o.rows = min(a.B * a.R - o.row0, a.rt);
      o.len = 0;
      o.n_cart = w.n_cart_all;
      o.cart_lo = w.cart_lo;
      o.row_lo = 0;
      o.t0 = k.t0;
      o.n = k.n;
      o.slot = seg + w.cta;
      return true;
    }
    if (w.off >= conv_units(a, w.c.n)) {  // the next conversation that has work
      do {
        ++w.b;
        w.c = conv_tiles_of(a, held_rows_of(a.pt, w.len_next));
        load_next_len(a, w);
      } while (w.c.n == 0);
      w.off = 0;
    }
    const int v = w.c.n + kStartUnits;
    const int seg = static_cast<int>(div_units(w.off, v));
    const int in = static_cast<int>(w.off - static_cast<long long>(seg) * v);
    const Cut k = cut_segment(w.x - in, w.c.n, w.x, w.hi);
    const bool at_lo = w.x == w.lo;
    const long long step = min(static_cast<long long>(v - in), w.hi - w.x);
    w.x += step;
    w.off += step;
    if (k.n <= 0) continue;
    const int part = seg % a.segs;
    o.own = 1;
    o.b = w.b;
    o.g = seg / a.segs;
    o.row0 = w.b * a.R + part * a.rt;
    o.rows = min(a.R - part * a.rt, a.rt);
    o.len = w.c.len;
    o.n_cart = w.c.n_cart;
    o.cart_lo = w.c.first_cart;
    o.row_lo = w.c.row_lo;
    o.t0 = k.t0;
    o.n = k.n;
    o.slot = a.stacked ? (w.b * a.Hkv + o.g) * a.segs + part + w.cta
                       : (k.n == w.c.n ? -1 : 2 * w.cta + (at_lo ? 0 : 1));
    return true;
  }
  return false;
}

// Row r of conversation b's rows: one that is nobody's (outside the window of
// every node, behind the sequence, an unused node's) becomes 0, since 0 times
// what is not finite is not 0; one that only some nodes see (a used node's, or
// one of the nodes - 1 cached rows from first_row() on, which the windows of
// deeper nodes leave behind) and that has values that are not finite has them
// set to 0 and its bit set in `bad`, for the query rows that see it.
__device__ __forceinline__ int v_row_kind(const TreeArgs& a, int b, int r, int len) {
  const bool cached = r < len;
  if (cached && a.window == 0) return kVKeep;
  const int i = r - (cached ? first_row(a, len) : len);
  if (i < 0) return kVZero;
  if (i >= (cached ? a.nodes - 1 : a.nodes)) return cached ? kVKeep : kVZero;
  const NodeSet* s = a.set + b * a.nodes + i;
  return __ldcg(cached ? &s->cached : &s->row);
}

// Thread i of a stream takes row i.  Both streams may do so for one tile: they
// write the same values, and a row's bit is set before a value of it is
// replaced.
template <int D>
__device__ __forceinline__ void clean_v_row(uint32_t sv, int row, int kind, unsigned* bad) {
  if (kind == kVZero) {
#pragma unroll
    for (int k = 0; k < D / 8; ++k)
      sts_u4(sv + (k >> 3) * 16384 + sw128_offset(row, k & 7), make_uint4(0, 0, 0, 0));
  } else if (kind >= 0) {
#pragma unroll 1
    for (int k = 0; k < D / 8; ++k) {
      const uint32_t at = sv + (k >> 3) * 16384 + sw128_offset(row, k & 7);
      const uint4 v = lds_u4(at);
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
        if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
      }
      if ((w[0] ^ v.x) | (w[1] ^ v.y) | (w[2] ^ v.z) | (w[3] ^ v.w)) {
        atomicOr(&bad[kind >> 5], 1u << (kind & 31));
        __threadfence_block();
        sts_u4(at, make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
}

// One online softmax per query row over a run's pieces: with S = Q K^T, the
// running maximum m (of the scaled logits in log2) and sum l, each 128-key
// tile gives P = 2^(S - m), l += sum P, O += P V, and O and l are scaled where
// m grew by more than 8.  Sums, maxima and O are f32; Q, K, V and P are bf16,
// what the tensor core multiplies.
//
// Bound by the tensor pipe where queries are many: 64 conversations with 64
// nodes behind 4096 rows, 198 us alone, pipe active for 71 % of the time, 1600
// TFLOP/s with the masked products (the rest is the exchange of S and P
// between a stream's products and its softmax, and pieces' starts and ends);
// four conversations with 25 nodes, G = 8, over 49k rows 114 us, 589 MB, 5.2
// TB/s, pipe active for 68 %.  Single tokens, 64 conversations: 42 us, 170 MB,
// 4.0 TB/s; there the loads of a CTA's next tile wait for the products of the
// one before, with 64 KB of keys and values per CTA.
template <int D, int NT>
__global__ void __launch_bounds__(TreeLayout<D, NT>::kThreads, 3 - NT)
    tree_attend_kernel(const __grid_constant__ CUtensorMap mQ,
                       const __grid_constant__ CUtensorMap mKc,
                       const __grid_constant__ CUtensorMap mVc,
                       const __grid_constant__ CUtensorMap mKp,
                       const __grid_constant__ CUtensorMap mVp,
                       const __grid_constant__ TreeArgs a) {
  using L = TreeLayout<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it
    if (threadIdx.x == 0) atomicOr(a.status, kDevErrSmemLayout);
    pdl_wait();
    return;
  }
  using Small = TreeSmall<L::kThreads>;
  Small& sh = *reinterpret_cast<Small*>(smem + L::kSmall);
  uint64_t* const bars = sh.bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&mQ);
    tma_prefetch_desc(&mKc);
    tma_prefetch_desc(&mVc);
    tma_prefetch_desc(&mKp);
    tma_prefetch_desc(&mVp);
  }
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int i = 0; i < kTNumBars; ++i)
      mbar_init(&bars[i], i == kTPFull0 || i == kTPFull1             ? 128
                          : i == kTPieceEmpty0 || i == kTPieceEmpty1 ? 1 + 4 * NT
                                                                     : 1);
    fence_mbar_init();
  }
  // ---- this CTA's run (the lengths are not the prep kernel's: it may still
  // be running)
  const Starts st = scan_starts<L::kThreads>(a, sh.scan);
  const long long chunk = div_units(st.total + a.n_ctas - 1, a.n_ctas);
  Walk walk;
  walk.lo = walk.x = min(chunk * blockIdx.x, st.total);
  walk.hi = min(walk.lo + chunk, st.total);
  walk.cart_units = st.cart_units;
  walk.cart_lo = st.cart_lo;
  walk.n_cart_all = (a.p + kTile - 1) / kTile - st.cart_lo;
  walk.cta = blockIdx.x;
  if (walk.lo >= walk.hi) {
    // (the merge reads what the prep kernel wrote before it waits for this grid)
    pdl_wait();
    pdl_release();
    return;
  }
  {
    const long long at = max(walk.x, walk.cart_units);
    if (at >= st.start && at < st.start + st.mine) {
      long long x = st.start;
      int b = st.b0;
      for (;; ++b) {
        const ConvTiles c = conv_tiles(a, b);
        const long long u = conv_units(a, c.n);
        if (at < x + u) {
          sh.begin_len = c.len;
          break;
        }
        x += u;
      }
      sh.begin_b = b;
      sh.begin_off = at - x;
    }
  }
  if (warp == 4 * NT + 1) {
    tmem_alloc(&sh.tmem, NT * 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t abort_s = smem_u32(&sh.abort_flag);
  const int g_log2 = __ffs(a.Hq / a.Hkv) - 1;
  constexpr int kS = L::kStages;

  if (warp == 4 * NT) {
    // ------------------------------------------------------------ producer --
    // The whole warp walks the run; lane 0 issues the tiled copies of the
    // queries and the cartridge, lane i those of a tile's i-th page.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, kDevErrTimeoutTma));
    };
    const int page_rows = 1 << a.pt.page_log2;
    const int tile_pages = kTile >> a.pt.page_log2;
    const int table_rows = a.pt.max_pages << a.pt.page_log2;
    bool waited = false;  // for the prep kernel
    auto after_prep = [&] {
      if (!waited) pdl_wait();
      waited = true;
    };
    walk.b = sh.begin_b;
    walk.off = sh.begin_off;
    if (walk.hi > walk.cart_units) {
      walk.c = conv_tiles_of(a, sh.begin_len);
      load_next_len(a, walk);
    }
    // Table entry of the page that this lane copies of tile t of piece q (-1
    // where it copies none), looked up a tile ahead.  (Bringing the pages of
    // later tiles into L2 as well made it slower: 337 -> 367 us one tile ahead
    // and 560 us three ahead for 64 histories of 8k rows, which stream at 96 %
    // of the copy bandwidth without.)
    auto look_up = [&](const Piece& q, int t) {
      const int ta = q.t0 + t;
      const int k = ((q.row_lo + ta - q.n_cart) * kTile >> a.pt.page_log2) + lane;
      return ta >= q.n_cart && lane < tile_pages && k < a.pt.max_pages
                 ? __ldg(a.pt.table + static_cast<long long>(q.b) * a.pt.max_pages + k)
                 : -1;
    };
    Piece o{}, o_next{};
    bool more = next_piece(a, walk, o), ok = true;
    int entry = more ? look_up(o, 0) : -1;
    int ring = 0, nq = 0, k_issued = 0, v_issued = 0;
    for (int it = 0; ok; ++it) {
      const int sl = it & 1;
      if (it >= 2) {
        ok = wait(&bars[kTPieceEmpty0 + sl], ((it >> 1) - 1) & 1);
        if (!ok) break;
      }
      if (!more) {
        if (lane == 0) {
          sh.pieces[sl].n = 0;
          mbar_arrive(&bars[kTPieceFull0 + sl]);
        }
        break;
      }
      o.ring = ring;
      o.bad[0] = o.bad[1] = o.bad[2] = o.bad[3] = 0;
      if (lane == 0) {
        sh.pieces[sl] = o;
        mbar_arrive(&bars[kTPieceFull0 + sl]);
      }
      __syncwarp();
      const int row_end = min(o.len + a.nodes, table_rows);
      for (int t = 0; t < o.n && ok; ++t, ++ring) {
        const int s = ring % kS, before = ring / kS - 1;  // ring slot, its earlier phase
        const int ta = o.t0 + t;
        const bool cart = ta < o.n_cart;
        const int r0 = cart ? 0 : (o.row_lo + ta - o.n_cart) * kTile;
        // pages of the tile: -1 behind the last row, n_pages (a box outside
        // the pool, which reads as 0) for one that is not there
        int page = -1;
        if (!cart && lane < tile_pages && r0 + lane * page_rows < row_end)
          page = static_cast<unsigned>(entry) < static_cast<unsigned>(a.pt.n_pages)
                     ? entry
                     : a.pt.n_pages;
        const unsigned gone = __ballot_sync(0xffffffffu, page == a.pt.n_pages);
        const uint32_t bytes =
            cart ? L::kTileBytes
                 : __popc(__ballot_sync(0xffffffffu, page >= 0)) * page_rows * D * 2;
        if (!cart && r0 + kTile > o.len) after_prep();  // it holds new rows
        auto load = [&](int base, const CUtensorMap* mc, const CUtensorMap* mp, uint64_t* bar) {
          uint8_t* dst = smem + base + s * L::kTileBytes;
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (cart) {
            if (lane == 0)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_4d(dst + h * 16384, mc, bar, h * 64, o.g, (o.cart_lo + ta) * kTile, 0);
          } else if (page >= 0) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(dst + h * 16384 + lane * page_rows * 128, mp, bar, h * 64, o.g, 0, page);
          }
        };
        if (before >= 0) {
          ok = wait(&bars[kTKEmpty0 + s], before & 1);
          if (!ok) break;
        }
        if (lane == 0) sh.absent[ring % kAbsentRing] = gone;
        load(L::kK, &mKc, &mKp, &bars[kTKFull0 + s]);
        k_issued = ring + 1;
        if (t == 0) {
          // the piece's queries, once the last piece's S products have read theirs
          after_prep();
          if (nq >= 1) {
            ok = wait(&bars[kTQEmpty], (nq - 1) & 1);
            if (!ok) break;
          }
          if (lane == 0) {
            // boxes of 32 rows, those that hold rows of the segment
            const int boxes = (o.rows + 31) / 32;
            mbar_arrive_expect_tx(&bars[kTQFull], boxes * 32 * D * 2);
            for (int x = 0; x < boxes; ++x)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_4d(smem + L::kQ + (x >> 2) * L::kTileBytes + h * 16384 + (x & 3) * 4096,
                            &mQ, &bars[kTQFull], h * 64, 0, o.g, (o.row0 + x * 32) >> g_log2);
          }
          ++nq;
        }
        // what comes next, while V's slot is waited for
        if (t + 1 < o.n) {
          entry = look_up(o, t + 1);
        } else {
          more = next_piece(a, walk, o_next);
          if (more) entry = look_up(o_next, 0);
        }
        if (before >= 0) {
          ok = wait(&bars[kTVEmpty0 + s], before & 1);
          if (!ok) break;
        }
        load(L::kV, &mVc, &mVp, &bars[kTVFull0 + s]);
        v_issued = ring + 1;
      }
      o = o_next;
    }
    after_prep();
    pdl_release();
    if (!ok && lane == 0) {
      // copies in flight get a bounded chance to land before the CTA ends
      if (nq > 0) mbar_wait(&bars[kTQFull], (nq - 1) & 1, 0u, nullptr, 0);
      for (int t = max(k_issued - kS, 0); t < k_issued; ++t)
        mbar_wait(&bars[kTKFull0 + t % kS], (t / kS) & 1, 0u, nullptr, 0);
      for (int t = max(v_issued - kS, 0); t < v_issued; ++t)
        mbar_wait(&bars[kTVFull0 + t % kS], (t / kS) & 1, 0u, nullptr, 0);
    }
    __syncwarp();
  } else if (warp == 4 * NT + 1) {
    // ----------------------------------------------------------------- MMA --
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, kDevErrTimeoutMma));
    };
    const uint32_t idS = idesc_bf16(128, 128, false, false);
    const uint32_t idPV = idesc_bf16(128, D, false, true);
    const uint64_t dQ0 = sdesc_sw128(smem_u32(smem + L::kQ), 16u, 1024u);
    const uint64_t dQ1 = desc_add(dQ0, L::kTileBytes);
    const uint64_t dK0 = sdesc_sw128(smem_u32(smem + L::kK), 16u, 1024u);
    const uint64_t dK1 = desc_add(dK0, L::kTileBytes);
    const uint64_t dV0 = sdesc_sw128(smem_u32(smem + L::kV), 16384u, 1024u);
    const uint64_t dV1 = desc_add(dV0, L::kTileBytes);
    // S of stream x from the keys of ring slot s
    auto issue_qk = [&](int x, int s) {
      const uint64_t dq = x ? dQ1 : dQ0, dk = s ? dK1 : dK0;
      const uint32_t ts = tmem + x * 128;
      umma_bf16_ss_w(ts, dq, dk, idS, 0u);
#pragma unroll
      for (int k = 1; k < D / 16; ++k) {
        const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
        umma_bf16_ss_w(ts, desc_add(dq, off), desc_add(dk, off), idS, 1u);
      }
      umma_commit_w(&bars[kTSFull0 + x]);
    };
    auto issue_pv = [&](int x, int s, bool acc) {
      const uint64_t dv = s ? dV1 : dV0;
      const uint32_t tp = tmem + x * 128, to = tmem + (NT + x) * 128;
      umma_bf16_ts_w(to, tp, dv, idPV, acc ? 1u : 0u);
#pragma unroll
      for (int k = 1; k < kTile / 16; ++k)
        umma_bf16_ts_w(to, tp + k * 8, desc_add(dv, k * 2048), idPV, 1u);
    };
    int nP[2] = {0, 0};
    bool ok = true;
    for (int it = 0; ok; ++it) {
      ok = wait(&bars[kTPieceFull0 + (it & 1)], (it >> 1) & 1);
      if (!ok) break;
      const Piece& sp = sh.pieces[it & 1];
      const int n = vld(sp.n), ring = vld(sp.ring);
      const bool two = NT == 2 && vld(sp.rows) > kTile;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kTPieceEmpty0 + (it & 1)]);
      if (n == 0) break;
      // Per tile t: PV_0(t), S_0(t+1), PV_1(t), S_1(t+1).  Products run in
      // issue order, so the commit that publishes S_x(t+1) also says that
      // PV_x(t) has read its weights and written O_x.
      ok = wait(&bars[kTQFull], it & 1) && wait(&bars[kTKFull0 + ring % kS], (ring / kS) & 1);
      if (!ok) break;
      tc_fence_after();
      issue_qk(0, ring % kS);
      if (two) issue_qk(1, ring % kS);
      umma_commit_w(&bars[kTKEmpty0 + ring % kS]);
      if (n == 1) umma_commit_w(&bars[kTQEmpty]);
      for (int t = 0; t < n && ok; ++t) {
        const int gt = ring + t, s = gt % kS, sn = (gt + 1) % kS;
        const bool next = t + 1 < n;
        ok = wait(&bars[kTVFull0 + s], (gt / kS) & 1);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          if (x == 1 && !two) break;
          ok = ok && wait(&bars[kTPFull0 + x], nP[x] & 1);
          if (!ok) break;
          ++nP[x];
          tc_fence_after();
          issue_pv(x, s, t > 0);
          if (!next) umma_commit_w(&bars[kTODone0 + x]);
          if (x == (two ? 1 : 0)) umma_commit_w(&bars[kTVEmpty0 + s]);
          if (next) {
            if (x == 0) {
              ok = wait(&bars[kTKFull0 + sn], ((gt + 1) / kS) & 1);
              if (!ok) break;
              tc_fence_after();
            }
            issue_qk(x, sn);
          }
        }
        if (ok && next) {
          umma_commit_w(&bars[kTKEmpty0 + sn]);
          if (t + 2 == n) umma_commit_w(&bars[kTQEmpty]);
        }
      }
    }
    // every product issued above completes before the CTA ends
    umma_commit_w(&bars[kTDrain]);
    mbar_wait(&bars[kTDrain], 0, 0u, nullptr, 0);
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax --
    pdl_wait();
    const int x = NT == 1 ? 0 : warp >> 2;  // the stream
    const int row = threadIdx.x & 127;  // TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_off;
    const uint32_t tO = tmem + (NT + x) * 128 + lane_off;
    uint8_t* const stg = smem + L::kStage + warp * 4096;
    int nS = 0, nO = 0;  // S tiles and pieces of this stream
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t err) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, err));
    };
    for (int it = 0; ok; ++it) {
      ok = wait(&bars[kTPieceFull0 + (it & 1)], (it >> 1) & 1, kDevErrTimeoutSoftmax);
      if (!ok) break;
      Piece& sp = sh.pieces[it & 1];
      const int n = vld(sp.n);
      if (n == 0) break;
      if (x * kTile >= vld(sp.rows)) {  // no rows for this stream
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kTPieceEmpty0 + (it & 1)]);
        continue;
      }
      // (the piece's fields are read where they are used, so that none takes a
      // register across the tile loop)
      // this thread's query row
      const int local = x * kTile + row;
      bool live = local < vld(sp.rows);
      const int grow = vld(sp.row0) + local;
      unsigned long long vis = 0;
      int first = 0;  // position of its first key
      if (live) {
        const int bt = grow >> g_log2;
        const unsigned long long anc = __ldcg(&a.set[bt].anc);
        vis = __ldcg(&a.set[bt].vis);
        live = anc != 0;
        if (a.window > 0)
          first = a.p + (vld(sp.own) ? vld(sp.len) : held_rows(a.pt, bt / a.nodes)) +
                  __popcll(anc) - a.window;
      }
      const unsigned live_rows = __ballot_sync(0xffffffffu, live);
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < n && ok; ++t) {
        // the tile's first key (a cartridge row or an own row), the keys before
        // `end` and from `from` on, and pages that are not there
        const int ta = vld(sp.t0) + t - vld(sp.n_cart);
        const bool cart = ta < 0;
        const int k0 = cart ? (vld(sp.cart_lo) + vld(sp.t0) + t) * kTile
                            : (vld(sp.row_lo) + ta) * kTile;
        const int end = (cart ? a.p : vld(sp.len)) - k0;
        const int from = first - (cart ? k0 : a.p + k0);
        // (it holds rows that not every node sees)
        const bool clean =
            !cart &&
            (end < kTile || (a.window > 0 && k0 < first_row(a, vld(sp.len)) + a.nodes - 1));
        int kind = kVKeep;
        if (clean) kind = v_row_kind(a, vld(sp.b), k0 + row, vld(sp.len));
        ok = wait(&bars[kTSFull0 + x], nS & 1, kDevErrTimeoutSoftmax);
        if (!ok) break;
        ++nS;
        tc_fence_after();
        if (__any_sync(0xffffffffu, kind != kVKeep)) {
          const int gt = vld(sp.ring) + t;
          ok = wait(&bars[kTVFull0 + gt % kS], (gt / kS) & 1, kDevErrTimeoutSoftmax);
          if (!ok) break;
          clean_v_row<D>(smem_u32(smem + L::kV + gt % kS * L::kTileBytes), row, kind, sp.bad);
          fence_proxy_async_smem();
        }
        if (live_rows) {
          // (one load: four of 32 columns, with the maximum taken after them, need
          // more registers than there are, and the calls 4 to 9 % more time)
          uint32_t r[4][32];
          float most;
          tmem_ld128_max(tS, r[0], r[1], r[2], r[3], most);
          tmem_ld_wait();
          tmem_max_fence(most);
          tmem_reg_fence(r[0]);
          tmem_reg_fence(r[1]);
          tmem_reg_fence(r[2]);
          tmem_reg_fence(r[3]);
          const unsigned gone =
              cart ? 0u
                   : *reinterpret_cast<volatile unsigned*>(
                         &sh.absent[(vld(sp.ring) + t) % kAbsentRing]);
          if (__any_sync(0xffffffffu, end < kTile || from > 0 || gone)) {
            most = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              unsigned w = low_bits(end - 32 * i) & ~low_bits(from - 32 * i);
              if (gone) {
                if (a.pt.page_log2 == 4) {
                  if (gone >> (2 * i) & 1) w &= 0xffff0000u;
                  if (gone >> (2 * i + 1) & 1) w &= 0xffffu;
                } else if (gone >> ((32 * i) >> a.pt.page_log2) & 1) {
                  w = 0;
                }
              }
              if (!cart) {
                const int d = 32 * i - end;  // node d sits in bit 0 of this word
                if (d >= 0)
                  w |= d < 64 ? static_cast<unsigned>(vis >> d) : 0u;
                else if (d > -32)
                  w |= static_cast<unsigned>(vis << -d);
              }
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(w >> c & 1u)) r[i][c] = __float_as_uint(-INFINITY);
              float v = fmax3(__uint_as_float(r[i][0]), __uint_as_float(r[i][1]),
                              __uint_as_float(r[i][2]));
#pragma unroll
              for (int c = 3; c < 31; c += 2)
                v = fmax3(v, __uint_as_float(r[i][c]), __uint_as_float(r[i][c + 1]));
              most = fmax3(most, v, __uint_as_float(r[i][31]));
            }
          }
          const float rmax = most * a.scale_log2;
          // the running maximum is kept until a row's grows by more than 8
          // (weights stay below 2^8), so O is rarely rescaled
          float alpha = 1.f;
          bool rescale = false;
          if (rmax > m + 8.f) {
            alpha = exp2_approx(m - rmax);
            m = rmax;
            rescale = t > 0;
          }
          const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
          const float mr = m == -INFINITY ? 0.f : m;  // no key yet: weights 0
          const float2 nm2 = make_float2(-mr, -mr);
          float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 e = __ffma2_rn(u2f2(r[q][2 * c], r[q][2 * c + 1]), sc2, nm2);
              const float2 w = make_float2(exp2_approx(e.x), exp2_approx(e.y));
              rs[c & 1] = __fadd2_rn(rs[c & 1], w);
              pk[c] = pack_bf16x2(w.x, w.y);
            }
            tmem_st16(tS + 16 * q, pk);
          }
          const float2 rs01 = __fadd2_rn(rs[0], rs[1]);
          l = l * alpha + (rs01.x + rs01.y);
          if (__any_sync(0xffffffffu, rescale)) {
            // (the stream's last PV has completed: the commit that published
            // this S follows it)
#pragma unroll 1
            for (int blk = 0; blk < D / 32; ++blk) {
              uint32_t v[32];
              tmem_ld32(tO + blk * 32, v);
              tmem_ld_wait();
              tmem_reg_fence(v);
              const float2 al2 = make_float2(alpha, alpha);
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const float2 y = __fmul2_rn(u2f2(v[c], v[c + 1]), al2);
                v[c] = __float_as_uint(y.x);
                v[c + 1] = __float_as_uint(y.y);
              }
              tmem_st32(tO + blk * 32, v);
            }
          }
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&bars[kTPFull0 + x]);
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue --
      ok = wait(&bars[kTODone0 + x], nO & 1, kDevErrTimeoutEpilogue);
      if (!ok) break;
      ++nO;
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int slot = vld(sp.slot), g = vld(sp.g), own = vld(sp.own), b = vld(sp.b);
      // rows that this one sees and whose value is not finite: new ones, and
      // cached ones from the first that its own window holds
      auto noted = [&](int i) {
        return static_cast<unsigned long long>(*reinterpret_cast<volatile unsigned*>(&sp.bad[i + 1]))
                   << 32 |
               *reinterpret_cast<volatile unsigned*>(&sp.bad[i]);
      };
      const unsigned long long bad = vis & noted(0);
      unsigned long long bad_cached = 0;
      if (live && own && a.window > 0)
        bad_cached = noted(2) & ~0ull << (first - a.p - first_row(a, vld(sp.len)));
      if (live_rows) {
        const int rows_cap = own ? min(a.R, a.rt) : min(a.B * a.R, a.rt);
        const int part0 = slot < 0 ? 0 : (own ? a.own0 : 0) + slot * rows_cap + (local - lane);
        // Through the warp's slice, so that stores cover whole sectors: 32 rows of
        // 128 bytes (32 f32 or 64 bf16 columns), 16-byte granule k of row r at
        // r*128 + (k ^ (r & 7))*16.  Lane l stores granule l % 8 of rows
        // l / 8 + 4*i.  (A loop: unrolled, the epilogue does not stay in the
        // instruction cache next to the tile loop and took 3 us a piece.)
        const bool f32 = slot >= 0;
        uint8_t* const my = stg + lane * 128;
        const int r1 = lane >> 3, k1 = lane & 7;
        const uint8_t* const from0 = stg + r1 * 128 + ((k1 ^ r1) << 4);
        const uint8_t* const from1 = stg + (r1 + 4) * 128 + ((k1 ^ (r1 + 4)) << 4);
        float* const part_to = a.part + static_cast<long long>(part0 + r1) * D + k1 * 4;
        __nv_bfloat16* const o_to =
            a.o + (static_cast<long long>((grow - lane) >> g_log2) * a.Hq + (g << g_log2)) * D +
            k1 * 8;
        const unsigned mine = live_rows >> r1;
        auto put = [&](int k, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
          *reinterpret_cast<uint4*>(my + ((k ^ (lane & 7)) << 4)) = make_uint4(x, y, z, w);
        };
#pragma unroll 1
        for (int h = 0; h < D / 64; ++h) {
          uint32_t v[64];
          {
            uint32_t(&v0)[32] = *reinterpret_cast<uint32_t(*)[32]>(v);
            uint32_t(&v1)[32] = *reinterpret_cast<uint32_t(*)[32]>(v + 32);
            tmem_ld32(tO + h * 64, v0);
            tmem_ld32(tO + h * 64 + 32, v1);
            tmem_ld_wait();
            tmem_reg_fence(v0);
            tmem_reg_fence(v1);
          }
#pragma unroll
          for (int c = 0; c < 64; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * inv);
          unsigned long long left = own ? bad : 0ull, left_cached = bad_cached;
          while (left | left_cached) {
            const __nv_bfloat16* y;
            if (left) {
              y = a.v_new + (static_cast<long long>(b) * a.nodes + __ffsll(left) - 1) * a.Hkv * D;
              left &= left - 1;
            } else {
              const int r = first_row(a, vld(sp.len)) + __ffsll(left_cached) - 1;
              const int page = page_of(a.pt, b, r);
              left_cached &= left_cached - 1;
              if (page < 0) continue;  // (cannot be: its rows were loaded as 0)
              y = a.v_pages + ((static_cast<long long>(page) << a.pt.page_log2) +
                               (r & ((1 << a.pt.page_log2) - 1))) * a.Hkv * D;
            }
            y += g * D + h * 64;
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              const float f = __bfloat162float(y[c]);
              if (!isfinite(f)) v[c] = __float_as_uint(__uint_as_float(v[c]) + f);
            }
          }
          if (f32) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                put(k, v[32 * q + 4 * k], v[32 * q + 4 * k + 1], v[32 * q + 4 * k + 2],
                    v[32 * q + 4 * k + 3]);
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4 y =
                    *reinterpret_cast<const uint4*>((i & 1 ? from1 : from0) + (i >> 1) * 1024);
                if (mine >> (4 * i) & 1)
                  *reinterpret_cast<uint4*>(part_to + i * 4 * D + h * 64 + q * 32) = y;
              }
              __syncwarp();
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              put(k, pack_bf16x2(__uint_as_float(v[8 * k]), __uint_as_float(v[8 * k + 1])),
                  pack_bf16x2(__uint_as_float(v[8 * k + 2]), __uint_as_float(v[8 * k + 3])),
                  pack_bf16x2(__uint_as_float(v[8 * k + 4]), __uint_as_float(v[8 * k + 5])),
                  pack_bf16x2(__uint_as_float(v[8 * k + 6]), __uint_as_float(v[8 * k + 7])));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 y =
                  *reinterpret_cast<const uint4*>((i & 1 ? from1 : from0) + (i >> 1) * 1024);
              const int r = r1 + 4 * i;
              if (mine >> (4 * i) & 1)
                *reinterpret_cast<uint4*>(
                    o_to + ((r >> g_log2) * a.Hq + (r & ((1 << g_log2) - 1))) * D + h * 64) = y;
            }
            __syncwarp();
          }
        }
        if (slot >= 0 && live)
          a.lse[part0 + lane] = l == 0.f ? -INFINITY : m + __log2f(l);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kTPieceEmpty0 + (it & 1)]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4 * NT + 1) tmem_dealloc(tmem, NT * 256);
}

// ---------------------------------------------------------------- merge ----
// Joins the parts that the pieces of a row's segments left, in an order that
// the schedule alone decides: o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M).
// Block (own segment, merge_rows of its rows), four rows per warp; where that
// leaves warps over, `slices` warps share four rows, each taking every
// slices-th pair of parts.  Bound by the latency of L2 (spans, then the first
// parts and log-sum-exps side by side, then two more parts of four rows at a
// time) and, for many rows, by its bandwidth: alone 12 us for 64 conversations
// with one node, 10 us for 25 nodes over four long histories, 16 us for 64
// conversations with 64 nodes.  (80 registers, three blocks per SM: 16 bytes
// spill at d = 128; with four per SM more do, and calls took up to 10 us more,
// that of 64 single tokens 1 us less.)
template <int D>
__global__ void __launch_bounds__(256, 3) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int E = D / 32;  // output columns per lane
  using Vec = std::conditional_t<E == 4, float4, float2>;
  __shared__ float s_num[8][4][D], s_den[8][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The lists and sets are the prep kernel's, which had ended before any CTA of
  // the attend kernel let this one start, so they are read before the wait.
  // Every block waits, so that this grid's end implies the attend kernel's.
  const int id = a.by_cut ? __ldcg(a.cut + blockIdx.x) : blockIdx.x;
  const int base = id < 0 ? a.R : id % a.segs * a.rt + blockIdx.y * a.merge_rows;
  const int rows = min(a.merge_rows, a.R - base);
  if (rows <= 0) {
    pdl_wait();
    return;
  }
  const int b = id / (a.Hkv * a.segs), g = id / a.segs % a.Hkv, G = a.Hq / a.Hkv;
  const int groups = (rows + 3) >> 2;
  const int slices = groups > 4 ? 1 : groups > 2 ? 2 : groups > 1 ? 4 : 8;
  const int slice = warp / groups, r0 = base + warp % groups * 4;
  // lane: its row is r0 + lane / 8
  const int mine = r0 + (lane >> 3);
  const int gr = b * a.R + mine;
  const int id_c = gr / a.rt * a.Hkv + g;
  const int stacks = a.stacked ? (a.B * a.R + a.rt - 1) / a.rt * a.Hkv : 0;
  const bool row_ok = slice < slices && mine < base + rows;
  const int2 sp = __ldcg(a.spans + stacks + id);
  int2 sc = make_int2(0, 0);
  if (a.stacked && row_ok) sc = __ldcg(a.spans + id_c);
  unsigned long long anc = 0;
  if (row_ok) anc = __ldcg(&a.set[b * a.nodes + mine / G].anc);
  pdl_wait();
  if (sp.y <= (a.stacked ? 0 : 1)) return;  // idle, or written by its one CTA
  const int n = anc ? sc.y + sp.y : 0;
  // row of part i of the lane's row
  const int rows_c = min(a.B * a.R, a.rt), rows_p = min(a.R, a.rt);
  auto locate = [&](int i) {
    if (i < sc.y) return (id_c + (sc.x >> 1) + i) * rows_c + gr % a.rt;
    i -= sc.y;
    const int slot = a.stacked ? id + (sp.x >> 1) + i : i ? 2 * ((sp.x >> 1) + i) : sp.x;
    return a.own0 + slot * rows_p + mine % a.rt;
  };
  // part that is the slice's u-th
  auto part = [&](int u) { return 2 * (slice + (u >> 1) * slices) + (u & 1); };
  // parts u0 + j and u0 + j + 1 of four rows, whose places lanes 8 r + j hold
  Vec v[8];
  auto load = [&](int at, int j) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int from = __shfl_sync(0xffffffffu, at, (q & 3) * 8 + j + (q >> 2));
      const float* out = a.part + static_cast<long long>(from) * D;
      v[q] = from >= 0 ? __ldcg(reinterpret_cast<const Vec*>(out) + lane) : Vec{};
    }
  };
  const int n_max = __reduce_max_sync(0xffffffffu, n);
  int i = part(lane & 7), at = i < n ? locate(i) : -1;
  load(at, 0);  // (on their way together with the log-sum-exps)
  float lse = at >= 0 ? __ldcg(a.lse + at) : -INFINITY, top = lse;
  if (slices > 1 || n > 8)
    for (int k = lane & 7; k < n; k += 8) top = fmaxf(top, __ldcg(a.lse + locate(k)));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (top == -INFINITY) top = 0.f;
  float num[4][E], den = 0.f;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int e = 0; e < E; ++e) num[r][e] = 0.f;
  for (int u0 = 0;;) {
    const float f = exp2_approx(lse - top);  // (0 where there is no part)
    den += f;
    for (int j = 0;;) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float w = __shfl_sync(0xffffffffu, f, (q & 3) * 8 + j + (q >> 2));
        const float* y = reinterpret_cast<const float*>(&v[q]);
#pragma unroll
        for (int e = 0; e < E; ++e) num[q & 3][e] = fmaf(w, y[e], num[q & 3][e]);
      }
      j += 2;
      if (j == 8 || part(u0 + j) >= n_max) break;
      load(at, j);
    }
    u0 += 8;
    if (part(u0) >= n_max) break;
    i = part(u0 + (lane & 7));
    at = i < n ? locate(i) : -1;
    load(at, 0);
    lse = at >= 0 ? __ldcg(a.lse + at) : -INFINITY;
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  if (slices > 1) {  // join the slices of a group of rows, in their order
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) s_num[warp][r][e * 32 + lane] = num[r][e];
    if ((lane & 7) == 0) s_den[warp][lane >> 3] = den;
    __syncthreads();
    if (slice > 0) return;
    for (int k = 1; k < slices; ++k) {
      const int w = warp + k * groups;
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < E; ++e) num[r][e] += s_num[w][r][e * 32 + lane];
      den += s_den[w][lane >> 3];
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float sum = __shfl_sync(0xffffffffu, den, r * 8);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (all logits -inf: 0, as in attend)
    if (!__shfl_sync(0xffffffffu, n, r * 8)) continue;
    const int t = (r0 + r) / G;
    __nv_bfloat16* o =
        a.o + ((static_cast<long long>(b) * a.nodes + t) * a.Hq + g * G + (r0 + r) % G) * D +
        lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(num[r][0] * inv, num[r][1] * inv),
                                                pack_bf16x2(num[r][2] * inv, num[r][3] * inv));
    else
      *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(num[r][0] * inv, num[r][1] * inv);
  }
}

// ------------------------------------------------------------- workspace ----
struct TreeWs {
  size_t qr, set, spans, cut, part, lse, total;
  int R, rt, segs, stacked, own0;
};

TreeWs tree_ws(int B, int nodes, int Hq, int Hkv, int d, int p) {
  TreeWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~static_cast<size_t>(255);
    return o;
  };
  const size_t n = static_cast<size_t>(B) * nodes;
  w.R = nodes * (Hq / Hkv);
  // Up to 128 rows: one query tile per CTA and two CTAs per SM, so that one
  // covers the other's starts and ends, although the cartridge is then staged
  // twice as often (in us, one against two tiles per CTA, 64 conversations, G =
  // 4: 24 nodes behind 4096 rows 134, 136, behind 8192 rows 195, 188; 32 nodes
  // 138, 161).  Above: two tiles that share the keys (40 nodes 242, 193; 64
  // nodes 254, 224; 25 nodes, G = 8, 49k rows 152, 118).
  w.rt = w.R > kTile ? 2 * kTile : kTile;
  w.segs = (w.R + w.rt - 1) / w.rt;
  // Stacking fills the query tiles that walk the cartridge with rows of
  // several conversations, which saves cartridge tiles; but then a conversation
  // has a segment more, and all rows have to be joined: about as much as 3 +
  // R/40 tiles of it.  Stacked against fused in us, 64 conversations, G = 4:
  // p = 1024, R = 4 47, 60; R = 64 72, 68; R = 96 88, 74; R = 160 132, 107;
  // p = 4096, R = 4 49, 118; R = 64 99, 125; R = 96 132, 133; R = 160 188, 204;
  // R = 192 216, 212.  Over p = 128 to 4096, 2 to 64 conversations and R = 4 to
  // 192 the rule loses 0.6 % against the better of the two, at most 13 %.  (All
  // at G = 4 and d = 128; elsewhere it is taken as it is.)
  const long long row_tiles = (static_cast<long long>(B) * w.R + w.rt - 1) / w.rt;
  const long long cart_tiles = (p + kTile - 1) / kTile;
  w.stacked = B > 1 && w.segs == 1 && 40 * cart_tiles * (B - row_tiles) > (120ll + w.R) * B;
  w.qr = take(n * Hq * d * 2);
  w.set = take(n * sizeof(NodeSet));
  // partial outputs: a slot per segment and cut, or two per run
  const size_t ctas = w.rt > kTile ? kTreeMaxCtas / 2 : kTreeMaxCtas;
  const size_t rows_p = std::min(w.R, w.rt);
  const size_t slots_p = w.stacked ? static_cast<size_t>(B) * Hkv * w.segs + ctas : 2 * ctas;
  const size_t all = static_cast<size_t>(B) * w.R;
  const size_t rows_c = w.stacked ? std::min<size_t>(all, w.rt) : 0;
  const size_t stacks = w.stacked ? (all + w.rt - 1) / w.rt * Hkv : 0;
  const size_t slots_c = w.stacked ? stacks + ctas : 0;
  w.spans = take((stacks + static_cast<size_t>(B) * Hkv * w.segs) * 8);
  w.cut = take(kTreeMaxCtas * 4);
  w.own0 = static_cast<int>(slots_c * rows_c);
  w.part = take((w.own0 + slots_p * rows_p) * d * 4);
  w.lse = take((w.own0 + slots_p * rows_p) * 4);
  w.total = off;
  return w;
}

int check_tree(int B, int nodes, int Hq, int Hkv, int d, int p, int page_rows, int max_pages) {
  if (B < 1 || nodes < 1 || nodes > kMaxNodes || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || p < 0 ||
      max_pages < 1 || page_log2_of(page_rows) < 0)
    return CART_ERR_GEOMETRY;
  const int G = Hq / Hkv;
  if ((G != 1 && G != 2 && G != 4 && G != 8) || Hq > 1024) return CART_ERR_GEOMETRY;
  if (d != 64 && d != 128) return CART_ERR_GEOMETRY;
  if (static_cast<long long>(B) * nodes > 65535) return CART_ERR_GEOMETRY;
  // positions must be exact in f32 (the rotation reduces its angles there)
  if (static_cast<long long>(max_pages) * page_rows + p + kMaxNodes >= (1ll << 24))
    return CART_ERR_GEOMETRY;
  return CART_OK;
}

struct TreeMaps {
  CUtensorMap q, kc, vc, kp, vp;
};

template <int D, int NT>
cudaError_t launch_attend(const TreeArgs& a, const TreeMaps& m, cudaStream_t st) {
  using L = TreeLayout<D, NT>;
  const cudaError_t e = set_smem_once<tree_attend_kernel<D, NT>>(L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(tree_attend_kernel<D, NT>, dim3(a.n_ctas), dim3(L::kThreads), L::kBytes,
                          st, m.q, m.kc, m.vc, m.kp, m.vp, a);
}

template <int D>
cudaError_t launch_tree(TreeArgs a, const Turns& turns, cudaStream_t st) {
  const int sms = sm_count();
  if (sms < 1) return cudaErrorInvalidValue;
  a.n_ctas = std::min(sms, kTreeMaxCtas / 2) * (a.rt > kTile ? 1 : 2);
  // The merge goes by own segments, or by the CTAs' cuts where those are fewer.
  // Runs per segment, about the parts of a row, set a block's rows: 32 (a warp
  // for every four) where they are few, less where warps can share them.  In
  // us, with 32, 16, 8 and 4 rows: 2.4 runs per segment 77, 80, 87, 104; 4.8
  // 126, 126, 128, 134; 9.5 34, 31, 33, 36; 19 55, 50, 48, 51; 38 35, 29, 25, 24
  // (G = 4, d = 128).
  const int own = a.B * a.Hkv * a.segs;
  const int runs = a.n_ctas / (a.stacked ? (a.B * a.R + a.rt - 1) / a.rt * a.Hkv : own);
  a.by_cut = !a.stacked && own > a.n_ctas;
  a.merge_rows = runs < 4 ? 32 : runs < 12 ? 16 : runs < 24 ? 8 : 4;
  // rotated queries [B*nodes, Hkv, G, d] as (d, G, Hkv, B*nodes): a
  // (64, G, 1, 32/G) box is 32 rows of one kv head; pools as (d, Hkv,
  // page_rows, n_pages), a box one page of one kv head
  TreeMaps m;
  const int G = a.Hq / a.Hkv;
  const uint64_t d = D, e2 = 2, hkv = a.Hkv;
  const uint64_t qdims[4] = {d, static_cast<uint64_t>(G), hkv,
                             static_cast<uint64_t>(a.B) * a.nodes};
  const uint64_t qstr[3] = {d * e2, G * d * e2, hkv * G * d * e2};
  const uint32_t qbox[4] = {64, static_cast<uint32_t>(G), 1, static_cast<uint32_t>(32 / G)};
  auto rows_map = [&](CUtensorMap* map, const void* base, uint64_t blocks, uint64_t rows,
                      uint32_t box_rows) {
    const uint64_t dims[4] = {d, hkv, rows, blocks};
    const uint64_t strides[3] = {d * e2, hkv * d * e2, rows * hkv * d * e2};
    const uint32_t box[4] = {64, 1, box_rows, 1};
    return encode_bf16_map4(map, base, dims, strides, box);
  };
  const uint32_t page_rows = 1u << a.pt.page_log2;
  if (!encode_bf16_map4(&m.q, a.qr, qdims, qstr, qbox) ||
      !rows_map(&m.kp, a.k_pages, a.pt.n_pages, page_rows, page_rows) ||
      !rows_map(&m.vp, a.v_pages, a.pt.n_pages, page_rows, page_rows))
    return cudaErrorInvalidValue;
  if (a.p == 0) {  // no cartridge tile is read
    m.kc = m.kp;
    m.vc = m.vp;
  } else if (!rows_map(&m.kc, a.kc, 1, a.p, kTile) || !rows_map(&m.vc, a.vc, 1, a.p, kTile)) {
    return cudaErrorInvalidValue;
  }
  // nodes per prep block: one for a few nodes (latency), more for many, whose
  // blocks then share a conversation's lookups
  const int per = std::min(kPrepNodes, (a.B * a.nodes + 4 * sms - 1) / (4 * sms));
  const int prep_blocks = a.B * ((a.nodes + per - 1) / per);
  if (a.window > 0)
    tree_prep_kernel<D, true>
        <<<1 + prep_blocks + a.B * cached_blocks(a.nodes), 256, 0, st>>>(a, turns, per);
  else
    tree_prep_kernel<D, false><<<1 + prep_blocks, 256, 0, st>>>(a, turns, per);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = a.rt > kTile ? launch_attend<D, 2>(a, m, st) : launch_attend<D, 1>(a, m, st);
  if (e != cudaSuccess) return e;
  return launch_dependent(tree_merge_kernel<D>,
                          dim3(a.by_cut ? a.n_ctas : own,
                               (std::min(a.R, a.rt) + a.merge_rows - 1) / a.merge_rows),
                          dim3(256), 0, st, a);
}

}  // namespace
}  // namespace cart

using namespace cart;

extern "C" {

size_t cart_attn_decode_tree_workspace_size(int B, int nodes, int Hq, int Hkv, int d, int p,
                                            int page_rows, int max_pages) {
  if (check_tree(B, nodes, Hq, Hkv, d, p, page_rows, max_pages)) return 0;
  return tree_ws(B, nodes, Hq, Hkv, d, p).total;
}

int cart_attn_decode_tree(int B, int nodes, int window, int Hq, int Hkv, int d, int p, float scale,
                          double rope_theta, const void* q, const void* k_new, const void* v_new,
                          const void* kc, const void* vc, void* k_pages, void* v_pages,
                          int n_pages, int page_rows, const int* table, int max_pages,
                          const int* lens, const int* parents, void* o, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int rc = check_tree(B, nodes, Hq, Hkv, d, p, page_rows, max_pages);
  if (rc) return rc;
  if (window < 0 || n_pages < 1 || n_pages > (1 << 30) || !std::isfinite(scale) || !(scale > 0.f) ||
      !std::isfinite(rope_theta) || !(rope_theta > 0.0))
    return CART_ERR_GEOMETRY;
  const void* ptrs[] = {q, k_new, v_new, k_pages, v_pages, o};
  for (const void* ptr : ptrs)
    if (!aligned_to(ptr, 16)) return CART_ERR_POINTER;
  if (p > 0 && (!aligned_to(kc, 16) || !aligned_to(vc, 16))) return CART_ERR_POINTER;
  if (!aligned_to(table, 4) || !aligned_to(lens, 4) || (parents && !aligned_to(parents, 4)))
    return CART_ERR_POINTER;
  const TreeWs w = tree_ws(B, nodes, Hq, Hkv, d, p);
  if (!aligned_to(workspace, 16) || workspace_bytes < w.total) return CART_ERR_WORKSPACE;
  rc = check_device();
  if (rc) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  TreeArgs a{};
  a.pt = PageTable{table, lens, max_pages, n_pages, page_log2_of(page_rows)};
  a.B = B;
  a.nodes = nodes;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.p = p;
  // positions lie below 2^24: a window from there on cuts nothing, and
  // differences with it might leave 32 bits
  a.window = window < (1 << 24) ? window : 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_new = static_cast<const __nv_bfloat16*>(k_new);
  a.v_new = static_cast<const __nv_bfloat16*>(v_new);
  a.kc = static_cast<const __nv_bfloat16*>(kc);
  a.vc = static_cast<const __nv_bfloat16*>(vc);
  a.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  a.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.parents = parents;
  a.qr = reinterpret_cast<__nv_bfloat16*>(ws + w.qr);
  a.set = reinterpret_cast<NodeSet*>(ws + w.set);
  a.R = w.R;
  a.rt = w.rt;
  a.segs = w.segs;
  a.stacked = w.stacked;
  a.spans = reinterpret_cast<int2*>(ws + w.spans);
  a.cut = reinterpret_cast<int*>(ws + w.cut);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.lse = reinterpret_cast<float*>(ws + w.lse);
  a.own0 = w.own0;
  a.status = device_status_ptr();
  if (!a.status) return CART_ERR_CUDA;
  // the turns of the last (d, theta) of this host thread
  static thread_local Turns turns;
  static thread_local int turns_d = 0;
  static thread_local double turns_theta = 0.0;
  if (turns_d != d || turns_theta != rope_theta) {
    const RopeFreqs f = make_rope_freqs(d, rope_theta);
    for (int j = 0; j < kMaxHeadDim / 2; ++j) turns.t[j] = f.turns[j];
    turns_d = d;
    turns_theta = rope_theta;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope tr("decode_tree", st);
  const cudaError_t e = d == 128 ? launch_tree<128>(a, turns, st) : launch_tree<64>(a, turns, st);
  return e == cudaSuccess ? CART_OK : CART_ERR_CUDA;
}

}  // extern "C"
