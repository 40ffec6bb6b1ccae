// tree.cu -- attention of a tree of drafted tokens per conversation over the
// shared cartridge, the conversation's paged rows and each token's ancestors
// (cart_attn_decode_tree).
//
// Three kernels, chained by programmatic dependent launch:
//   prep    one block per (conversation, node): the tree's ancestor sets, the
//           node's queries rotated into the workspace, its rotated key and
//           value written to its page row, its output set to 0 if unused.
//           One more block writes the start of every conversation's work.
//   attend  persistent, one CTA per SM: tcgen05 products over 128-key tiles.
//   merge   joins the parts of rows whose keys more than one CTA walked.
//
// Work.  The query rows of conversation b and kv head g are r = t*G + hh (t
// the node, hh the head of the group): R = nodes*G rows that see the same
// cached keys.  A segment is up to 256 of them (two 128-row tiles) with the
// key tiles they walk:
//   fused    (R >= 256, or B == 1, or p == 0) cartridge tiles, then the
//            conversation's own rows, cached and new: one segment per
//            (conversation, kv head, 256 rows).
//   stacked  (else) the rows of all conversations, stacked 256 at a time,
//            against the cartridge, so that it is read once for many of
//            them; and one segment per (conversation, kv head) against its
//            own rows.
// New rows lie behind the cached ones in the same pages, so they share the
// last tiles; a row's ancestor set masks them.
//
// The tiles of all segments, one after the other, are cut into equal runs,
// one per CTA (a segment counts one tile more for its start and end), so
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

#include "internal.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cart {
namespace {

// A node's ancestors and itself (0: unused), and those of them in its window.
struct NodeSet {
  unsigned long long anc, vis;
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
  // ---- schedule
  int R, pairs, stacked, n_ctas;
  long long* start;         // [B + 1] first unit of each conversation, then the end
  int* cart_lo;             // first cartridge tile of the stacked segments
  // ---- partial outputs
  float *part_c, *part_p, *lse_c, *lse_p;
};

struct Turns {
  float2 t[kMaxHeadDim / 2];
};

// ------------------------------------------------------------- schedule ----
// Key tiles of conversation b's own segments (n == 0: it has no used node):
// cartridge tiles cart_lo .. n_ct - 1 (fused only), then tiles of 128 own rows
// from row_lo on.  first_cart: the first cartridge tile any of its nodes sees.
struct ConvTiles {
  int len, first_cart, n_cart, row_lo, n;
};
__device__ __forceinline__ ConvTiles conv_tiles(const TreeArgs& a, int b) {
  ConvTiles c;
  c.len = held_rows(a.pt, b);
  const int rows = a.pt.max_pages << a.pt.page_log2, n_ct = (a.p + kTile - 1) / kTile;
  // position of the first key that the shallowest node sees
  const int lo = a.window > 0 ? a.p + c.len - a.window + 1 : 0;
  c.first_cart = lo > 0 ? min(lo / kTile, n_ct) : 0;
  c.n_cart = a.stacked ? 0 : n_ct - c.first_cart;
  c.row_lo = lo > a.p ? (lo - a.p) / kTile : 0;
  c.n = c.len < 0 || c.len >= rows
            ? 0
            : c.n_cart + (min(c.len + a.nodes, rows) + kTile - 1) / kTile - c.row_lo;
  return c;
}
// A segment of n tiles is n + 1 units of the schedule.
__device__ __forceinline__ long long conv_units(const TreeArgs& a, int n) {
  return n > 0 ? static_cast<long long>(n + 1) * a.Hkv * a.pairs : 0;
}

// The schedule as every thread of a block needs it: the first unit of the
// thread's conversations b0 .. b1 - 1 and the units they have, the stacked
// segments' first cartridge tile and units (units 0 .. cart_units - 1), and
// the number of all units.
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
  const int stacks = (a.B * a.R + 2 * kTile - 1) / (2 * kTile);
  r.cart_units = a.stacked && n_c > 0 ? static_cast<long long>(n_c + 1) * stacks * a.Hkv : 0;
  r.start = r.cart_units + before + x - r.mine;
  r.total = r.cart_units + all;
  return r;
}

// For the merge: the first unit of every conversation, the total, and the
// stacked segments' first cartridge tile.
__device__ __forceinline__ void write_starts(const TreeArgs& a) {
  __shared__ StartsSmem<256> s;
  const Starts r = scan_starts<256>(a, s);
  long long x = r.start;
  for (int b = r.b0; b < r.b1; ++b) {
    a.start[b] = x;
    x += conv_units(a, conv_tiles(a, b).n);
  }
  if (threadIdx.x == 0) {
    a.start[a.B] = r.total;
    *a.cart_lo = r.cart_lo;
  }
}

// Tiles [t0, t0 + n) of a segment of `tiles` tiles (tiles + 1 units from unit
// `first`) that lie in the run [lo, hi) of one CTA.
struct Cut {
  int t0, n;
  bool at_lo;  // the piece begins where the run does
};
__device__ __forceinline__ Cut cut_segment(long long first, int tiles, long long lo, long long hi) {
  const long long u0 = max(lo - first, 0ll), u1 = min(hi - first, static_cast<long long>(tiles + 1));
  Cut c;
  c.t0 = static_cast<int>(max(u0, 1ll) - 1);
  c.n = static_cast<int>(u1 - 1) - c.t0;
  c.at_lo = lo >= first;
  return c;
}

// ----------------------------------------------------------------- prep ----
// Rotates one head row x (D values) into y: lane l holds pairs j and j + D/2
// for j = l * D/64 .. + D/64 - 1.
template <int D>
__device__ __forceinline__ void rotate_row(const __nv_bfloat16* x, __nv_bfloat16* y,
                                           const float2 (&cs)[D / 64], int lane) {
  if constexpr (D == 128) {
    const uint32_t a = __ldg(reinterpret_cast<const uint32_t*>(x) + lane);
    const uint32_t b = __ldg(reinterpret_cast<const uint32_t*>(x) + 32 + lane);
    const float2 fa = bf16x2_to_float2(a), fb = bf16x2_to_float2(b);
    float2 ya, yb;
    rope_pair(fa.x, fb.x, cs[0], ya.x, yb.x);
    rope_pair(fa.y, fb.y, cs[1], ya.y, yb.y);
    reinterpret_cast<uint32_t*>(y)[lane] = pack_bf16x2(ya.x, ya.y);
    reinterpret_cast<uint32_t*>(y)[32 + lane] = pack_bf16x2(yb.x, yb.y);
  } else {
    float ya, yb;
    rope_pair(__bfloat162float(x[lane]), __bfloat162float(x[32 + lane]), cs[0], ya, yb);
    y[lane] = __float2bfloat16_rn(ya);
    y[32 + lane] = __float2bfloat16_rn(yb);
  }
}

template <int D>
__global__ void __launch_bounds__(256) tree_prep_kernel(const TreeArgs a, const Turns f) {
  pdl_release();
  if (blockIdx.x == a.B * a.nodes) {
    write_starts(a);
    return;
  }
  __shared__ TreeSmem tree;
  const int t = blockIdx.x % a.nodes, b = blockIdx.x / a.nodes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = held_rows(a.pt, b);
  const int node = threadIdx.x;
  const int page = len >= 0 && node < a.nodes ? page_of(a.pt, b, len + node) : -1;
  const bool lost = tree_ancestors(
      tree, a.parents ? a.parents + static_cast<long long>(b) * a.nodes : nullptr, a.nodes,
      page >= 0);
  if (lost && len >= 0 && node == t) atomicOr(a.status, kDevErrNoPage);
  const unsigned long long anc = tree.anc[t];
  const long long bt = static_cast<long long>(b) * a.nodes + t;
  if (threadIdx.x == 0) {
    // nearer ancestors have higher numbers: a window keeps the top ones
    unsigned long long vis = anc;
    if (a.window > 0)
      for (int n = __popcll(vis); n > a.window; --n) vis &= vis - 1;
    a.set[bt] = NodeSet{anc, vis};
  }
  if (!anc) {
    uint4* o = reinterpret_cast<uint4*>(a.o + bt * a.Hq * D);
    for (int i = threadIdx.x; i < a.Hq * D / 8; i += blockDim.x) o[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int pos = a.p + len + __popcll(anc) - 1;
  float2 cs[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) cs[i] = rope_cs_turns(f.t[lane * (D / 64) + i], pos);
  const int my_page = page_of(a.pt, b, len + t);
  const long long row =
      ((static_cast<long long>(my_page) << a.pt.page_log2) +
       ((len + t) & ((1 << a.pt.page_log2) - 1))) * a.Hkv * D;
  for (int h = warp; h < a.Hq + 2 * a.Hkv; h += 8) {
    if (h < a.Hq) {
      rotate_row<D>(a.q + (bt * a.Hq + h) * D, a.qr + (bt * a.Hq + h) * D, cs, lane);
    } else if (h < a.Hq + a.Hkv) {
      const int g = h - a.Hq;
      rotate_row<D>(a.k_new + (bt * a.Hkv + g) * D, a.k_pages + row + g * D, cs, lane);
    } else {
      const int g = h - a.Hq - a.Hkv;
      const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v_new + (bt * a.Hkv + g) * D);
      uint32_t* y = reinterpret_cast<uint32_t*>(a.v_pages + row + g * D);
      for (int i = lane; i < D / 2; i += 32) y[i] = __ldg(v + i);
    }
  }
}

// --------------------------------------------------------------- attend ----
constexpr int kTreeThreads = 320;
constexpr int kTreeMaxCtas = 160;  // bound of the workspace; one CTA per SM
constexpr int kAbsentRing = 8;

template <int D>
struct TreeLayout {
  static constexpr int kTileBytes = kTile * D * 2;  // one 128-row Q, K or V tile
  static constexpr int kQ = 0;                      // Q_A, Q_B
  static constexpr int kK = kQ + 2 * kTileBytes;    // K ring, 2 stages
  static constexpr int kV = kK + 2 * kTileBytes;    // V ring, 2 stages
  static constexpr int kStage = kV + 2 * kTileBytes;  // output staging, 4 KB per softmax warp
  static constexpr int kSmall = kStage + 8 * 4096;  // TreeSmall
  static constexpr int kBytes = kSmall + 3072;
};
static_assert(TreeLayout<kMaxHeadDim>::kBytes <= 232448, "shared memory of one CTA");

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
  int split;       // the two streams share one query tile and take tiles in turn
  unsigned bad[2]; // new rows whose value is not finite
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
  kTPair0,       // warps w and w + 4 of a split piece (64 arrivals)
  kTPair1,
  kTPair2,
  kTPair3,
  kTDrain,
  kTNumBars
};

// The shared memory next to the tiles.
struct TreeSmall {
  float2 stats[2][kTile];  // split pieces: (m, l) of each stream's rows
  uint64_t bars[kTNumBars];
  StartsSmem<kTreeThreads> scan;
  long long begin_off;
  int begin_b, abort_flag;
  uint32_t tmem;
  Piece pieces[2];
  unsigned absent[kAbsentRing];
};
static_assert(sizeof(TreeSmall) <= 3072, "shared memory next to the tiles");

__device__ __forceinline__ unsigned low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// The pieces of one CTA's run, in order.
struct Walk {
  long long x, lo, hi, cart_units;
  int cta, cart_lo, n_cart_all, b;
  long long off;  // units of conversation b that lie before x
  ConvTiles c;
};

// The next piece that has tiles; false at the run's end.
__device__ __forceinline__ bool next_piece(const TreeArgs& a, Walk& w, Piece& o) {
  while (w.x < w.hi) {
    if (w.x < w.cart_units) {
      const int v = w.n_cart_all + 1;
      const int seg = static_cast<int>(w.x / v);
      const long long first = static_cast<long long>(seg) * v;
      const Cut k = cut_segment(first, w.n_cart_all, w.x, w.hi);
      w.x = min(first + v, w.hi);
      if (k.n <= 0) continue;
      o.own = 0;
      o.b = 0;
      o.g = seg % a.Hkv;
      o.row0 = seg / a.Hkv * 2 * kTile;
      o.rows = min(a.B * a.R - o.row0, 2 * kTile);
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
        w.c = conv_tiles(a, ++w.b);
      } while (w.c.n == 0);
      w.off = 0;
    }
    const int v = w.c.n + 1;
    const int seg = static_cast<int>(w.off / v), in = static_cast<int>(w.off % v);
    const Cut k = cut_segment(w.x - in, w.c.n, w.x, w.hi);
    const bool at_lo = w.x == w.lo;
    const long long step = min(static_cast<long long>(v - in), w.hi - w.x);
    w.x += step;
    w.off += step;
    if (k.n <= 0) continue;
    const int pair = seg % a.pairs;
    o.own = 1;
    o.b = w.b;
    o.g = seg / a.pairs;
    o.row0 = w.b * a.R + pair * 2 * kTile;
    o.rows = min(a.R - pair * 2 * kTile, 2 * kTile);
    o.len = w.c.len;
    o.n_cart = w.c.n_cart;
    o.cart_lo = w.c.first_cart;
    o.row_lo = w.c.row_lo;
    o.t0 = k.t0;
    o.n = k.n;
    o.slot = a.stacked ? (w.b * a.Hkv + o.g) * a.pairs + pair + w.cta
                       : (k.n == w.c.n ? -1 : 2 * w.cta + (at_lo ? 0 : 1));
    return true;
  }
  return false;
}

// Values of staged V rows that must not reach the products: rows that are
// nobody's (outside the window of every node, behind the sequence, unused
// nodes) become 0, and in rows of used nodes what is not finite becomes 0
// and is noted in bad (a bit per node), to be added to the rows that see it.
// Thread i of a stream takes row i.  Both streams may do so for one tile:
// they write the same values, and a bit is set before its value is replaced.
template <int D>
__device__ __forceinline__ void clean_v_row(const TreeArgs& a, uint32_t sv, int row, int r0,
                                            int lo_row, int len, int b, unsigned* bad) {
  const int r = r0 + row;
  if (r >= lo_row && r < len) return;
  const int node = r - len;
  const bool used = node >= 0 && node < a.nodes &&
                    __ldcg(&a.set[static_cast<long long>(b) * a.nodes + node].anc) != 0;
  bool noted = false;
#pragma unroll 1
  for (int k = 0; k < D / 8; ++k) {
    const uint32_t at = sv + (k >> 3) * 16384 + sw128_offset(row, k & 7);
    if (!used) {
      sts_u4(at, make_uint4(0, 0, 0, 0));
      continue;
    }
    const uint4 v = lds_u4(at);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7f80u) == 0x7f80u) {
        w[i] &= 0xffff0000u;
        any = true;
      }
      if ((w[i] & 0x7f800000u) == 0x7f800000u) {
        w[i] &= 0xffffu;
        any = true;
      }
    }
    if (any) {
      if (!noted) {
        atomicOr(&bad[node >> 5], 1u << (node & 31));
        __threadfence_block();
        noted = true;
      }
      sts_u4(at, make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_attend_kernel(const __grid_constant__ CUtensorMap mQ,
                       const __grid_constant__ CUtensorMap mKc,
                       const __grid_constant__ CUtensorMap mVc,
                       const __grid_constant__ CUtensorMap mKp,
                       const __grid_constant__ CUtensorMap mVp,
                       const __grid_constant__ TreeArgs a) {
  using L = TreeLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it
    if (threadIdx.x == 0) atomicOr(a.status, kDevErrSmemLayout);
    pdl_wait();
    return;
  }
  TreeSmall& sh = *reinterpret_cast<TreeSmall*>(smem + L::kSmall);
  uint64_t* const bars = sh.bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int i = 0; i < kTNumBars; ++i)
      mbar_init(&bars[i], i == kTPFull0 || i == kTPFull1           ? 128
                          : i == kTPieceEmpty0 || i == kTPieceEmpty1 ? 9
                          : i >= kTPair0 && i <= kTPair3             ? 64
                                                                     : 1);
    fence_mbar_init();
  }
  // ---- this CTA's run (the lengths are not the prep kernel's: it may still
  // be running)
  const Starts st = scan_starts<kTreeThreads>(a, sh.scan);
  const long long chunk = (st.total + gridDim.x - 1) / gridDim.x;
  Walk walk;
  walk.lo = walk.x = min(chunk * blockIdx.x, st.total);
  walk.hi = min(walk.lo + chunk, st.total);
  walk.cart_units = st.cart_units;
  walk.cart_lo = st.cart_lo;
  walk.n_cart_all = (a.p + kTile - 1) / kTile - st.cart_lo;
  walk.cta = blockIdx.x;
  if (walk.lo >= walk.hi) {
    pdl_release();
    pdl_wait();  // this grid's end implies the prep kernel's
    return;
  }
  {
    const long long at = max(walk.x, st.cart_units);
    if (at >= st.start && at < st.start + st.mine) {
      long long x = st.start;
      int b = st.b0;
      for (;; ++b) {
        const long long u = conv_units(a, conv_tiles(a, b).n);
        if (at < x + u) break;
        x += u;
      }
      sh.begin_b = b;
      sh.begin_off = at - x;
    }
  }
  if (warp == 9) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t abort_s = smem_u32(&sh.abort_flag);
  const int g_log2 = __ffs(a.Hq / a.Hkv) - 1;

  if (warp == 8) {
    // ------------------------------------------------------------ producer --
    // The whole warp walks the run; lane 0 issues the tiled copies of the
    // queries and the cartridge, lane i those of a tile's i-th page.
    if (lane == 0) {
      tma_prefetch_desc(&mQ);
      tma_prefetch_desc(&mKc);
      tma_prefetch_desc(&mVc);
      tma_prefetch_desc(&mKp);
      tma_prefetch_desc(&mVp);
    }
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
    if (walk.hi > walk.cart_units) walk.c = conv_tiles(a, walk.b);
    Piece o;
    bool more = next_piece(a, walk, o), ok = true;
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
      o.split = o.rows <= kTile;
      o.bad[0] = o.bad[1] = 0;
      if (lane == 0) {
        sh.pieces[sl] = o;
        mbar_arrive(&bars[kTPieceFull0 + sl]);
      }
      __syncwarp();
      const int row_end = min(o.len + a.nodes, table_rows);
      for (int t = 0; t < o.n && ok; ++t, ++ring) {
        const int s = ring & 1;
        const int ta = o.t0 + t;
        const bool cart = ta < o.n_cart;
        const int r0 = cart ? 0 : (o.row_lo + ta - o.n_cart) * kTile;
        // pages of the tile: -1 behind the last row, n_pages (a box outside
        // the pool, which reads as 0) for one that is not there
        int page = -1;
        if (!cart && lane < tile_pages && r0 + lane * page_rows < row_end) {
          page = page_of(a.pt, o.b, r0 + lane * page_rows);
          if (page < 0) page = a.pt.n_pages;
        }
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
        if (ring >= 2) {
          ok = wait(&bars[kTKEmpty0 + s], ((ring >> 1) - 1) & 1);
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
            const int tiles = o.split ? 1 : 2;
            mbar_arrive_expect_tx(&bars[kTQFull], tiles * L::kTileBytes);
            for (int x = 0; x < tiles; ++x)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_4d(smem + L::kQ + x * L::kTileBytes + h * 16384, &mQ, &bars[kTQFull],
                            h * 64, 0, o.g, (o.row0 + x * kTile) >> g_log2);
          }
          ++nq;
        }
        if (ring >= 2) {
          ok = wait(&bars[kTVEmpty0 + s], ((ring >> 1) - 1) & 1);
          if (!ok) break;
        }
        load(L::kV, &mVc, &mVp, &bars[kTVFull0 + s]);
        v_issued = ring + 1;
      }
      if (ok) more = next_piece(a, walk, o);
    }
    after_prep();
    pdl_release();
    if (!ok && lane == 0) {
      // copies in flight get a bounded chance to land before the CTA ends
      if (nq > 0) mbar_wait(&bars[kTQFull], (nq - 1) & 1, 0u, nullptr, 0);
      for (int t = max(k_issued - 2, 0); t < k_issued; ++t)
        mbar_wait(&bars[kTKFull0 + (t & 1)], (t >> 1) & 1, 0u, nullptr, 0);
      for (int t = max(v_issued - 2, 0); t < v_issued; ++t)
        mbar_wait(&bars[kTVFull0 + (t & 1)], (t >> 1) & 1, 0u, nullptr, 0);
    }
    __syncwarp();
  } else if (warp == 9) {
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
    // S of stream x = Q tile y times the keys of ring slot s
    auto issue_qk = [&](int x, int y, int s) {
      const uint64_t dq = y ? dQ1 : dQ0, dk = s ? dK1 : dK0;
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
      const uint32_t tp = tmem + x * 128, to = tmem + 256 + x * 128;
      umma_bf16_ts_w(to, tp, dv, idPV, acc ? 1u : 0u);
#pragma unroll
      for (int k = 1; k < kTile / 16; ++k)
        umma_bf16_ts_w(to, tp + k * 8, desc_add(dv, k * 2048), idPV, 1u);
    };
    int nP0 = 0, nP1 = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      ok = wait(&bars[kTPieceFull0 + (it & 1)], (it >> 1) & 1);
      if (!ok) break;
      const Piece& sp = sh.pieces[it & 1];
      const int n = vld(sp.n), split = vld(sp.split), ring = vld(sp.ring);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kTPieceEmpty0 + (it & 1)]);
      if (n == 0) break;
      // S of the tiles that the streams begin with
      ok = wait(&bars[kTQFull], it & 1) && wait(&bars[kTKFull0 + (ring & 1)], (ring >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      issue_qk(0, 0, ring & 1);
      if (!split) issue_qk(1, 1, ring & 1);
      umma_commit_w(&bars[kTKEmpty0 + (ring & 1)]);
      if (split && n > 1) {
        ok = wait(&bars[kTKFull0 + ((ring + 1) & 1)], ((ring + 1) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        issue_qk(1, 0, (ring + 1) & 1);
        umma_commit_w(&bars[kTKEmpty0 + ((ring + 1) & 1)]);
      }
      const int ahead = split ? 2 : 1;  // a stream's next tile
      if (n <= ahead) umma_commit_w(&bars[kTQEmpty]);
      for (int t = 0; t < n && ok; ++t) {
        const int gt = ring + t, s = gt & 1, gn = gt + ahead;
        const bool next = t + ahead < n;
        ok = wait(&bars[kTVFull0 + s], (gt >> 1) & 1);
        if (!ok) break;
        if (!split) {
          ok = wait(&bars[kTPFull0], nP0 & 1);
          if (!ok) break;
          ++nP0;
          tc_fence_after();
          issue_pv(0, s, t > 0);
          if (!next) umma_commit_w(&bars[kTODone0]);
          if (next) {
            ok = wait(&bars[kTKFull0 + (gn & 1)], (gn >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            issue_qk(0, 0, gn & 1);
          }
          ok = wait(&bars[kTPFull1], nP1 & 1);
          if (!ok) break;
          ++nP1;
          tc_fence_after();
          issue_pv(1, s, t > 0);
          if (!next) umma_commit_w(&bars[kTODone1]);
          if (next) issue_qk(1, 1, gn & 1);
        } else {
          const int x = t & 1;
          ok = wait(&bars[kTPFull0 + x], (x ? nP1 : nP0) & 1);
          if (!ok) break;
          if (x)
            ++nP1;
          else
            ++nP0;
          tc_fence_after();
          issue_pv(x, s, t >= 2);
          if (!next) umma_commit_w(&bars[kTODone0 + x]);
          if (next) {
            umma_commit_w(&bars[kTVEmpty0 + s]);  // before the keys' wait: V of tile t + 2 may come
            ok = wait(&bars[kTKFull0 + (gn & 1)], (gn >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            issue_qk(x, 0, gn & 1);
          }
        }
        if (!(split && next)) umma_commit_w(&bars[kTVEmpty0 + s]);
        if (next) {
          umma_commit_w(&bars[kTKEmpty0 + (gn & 1)]);
          if (t + ahead == n - 1) umma_commit_w(&bars[kTQEmpty]);
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
    const int x = warp >> 2;
    const int row = threadIdx.x & 127;  // TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_off;
    const uint32_t tO0 = tmem + 256 + lane_off;  // O of stream 0; stream 1's 128 columns on
    const uint32_t tO = tO0 + x * 128;
    uint8_t* const stg = smem + L::kStage + warp * 4096;
    int nS = 0, nO0 = 0, nO1 = 0, n_pair = 0;
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
      const int split = vld(sp.split), own = vld(sp.own), len = vld(sp.len), b = vld(sp.b);
      const int ring = vld(sp.ring), n_cart = vld(sp.n_cart), t0 = vld(sp.t0);
      const int cart_lo = vld(sp.cart_lo), row_lo = vld(sp.row_lo);
      const int step = split ? 2 : 1;
      // this thread's query row
      const int local = split ? row : x * kTile + row;
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
          first = a.p + (own ? len : held_rows(a.pt, bt / a.nodes)) + __popcll(anc) - a.window;
      }
      const unsigned live_rows = __ballot_sync(0xffffffffu, live);
      const int lo_row = a.window > 0 ? len - a.window + 1 : 0;  // of the shallowest node
      float m = -INFINITY, l = 0.f;
      for (int t = split ? x : 0; t < n && ok; t += step) {
        ok = wait(&bars[kTSFull0 + x], nS & 1, kDevErrTimeoutSoftmax);
        if (!ok) break;
        ++nS;
        tc_fence_after();
        const int ta = t0 + t, gt = ring + t;
        const bool cart = ta < n_cart;
        const int k0 = cart ? (cart_lo + ta) * kTile : (row_lo + ta - n_cart) * kTile;
        if (!cart && (k0 + kTile > len || k0 < lo_row)) {
          ok = wait(&bars[kTVFull0 + (gt & 1)], (gt >> 1) & 1, kDevErrTimeoutSoftmax);
          if (!ok) break;
          clean_v_row<D>(a, smem_u32(smem + L::kV + (gt & 1) * L::kTileBytes), row, k0, lo_row,
                         len, b, sp.bad);
          fence_proxy_async_smem();
        }
        if (live_rows) {
          uint32_t r[4][32];
          tmem_ld32(tS, r[0]);
          tmem_ld32(tS + 32, r[1]);
          tmem_ld32(tS + 64, r[2]);
          tmem_ld32(tS + 96, r[3]);
          tmem_ld_wait();
          tmem_reg_fence(r[0]);
          tmem_reg_fence(r[1]);
          tmem_reg_fence(r[2]);
          tmem_reg_fence(r[3]);
          // keys of the tile before `end` and from `from` on, on pages that
          // are there, and new rows by the node's set
          const int end = (cart ? a.p : len) - k0;
          const int from = first - (cart ? k0 : a.p + k0);
          const unsigned gone =
              cart ? 0u : *reinterpret_cast<volatile unsigned*>(&sh.absent[gt % kAbsentRing]);
          if (__any_sync(0xffffffffu, end < kTile || from > 0 || gone)) {
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
            }
          }
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v = fmax3(__uint_as_float(r[q][0]), __uint_as_float(r[q][1]),
                            __uint_as_float(r[q][2]));
#pragma unroll
            for (int c = 3; c < 31; c += 2)
              v = fmax3(v, __uint_as_float(r[q][c]), __uint_as_float(r[q][c + 1]));
            mx[q] = fmaxf(v, __uint_as_float(r[q][31]));
          }
          const float rmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
          // the running maximum is kept until a row's grows by more than 8
          // (weights stay below 2^8), so O is rarely rescaled
          float alpha = 1.f;
          bool rescale = false;
          if (rmax > m + 8.f) {
            alpha = exp2_approx(m - rmax);
            m = rmax;
            rescale = t >= step;
          }
          const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
          const float mr = m == -INFINITY ? 0.f : m;  // no key yet: weights 0
          const float2 nm2 = make_float2(-mr, -mr);
          float2 rs[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                          make_float2(0.f, 0.f)};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 e = __ffma2_rn(u2f2(r[q][2 * c], r[q][2 * c + 1]), sc2, nm2);
              const float2 w = make_float2(exp2_approx(e.x), exp2_approx(e.y));
              rs[c & 3] = __fadd2_rn(rs[c & 3], w);
              pk[c] = pack_bf16x2(w.x, w.y);
            }
            tmem_st16(tS + 16 * q, pk);
          }
          const float2 rs01 = __fadd2_rn(rs[0], rs[1]), rs23 = __fadd2_rn(rs[2], rs[3]);
          l = l * alpha + ((rs01.x + rs01.y) + (rs23.x + rs23.y));
          if (__any_sync(0xffffffffu, rescale)) {
            // (the stream's last PV has completed: the commit that published
            // this S follows it)
#pragma unroll
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
      // The output is c0 * O_0 + c1 * O_1 of the streams (one of them alone
      // unless the piece is split, where warps w and w + 4 hold the same rows
      // and each writes half of the columns).
      const bool two = split && n > 1;
      float c0, c1 = 0.f, lse;
      if (split) {
        sh.stats[x][row] = make_float2(m, l);
        mbar_arrive(&bars[kTPair0 + (warp & 3)]);
        ok = wait(&bars[kTPair0 + (warp & 3)], n_pair & 1, kDevErrTimeoutEpilogue);
        if (!ok) break;
        ++n_pair;
        const float2 s0 = sh.stats[0][row], s1 = sh.stats[1][row];
        const float top = fmaxf(s0.x, s1.x), base = top == -INFINITY ? 0.f : top;
        const float f0 = exp2_approx(s0.x - base), f1 = exp2_approx(s1.x - base);
        const float sum = s0.y * f0 + s1.y * f1;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        c0 = f0 * inv;
        c1 = f1 * inv;
        lse = sum == 0.f ? -INFINITY : top + __log2f(sum);
      } else {
        c0 = l == 0.f ? 0.f : 1.f / l;
        lse = l == 0.f ? -INFINITY : m + __log2f(l);
      }
      if (split || x == 0) {
        ok = wait(&bars[kTODone0], nO0 & 1, kDevErrTimeoutEpilogue);
        if (!ok) break;
      }
      if (two || (!split && x == 1)) {
        ok = wait(&bars[kTODone1], nO1 & 1, kDevErrTimeoutEpilogue);
        if (!ok) break;
      }
      ++nO0;
      if (two || !split) ++nO1;
      tc_fence_after();
      const int slot = vld(sp.slot), g = vld(sp.g);
      // new rows that this one sees and whose value is not finite
      const unsigned long long bad =
          vis & (static_cast<unsigned long long>(*reinterpret_cast<volatile unsigned*>(&sp.bad[1]))
                     << 32 |
                 *reinterpret_cast<volatile unsigned*>(&sp.bad[0]));
      if (live_rows) {
        const int blk_lo = split ? x * (D / 64) : 0, blk_hi = split ? blk_lo + D / 64 : D / 32;
        const int rows_cap = own ? min(a.R, 2 * kTile) : min(a.B * a.R, 2 * kTile);
        const long long part0 =
            slot < 0 ? 0 : static_cast<long long>(slot) * rows_cap + (local - lane);
        float* const part = own ? a.part_p : a.part_c;
#pragma unroll 1
        for (int blk = blk_lo; blk < blk_hi; ++blk) {
          uint32_t v[32];
          tmem_ld32((split ? tO0 : tO) + blk * 32, v);
          tmem_ld_wait();
          tmem_reg_fence(v);
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * c0);
          if (two) {
            uint32_t y[32];
            tmem_ld32(tO0 + 128 + blk * 32, y);
            tmem_ld_wait();
            tmem_reg_fence(y);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              v[c] = __float_as_uint(fmaf(__uint_as_float(y[c]), c1, __uint_as_float(v[c])));
          }
          for (unsigned long long left = own ? bad : 0ull; left; left &= left - 1) {
            const __nv_bfloat16* y =
                a.v_new + ((static_cast<long long>(b) * a.nodes + __ffsll(left) - 1) * a.Hkv + g) * D +
                blk * 32;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float f = __bfloat162float(y[c]);
              if (!isfinite(f)) v[c] = __float_as_uint(__uint_as_float(v[c]) + f);
            }
          }
          // through the warp's slice, so that stores cover whole sectors: 16-byte
          // granule k of staged row r sits at r*128 + (k ^ (r & 7))*16
          uint8_t* my = stg + lane * 128;
          if (slot >= 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(my + ((k ^ (lane & 7)) << 4)) =
                  make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(my + ((k ^ (lane & 7)) << 4)) = make_uint4(
                  pack_bf16x2(__uint_as_float(v[8 * k]), __uint_as_float(v[8 * k + 1])),
                  pack_bf16x2(__uint_as_float(v[8 * k + 2]), __uint_as_float(v[8 * k + 3])),
                  pack_bf16x2(__uint_as_float(v[8 * k + 4]), __uint_as_float(v[8 * k + 5])),
                  pack_bf16x2(__uint_as_float(v[8 * k + 6]), __uint_as_float(v[8 * k + 7])));
          }
          __syncwarp();
          const int gpr = slot >= 0 ? 8 : 4;
          for (int i = lane; i < 32 * gpr; i += 32) {
            const int r = i / gpr, k = i % gpr;
            if (!(live_rows >> r & 1)) continue;
            const uint4 y = *reinterpret_cast<const uint4*>(stg + r * 128 + ((k ^ (r & 7)) << 4));
            if (slot >= 0) {
              *reinterpret_cast<uint4*>(part + (part0 + r) * D + blk * 32 + k * 4) = y;
            } else {
              const int gr = grow - lane + r;
              const long long off = (static_cast<long long>(gr >> g_log2) * a.Hq + (g << g_log2) +
                                     (gr & ((1 << g_log2) - 1))) * D;
              *reinterpret_cast<uint4*>(a.o + off + blk * 32 + k * 8) = y;
            }
          }
          __syncwarp();
        }
        if (slot >= 0 && live && (!split || x == 0))
          (own ? a.lse_p : a.lse_c)[part0 + lane] = lse;
      }
      if (split) {
        // both warps have read O of both streams (the next piece's products
        // wait for their weights) and the other's statistics
        tc_fence_before();
        mbar_arrive(&bars[kTPair0 + (warp & 3)]);
        ok = wait(&bars[kTPair0 + (warp & 3)], n_pair & 1, kDevErrTimeoutEpilogue);
        ++n_pair;
        tc_fence_after();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kTPieceEmpty0 + (it & 1)]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- merge ----
// One warp per output row: the parts that the pieces of its segments left,
// in the order of the CTAs (o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M)).
// Rows that one piece wrote whole have none.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int E = D / 32;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int rows = a.B * a.nodes * a.Hq, G = a.Hq / a.Hkv;
  const long long total = a.start[a.B];
  const long long chunk = (total + a.n_ctas - 1) / a.n_ctas;
  const int cart_lo = *a.cart_lo, n_c = (a.p + kTile - 1) / kTile - cart_lo;
  for (int w = (blockIdx.x * 256 + threadIdx.x) >> 5; w < rows; w += gridDim.x * 8) {
    // rows of one (conversation, kv head) follow one another
    const int b = w / (a.nodes * a.Hq), g = w / a.R % a.Hkv, r = w % a.R;
    const int bt = b * a.nodes + r / G;
    if (!__ldcg(&a.set[bt].anc)) continue;
    const ConvTiles c = conv_tiles(a, b);
    const int pair = r / (2 * kTile);
    // its segments: [0] stacked rows against the cartridge, [1] own rows
    long long first[2];
    int tiles[2], id[2];
    const int gr = b * a.R + r;
    id[0] = gr / (2 * kTile) * a.Hkv + g;
    tiles[0] = a.stacked ? n_c : 0;
    first[0] = static_cast<long long>(id[0]) * (n_c + 1);
    id[1] = (b * a.Hkv + g) * a.pairs + pair;
    tiles[1] = c.n;
    first[1] = a.start[b] + static_cast<long long>(g * a.pairs + pair) * (c.n + 1);
    int c_lo[2], n_part[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      c_lo[s] = static_cast<int>(first[s] / chunk);
      const int c_hi = static_cast<int>((first[s] + tiles[s]) / chunk);
      // (a run may hold the segment's start alone, without a tile)
      if (tiles[s] > 0 &&
          cut_segment(first[s], tiles[s], c_lo[s] * chunk, (c_lo[s] + 1) * chunk).n <= 0)
        ++c_lo[s];
      n_part[s] = tiles[s] > 0 ? c_hi - c_lo[s] + 1 : 0;
    }
    if (!a.stacked && n_part[1] == 1) continue;  // written by the piece
    const int n = n_part[0] + n_part[1];
    const float *out = nullptr, *lse_at = nullptr;
    auto locate = [&](int i) {
      if (i < n_part[0]) {
        const long long at = static_cast<long long>(id[0] + c_lo[0] + i) *
                                 min(a.B * a.R, 2 * kTile) + gr % (2 * kTile);
        out = a.part_c + at * D;
        lse_at = a.lse_c + at;
      } else {
        const int cta = c_lo[1] + i - n_part[0];
        const long long slot =
            a.stacked ? id[1] + cta : 2 * cta + (cta * chunk >= first[1] ? 0 : 1);
        const long long at = slot * min(a.R, 2 * kTile) + r % (2 * kTile);
        out = a.part_p + at * D;
        lse_at = a.lse_p + at;
      }
    };
    float top = -INFINITY;
    for (int i = lane; i < n; i += 32) {
      locate(i);
      top = fmaxf(top, __ldcg(lse_at));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == -INFINITY) top = 0.f;
    float num[E], den = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) num[e] = 0.f;
    for (int i = 0; i < n; ++i) {
      locate(i);
      const float f = exp2_approx(__ldcg(lse_at) - top);
      den += f;
      if constexpr (E == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(out) + lane);
        num[0] = fmaf(f, v.x, num[0]);
        num[1] = fmaf(f, v.y, num[1]);
        num[2] = fmaf(f, v.z, num[2]);
        num[3] = fmaf(f, v.w, num[3]);
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(out) + lane);
        num[0] = fmaf(f, v.x, num[0]);
        num[1] = fmaf(f, v.y, num[1]);
      }
    }
    const float inv = 1.f / den;
    __nv_bfloat16* o = a.o + (static_cast<long long>(bt) * a.Hq + g * G + r % G) * D + lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(num[0] * inv, num[1] * inv),
                                                pack_bf16x2(num[2] * inv, num[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(num[0] * inv, num[1] * inv);
  }
}

// ------------------------------------------------------------- workspace ----
struct TreeWs {
  size_t qr, set, start, cart_lo, part_c, part_p, lse_c, lse_p, total;
  int R, pairs, stacked;
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
  w.pairs = (w.R + 2 * kTile - 1) / (2 * kTile);
  // Stacking reads the cartridge once for 256 rows of several conversations;
  // with 256 rows of one conversation nothing is left to stack, and joining
  // the two kinds of segments would only cost.
  w.stacked = p > 0 && B > 1 && w.R < 2 * kTile;
  w.qr = take(n * Hq * d * 2);
  w.set = take(n * sizeof(NodeSet));
  w.start = take((static_cast<size_t>(B) + 1) * 8);
  w.cart_lo = take(4);
  // partial outputs: a slot per segment and cut, or two per run
  const size_t rows_p = std::min(w.R, 2 * kTile);
  const size_t slots_p =
      w.stacked ? static_cast<size_t>(B) * Hkv * w.pairs + kTreeMaxCtas : 2 * kTreeMaxCtas;
  const size_t rows_c = w.stacked ? std::min<size_t>(static_cast<size_t>(B) * w.R, 2 * kTile) : 0;
  const size_t slots_c =
      w.stacked
          ? (static_cast<size_t>(B) * w.R + 2 * kTile - 1) / (2 * kTile) * Hkv + kTreeMaxCtas
          : 0;
  w.part_c = take(slots_c * rows_c * d * 4);
  w.part_p = take(slots_p * rows_p * d * 4);
  w.lse_c = take(slots_c * rows_c * 4);
  w.lse_p = take(slots_p * rows_p * 4);
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

template <int D>
cudaError_t launch_tree(TreeArgs a, const RopeFreqs& f, cudaStream_t st) {
  const int sms = sm_count();
  if (sms < 1) return cudaErrorInvalidValue;
  a.n_ctas = std::min(sms, kTreeMaxCtas);
  // rotated queries [B*nodes, Hkv, G, d] as (d, G, Hkv, B*nodes): a
  // (64, G, 1, 128/G) box is 128 rows of one kv head; pools as (d, Hkv,
  // page_rows, n_pages), a box one page of one kv head
  CUtensorMap mQ, mKc, mVc, mKp, mVp;
  const int G = a.Hq / a.Hkv;
  const uint64_t d = D, e2 = 2, hkv = a.Hkv;
  const uint64_t qdims[4] = {d, static_cast<uint64_t>(G), hkv,
                             static_cast<uint64_t>(a.B) * a.nodes};
  const uint64_t qstr[3] = {d * e2, G * d * e2, hkv * G * d * e2};
  const uint32_t qbox[4] = {64, static_cast<uint32_t>(G), 1, static_cast<uint32_t>(kTile / G)};
  const unsigned page_rows = 1u << a.pt.page_log2;
  if (!make_bf16_map4(&mQ, a.qr, qdims, qstr, qbox) ||
      !make_bf16_rows_map(&mKp, a.k_pages, a.pt.n_pages, page_rows, a.Hkv, D, page_rows) ||
      !make_bf16_rows_map(&mVp, a.v_pages, a.pt.n_pages, page_rows, a.Hkv, D, page_rows))
    return cudaErrorInvalidValue;
  if (a.p == 0) {  // no cartridge tile is read
    mKc = mKp;
    mVc = mVp;
  } else if (!make_bf16_rows_map(&mKc, a.kc, 1, a.p, a.Hkv, D, kTile) ||
             !make_bf16_rows_map(&mVc, a.vc, 1, a.p, a.Hkv, D, kTile)) {
    return cudaErrorInvalidValue;
  }
  Turns turns;
  for (int j = 0; j < kMaxHeadDim / 2; ++j) turns.t[j] = f.turns[j];
  using L = TreeLayout<D>;
  cudaError_t e = set_smem_once<tree_attend_kernel<D>>(L::kBytes);
  if (e != cudaSuccess) return e;
  tree_prep_kernel<D><<<a.B * a.nodes + 1, 256, 0, st>>>(a, turns);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_dependent(tree_attend_kernel<D>, dim3(a.n_ctas), dim3(kTreeThreads), L::kBytes, st,
                       mQ, mKc, mVc, mKp, mVp, a);
  if (e != cudaSuccess) return e;
  const int blocks = (a.B * a.nodes * a.Hq + 7) / 8;
  return launch_dependent(tree_merge_kernel<D>, dim3(std::min(blocks, 8 * sms)), dim3(256), 0, st,
                          a);
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
  if (!aligned_to(table, 4) || !aligned_to(lens, 4) || (parents && !aligned_to(parents, 4))) return CART_ERR_POINTER;
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
  a.window = window;
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
  a.pairs = w.pairs;
  a.stacked = w.stacked;
  a.start = reinterpret_cast<long long*>(ws + w.start);
  a.cart_lo = reinterpret_cast<int*>(ws + w.cart_lo);
  a.part_c = reinterpret_cast<float*>(ws + w.part_c);
  a.part_p = reinterpret_cast<float*>(ws + w.part_p);
  a.lse_c = reinterpret_cast<float*>(ws + w.lse_c);
  a.lse_p = reinterpret_cast<float*>(ws + w.lse_p);
  a.status = device_status_ptr();
  if (!a.status) return CART_ERR_CUDA;
  const RopeFreqs f = make_rope_freqs(d, rope_theta);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope tr("decode_tree", st);
  const cudaError_t e = d == 128 ? launch_tree<128>(a, f, st) : launch_tree<64>(a, f, st);
  return e == cudaSuccess ? CART_OK : CART_ERR_CUDA;
}

}  // extern "C"
