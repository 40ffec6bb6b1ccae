// step.cu -- one new token per conversation over the shared cartridge and paged
// private rows, with the attention weights that the rows get added up
// (cart_attn_decode_paged).
//
// Three kernels, chained by programmatic dependent launch; the first two run at
// once, on SMs of their own:
//   rows    the cached private rows, bound by HBM: S^T = K Q^T and O^T = V^T P^T
//           on tcgen05, so that the keys fill the 128 rows of a product and the
//           few queries its columns.  A tile is 128 key rows, 32 of each of four
//           kv heads (64 of two, 128 of one), its columns the queries of those
//           heads as three bf16 terms each, which hold all 24 bits of f32; what a
//           key's row meets of another head's queries is not read.  Warp w has
//           the keys 32w .. 32w + 31 of a tile, one a thread, and a maximum, sums
//           and an O^T of its own.  K and V tiles come through one ring of 192 KB.
//           All conversations' rows, one after the other, are cut into equal
//           runs, one per CTA and SM.
//   cart    the B * G stacked query rows of each kv head against the cartridge,
//           as tcgen05 products: 128 rows and 48 keys at a time, Q resident as
//           two bf16 terms (2^-16 of it, and the hardware's sine and cosine, 5e-7;
//           with a third, two CTAs do not fit an SM), S and O in TMEM.  The key
//           tiles of each (kv head, row tile) are cut into equal pieces, one or more
//           per CTA; two CTAs an SM, on the SMs that the rows' kernel, launched
//           first, leaves.
//   join    the new token: its rotated key and its value to its row, its logits;
//           joins them and a (conversation, kv head)'s parts by their log-sum-exps;
//           adds exp2(logit - log-sum-exp) of the group's heads to each row's weights.
//
// The rows' kernel is launched plainly and starts behind all that came before the
// call: so cart, and join ahead of its wait, may read the call's inputs, and join may
// write what no other kernel of the call looks at: the new row (the rows' kernel
// loads it with its neighbours and takes nothing from it) and the outputs of
// conversations that sit the step out (o may be q: nothing is taken from their
// queries either).  Launched as a dependent itself, it would leave cart and join
// racing what came before the call.
//
// The whole, 32 query heads over 8, d 128, with weights: 96 conversations of up to
// 1500 rows over a cartridge of 2048 in 68 us, 61 without weights, of which 46 are the
// bytes' at a copy's rate.  Stamps of an earlier form that took 75 us: the first loads
// leave after 4.7 us (schedule, pages), the first S^T is there at 7; the rows end at 57
// (5.8 TB/s from the first load on, at 128 SMs), the cartridge by then; the log-sum-exps
// are joined at 63, the weights and outputs out at 70.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "internal.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cart {
namespace {

// Raises a kernel's shared-memory limit as set_smem_once does, and asks for the
// largest shared part of an SM's first-level cache: what the first CTA on an SM
// was given decides whether a second one fits.
template <auto Kernel>
cudaError_t set_shared_once(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) e = set_smem_once<Kernel>(bytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

constexpr int kMaxGroup = 8;  // query heads of a kv head
// (a window or sinks beyond every place are that many)
constexpr int kMostPlaces = 1 << 25;

struct StepArgs {
  PageTable pt;
  int B, Hq, Hkv, G, p, window, sinks;
  float scale_log2;
  const int* pos;  // null: p + lens
  const __nv_bfloat16 *q, *k_new, *v_new, *kc, *vc;
  __nv_bfloat16 *k_pages, *v_pages, *o;
  float* weights;  // [B, Hkv, weight_rows], or null
  int weight_rows;
  uint32_t* status;
  // ---- cart: row tiles, key tiles, pieces that the key tiles of a (kv head, row
  // tile) are cut into, pieces of a CTA
  int row_tiles, key_tiles, cart_parts, cart_each;
  float *cart_o, *cart_lse;  // [Hkv * row_tiles, cart_parts, d / 4, 128] float4; [.., 128]
  // ---- rows: heads of a unit (of which a conversation has `units`), 32-row
  // groups of a tile (heads * groups is 4), CTAs
  int heads, units, groups, row_ctas;
  int join_heads;            // heads of a block of the joining kernel: `heads` or 1
  long long* starts;         // [B + 1]: chunks of a unit before each conversation's
  float *row_o, *row_lse;    // [slots, groups, heads, G, d], [.., G]
  int cap;                   // most private rows
  int logit_rows;            // ... in whole groups of 32, as they are written and read
  float* logits;             // [B, Hkv, G, logit_rows], log2 domain, by the order of groups seen
};

struct Turns {
  float2 t[kMaxHeadDim / 2];
};

// Softmax weights of values enter the products as two bf16 terms, good to 2^-15 of
// them, so that outputs are as exact as their own rounding to bf16 allows (0.0017 of
// them in all; 0.0023 with one term, at the same speed to within 3%).  The first is
// cut off below the weight, so that both are above 0 where it is, and a value that
// is infinite stays so.
__device__ __forceinline__ float below(float w) { return w * 0x1.fffffep-1f; }
// ... of two weights, each term's in a word
__device__ __forceinline__ void split_weights(float2 w, uint32_t& first, uint32_t& second) {
  const float2 y = __fmul2_rn(w, make_float2(0x1.fffffep-1f, 0x1.fffffep-1f));
  first = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
  const float2 f = bf16x2_to_float2(first);
  second = pack_bf16x2(w.x - f.x, w.y - f.y);
}

// The step of conversation b: the row of its new token (-1: idle, or its table
// has no place for it); the cached rows that it sees: those below `low` and from
// `high` to row - 1, in n groups of 32: those below g_low and from g_high on.
// (Whether the row has a page is looked up where the token is taken.)
struct StepOf {
  int row, low, high, g_low, g_high, n;
  __device__ __forceinline__ int group(int i) const { return i < g_low ? i : i - g_low + g_high; }
  __device__ __forceinline__ bool sees(int r) const { return r < row && (r < low || r >= high); }
  // ... rows r .. r + 31, a bit each
  __device__ __forceinline__ unsigned sees32(int r) const {
    auto below = [&](int x) {
      return x - r >= 32 ? 0xffffffffu : x > r ? (1u << (x - r)) - 1 : 0u;
    };
    return below(row) & (below(low) | ~below(high));
  }
};
__device__ __forceinline__ StepOf step_of(const StepArgs& a, int b) {
  StepOf s;
  const int len = held_rows(a.pt, b);
  s.row = len < a.cap ? len : -1;
  s.high = a.window > 0 ? max(s.row - a.window + 1, 0) : 0;
  s.low = min(max(a.sinks - a.p, 0), s.high);
  s.g_high = s.high >> 5;
  s.g_low = min((s.low + 31) >> 5, s.g_high);
  s.n = s.row < 0 ? 0 : s.g_low + max(((s.row + 31) >> 5) - s.g_high, 0);
  return s;
}
__device__ __forceinline__ int position_of(const StepArgs& a, int b, int row) {
  return min(max(a.pos ? __ldg(a.pos + b) : a.p + row, 0), (1 << 24) - 1);
}

// ----------------------------------------------------------------- cart ----
constexpr int kCartThreads = 192;  // four softmax warps, TMA warp, MMA warp
constexpr int kCartKeys = 48;      // keys of a tile
constexpr int kCartSColumns = 64;  // of TMEM, from one buffer of S to the next

template <int D>
struct CartSmem {
  static constexpr int kQBytes = kTile * D * 2, kKBytes = kCartKeys * D * 2;
  static constexpr int kQ = 0;                 // two terms
  static constexpr int kK = kQ + 2 * kQBytes;  // two of each
  static constexpr int kV = kK + 2 * kKBytes;
  static constexpr int kShared = kV + 2 * kKBytes;  // a CartShared
  static constexpr int kAlloc = kShared + 256;  // starts 1024-aligned (checked at entry)
};

enum CartBar {
  kCKFull0 = 0,               // keys of buffer x have landed
  kCKEmpty0 = kCKFull0 + 2,   // ... have been read
  kCVFull0 = kCKEmpty0 + 2,   // values, the same
  kCVEmpty0 = kCVFull0 + 2,
  kCSFull0 = kCVEmpty0 + 2,   // S of buffer x is in TMEM
  kCPFull0 = kCSFull0 + 2,    // its weights are (128 arrivals); by buffer, since those
                              // of the next tile may come before these are waited for
  kCPvDone = kCPFull0 + 2,    // O has a tile's
  kCODone,                    // O has those of the piece's last tile (waits for this one
                              // may come two tiles after the last for the one before)
  kCDrain,
  kCBars
};

// (no static shared memory: it would take 1 KB before aligned tiles)
struct CartShared {
  uint64_t bars[kCBars];
  uint32_t tmem;
  int abort, first;
};
static_assert(sizeof(CartShared) <= 256, "cart barrier area");

struct CartMaps {
  CUtensorMap k, v;
};

// Bound by latency: what it reads comes behind the rows' traffic, about 2 us a load,
// so keys and values have two buffers each, of 48 keys, which two CTAs an SM just
// hold.  (One buffer each of 64 keys: 108 us in all with 12 SMs for 768 tiles of 64
// keys, against 90.)
template <int D>
__global__ void __launch_bounds__(kCartThreads, 2)
    step_cart_kernel(const __grid_constant__ CartMaps maps, const __grid_constant__ StepArgs a,
                     const __grid_constant__ Turns f) {
  using L = CartSmem<D>;
  constexpr int HALF = D / 2;
  extern __shared__ __align__(1024) uint8_t step_smem[];
  uint8_t* const smem = step_smem;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(a.status, kDevErrSmemLayout);
    return;
  }
  CartShared& sh = *reinterpret_cast<CartShared*>(smem + L::kShared);
  uint64_t* const bars = sh.bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t abort_s = smem_u32(&sh.abort);
  pdl_release();
  if (threadIdx.x == 0) {
    sh.abort = 0;
    for (int s = 0; s < kCBars; ++s)
      mbar_init(&bars[s], s == kCPFull0 || s == kCPFull0 + 1 ? 128 : 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 128) {
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == 5) {
    tmem_alloc(&sh.tmem, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem, tO = tmem, tS = tmem + 128;
  const int total = a.Hkv * a.row_tiles * a.cart_parts;
  const int lo = min(blockIdx.x * a.cart_each, total), hi = min(lo + a.cart_each, total);
  const int R = a.B * a.G;
  int step = 0, pieces = 0;  // tiles walked, and pieces that had any, in every role
  bool ok = true;
  const int least = a.key_tiles / a.cart_parts, over = a.key_tiles - least * a.cart_parts;
  for (int u = lo; u < hi; ++u) {
    const int seg = u / a.cart_parts, part = u - seg * a.cart_parts;
    const int t0 = part * least + min(part, over), t1 = t0 + least + (part < over);
    const int g = seg / a.row_tiles, row0 = (seg - g * a.row_tiles) * kTile;
    // ---- the tile's queries, rotated, as two terms; what they see.  D / 16 threads
    // have a row, pairs 8c .. 8c + 7 each; the angles, which a conversation's heads
    // share, are worked out in the space of the keys and values, for as many rows
    // at a time as have theirs there.
    if (threadIdx.x == 0) sh.first = 0x7fffffff;
    constexpr int kChunks = HALF / 8, kAhead = 2;  // loads that a thread has in flight
    const int rows = min(R - row0, kTile), turn_rows = a.G >= 3 ? kTile : 32;
    static_assert((kTile / 3 + 2) * HALF * 8 <= 4 * L::kKBytes && 32 * HALF * 8 <= 4 * L::kKBytes,
                  "angles of a turn's conversations");
    float2* const angles = reinterpret_cast<float2*>(smem + L::kK);
    const uint32_t qs = smem_u32(smem + L::kQ);
    for (int r0 = 0; r0 < rows; r0 += turn_rows) {
      const int n_rows = min(rows - r0, turn_rows), b0 = (row0 + r0) / a.G;
      for (int e0 = threadIdx.x; e0 - static_cast<int>(threadIdx.x) < n_rows * kChunks;
           e0 += kAhead * kCartThreads) {
        uint4 l4[kAhead], h4[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int e = e0 + i * kCartThreads, r = row0 + r0 + e / kChunks;
          if (e < n_rows * kChunks) {
            const __nv_bfloat16* x =
                a.q + (static_cast<long long>(r / a.G) * a.Hq + g * a.G + r % a.G) * D +
                e % kChunks * 8;
            l4[i] = __ldg(reinterpret_cast<const uint4*>(x));
            h4[i] = __ldg(reinterpret_cast<const uint4*>(x + HALF));
          }
        }
        if (e0 == static_cast<int>(threadIdx.x)) {
          if (r0 > 0) __syncthreads();
          const int n = (row0 + r0 + n_rows - 1) / a.G - b0 + 1;
#pragma unroll 4
          for (int k = threadIdx.x; k < n * HALF; k += kCartThreads) {
            const int b = b0 + k / HALF;
            angles[k] =
                rope_cs_turns_fast(f.t[k % HALF], position_of(a, b, max(held_rows(a.pt, b), 0)));
          }
          __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int e = e0 + i * kCartThreads, r = r0 + e / kChunks, c = e % kChunks;
          if (e >= n_rows * kChunks) continue;
          const float2* cs = angles + ((row0 + r) / a.G - b0) * HALF + 8 * c;
          const uint32_t pl[4] = {l4[i].x, l4[i].y, l4[i].z, l4[i].w};
          const uint32_t ph[4] = {h4[i].x, h4[i].y, h4[i].z, h4[i].w};
          uint32_t yl[2][4], yh[2][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 fl = bf16x2_to_float2(pl[k]), fh = bf16x2_to_float2(ph[k]);
            float2 v, w;
            rope_pair(fl.x, fh.x, cs[2 * k], v.x, w.x);
            rope_pair(fl.y, fh.y, cs[2 * k + 1], v.y, w.y);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              yl[m][k] = pack_bf16x2(v.x, v.y);
              yh[m][k] = pack_bf16x2(w.x, w.y);
              const float2 dv = bf16x2_to_float2(yl[m][k]), dw = bf16x2_to_float2(yh[m][k]);
              v.x -= dv.x;
              v.y -= dv.y;
              w.x -= dw.x;
              w.y -= dw.y;
            }
          }
          // (rows of 128 bytes, 64 elements; d = 128 has a second block)
          const uint32_t o0 = sw128_offset(r, c);
          const uint32_t o1 = D == 128 ? 16384u + sw128_offset(r, c) : sw128_offset(r, c + 4);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            sts_u4(qs + m * L::kQBytes + o0, make_uint4(yl[m][0], yl[m][1], yl[m][2], yl[m][3]));
            sts_u4(qs + m * L::kQBytes + o1, make_uint4(yh[m][0], yh[m][1], yh[m][2], yh[m][3]));
          }
        }
      }
    }
    fence_proxy_async_smem();
    const int row = threadIdx.x;
    int first = 0x7fffffff;  // first key in the row's window
    if (row < kTile) {
      if (row < rows) {
        const StepOf s = step_of(a, (row0 + row) / a.G);
        if (s.row >= 0) first = a.window > 0 ? a.p + s.row - a.window + 1 : 0;
      }
      if (a.window > 0) {
        const int w = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) atomicMin(&sh.first, w);
      }
    }
    __syncthreads();
    // tiles that some row sees
    const int low = a.window > 0 ? *const_cast<volatile int*>(&sh.first) : 0;
    auto seen = [&](int t) { return t * kCartKeys < a.sinks || (t + 1) * kCartKeys > low; };
    int n = 0;
    for (int t = t0; t < t1; ++t) n += seen(t);
    if (warp == 4) {
      // ---------------------------------------------------------- producer --
      if (lane == 0) {
        int s = step;
        for (int t = t0; t < t1 && ok; ++t) {
          if (!seen(t)) continue;
          const int x = s & 1;
          const uint32_t last = ((s >> 1) - 1) & 1;
          if (s >= 2)
            ok = mbar_wait(&bars[kCKEmpty0 + x], last, abort_s, a.status, kDevErrTimeoutTma);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars[kCKFull0 + x], L::kKBytes);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(smem + L::kK + x * L::kKBytes + h * kCartKeys * 128, &maps.k,
                        &bars[kCKFull0 + x], h * 64, g, t * kCartKeys, 0);
          if (s >= 2)
            ok = mbar_wait(&bars[kCVEmpty0 + x], last, abort_s, a.status, kDevErrTimeoutTma);
          if (!ok) {
            mbar_wait(&bars[kCKFull0 + x], (s >> 1) & 1, 0u, nullptr, 0);
            break;
          }
          mbar_arrive_expect_tx(&bars[kCVFull0 + x], L::kKBytes);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(smem + L::kV + x * L::kKBytes + h * kCartKeys * 128, &maps.v,
                        &bars[kCVFull0 + x], h * 64, g, t * kCartKeys, 0);
          ++s;
        }
        // (whatever went wrong: the last copies land before the CTA ends)
        for (int i = max(s - 2, step); i < s; ++i) {
          mbar_wait(&bars[kCKFull0 + (i & 1)], (i >> 1) & 1, 0u, nullptr, 0);
          mbar_wait(&bars[kCVFull0 + (i & 1)], (i >> 1) & 1, 0u, nullptr, 0);
        }
      }
      __syncwarp();
    } else if (warp == 5) {
      // --------------------------------------------------------------- MMA --
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, kDevErrTimeoutMma));
      };
      const uint32_t idS = idesc_bf16(128, kCartKeys, false, false);
      const uint32_t idPV = idesc_bf16(128, D, false, true);
      const uint64_t dQ = sdesc_sw128(smem_u32(smem + L::kQ), 16u, 1024u);
      const uint64_t dK = sdesc_sw128(smem_u32(smem + L::kK), 16u, 1024u);
      const uint64_t dV = sdesc_sw128(smem_u32(smem + L::kV), kCartKeys * 128u, 1024u);
      auto issue_s = [&](int s) {
        const uint64_t dk = desc_add(dK, (s & 1) * L::kKBytes);
#pragma unroll
        for (int m = 1; m >= 0; --m)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_bf16_ss_w(tS + (s & 1) * kCartSColumns,
                           desc_add(dQ, m * L::kQBytes + (k >> 2) * 16384 + (k & 3) * 32),
                           desc_add(dk, (k >> 2) * kCartKeys * 128 + (k & 3) * 32), idS,
                           m == 1 && k == 0 ? 0u : 1u);
        umma_commit_w(&bars[kCSFull0 + (s & 1)]);
        umma_commit_w(&bars[kCKEmpty0 + (s & 1)]);
      };
      for (int t = 0; t < n && ok; ++t) {
        const int s = step + t;
        if (t == 0) {
          ok = wait(&bars[kCKFull0 + (s & 1)], (s >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          issue_s(s);
        }
        if (t + 1 < n) {  // over the weights of tile t - 1, read by the product before
          ok = wait(&bars[kCKFull0 + ((s + 1) & 1)], ((s + 1) >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          issue_s(s + 1);
        }
        ok = wait(&bars[kCVFull0 + (s & 1)], (s >> 1) & 1) &&
             wait(&bars[kCPFull0 + (s & 1)], (s >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int m = 1; m >= 0; --m)  // (the smaller terms first)
#pragma unroll
          for (int k = 0; k < kCartKeys / 16; ++k)
            umma_bf16_ts_w(tO, tS + (s & 1) * kCartSColumns + m * (kCartKeys / 2) + k * 8,
                           desc_add(dV, (s & 1) * L::kKBytes + k * 2048), idPV,
                           t > 0 || m == 0 || k > 0 ? 1u : 0u);
        umma_commit_w(&bars[kCVEmpty0 + (s & 1)]);
        umma_commit_w(&bars[kCPvDone]);
        if (t == n - 1) umma_commit_w(&bars[kCODone]);
      }
    } else {
      // ----------------------------------------------------------- softmax --
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t err) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, err));
      };
      const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
      const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
      float m = -INFINITY, l = 0.f;
      int i = 0;  // tiles of this piece walked
      for (int t = t0; t < t1 && ok; ++t) {
        if (!seen(t)) continue;
        const int s = step + i;
        ok = wait(&bars[kCSFull0 + (s & 1)], (s >> 1) & 1, kDevErrTimeoutSoftmax);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ts = tS + (s & 1) * kCartSColumns + lane_off;
        // the row sees the keys up to `end` that are sinks or in its window
        const int k0 = t * kCartKeys;
        const int end = first == 0x7fffffff ? 0 : min(a.p - k0, kCartKeys);
        const int from = first > k0 ? min(first - k0, kCartKeys) : 0;
        const int sink = min(max(a.sinks - k0, 0), kCartKeys);
        const bool cut = __any_sync(0xffffffffu, end < kCartKeys || from > sink);
        float v[kCartKeys];
        {
          uint32_t r[32], z[16];
          tmem_ld32(ts, r);
          tmem_ld16(ts + 32, z);
          tmem_ld_wait();
          tmem_reg_fence(r);
          tmem_reg_fence16(z);
#pragma unroll
          for (int c = 0; c < kCartKeys; ++c) v[c] = __uint_as_float(c < 32 ? r[c & 31] : z[c & 15]);
        }
        if (cut) {
#pragma unroll
          for (int c = 0; c < kCartKeys; ++c)
            if (c >= end || (c < from && c >= sink)) v[c] = -INFINITY;
        }
        float mx[2] = {v[0], v[1]};
#pragma unroll
        for (int c = 2; c < kCartKeys - 2; c += 4) {
          mx[0] = fmax3(mx[0], v[c], v[c + 1]);
          mx[1] = fmax3(mx[1], v[c + 2], v[c + 3]);
        }
        float top = fmax3(fmaxf(mx[0], mx[1]), v[kCartKeys - 2], v[kCartKeys - 1]);
        top *= a.scale_log2;
        // (the maximum is renewed where it grows by more than 8: weights stay
        // below 2^8)
        float alpha = 1.f;
        bool rescale = false;
        if (top > m + 8.f) {
          alpha = exp2_approx(m - top);
          m = top;
          rescale = i > 0;
        }
        const float mr = m == -INFINITY ? 0.f : m;  // (nothing seen yet: weights 0)
        const float2 nm2 = make_float2(-mr, -mr);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[kCartKeys];  // first terms, second terms
#pragma unroll
        for (int c = 0; c < kCartKeys / 2; ++c) {
          const float2 x = __ffma2_rn(make_float2(v[2 * c], v[2 * c + 1]), sc2, nm2);
          const float2 w = make_float2(exp2_approx(x.x), exp2_approx(x.y));
          sum[c & 1] = __fadd2_rn(sum[c & 1], w);
          split_weights(w, pk[c], pk[kCartKeys / 2 + c]);
        }
        tmem_st32(ts, pk);  // (over columns that have been read)
        tmem_st16(ts + 32, pk + 32);
        l = l * alpha + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
        if (__any_sync(0xffffffffu, rescale)) {
          ok = wait(&bars[kCPvDone], (s - 1) & 1, kDevErrTimeoutSoftmax);
          if (!ok) break;
          tc_fence_after();
          const float2 al2 = make_float2(alpha, alpha);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + lane_off + c * 32, o);
            tmem_ld_wait();
            tmem_reg_fence(o);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 v = __fmul2_rn(u2f2(o[e], o[e + 1]), al2);
              o[e] = __float_as_uint(v.x);
              o[e + 1] = __float_as_uint(v.y);
            }
            tmem_st32(tO + lane_off + c * 32, o);
          }
        }
        // values of keys that none of the rows sees may be anything, and 0 times
        // them need not be 0
        const int z0 = max(a.sinks - k0, 0), z1 = min(low - k0, kCartKeys);
        if (z0 < z1) {
          ok = wait(&bars[kCVFull0 + (s & 1)], (s >> 1) & 1, kDevErrTimeoutSoftmax);
          if (!ok) break;
          const uint32_t vs = smem_u32(smem + L::kV + (s & 1) * L::kKBytes);
          for (int e = row; e < (z1 - z0) * (D / 8); e += 128) {
            const int j = z0 + e / (D / 8), c = e % (D / 8);
            sts_u4(vs + (c >> 3) * kCartKeys * 128 + j * 128 + (c & 7) * 16,
                   make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars[kCPFull0 + (s & 1)]);
        ++i;
      }
      // ---- the piece's part: column blocks of four by row
      const long long slot = u;
      if (ok && n > 0) ok = wait(&bars[kCODone], pieces & 1, kDevErrTimeoutEpilogue);
      if (ok) {
        tc_fence_after();
        const bool any = l > 0.f || l != l;
        const float inv = any ? 1.f / l : 0.f;
        float4* out = reinterpret_cast<float4*>(a.cart_o) + slot * (D / 4) * kTile + row;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(tO + lane_off + c * 32, o);
            tmem_ld_wait();
            tmem_reg_fence(o);
          }
          if (row < rows)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              out[(c * 8 + e / 4) * kTile] =
                  any ? make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                    __uint_as_float(o[e + 2]) * inv,
                                    __uint_as_float(o[e + 3]) * inv)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        a.cart_lse[slot * kTile + row] = any ? m + __log2f(l) : -INFINITY;
        tc_fence_before();
      }
    }
    step += n;
    pieces += n > 0;
    // every role is done with the piece's Q, barriers and O; one that gave up
    // ends them all
    ok = !__syncthreads_or(!ok);
    tc_fence_after();
    if (!ok) break;
  }
  if (warp == 5) {  // every product issued completes before the CTA ends
    umma_commit_w(&bars[kCDrain]);
    mbar_wait(&bars[kCDrain], 0, 0u, nullptr, 0);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, 256);
  // the next kernel waits for this one alone: it has waited for the rows'
  pdl_wait();
}

// ----------------------------------------------------------------- rows ----
constexpr int kRowThreads = 192;   // four warps of keys, TMA warp, MMA warp
constexpr int kRowHeads = 4;       // most heads of a unit
constexpr int kTerms = 3;          // of a query
constexpr int kHeadColumns = kTerms * kMaxGroup;
constexpr int kTileInfos = 4;

// What the roles know of a tile: conversation, first head, first key's number
// among the groups seen, times 32; whether it opens and closes a piece and is the
// run's last (kNone: the run has none); the slot of the piece's parts; the rows of
// each group that are there and seen.
enum TileFlags { kOpens = 1, kCloses = 2, kLast = 4, kNone = 8 };
struct TileInfo {
  int b, h0, v0, flags, slot;
  unsigned bits[kRowHeads];
};

template <int D>
struct RowSmem {
  static constexpr int kTileBytes = kTile * D * 2;          // a K or V tile
  static constexpr int kSlots = 6 * 128 / D;                // of the ring
  static constexpr int kQHalf = kRowHeads * kHeadColumns * 128;  // 64 dims of all columns
  // weights: two buffers, 2 KB for two warps, eight rows of each term (a product
  // has at least 16 columns: the second term costs none)
  static constexpr int kP = kSlots * kTileBytes;
  static constexpr int kQ = kP + 2 * 4096;
  static constexpr int kShared = kQ + (D / 64) * kQHalf;  // a RowShared
  static constexpr int kAlloc = kShared + 3072;           // starts 1024-aligned
};

enum RowBar {
  kRFull0 = 0,                  // ring slot has landed (12 slots at most)
  kREmpty0 = kRFull0 + 12,
  kRInfoFull0 = kREmpty0 + 12,  // info of a tile
  kRInfoEmpty0 = kRInfoFull0 + kTileInfos,  // four warps and the MMA warp have read it
  kRQReady = kRInfoEmpty0 + kTileInfos,     // a piece's queries are staged (128 arrivals)
  kRSFull0,                     // S^T of buffer x is in TMEM
  kRPFull0 = kRSFull0 + 2,      // its weights are in shared memory (128 arrivals)
  kRPvDone = kRPFull0 + 2,      // O^T has a tile's
  kRODone,                      // ... a piece's last tile's
  kRExchange,                   // the four warps have left their factors (4 arrivals)
  kRDrain,
  kRBars
};

struct RowShared {
  float2 angles[kTileInfos][kMaxHeadDim / 2];  // of a piece, beside its first tile's info
  uint64_t bars[kRBars];
  long long scan[kRowThreads / 32];
  TileInfo info[kTileInfos];
  float factor[2][4][kMaxGroup];  // what each warp's O^T is multiplied by, by tile
  float inverse[4][kMaxGroup];    // ... in the end (a warp may be a tile ahead of another)
  int rescale[2][4];
  uint32_t tmem;
  int run_b, run_unit, run_at, abort;  // (where the run begins)
};
static_assert(sizeof(RowShared) <= 3072, "rows barrier area");

struct RowMaps {
  CUtensorMap k, v;  // (d, page_rows, Hkv, pages), box 64 x 32 x heads, or 64 x 16 x 1
};

// Tiles of one unit of a conversation that sees n groups, and what they cost in
// the schedule: the change from one unit's queries and sums to another's takes
// about as long as that many tiles (2 / 3 / 4 / 5 / 6, in all: 68.8 / 68.9 / 69.9 / 70.4
// / 70.6 us at 96 conversations, 115.3 / 115.1 / 114.9 / 114.3 / 113.6 at 4 long ones,
// 89.6 / 88.6 / 89.2 / 90.4 / 90.1 at 200 in a window).
constexpr int kStart = 3;
__device__ __forceinline__ int tiles_of(const StepArgs& a, int n) {
  return (n + a.groups - 1) / a.groups;
}
__device__ __forceinline__ int cost_of(int tiles) { return tiles > 0 ? tiles + kStart : 0; }
// x / y for x >= 0, y > 0; the 64-bit division takes several times as long as the
// 32-bit one that nearly every schedule gets by with.
__device__ __forceinline__ long long div_units(long long x, long long y) {
  return ((x | y) >> 31) == 0 ? static_cast<unsigned>(x) / static_cast<unsigned>(y) : x / y;
}

// The largest of a warp's values (NaN left out).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Row v of a tile is a key, its logits with the unit's queries a row of S^T in TMEM:
// no thread shares a key, and the sums of a query over keys are the tensor pipe's
// (O^T) and one addition a tile.  The maxima that the weights are taken relative to
// are a warp's own, renewed where one grows by more than 8, so warps wait for each
// other only to renew O^T (its lanes are dims, all warps').  Bound by HBM but for the
// start (7 us until the first S^T) and the changes of units: 305 MB take 59 us alone
// on 128 SMs (ncu: DRAM 66% of its peak, tensor pipe 12%).
// GQ: query heads of a kv head, 4 or 8 at most.
template <int D, int GQ>
__global__ void __launch_bounds__(kRowThreads, 1)
    step_rows_kernel(const __grid_constant__ RowMaps maps, const __grid_constant__ StepArgs a,
                     const __grid_constant__ Turns f) {
  using L = RowSmem<D>;
  constexpr int HALF = D / 2, NS = L::kSlots;
  extern __shared__ __align__(1024) uint8_t step_smem[];
  uint8_t* const smem = step_smem;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(a.status, kDevErrSmemLayout);
    return;
  }
  RowShared& sh = *reinterpret_cast<RowShared*>(smem + L::kShared);
  uint64_t* const bars = sh.bars;
  TileInfo* const info = sh.info;
  auto& factor = sh.factor;
  auto& rescale = sh.rescale;
  auto& inverse = sh.inverse;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t abort_s = smem_u32(&sh.abort);
  if (tid == 0) {
    sh.abort = 0;
    for (int s = 0; s < kRBars; ++s)
      mbar_init(&bars[s], s == kRQReady || s == kRPFull0 || s == kRPFull0 + 1 ? 128
                          : s >= kRInfoEmpty0 && s < kRInfoEmpty0 + kTileInfos ? 5
                          : s == kRExchange                                    ? 4
                                                                               : 1);
    fence_mbar_init();
  }
  pdl_release();  // (the cartridge's kernel runs beside this one)
  if (tid == 128) {
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == 5) {
    tmem_alloc(&sh.tmem, 256);
    tmem_relinquish();
  }
  // ---- the tiles of all conversations, and this CTA's run of them
  const int per = (a.B + kRowThreads - 1) / kRowThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += static_cast<long long>(cost_of(tiles_of(a, step_of(a, b).n))) * a.units;
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh.scan[warp] = x;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  long long total = 0, start = x - mine;
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) {
    start += w < warp ? sh.scan[w] : 0;
    total += sh.scan[w];
  }
  const long long chunk = div_units(total + a.row_ctas - 1, a.row_ctas);
  const long long lo = min(blockIdx.x * chunk, total), hi = min(lo + chunk, total);
  if (lo < hi && start <= lo && lo < start + mine) {  // (one thread)
    long long at = start;
    int b = b0;
    for (;; ++b) {
      const long long n = static_cast<long long>(cost_of(tiles_of(a, step_of(a, b).n))) * a.units;
      if (lo < at + n) break;
      at += n;
    }
    const int cost = cost_of(tiles_of(a, step_of(a, b).n));
    const long long off = lo - at;
    sh.run_b = b;
    sh.run_unit = static_cast<int>(div_units(off, cost));
    sh.run_at = static_cast<int>(off - static_cast<long long>(sh.run_unit) * cost);
  }
  if (blockIdx.x == 0) {  // for the last kernel
    long long at = start;
    for (int b = b0; b < b1; ++b) {
      a.starts[b] = at;
      at += static_cast<long long>(cost_of(tiles_of(a, step_of(a, b).n))) * a.units;
    }
    if (tid == 0) a.starts[a.B] = total;
  }
  __syncthreads();
  // TMEM: two buffers of S^T, then the four O^T (16 columns each, eight of a term)
  const uint32_t tS = tmem, tO = tmem + 192;
  constexpr int kSBuffer = 96;

  if (warp == 4) {
    // ------------------------------------------------------------ producer --
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, kDevErrTimeoutTma));
    };
    int b = vld(sh.run_b), n = 0, loads = 0;  // tiles handed on, ring slots filled
    long long left = hi - lo;                 // units to go
    bool ok = true;
    int unit = 0, at = 0;  // of the conversation, and in its cost
    StepOf s{};
    if (left > 0) {
      s = step_of(a, b);
      unit = vld(sh.run_unit);
      at = vld(sh.run_at);
    }
    // boxes: a group's 32 rows of all heads, or, in pages of 16, 16 rows of one
    const bool small = a.pt.page_log2 == 4;
    const int lanes = small ? 2 * a.groups : a.groups;  // that issue boxes
    const int group_of = small ? lane >> 1 : lane;
    const int lane_bytes = a.heads * (small ? 2048 : 4096) * (D / 64);
    const int mask = (1 << a.pt.page_log2) - 1;
    // (rows are read once a step; the cartridge, the logits and the parts stay in L2
    // for it: 88 / 140 / 112 us without, 81 / 130 / 102 us with, at 96, 4 and 200
    // conversations of 8, 8 and 4 kv heads)
    const uint64_t policy = evict_first_policy();
    while (ok && left > 0) {
      const int all = tiles_of(a, s.n);
      if (all == 0) {  // idle, or nothing cached
        s = step_of(a, ++b);
        continue;
      }
      const int h0 = unit * a.heads;
      const int end = static_cast<int>(min(static_cast<long long>(cost_of(all)), at + left));
      const int t0 = max(at - kStart, 0), t1 = end - kStart;
      left -= end - at;
      // (what is left holds tiles if it is more than a start)
      const bool more = left > kStart;
      const int* pages = a.pt.table + static_cast<long long>(b) * a.pt.max_pages;
      // a tile's boxes, a lane each: first row, and that row's page
      auto row_of = [&](int t) {
        const int i = t * a.groups + group_of;
        return lane < lanes && i < s.n ? s.group(i) * 32 + (small ? (lane & 1) * 16 : 0) : -1;
      };
      auto look_up = [&](int r) {  // (the second half of the last group may be past the table)
        return r < 0 || (r >> a.pt.page_log2) >= a.pt.max_pages
                   ? -1
                   : __ldg(pages + (r >> a.pt.page_log2));
      };
      int row = row_of(t0), page = look_up(row);
      // the next conversation's, before they are needed
      const StepOf next = unit + 1 == a.units && b + 1 < a.B ? step_of(a, b + 1) : s;
      // the piece's slot: the run's first piece, its last one, or a whole unit
      const bool goes_on = t1 < all;
      const int slot = t0 > 0 || (goes_on && n == 0) ? 2 * blockIdx.x
                       : goes_on                     ? 2 * blockIdx.x + 1
                                                     : 2 * a.row_ctas + b * a.units + unit;
      if (t0 < t1 && n > 0) {  // its queries on their way to L2 (the run's first are asked for)
        const int heads = min(a.heads, a.Hkv - h0);
        const char* q = reinterpret_cast<const char*>(
            a.q + (static_cast<long long>(b) * a.Hq + h0 * a.G) * D);
        for (int e = lane * 128; e < heads * a.G * D * 2; e += 32 * 128) prefetch_l2(q + e);
      }
      for (int t = t0; t < t1; ++t, ++n) {
        const int row_next = t + 1 < t1 ? row_of(t + 1) : -1, page_next = look_up(row_next);
        const bool there = row >= 0 && is_page(page, a.pt.n_pages);
        unsigned bits = there ? s.sees32(row) & (small ? 0xffffu : 0xffffffffu) : 0u;
        if (small) bits |= __shfl_down_sync(0xffffffffu, bits, 1) << 16;  // (even lanes')
        const unsigned boxes = __ballot_sync(0xffffffffu, there);
        // a K or V tile into the next slot
        auto load = [&](const CUtensorMap* m) {
          const int sl = loads % NS;
          if (loads >= NS && !wait(&bars[kREmpty0 + sl], (loads / NS - 1) & 1)) return false;
          if (lane == 0) mbar_arrive_expect_tx(&bars[kRFull0 + sl], __popc(boxes) * lane_bytes);
          __syncwarp();
          if (there) {
            uint8_t* const to = smem + sl * L::kTileBytes + group_of * a.heads * 4096;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              if (!small) {
                tma_load_4d_hint(to + h * 16384, m, &bars[kRFull0 + sl], h * 64, row & mask, h0,
                                 page, policy);
              } else {
                for (int i = 0; i < a.heads; ++i)
                  tma_load_4d_hint(to + h * 16384 + i * 4096 + (lane & 1) * 2048, m,
                                   &bars[kRFull0 + sl], h * 64, 0, h0 + i, page, policy);
              }
            }
          }
          __syncwarp();
          ++loads;
          return true;
        };
        ok = load(&maps.k);
        if (!ok) break;
        const int ti = n % kTileInfos;
        if (n >= kTileInfos) {
          ok = wait(&bars[kRInfoEmpty0 + ti], (n / kTileInfos - 1) & 1);
          if (!ok) break;
        }
        TileInfo& o = info[ti];
        if (lane < lanes && (!small || !(lane & 1))) o.bits[group_of] = bits;
        if (lane == 0) {
          o.b = b;
          o.h0 = h0;
          o.v0 = t * a.groups * 32;
          o.flags = (t == t0 ? kOpens : 0) | (t + 1 < t1 ? 0 : more ? kCloses : kCloses | kLast);
          o.slot = slot;
        }
        if (t == t0 && n > 0) {  // the piece's angles (the key warps have the first one's)
          const int pos = position_of(a, b, s.row);
#pragma unroll 1
          for (int e = lane; e < HALF; e += 32) sh.angles[ti][e] = rope_cs_turns(f.t[e], pos);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kRInfoFull0 + ti]);
        ok = load(&maps.v);
        if (!ok) break;
        row = row_next;
        page = page_next;
      }
      at = 0;
      if (++unit == a.units) {
        unit = 0;
        ++b;
        s = next;
      }
    }
    if (ok && n == 0 && lane == 0) {  // a run without tiles
      info[0].flags = kNone;
      mbar_arrive(&bars[kRInfoFull0]);
    }
    if (lane == 0)  // the last copies land before the CTA ends
      for (int i = max(loads - NS, 0); i < loads; ++i)
        mbar_wait(&bars[kRFull0 + i % NS], (i / NS) & 1, 0u, nullptr, 0);
    __syncwarp();
  } else if (warp == 5) {
    // ----------------------------------------------------------------- MMA --
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, kDevErrTimeoutMma));
    };
    const uint32_t idS = idesc_bf16(128, a.heads == 1 ? 32 : a.heads * kHeadColumns, false, false);
    const uint32_t idO = idesc_bf16(128, 16, true, false);
    const uint64_t dK = sdesc_sw128(smem_u32(smem), 16u, 1024u);
    // (64 dims: the product's upper 64 rows are the next warp's values, unread)
    const uint64_t dV = sdesc_sw128(smem_u32(smem), D == 128 ? 16384u : 4096u, 1024u);
    const uint64_t dQ = sdesc_sw128(smem_u32(smem + L::kQ), 16u, 1024u);
    const uint64_t dP = sdesc_sw128(smem_u32(smem + L::kP), 16u, 1024u);
    auto issue_s = [&](int n) {
      const int e = 2 * n, sl = e % NS;
      if (!wait(&bars[kRFull0 + sl], (e / NS) & 1)) return false;
      tc_fence_after();
      const uint64_t dk = desc_add(dK, sl * L::kTileBytes);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        umma_bf16_ss_w(tS + (n & 1) * kSBuffer, desc_add(dk, (k >> 2) * 16384 + (k & 3) * 32),
                       desc_add(dQ, (k >> 2) * L::kQHalf + (k & 3) * 32), idS, k > 0 ? 1u : 0u);
      umma_commit_w(&bars[kRSFull0 + (n & 1)]);
      umma_commit_w(&bars[kREmpty0 + sl]);
      return true;
    };
    bool ok = true;
    int pieces = 0;
    auto flags_of = [&](int n) {
      const int ti = n % kTileInfos;
      if (!wait(&bars[kRInfoFull0 + ti], (n / kTileInfos) & 1)) return -1;
      const int fl = vld(info[ti].flags);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kRInfoEmpty0 + ti]);
      return fl;
    };
    int fl = flags_of(0);
    for (int n = 0; ok; ++n) {
      const int now = fl;
      if (now < 0 || (now & kNone)) break;
      if (now & kOpens) {  // a piece's first tile: its queries
        ok = wait(&bars[kRQReady], pieces & 1) && issue_s(n);
        ++pieces;
        if (!ok) break;
      }
      if (!(now & kLast)) {
        fl = flags_of(n + 1);
        ok = fl >= 0;
        if (!ok) break;
        // (of the same piece: over the S^T before, whose weights have been used)
        if (!(fl & kOpens)) ok = issue_s(n + 1);
        if (!ok) break;
      }
      const int e = 2 * n + 1, sl = e % NS;
      ok = wait(&bars[kRFull0 + sl], (e / NS) & 1) && wait(&bars[kRPFull0 + (n & 1)], (n >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint64_t dv = desc_add(dV, sl * L::kTileBytes), dp = desc_add(dP, (n & 1) * 4096);
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          umma_bf16_ss_w(tO + w * 16, desc_add(dv, w * 4096 + k * 2048),
                         desc_add(dp, (w >> 1) * 2048 + (w & 1) * 64 + k * 32), idO,
                         (now & kOpens) && k == 0 ? 0u : 1u);
      umma_commit_w(&bars[kREmpty0 + sl]);
      umma_commit_w(&bars[kRPvDone]);
      if (now & kCloses) umma_commit_w(&bars[kRODone]);
      if (now & kLast) break;
    }
    // every product issued above completes before the CTA ends
    umma_commit_w(&bars[kRDrain]);
    mbar_wait(&bars[kRDrain], 0, 0u, nullptr, 0);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- keys --
    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t err) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, err));
    };
    const int h = warp % a.heads, grp = warp / a.heads;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    bool ok = true;
    float m[GQ], l[GQ];  // the warp's maxima, the thread's sums
    int exchanges = 0, pieces = 0;
    // A piece's queries: four threads a row, over all terms.  (The products of the
    // piece before have read theirs: its last S^T is there.)  The run's first ones
    // are worked on while its pages are looked up, their angles here.
    auto stage_queries = [&](int ti, int b, int h0, bool first) {
      const int qi = tid >> 2, part = tid & 3, qh = qi / kMaxGroup, qq = qi % kMaxGroup;
      const bool mine = qh < a.heads && qq < a.G && h0 + qh < a.Hkv;
      uint4 l4[HALF / 32], h4[HALF / 32];
      if (mine) {
        const __nv_bfloat16* src =
            a.q + (static_cast<long long>(b) * a.Hq + (h0 + qh) * a.G + qq) * D;
#pragma unroll
        for (int c = 0; c < HALF / 32; ++c) {  // pairs 8j .. 8j + 7
          const int j = part * (HALF / 32) + c;
          l4[c] = __ldg(reinterpret_cast<const uint4*>(src + 8 * j));
          h4[c] = __ldg(reinterpret_cast<const uint4*>(src + HALF + 8 * j));
        }
      }
      if (first) {
        if (tid < HALF)
          sh.angles[ti][tid] = rope_cs_turns(f.t[tid], position_of(a, b, step_of(a, b).row));
        asm volatile("bar.sync 1, 128;" ::: "memory");
      }
      if (mine) {
        const uint32_t qs = smem_u32(smem + L::kQ);
#pragma unroll
        for (int c = 0; c < HALF / 32; ++c) {
          const int j = part * (HALF / 32) + c;
          const uint32_t pl[4] = {l4[c].x, l4[c].y, l4[c].z, l4[c].w};
          const uint32_t ph[4] = {h4[c].x, h4[c].y, h4[c].z, h4[c].w};
          uint32_t yl[kTerms][4], yh[kTerms][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 fl = bf16x2_to_float2(pl[k]), fh = bf16x2_to_float2(ph[k]);
            float2 u, w;
            rope_pair(fl.x, fh.x, sh.angles[ti][8 * j + 2 * k], u.x, w.x);
            rope_pair(fl.y, fh.y, sh.angles[ti][8 * j + 2 * k + 1], u.y, w.y);
#pragma unroll
            for (int s = 0; s < kTerms; ++s) {  // what the terms before leave, exactly
              yl[s][k] = pack_bf16x2(u.x, u.y);
              yh[s][k] = pack_bf16x2(w.x, w.y);
              const float2 du = bf16x2_to_float2(yl[s][k]), dw = bf16x2_to_float2(yh[s][k]);
              u.x -= du.x;
              u.y -= du.y;
              w.x -= dw.x;
              w.y -= dw.y;
            }
          }
#pragma unroll
          for (int s = 0; s < kTerms; ++s) {
            const int col = qh * kHeadColumns + s * kMaxGroup + qq;  // a row of 128 bytes
            sts_u4(qs + sw128_offset(col, j), make_uint4(yl[s][0], yl[s][1], yl[s][2], yl[s][3]));
            sts_u4(qs + (D == 128 ? L::kQHalf + sw128_offset(col, j) : sw128_offset(col, j + 4)),
                   make_uint4(yh[s][0], yh[s][1], yh[s][2], yh[s][3]));
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars[kRQReady]);
    };
    if (lo < hi) stage_queries(0, vld(sh.run_b), vld(sh.run_unit) * a.heads, true);
    for (int n = 0; ok; ++n) {
      const int ti = n % kTileInfos, x = n & 1;
      ok = wait(&bars[kRInfoFull0 + ti], (n / kTileInfos) & 1, kDevErrTimeoutSoftmax);
      if (!ok) break;
      const TileInfo& in = info[ti];
      const int flags = vld(in.flags);
      if (flags & kNone) break;
      const int b = vld(in.b), h0 = vld(in.h0), v0 = vld(in.v0), slot = vld(in.slot);
      const bool opens = flags & kOpens, closes = flags & kCloses;
      const unsigned bits = *const_cast<const volatile unsigned*>(&in.bits[grp]);
      const int g = h0 + h;
      if (opens) {
#pragma unroll
        for (int q = 0; q < GQ; ++q) {
          m[q] = -INFINITY;
          l[q] = 0.f;
        }
      }
      ok = wait(&bars[kRSFull0 + x], (n >> 1) & 1, kDevErrTimeoutSoftmax);
      if (!ok) break;
      tc_fence_after();
      uint32_t r[32];
      tmem_ld32(tS + x * kSBuffer + h * kHeadColumns + lane_off, r);
      tmem_ld_wait();
      tmem_reg_fence(r);
      const bool seen = bits >> lane & 1;
      float s[GQ];
#pragma unroll
      for (int q = 0; q < GQ; ++q) {
        const float v = __uint_as_float(r[q]) +
                        (__uint_as_float(r[8 + q]) + __uint_as_float(r[16 + q]));
        s[q] = seen && q < a.G ? v * a.scale_log2 : -INFINITY;
      }
      // ---- maxima, renewed where they grow by more than 8 (the weights stay below
      // 2^8): every O^T spans the lanes of all warps, so the factors are exchanged
      float top[GQ];
      bool grows = false;
#pragma unroll
      for (int q = 0; q < GQ; ++q) top[q] = warp_max(s[q]);
#pragma unroll
      for (int q = 0; q < GQ; ++q) grows |= top[q] > m[q] + 8.f;
      if (grows) {
#pragma unroll
        for (int q = 0; q < GQ; ++q) {
          const bool up = top[q] > m[q] + 8.f;
          const float alpha = up ? exp2_approx(m[q] - top[q]) : 1.f;
          m[q] = up ? top[q] : m[q];
          l[q] *= alpha;
          if (lane == q) factor[x][warp][q] = alpha;
        }
      }
      __syncwarp();
      if (lane == 0) {
        rescale[x][warp] = grows && !opens;
        mbar_arrive(&bars[kRExchange]);
      }
      // ---- weights as B: row q of 128 bytes, and q + 8, this key's two bytes
      {
        const uint32_t ps = smem_u32(smem + L::kP) + x * 4096 + (warp >> 1) * 2048;
#pragma unroll
        for (int q = 0; q < GQ; ++q) {
          const float p = exp2_approx(s[q] - (m[q] == -INFINITY ? 0.f : m[q]));
          l[q] += p;
          const uint32_t at =
              ps + q * 128 + ((((warp & 1) * 4 + (lane >> 3)) ^ q) << 4) + (lane & 7) * 2;
          const uint32_t first = __float_as_uint(below(p)) >> 16;
          sts_u16(at, static_cast<uint16_t>(first));
          sts_u16(at + 1024, __bfloat16_as_ushort(
                                 __float2bfloat16_rn(p - __uint_as_float(first << 16))));
        }
      }
      if (a.logits && g < a.Hkv && v0 + grp * 32 + lane < a.logit_rows) {
        float* lg = a.logits + (static_cast<long long>(b) * a.Hkv + g) * a.G * a.logit_rows + v0 +
                    grp * 32 + lane;
#pragma unroll
        for (int q = 0; q < GQ; ++q)
          if (q < a.G) lg[static_cast<long long>(q) * a.logit_rows] = s[q];
      }
      if (bits != 0xffffffffu) {
        // values of rows that are not seen may be anything, and 0 times them need
        // not be 0
        const int e = 2 * n + 1, sl = e % NS;
        ok = wait(&bars[kRFull0 + sl], (e / NS) & 1, kDevErrTimeoutSoftmax);
        if (!ok) break;
        if (!seen) {
          const uint32_t at = smem_u32(smem + sl * L::kTileBytes) + warp * 4096 + lane * 128;
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              sts_u4(at + k * 16384 + c * 16, make_uint4(0u, 0u, 0u, 0u));
        }
      }
      ok = wait(&bars[kRExchange], exchanges & 1, kDevErrTimeoutSoftmax);
      ++exchanges;
      if (!ok) break;
      int any = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) any |= vld(rescale[x][w]);
      if (any) {
        // (the product before the last one is done: S^T of this tile came after it)
        ok = wait(&bars[kRPvDone], (n - 1) & 1, kDevErrTimeoutSoftmax);
        if (!ok) break;
        tc_fence_after();
        for (int w = 0; w < 4; ++w) {
          if (!vld(rescale[x][w])) continue;
          uint32_t o[16];
          tmem_ld16(tO + w * 16 + lane_off, o);
          tmem_ld_wait();
          tmem_reg_fence16(o);
#pragma unroll
          for (int q = 0; q < GQ; ++q) {
            const float f = *const_cast<const volatile float*>(&factor[x][w][q]);
            o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
            o[8 + q] = __float_as_uint(__uint_as_float(o[8 + q]) * f);
          }
          tmem_st16(tO + w * 16 + lane_off, o);
        }
        tmem_st_wait();
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&bars[kRPFull0 + x]);
      if (closes) {
        if (!(flags & kLast)) {  // the next piece's queries meanwhile
          const int next = (n + 1) % kTileInfos;
          ok = wait(&bars[kRInfoFull0 + next], ((n + 1) / kTileInfos) & 1, kDevErrTimeoutSoftmax);
          if (!ok) break;
          stage_queries(next, vld(info[next].b), vld(info[next].h0), false);
        }
        // ---- the piece's parts: one of each warp, by all four (lane = dim)
        float sum = 0.f, most = 0.f;  // of query `lane`
#pragma unroll
        for (int q = 0; q < GQ; ++q) {
          float y = l[q];
#pragma unroll
          for (int w = 16; w; w >>= 1) y += __shfl_xor_sync(0xffffffffu, y, w);
          sum = lane == q ? y : sum;
          most = lane == q ? m[q] : most;
        }
        // (the last piece's are read: everyone has come to this tile's exchange)
        if (lane < GQ) {
          const bool some = sum > 0.f || sum != sum;
          inverse[warp][lane] = some ? 1.f / sum : 0.f;
          if (lane < a.G && g < a.Hkv)
            a.row_lse[((static_cast<long long>(slot) * a.groups + grp) * a.heads + h) * a.G + lane] =
                some ? most + __log2f(sum) : -INFINITY;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kRExchange]);
        ok = wait(&bars[kRODone], pieces & 1, kDevErrTimeoutEpilogue) &&
             wait(&bars[kRExchange], exchanges & 1, kDevErrTimeoutEpilogue);
        ++exchanges;
        ++pieces;
        if (!ok) break;
        tc_fence_after();
        const int dim = warp * 32 + lane;
        for (int w = 0; w < 4; ++w) {
          const int wh = w % a.heads, wg = w / a.heads;
          uint32_t o[16];
          tmem_ld16(tO + w * 16 + lane_off, o);
          tmem_ld_wait();
          tmem_reg_fence16(o);
          if (h0 + wh < a.Hkv && dim < D) {
            float* out = a.row_o +
                         ((static_cast<long long>(slot) * a.groups + wg) * a.heads + wh) * a.G * D +
                         dim;
#pragma unroll
            for (int q = 0; q < GQ; ++q) {
              const float inv = *const_cast<const volatile float*>(&inverse[w][q]);
              if (q < a.G)
                out[q * D] =
                    inv == 0.f ? 0.f : (__uint_as_float(o[q]) + __uint_as_float(o[8 + q])) * inv;
            }
          }
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kRInfoEmpty0 + ti]);
      if (flags & kLast) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, 256);
}

// ----------------------------------------------------------------- join ----
constexpr int kJoinThreads = 512;
constexpr int kJoinParts = 32;                      // parts joined at a time
constexpr int kJoinHeads = kRowHeads * kMaxGroup;   // most query heads of a block

// Block (heads, conversation), the heads a unit's or one: the new token's row and
// logits, a warp per query head, before what the other kernels leave is waited
// for; then the parts' common log-sum-exp; then the output, some threads per
// column of four, the parts' weights and places settled before.  The cached rows'
// weights are spread over further blocks, which repeat what leads to the log-sum-exp,
// while the GPU has room for them at once; else they follow the output (96
// conversations of four-head units: 76.1 us in all, 80.4 with further blocks all the
// same).  Bound by latency: the schedule, the parts' log-sum-exps, the parts and
// logits (L2), one after the other; 12 us behind the last row of those
// conversations.  (Blocks of a head each: 128 threads 88.0, 256 95, 512 102.7; of four
// heads 512 threads 88.5 us in all, at an earlier state.)
// GQ as above: the fewer registers for four take 1.6 us off the 76.2 of 96
// conversations.
template <int D, int GQ>
__global__ void __launch_bounds__(kJoinThreads, 2)
    step_join_kernel(const __grid_constant__ StepArgs a, const __grid_constant__ Turns f) {
  constexpr int HALF = D / 2;
  __shared__ float fresh[kJoinHeads], total[kJoinHeads];
  __shared__ long long cart_at[kJoinHeads];
  __shared__ float4 acc[kJoinThreads];
  __shared__ float weight[kJoinHeads][kJoinParts];
  __shared__ const float4* place[kJoinHeads][kJoinParts];
  const int g0 = blockIdx.x * a.join_heads, b = blockIdx.y;
  const int heads = min(a.join_heads, a.Hkv - g0), nq = heads * a.G;  // query heads
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_release();
  const StepOf s = step_of(a, b);
  const int page = s.row < 0 ? -1 : page_of(a.pt, b, s.row);
  __nv_bfloat16* out = a.o + (static_cast<long long>(b) * a.Hq + g0 * a.G) * D;
  if (page < 0) {
    if (blockIdx.z > 0) {
      pdl_wait();
      return;
    }
    if (g0 == 0 && tid == 0 && __ldg(a.pt.lens + b) >= 0) atomicOr(a.status, kDevErrNoPage);
    for (int e = tid; e < nq * D; e += kJoinThreads) out[e] = __float2bfloat16_rn(0.f);
    pdl_wait();
    return;
  }
  // ---- the new token: its key as the cache holds it, its logits
  const long long from = (static_cast<long long>(b) * a.Hkv + g0) * D;
  {
    const int pos = position_of(a, b, s.row);
    float2 cs[HALF / 32];
#pragma unroll
    for (int e = 0; e < HALF / 32; ++e) cs[e] = rope_cs_turns(f.t[lane + 32 * e], pos);
    const long long at = ((static_cast<long long>(page) << a.pt.page_log2) +
                          (s.row & ((1 << a.pt.page_log2) - 1))) * a.Hkv * D + g0 * D;
    for (int q = warp; q < nq; q += kJoinThreads / 32) {
      const int h = q / a.G;
      const __nv_bfloat16* k = a.k_new + from + h * D;
      const __nv_bfloat16* x = a.q + (static_cast<long long>(b) * a.Hq + g0 * a.G + q) * D;
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < HALF / 32; ++e) {
        const int j = lane + 32 * e;
        float k0, k1, q0, q1;
        rope_pair(__bfloat162float(k[j]), __bfloat162float(k[j + HALF]), cs[e], k0, k1);
        rope_pair(__bfloat162float(x[j]), __bfloat162float(x[j + HALF]), cs[e], q0, q1);
        const __nv_bfloat16 z0 = __float2bfloat16_rn(k0), z1 = __float2bfloat16_rn(k1);
        if (q % a.G == 0 && blockIdx.z == 0) {
          a.k_pages[at + h * D + j] = z0;
          a.k_pages[at + h * D + j + HALF] = z1;
        }
        dot = fmaf(q0, __bfloat162float(z0), fmaf(q1, __bfloat162float(z1), dot));
      }
#pragma unroll
      for (int w = 16; w; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
      if (lane == 0) fresh[q] = dot * a.scale_log2;
    }
    if (tid < heads * (D / 8) && blockIdx.z == 0)
      *reinterpret_cast<uint4*>(a.v_pages + at + tid * 8) =
          __ldg(reinterpret_cast<const uint4*>(a.v_new + from + tid * 8));
  }
  // ---- parts of the cartridge, by the tile that holds the query's row: the first
  // one's place in cart_lse
  if (tid < nq) {
    const int R = b * a.G + tid % a.G, seg = (g0 + tid / a.G) * a.row_tiles + R / kTile;
    cart_at[tid] = static_cast<long long>(seg) * a.cart_parts * kTile + R % kTile;
  }
  const int unit = g0 / a.heads, cost = cost_of(tiles_of(a, s.n));
  const int groups_log2 = a.groups == 4 ? 2 : a.groups - 1;
  pdl_wait();
  // ---- and of the cached rows: those of the runs that hold the unit
  const long long start = __ldcg(a.starts + b), units = __ldcg(a.starts + a.B);
  const long long u0 = start + static_cast<long long>(unit) * cost;
  const long long chunk = max(div_units(units + a.row_ctas - 1, a.row_ctas), 1ll);
  // (a run may hold the unit's start alone)
  const int c0 = static_cast<int>(div_units(u0 + kStart, chunk));
  const int c1 = cost > 0 ? static_cast<int>(div_units(u0 + cost - 1, chunk)) : c0 - 1;
  const bool opens = u0 <= c0 * chunk;  // the unit's first tile is its run's first
  const int n_row = (c1 - c0 + 1) << groups_log2, n = n_row + a.cart_parts;
  auto row_part = [&](int q, int i) -> long long {
    const int c = c0 + (i >> groups_log2), k = i & (a.groups - 1);
    const long long slot = c0 == c1 ? 2 * a.row_ctas + static_cast<long long>(b) * a.units + unit
                           : c > c0 || opens ? 2 * c
                                             : 2 * c + 1;
    return (((slot << groups_log2) + k) * a.heads + g0 - unit * a.heads) * a.G + q;
  };
  auto place_of = [&](int q, int i) {
    return reinterpret_cast<const float4*>(
        i < n_row ? a.row_o + row_part(q, i) * D
                  : a.cart_o + ((cart_at[q] / kTile + i - n_row) * (D / 4) * kTile +
                                cart_at[q] % kTile) * 4);
  };
  auto lse_of = [&](int q, int i) {
    return i < n_row ? __ldcg(a.row_lse + row_part(q, i))
                     : __ldcg(a.cart_lse + cart_at[q] + static_cast<long long>(i - n_row) * kTile);
  };
  __syncthreads();
  for (int q = warp; q < nq; q += kJoinThreads / 32) {
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i <= n; i += 32) {
      const float x = i < n ? lse_of(q, i) : fresh[q], top = fmaxf(m, x);
      if (i < min(n, kJoinParts)) weight[q][i] = x;  // (for below)
      if (top != -INFINITY || x != x) {
        l = l * exp2_approx(m - top) + exp2_approx(x - top);
        m = top;
      }
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, w), l2 = __shfl_xor_sync(0xffffffffu, l, w);
      const float top = fmaxf(m, m2);
      l = (m == -INFINITY && l == 0.f ? 0.f : l * exp2_approx(m - top)) +
          (m2 == -INFINITY && l2 == 0.f ? 0.f : l2 * exp2_approx(m2 - top));
      m = top;
    }
    // (no logit above -inf: every weight is 0)
    const float all_of = l == 0.f ? INFINITY : m + __log2f(l);
    if (lane == 0) {
      total[q] = all_of;
    }
    // ---- the first parts' weights and places
    __syncwarp();
    for (int i = lane; i < min(n, kJoinParts); i += 32) {
      weight[q][i] = exp2_approx(weight[q][i] - all_of);
      place[q][i] = place_of(q, i);
    }
  }
  __syncthreads();
  if (blockIdx.z == 0) {
    if (a.weights && tid < heads) {  // of the new row
      float x = 0.f;
      for (int q = tid * a.G; q < (tid + 1) * a.G; ++q) x += exp2_approx(fresh[q] - total[q]);
      a.weights[(static_cast<long long>(b) * a.Hkv + g0 + tid) * a.weight_rows + s.row] = x;
    }
    const int cols = nq * (D / 4), each = max(kJoinThreads / cols, 1);
    const int turn = tid / cols;  // (below `each`, or idle; 0 where there are more columns)
    for (int col0 = 0; col0 < cols; col0 += kJoinThreads) {
      const int col = col0 + (each > 1 ? tid % cols : tid);
      const int q = col / (D / 4), j = col % (D / 4);
      const bool mine = turn < each && col < cols;
      const uint2 v2 = mine && turn == 0 ? __ldg(reinterpret_cast<const uint2*>(
                                               a.v_new + from + q / a.G * D + 4 * j))
                                         : make_uint2(0u, 0u);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = 0; i0 < n; i0 += kJoinParts) {
        if (n > kJoinParts && (col0 > 0 || i0 > 0)) {  // (the first ones are there)
          __syncthreads();
          for (int e = tid; e < nq * kJoinParts; e += kJoinThreads) {
            const int qq = e / kJoinParts, k = e % kJoinParts, i = i0 + k;
            if (i >= n) continue;
            weight[qq][k] = exp2_approx(lse_of(qq, i) - total[qq]);
            place[qq][k] = place_of(qq, i);
          }
          __syncthreads();
        }
        if (mine) {
          const int here = min(n - i0, kJoinParts);
#pragma unroll 8
          for (int k = turn; k < here; k += each) {
            const float w = weight[q][k];
            const float4 v = __ldcg(place[q][k] + (i0 + k < n_row ? j : j * kTile));
            // (a part of no weight may hold anything)
            x.x += w == 0.f ? 0.f : w * v.x;
            x.y += w == 0.f ? 0.f : w * v.y;
            x.z += w == 0.f ? 0.f : w * v.z;
            x.w += w == 0.f ? 0.f : w * v.w;
          }
        }
      }
      if (each > 1) {
        acc[tid] = x;
        __syncthreads();
        if (turn == 0)
          for (int k = 1; k < each; ++k) {
            const float4 v = acc[k * cols + col];
            x.x += v.x;
            x.y += v.y;
            x.z += v.z;
            x.w += v.w;
          }
      }
      if (mine && turn == 0) {
        const float w = exp2_approx(fresh[q] - total[q]);  // of the new token
        const float2 lo = bf16x2_to_float2(v2.x), hi = bf16x2_to_float2(v2.y);
        if (w != 0.f) {
          x.x = fmaf(w, lo.x, x.x);
          x.y = fmaf(w, lo.y, x.y);
          x.z = fmaf(w, hi.x, x.z);
          x.w = fmaf(w, hi.y, x.w);
        }
        *reinterpret_cast<uint2*>(out + q * D + 4 * j) =
            make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
      }
    }
  }
  // ---- the cached rows' weights, four rows a thread; by the blocks behind the
  // first where there are any
  if (a.weights && (gridDim.z == 1 || blockIdx.z > 0)) {
    const int parts = max(static_cast<int>(gridDim.z) - 1, 1);
    const int part = max(static_cast<int>(blockIdx.z) - 1, 0);
    const int G = a.G, per = s.n * 8;
    const bool wide = (a.weight_rows & 3) == 0;
#pragma unroll 1
    for (int e = part * kJoinThreads + tid; e < heads * per; e += parts * kJoinThreads) {
      const int h = e / per, v = (e - h * per) * 4, r = s.group(v >> 5) * 32 + (v & 31);
      const long long bg = static_cast<long long>(b) * a.Hkv + g0 + h;
      const float* lg = a.logits + bg * G * a.logit_rows + v;
      float* w = a.weights + bg * a.weight_rows + r;
      const bool all = wide && s.sees(r) && s.sees(r + 3) && (r >= s.high || r + 3 < s.low);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      float4 x[GQ];
      if (all) y = *reinterpret_cast<const float4*>(w);
#pragma unroll
      for (int q = 0; q < GQ; ++q)
        if (q < G)
          x[q] = __ldcg(
              reinterpret_cast<const float4*>(lg + static_cast<long long>(q) * a.logit_rows));
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < GQ; ++q)
        if (q < G) {
          const float t = total[h * G + q];
          sum.x += exp2_approx(x[q].x - t);
          sum.y += exp2_approx(x[q].y - t);
          sum.z += exp2_approx(x[q].z - t);
          sum.w += exp2_approx(x[q].w - t);
        }
      if (all) {
        *reinterpret_cast<float4*>(w) =
            make_float4(y.x + sum.x, y.y + sum.y, y.z + sum.z, y.w + sum.w);
      } else {
        const float part[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (s.sees(r + k)) w[k] += part[k];
      }
    }
  }
}

struct StepWs {
  size_t cart_o, cart_lse, row_o, row_lse, starts, logits, total;
  int row_tiles, key_tiles, cart_parts, cart_each, cart_ctas;
  int heads, units, groups, row_ctas, logit_rows;
};

struct CartCut {
  int parts, each;
};
// Pieces that the key tiles of a (kv head, row tile), a segment, are cut into, and
// how many a CTA has: as many SMs are the cartridge's kernel's as let both kernels
// end together, going by what they were seen to take side by side, the tables half
// full (`row_bytes`: their keys and values).  A CTA takes 16 us + 8 us a piece + 1.1
// us a tile; the rows 8 us + their bytes at 0.05 TB/s an SM, 6.3 TB/s at most; and
// a piece 0.3 us where it is joined.  The cartridge's own time counts a quarter
// beside: a table may hold far fewer rows than it names, and SMs that the rows do
// not need cost them nothing (96 conversations of up to 1500 rows, tables of 2048 to
// 32768: 68 us, 85 without that quarter).  In all, at 96 conversations (24 segments of 43
// tiles), 1 / 2 / 3 / 4 pieces of one a CTA took 87.4 / 75.3 / 78.3 / 83 us, at 200 (44
// of 22) 93 / 99 / 116 / 145, at 4 of up to 49k rows (8 of 171) 3 / 5 / 7 126 / 119.4 /
// 119.1, at one of 200 (8 of 11) 1 / 3 / 5 / 11 26.8 / 20.5 / 19.5 / 21.1.
CartCut cart_cut(int segments, int key_tiles, double row_bytes, int sms) {
  CartCut best{1, segments};
  double best_us = 0.0, best_cart = 0.0;
  const int most = std::max(2 * (sms - 1), 1);  // CTAs
  // (where a CTA has several segments anyway, whole ones: less to join)
  const int finest = segments >= 4 * most ? 1 : std::max(most / segments, 4);
  for (int n = 1; n <= std::min(key_tiles, finest); ++n) {
    const int tiles = (key_tiles + n - 1) / n, pieces = segments * n;
    for (int each = (pieces + most - 1) / most; each <= pieces; ++each) {
      const int ctas = (pieces + each - 1) / each, left = sms - (ctas + 1) / 2;
      const double cart = 16.0 + each * (8.0 + 1.1 * tiles);
      const double rows = 8.0 + row_bytes * 1e-6 / std::min(0.05 * std::max(left, 1), 6.3);
      const double us = std::max(cart, rows) + 0.25 * cart + 0.3 * n;
      if (best_us == 0.0 || us < best_us || (us == best_us && cart < best_cart)) {
        best = CartCut{n, each};
        best_us = us;
        best_cart = cart;
      }
      if (1.25 * cart > best_us) break;  // (and longer with more each)
    }
  }
  return best;
}

// (every size goes by the GPU's multiprocessors: the grids do)
StepWs step_ws(int B, int Hq, int Hkv, int d, int p, int cap, bool weights) {
  StepWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~static_cast<size_t>(255);
    return o;
  };
  const int sms = std::max(sm_count(), 1), G = Hq / Hkv;
  w.row_tiles = (B * G + kTile - 1) / kTile;
  w.key_tiles = (p + kCartKeys - 1) / kCartKeys;
  if (w.key_tiles > 0) {
    const int segments = Hkv * w.row_tiles;
    const CartCut cut =
        cart_cut(segments, w.key_tiles, static_cast<double>(B) * Hkv * d * 2 * cap, sms);
    w.cart_parts = cut.parts;
    w.cart_each = cut.each;
    w.cart_ctas = (segments * cut.parts + cut.each - 1) / cut.each;
  }
  w.heads = Hkv > 2 ? 4 : Hkv;  // (a unit's heads beyond the last one are not read)
  w.units = (Hkv + w.heads - 1) / w.heads;
  w.groups = kRowHeads / w.heads;
  w.row_ctas = std::max(sms - (w.cart_ctas + 1) / 2, 1);
  const size_t segments = static_cast<size_t>(Hkv) * w.row_tiles;
  w.cart_o = take(segments * w.cart_parts * kTile * d * 4);
  w.cart_lse = take(segments * w.cart_parts * kTile * 4);
  const size_t parts =
      (2 * static_cast<size_t>(w.row_ctas) + static_cast<size_t>(B) * w.units) * kRowHeads;
  w.row_o = take(parts * G * d * 4);
  w.row_lse = take(parts * G * 4);
  w.starts = take((static_cast<size_t>(B) + 1) * 8);
  w.logit_rows = (cap + 31) & ~31;
  w.logits = take(weights ? static_cast<size_t>(B) * Hq * w.logit_rows * 4 : 0);
  w.total = off;
  return w;
}

int check_step(int B, int window, int sinks, int Hq, int Hkv, int d, int p, float scale,
               double theta, int n_pages, int page_rows, int max_pages) {
  int rc = check_tables(B, max_pages, n_pages, page_rows);
  if (rc) return rc;
  if (Hq < 1 || Hkv < 1 || Hkv > 65535 || Hq % Hkv != 0 || Hq / Hkv > kMaxGroup ||
      (d != 64 && d != 128) || p < 0 || window < 0 || sinks < 0)
    return CART_ERR_GEOMETRY;
  if (!std::isfinite(scale) || !(scale > 0.f) || !(theta > 0.0) || !std::isfinite(theta))
    return CART_ERR_GEOMETRY;
  if (static_cast<long long>(p) + static_cast<long long>(max_pages) * page_rows >= (1ll << 24))
    return CART_ERR_GEOMETRY;
  // tiles of the cartridge's products are counted in 32 bits
  const long long row_tiles = (static_cast<long long>(B) * (Hq / Hkv) + kTile - 1) / kTile;
  if (row_tiles * Hkv > (1ll << 30) / (p / kCartKeys + 1)) return CART_ERR_GEOMETRY;
  return CART_OK;
}

template <int D>
cudaError_t launch_step(const StepArgs& a, const StepWs& w, const Turns& f, cudaStream_t st) {
  using C = CartSmem<D>;
  using L = RowSmem<D>;
  static_assert(L::kAlloc <= 232448 && C::kAlloc + L::kAlloc > 232448, "an SM for the rows alone");
  static_assert(2 * (C::kAlloc + 1024) <= 233472, "two CTAs of the cartridge's kernel an SM");
  const uint64_t page_rows = 1ull << a.pt.page_log2, row = static_cast<uint64_t>(a.Hkv) * D * 2;
  const bool small = page_rows == 16;
  RowMaps rows;
  {
    const uint64_t dims[4] = {D, page_rows, static_cast<uint64_t>(a.Hkv),
                              static_cast<uint64_t>(a.pt.n_pages)};
    const uint64_t strides[3] = {row, D * 2, row * page_rows};
    const uint32_t box[4] = {64, small ? 16u : 32u, small ? 1u : static_cast<uint32_t>(a.heads), 1};
    if (!encode_bf16_map4(&rows.k, a.k_pages, dims, strides, box) ||
        !encode_bf16_map4(&rows.v, a.v_pages, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = a.G > 4 ? set_shared_once<step_rows_kernel<D, 8>>(L::kAlloc)
                          : set_shared_once<step_rows_kernel<D, 4>>(L::kAlloc);
  if (e != cudaSuccess) return e;
  auto* rows_kernel = a.G > 4 ? step_rows_kernel<D, 8> : step_rows_kernel<D, 4>;
  rows_kernel<<<w.row_ctas, kRowThreads, L::kAlloc, st>>>(rows, a, f);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (w.cart_ctas > 0) {
    const uint64_t dims[4] = {D, static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.p), 1};
    const uint64_t strides[3] = {D * 2, row, row * a.p};
    const uint32_t box[4] = {64, 1, kCartKeys, 1};
    CartMaps cart;
    if (!encode_bf16_map4(&cart.k, a.kc, dims, strides, box) ||
        !encode_bf16_map4(&cart.v, a.vc, dims, strides, box))
      return cudaErrorInvalidValue;
    e = set_shared_once<step_cart_kernel<D>>(C::kAlloc);
    if (e == cudaSuccess)
      e = launch_dependent(step_cart_kernel<D>, dim3(w.cart_ctas), dim3(kCartThreads), C::kAlloc,
                           st, cart, a, f);
    if (e != cudaSuccess) return e;
  }
  // blocks of the joining kernel: a unit's heads each where that leaves enough of
  // them for the GPU, else one (in all, units against heads, 75.5 against 87.4 us at 96
  // conversations, 93.6 / 105.1 at 200, 134.1 / 121.5 at 4 long ones, 21.9 / 19.3 at one)
  StepArgs join = a;
  join.join_heads = a.B * a.units >= sm_count() ? a.heads : 1;
  const int across = (a.Hkv + join.join_heads - 1) / join.join_heads;
  // ... and as many for the rows' weights as the GPU takes at once, at most one for
  // every 4 * kJoinThreads rows that a table can name; none where the output takes
  // the queries' place, which they would read after it is written
  const auto at = [](const __nv_bfloat16* x) { return reinterpret_cast<uintptr_t>(x); };
  const uintptr_t bytes = static_cast<uintptr_t>(a.B) * a.Hq * D * 2;
  const bool in_place = at(a.o) < at(a.q) + bytes && at(a.q) < at(a.o) + bytes;
  const int deep =
      a.weights && !in_place
          ? std::max(1, std::min((a.cap + 4 * kJoinThreads - 1) / (4 * kJoinThreads),
                                 2 * sm_count() / (across * a.B) - 1) + 1)
          : 1;
  return launch_dependent(a.G > 4 ? step_join_kernel<D, 8> : step_join_kernel<D, 4>,
                          dim3(across, a.B, deep), dim3(kJoinThreads), 0, st, join, f);
}

}  // namespace
}  // namespace cart

using namespace cart;

extern "C" {

size_t cart_attn_decode_paged_workspace_size(int B, int Hq, int Hkv, int d, int p, int page_rows,
                                             int max_pages, int weights) {
  if (check_step(B, 0, 0, Hq, Hkv, d, p, 1.f, 1.0, 1, page_rows, max_pages)) return 0;
  return step_ws(B, Hq, Hkv, d, p, max_pages * page_rows, weights != 0).total;
}

int cart_attn_decode_paged(int B, int window, int sinks, int Hq, int Hkv, int d, int p, float scale,
                           double rope_theta, const void* q, const void* k_new, const void* v_new,
                           const void* kc, const void* vc, void* k_pages, void* v_pages,
                           int n_pages, int page_rows, const int* table, int max_pages,
                           const int* lens, const int* pos, float* weights, int weight_rows,
                           void* o, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_step(B, window, sinks, Hq, Hkv, d, p, scale, rope_theta, n_pages, page_rows,
                      max_pages);
  if (rc) return rc;
  if (weights && weight_rows < max_pages * page_rows) return CART_ERR_GEOMETRY;
  const void* ptrs[] = {q, k_new, v_new, k_pages, v_pages, o};
  for (const void* ptr : ptrs)
    if (!aligned_to(ptr, 16)) return CART_ERR_POINTER;
  if (p > 0 && (!aligned_to(kc, 16) || !aligned_to(vc, 16))) return CART_ERR_POINTER;
  if (!aligned_to(table, 4) || !aligned_to(lens, 4) || (pos && !aligned_to(pos, 4)) ||
      (weights && !aligned_to(weights, 16)))
    return CART_ERR_POINTER;
  const StepWs w = step_ws(B, Hq, Hkv, d, p, max_pages * page_rows, weights != nullptr);
  if (!aligned_to(workspace, 16) || workspace_bytes < w.total) return CART_ERR_WORKSPACE;
  rc = check_device();
  if (rc) return rc;
  char* ws = static_cast<char*>(workspace);
  StepArgs a{};
  a.pt = PageTable{table, lens, max_pages, n_pages, page_log2_of(page_rows)};
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.p = p;
  a.window = std::min(window, kMostPlaces);
  a.sinks = std::min(sinks, kMostPlaces);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.pos = pos;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_new = static_cast<const __nv_bfloat16*>(k_new);
  a.v_new = static_cast<const __nv_bfloat16*>(v_new);
  a.kc = static_cast<const __nv_bfloat16*>(kc);
  a.vc = static_cast<const __nv_bfloat16*>(vc);
  a.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  a.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.weights = weights;
  a.weight_rows = weight_rows;
  a.status = device_status_ptr();
  a.row_tiles = w.row_tiles;
  a.key_tiles = w.key_tiles;
  a.cart_parts = w.cart_parts;
  a.cart_each = w.cart_each;
  a.cart_o = reinterpret_cast<float*>(ws + w.cart_o);
  a.cart_lse = reinterpret_cast<float*>(ws + w.cart_lse);
  a.heads = w.heads;
  a.units = w.units;
  a.groups = w.groups;
  a.row_ctas = w.row_ctas;
  a.starts = reinterpret_cast<long long*>(ws + w.starts);
  a.row_o = reinterpret_cast<float*>(ws + w.row_o);
  a.row_lse = reinterpret_cast<float*>(ws + w.row_lse);
  a.cap = max_pages * page_rows;
  a.logit_rows = w.logit_rows;
  a.logits = weights ? reinterpret_cast<float*>(ws + w.logits) : nullptr;
  const RopeFreqs f = make_rope_freqs(d, rope_theta);
  Turns turns{};
  for (int j = 0; j < d / 2; ++j) turns.t[j] = f.turns[j];
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope tr("decode_paged", st);
  const cudaError_t e =
      d == 128 ? launch_step<128>(a, w, turns, st) : launch_step<64>(a, w, turns, st);
  return e == cudaSuccess ? CART_OK : CART_ERR_CUDA;
}

}  // extern "C"
