// weights.cu -- the attention weight that each key gets from a conversation's
// last queries, by the log-sum-exps that their attention came with
// (cart_attn_weights).
//
// With q~ = R(position) q and the cache's keys k~, the weight of key j is the
// sum over the queries i that see it and the heads of its group of
// exp(scale * q~_i . k~_j - lse_i): no maximum, no sum to wait for.  The result
// is f32 and the keys are bf16, so q~ enters as three bf16 terms that hold all
// of its 24 bits: S^T = K (Q_0 + Q_1 + Q_2)^T, three products of one key tile
// into one accumulator (two terms leave 2.8e-6 of the weights).
//
//   prep    the terms [3][B, Hkv, columns, d] and -lse * log2(e) [B, Hkv,
//           columns], column i * G + hh, padded to whole tiles of 128; one more
//           block adds up the schedule.
//   weigh   persistent, one CTA per SM.  A segment is 128 columns of one
//           (conversation, kv head) and the key tiles that they see; its Q terms
//           stay in shared memory (96 KB at d = 128) while its key tiles stream
//           by (the other way round a step would load 96 KB of Q terms for 1536
//           clocks of products, all that an SM's way to L2 has).  All segments'
//           tiles, one after the other, are cut into equal runs, one per CTA,
//           from the lengths on the device.  Warps 0-3 and 4-7 take every other
//           tile, a thread its key: TMEM lane = key, 128 columns, sums in
//           registers.
//   finish  where a (conversation, kv head) has more than 128 columns, or a
//           window leaves tiles out: the columns' parts added up in order.
//
// Bound by the tensor pipe.  32 heads over 8, d 128: the last 32 queries of 64
// conversations over 4096 and up to 1031 keys take 164 us, weigh 155 of them (the
// three products of the keys that are seen at 1470 TFLOP/s); 1024 queries of 4 over
// 2048 and up to 1200 keys 141 us: prep 18 (100 MB of terms written), weigh 120
// (1460 TFLOP/s), finish 9.
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

constexpr int kTerms = 3;
// (a window or sinks beyond every place are that many)
constexpr int kMostPlaces = 1 << 25;

struct WeighArgs {
  PageTable pt;
  int B, T, Hq, Hkv, G, p, window, sinks, accumulate;
  float scale_log2;
  const int* pos;  // null: p + lens - T
  const __nv_bfloat16* q;
  const float* lse;  // [B, Hq, T]
  float *weights, *cart;
  int weight_rows;
  int n_qt;                // column tiles of a (conversation, kv head)
  __nv_bfloat16* terms;    // [3][B, Hkv, n_qt * 128, d]
  long long term_elems;
  float* nlse2;            // [B, Hkv, n_qt * 128]
  long long* starts;       // [B + 1]: units of the schedule before each conversation
  float* part;             // [B, Hkv, n_qt, slots]; null: written at once
  int n_ct, slots;         // cartridge tiles; 128 * (all key tiles a table can name)
  uint32_t* status;
};

// Key tiles that queries at places x0 .. x1 see, as four runs: cartridge tiles
// below sk_c and from lo_c to n_ct, own tiles below sk_r and from lo_r to hi_r.
struct Tiles {
  int sk_c, lo_c, n_ct, sk_r, lo_r, hi_r, n;
  __device__ __forceinline__ bool own(int t) const { return t >= sk_c + n_ct - lo_c; }
  __device__ __forceinline__ int at(int t) const {  // number of tile t among its kind
    const int c = sk_c + n_ct - lo_c;
    if (t < c) return t < sk_c ? t : lo_c + t - sk_c;
    return t - c < sk_r ? t - c : lo_r + t - c - sk_r;
  }
  __device__ __forceinline__ bool has(bool own, int i) const {
    return own ? i < sk_r || (i >= lo_r && i < hi_r) : i < sk_c || i >= lo_c;
  }
};
__device__ __forceinline__ Tiles tiles_of(const WeighArgs& a, int x0, int x1) {
  Tiles k;
  const int low = a.window > 0 ? max(x0 - a.window + 1, 0) : 0;  // first place in the window
  k.n_ct = a.n_ct;
  k.lo_c = min(low / kTile, k.n_ct);
  k.sk_c = min((min(a.sinks, a.p) + kTile - 1) / kTile, k.lo_c);
  k.hi_r = (x1 - a.p) / kTile + 1;
  k.lo_r = low > a.p ? (low - a.p) / kTile : 0;
  k.sk_r = a.sinks > a.p ? min((a.sinks - a.p + kTile - 1) / kTile, k.lo_r) : 0;
  k.n = k.sk_c + k.n_ct - k.lo_c + k.sk_r + k.hi_r - k.lo_r;
  return k;
}
// The tiles of column tile qt of a conversation that holds `rows` rows (n == 0:
// none of its queries is there).
__device__ __forceinline__ Tiles column_tiles(const WeighArgs& a, int rows, int qt) {
  const int i0 = max(qt * kTile / a.G, a.T - rows);
  const int i1 = (min((qt + 1) * kTile, a.T * a.G) - 1) / a.G;
  if (i0 > i1 || rows <= 0) {
    Tiles none{};
    return none;
  }
  return tiles_of(a, a.p + rows - a.T + i0, a.p + rows - a.T + i1);
}
// A segment of n tiles is n + kStartUnits units of the schedule (0 / 1 / 2 / 3 / 4:
// whole prompts 150.5 / 147.4 / 146.9 / 147.2 / 145.8 us, 32 queries of 64 conversations
// 170.5 / 170.1 / 170.9 / 169.3 / 168.8).
constexpr int kStartUnits = 4;
__device__ __forceinline__ int segment_units(int n) { return n > 0 ? n + kStartUnits : 0; }

struct Turns {
  float2 t[kMaxHeadDim / 2];
};

// ----------------------------------------------------------------- prep ----
constexpr int kPrepThreads = 256;
constexpr int kPrepQueries = 4;  // per block

// Units before each conversation, by one block.
__device__ __forceinline__ void write_starts(const WeighArgs& a) {
  __shared__ long long sums[kPrepThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPrepThreads) {
    const int b = b0 + tid, rows = b < a.B ? held_rows(a.pt, b) : 0;
    long long n = 0;
    for (int qt = 0; qt < a.n_qt && rows > 0; ++qt)
      n += segment_units(column_tiles(a, rows, qt).n);
    n *= a.Hkv;
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long all = 0, mine = before;
    for (int w = 0; w < kPrepThreads / 32; ++w) {
      mine += w < warp ? sums[w] : 0;
      all += sums[w];
    }
    if (b < a.B) a.starts[b] = mine + x - n;
    before += all;
  }
  if (tid == 0) a.starts[a.B] = before;
}

// Block 0: the schedule; the others four queries of a conversation each.
// Queries that are not there, and the padding, are masked where they are used.
template <int D>
__global__ void __launch_bounds__(kPrepThreads)
    weigh_prep_kernel(const __grid_constant__ WeighArgs a, const __grid_constant__ Turns f) {
  constexpr int HALF = D / 2;
  pdl_release();
  if (blockIdx.x == 0) {
    write_starts(a);
    return;
  }
  __shared__ float2 cs[kPrepQueries][HALF];
  const int groups = (a.T + kPrepQueries - 1) / kPrepQueries, tid = threadIdx.x;
  const int b = (blockIdx.x - 1) / groups, t0 = (blockIdx.x - 1) % groups * kPrepQueries;
  const int rows = max(held_rows(a.pt, b), 0), nt = min(kPrepQueries, a.T - t0);
  // (written by nobody else: no query looks at the cartridge)
  if (rows == 0 && t0 == 0 && !a.part && !a.accumulate)
    for (long long e = tid; e < static_cast<long long>(a.Hkv) * a.p; e += kPrepThreads)
      a.cart[static_cast<long long>(b) * a.Hkv * a.p + e] = 0.f;
  if (t0 + nt <= a.T - rows) return;  // none of them is there
  const long long first =
      a.pos ? static_cast<long long>(__ldg(a.pos + b)) : static_cast<long long>(a.p) + rows - a.T;
  for (int e = tid; e < nt * HALF; e += kPrepThreads) {
    const int t = e / HALF, j = e % HALF;
    cs[t][j] = rope_cs_turns(
        f.t[j], static_cast<int>(min(max(first + t0 + t, 0ll), (1ll << 24) - 1)));
  }
  __syncthreads();
  constexpr int kPer = HALF / 8;  // pieces of a head's row: eight pairs
  for (int e = tid; e < nt * a.Hq * kPer; e += kPrepThreads) {
    const int j0 = e % kPer * 8, th = e / kPer, t = th / a.Hq, h = th % a.Hq;
    const __nv_bfloat16* x =
        a.q + ((static_cast<long long>(b) * a.T + t0 + t) * a.Hq + h) * D + j0;
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(x));
    const uint4 hi = __ldg(reinterpret_cast<const uint4*>(x + HALF));
    const uint32_t pl[4] = {lo.x, lo.y, lo.z, lo.w}, ph[4] = {hi.x, hi.y, hi.z, hi.w};
    uint32_t yl[kTerms][4], yh[kTerms][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 fl = bf16x2_to_float2(pl[k]), fh = bf16x2_to_float2(ph[k]);
      float2 u, w;
      rope_pair(fl.x, fh.x, cs[t][j0 + 2 * k], u.x, w.x);
      rope_pair(fl.y, fh.y, cs[t][j0 + 2 * k + 1], u.y, w.y);
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
    const long long col = (static_cast<long long>(b) * a.Hkv + h / a.G) * a.n_qt * kTile +
                          (t0 + t) * a.G + h % a.G;
#pragma unroll
    for (int s = 0; s < kTerms; ++s) {
      __nv_bfloat16* y = a.terms + s * a.term_elems + col * D + j0;
      *reinterpret_cast<uint4*>(y) = make_uint4(yl[s][0], yl[s][1], yl[s][2], yl[s][3]);
      *reinterpret_cast<uint4*>(y + HALF) = make_uint4(yh[s][0], yh[s][1], yh[s][2], yh[s][3]);
    }
    if (j0 == 0) {
      const float lse = __ldg(a.lse + (static_cast<long long>(b) * a.Hq + h) * a.T + t0 + t);
      // (-inf: every logit was, and the query gives no weight)
      a.nlse2[col] = lse == -INFINITY ? -INFINITY : -1.4426950408889634f * lse;
    }
  }
}

// ---------------------------------------------------------------- weigh ----
constexpr int kWeighThreads = 320;  // two warpgroups of keys, TMA warp, MMA warp
constexpr int kWeighStages = 4;     // key tiles
constexpr int kWeighSlots = 2;      // pieces published ahead

template <int D>
struct WeighSmem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kTerms * kTileBytes;
  static constexpr int kVec = kK + kWeighStages * kTileBytes;  // -lse2 of a piece's columns
  static constexpr int kBytes = kVec + kWeighSlots * 512;
  static constexpr int kAlloc = kBytes + 1024;  // slack for 1024-byte alignment
  static_assert(kAlloc <= 232448 - 512, "shared memory above the limit");
};

enum WeighBar {
  kWQFull = 0,                      // TMA: a piece's Q terms
  kWQEmpty,                         // its last product has read them
  kWKFull0,
  kWKEmpty0 = kWKFull0 + kWeighStages,
  kWSFull0 = kWKEmpty0 + kWeighStages,  // S^T of buffer x is in TMEM
  kWSEmpty0 = kWSFull0 + 4,             // its warpgroup has read it (4 warps)
  kWPieceFull0 = kWSEmpty0 + 4,         // piece and -lse2 of slot x are there
  kWPieceEmpty0 = kWPieceFull0 + kWeighSlots,  // the MMA warp and 8 warps are done with it
  kWDrain = kWPieceEmpty0 + kWeighSlots,
  kWBars
};

// Tiles t0 .. t0 + n - 1 of a segment (n == 0: no more).
struct WeighPiece {
  int b, g, qt, t0, n;
};
struct WeighShared {
  uint64_t bars[kWBars];
  uint32_t tmem;
  int abort;
  WeighPiece piece[kWeighSlots];
};

struct WeighMaps {
  CUtensorMap q[kTerms], kc, kp;
};

template <int D>
__global__ void __launch_bounds__(kWeighThreads, 1)
    weigh_kernel(const __grid_constant__ WeighMaps maps, const __grid_constant__ WeighArgs a) {
  using L = WeighSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ WeighShared sh;
  uint64_t* const bars = sh.bars;
  float* const vec = reinterpret_cast<float*>(smem + L::kVec);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t abort_s = smem_u32(&sh.abort);
  if (threadIdx.x == 0) {
    sh.abort = 0;
    mbar_init(&bars[kWQFull], 1);
    mbar_init(&bars[kWQEmpty], 1);
    for (int s = 0; s < kWeighStages; ++s) {
      mbar_init(&bars[kWKFull0 + s], 1);
      mbar_init(&bars[kWKEmpty0 + s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars[kWSFull0 + s], 1);
      mbar_init(&bars[kWSEmpty0 + s], 4);
    }
    for (int s = 0; s < kWeighSlots; ++s) {
      mbar_init(&bars[kWPieceFull0 + s], 1);
      mbar_init(&bars[kWPieceEmpty0 + s], 9);
    }
    mbar_init(&bars[kWDrain], 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();  // the terms and the schedule; nothing above touches global memory

  if (warp == 8) {
    // ------------------------------------------------------------ producer --
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, kDevErrTimeoutTma));
    };
    const long long total = __ldcg(a.starts + a.B);
    const long long chunk = (total + gridDim.x - 1) / gridDim.x;
    const long long lo = min(blockIdx.x * chunk, total), hi = min(lo + chunk, total);
    int left = static_cast<int>(min(hi - lo, 0x7fffffffll));  // units to go
    // the conversation, column tile, kv head and unit of it that the run starts in
    int b = 0, qt = 0, g = 0, unit = 0;
    if (left > 0) {
      int z = a.B;
      while (z - b > 1) {  // the last conversation that starts at or before lo
        const int mid = (b + z) >> 1;
        if (__ldcg(a.starts + mid) <= lo)
          b = mid;
        else
          z = mid;
      }
      long long off = lo - __ldcg(a.starts + b);
      const int rows = held_rows(a.pt, b);
      for (; qt < a.n_qt; ++qt) {
        const int u = segment_units(column_tiles(a, rows, qt).n);
        const long long all = static_cast<long long>(u) * a.Hkv;
        if (off < all) {
          g = static_cast<int>(off / u);
          unit = static_cast<int>(off - static_cast<long long>(g) * u);
          break;
        }
        off -= all;
      }
    }
    int it = 0, step = 0, q_issued = 0, k_issued = 0;
    bool ok = true;
    while (ok) {
      // the next piece of the run that has tiles
      WeighPiece pc{0, 0, 0, 0, 0};
      Tiles tl{};
      int rows = 0;
      while (left > 0 && b < a.B) {
        rows = held_rows(a.pt, b);
        tl = qt < a.n_qt ? column_tiles(a, rows, qt) : Tiles{};
        const int u = segment_units(tl.n);
        if (u == 0) {  // nothing here: the next column tile, or conversation
          g = 0;
          unit = 0;
          if (++qt >= a.n_qt) {
            qt = 0;
            ++b;
          }
          continue;
        }
        const int end = min(u, unit + left), t0 = max(unit - kStartUnits, 0);
        pc = WeighPiece{b, g, qt, t0, end - kStartUnits - t0};
        left -= end - unit;
        unit = 0;
        if (++g == a.Hkv) {
          g = 0;
          if (++qt >= a.n_qt) {
            qt = 0;
            ++b;
          }
        }
        if (pc.n > 0) break;
      }
      const int sl = it % kWeighSlots;
      if (it >= kWeighSlots) {
        ok = wait(&bars[kWPieceEmpty0 + sl], (it / kWeighSlots - 1) & 1);
        if (!ok) break;
      }
      const long long bg = static_cast<long long>(pc.b) * a.Hkv + pc.g;
      const long long col = bg * a.n_qt * kTile + static_cast<long long>(pc.qt) * kTile;
      if (pc.n <= 0) pc.n = 0;
      if (lane == 0) {
        sh.piece[sl] = pc;
        mbar_arrive_expect_tx(&bars[kWPieceFull0 + sl], pc.n ? 512 : 0);
        if (pc.n) bulk_load(vec + sl * kTile, a.nlse2 + col, 512, &bars[kWPieceFull0 + sl]);
      }
      ++it;
      if (pc.n == 0) break;
      if (q_issued > 0) {
        ok = wait(&bars[kWQEmpty], (q_issued - 1) & 1);
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[kWQFull], kTerms * L::kTileBytes);
        for (int s = 0; s < kTerms; ++s)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(smem + L::kQ + s * L::kTileBytes + h * 16384, &maps.q[s], &bars[kWQFull],
                        h * 64, 0, static_cast<int>(col), 0);
      }
      ++q_issued;
      const int per_log2 = 7 - a.pt.page_log2;  // pages of a tile
      for (int t = pc.t0; t < pc.t0 + pc.n && ok; ++t, ++step) {
        const bool own = tl.own(t);
        const int row0 = tl.at(t) * kTile;
        // the pages of the tile's rows, a lane each
        int page = -1;
        if (own && lane < 1 << per_log2) {
          const int r = row0 + (lane << a.pt.page_log2);
          if (r < rows) page = page_of(a.pt, pc.b, r);
        }
        const unsigned there = __ballot_sync(0xffffffffu, page >= 0);
        const int st = step % kWeighStages;
        if (step >= kWeighStages) {
          ok = wait(&bars[kWKEmpty0 + st], (step / kWeighStages - 1) & 1);
          if (!ok) break;
        }
        uint8_t* dst = smem + L::kK + st * L::kTileBytes;
        if (lane == 0)
          mbar_arrive_expect_tx(&bars[kWKFull0 + st],
                                own ? (__popc(there) * L::kTileBytes) >> per_log2 : L::kTileBytes);
        __syncwarp();
        if (own) {
          if (page >= 0)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(dst + h * 16384 + (lane << a.pt.page_log2) * 128, &maps.kp,
                          &bars[kWKFull0 + st], h * 64, pc.g, 0, page);
        } else if (lane == 0) {
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(dst + h * 16384, &maps.kc, &bars[kWKFull0 + st], h * 64, pc.g, row0, 0);
        }
        __syncwarp();
        k_issued = step + 1;
      }
    }
    pdl_release();
    if (!ok && lane == 0) {
      // copies in flight get a bounded chance to land before the CTA ends
      if (q_issued > 0) mbar_wait(&bars[kWQFull], (q_issued - 1) & 1, 0u, nullptr, 0);
      for (int t = max(k_issued - kWeighStages, 0); t < k_issued; ++t)
        mbar_wait(&bars[kWKFull0 + t % kWeighStages], (t / kWeighStages) & 1, 0u, nullptr, 0);
      for (int t = max(it - kWeighSlots, 0); t < it; ++t)
        mbar_wait(&bars[kWPieceFull0 + t % kWeighSlots], (t / kWeighSlots) & 1, 0u, nullptr, 0);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ----------------------------------------------------------------- MMA --
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_s, a.status, kDevErrTimeoutMma));
    };
    const uint32_t id = idesc_bf16(128, 128, false, false);
    const uint64_t dQ = sdesc_sw128(smem_u32(smem + L::kQ), 16u, 1024u);
    const uint64_t dK = sdesc_sw128(smem_u32(smem + L::kK), 16u, 1024u);
    int step = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int sl = it % kWeighSlots;
      ok = wait(&bars[kWPieceFull0 + sl], (it / kWeighSlots) & 1);
      if (!ok) break;
      const int n = vld(sh.piece[sl].n);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kWPieceEmpty0 + sl]);
      if (n == 0) break;
      ok = wait(&bars[kWQFull], it & 1);
      for (int t = 0; t < n && ok; ++t, ++step) {
        const int st = step % kWeighStages, x = step & 3;
        ok = wait(&bars[kWKFull0 + st], (step / kWeighStages) & 1) &&
             (step < 4 || wait(&bars[kWSEmpty0 + x], ((step >> 2) - 1) & 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t dk = desc_add(dK, st * L::kTileBytes);
        // the smallest terms first
#pragma unroll
        for (int s = kTerms - 1; s >= 0; --s)
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
            umma_bf16_ss_w(tmem + x * 128, desc_add(dk, off),
                           desc_add(dQ, s * L::kTileBytes + off), id,
                           s == kTerms - 1 && k == 0 ? 0u : 1u);
          }
        umma_commit_w(&bars[kWSFull0 + x]);
        umma_commit_w(&bars[kWKEmpty0 + st]);
      }
      if (ok) umma_commit_w(&bars[kWQEmpty]);
    }
    // every product issued above completes before the CTA ends
    umma_commit_w(&bars[kWDrain]);
    mbar_wait(&bars[kWDrain], 0, 0u, nullptr, 0);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- keys --
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu,
                        mbar_wait(bar, parity, abort_s, a.status, kDevErrTimeoutSoftmax));
    };
    const int wg = warp >> 2, row = threadIdx.x & 127;  // TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
    int step = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int sl = it % kWeighSlots;
      ok = wait(&bars[kWPieceFull0 + sl], (it / kWeighSlots) & 1);
      if (!ok) break;
      const WeighPiece pc = {vld(sh.piece[sl].b), vld(sh.piece[sl].g), vld(sh.piece[sl].qt),
                             vld(sh.piece[sl].t0), vld(sh.piece[sl].n)};
      if (pc.n == 0) break;
      const int rows = held_rows(a.pt, pc.b);
      const Tiles tl = column_tiles(a, rows, pc.qt);
      const long long bg = static_cast<long long>(pc.b) * a.Hkv + pc.g;
      const int x_first = a.p + rows - a.T;  // place of query 0
      const uint32_t vec_s = smem_u32(vec + sl * kTile);
      for (int t = 0; t < pc.n && ok; ++t) {
        const int s = step + t;
        if ((s & 1) != wg) continue;
        const bool own = tl.own(pc.t0 + t);
        const int r = tl.at(pc.t0 + t) * kTile + row, y = own ? a.p + r : r;
        const bool key = own ? r < rows : r < a.p;
        const bool there = key && (!own || page_of(a.pt, pc.b, r) >= 0);
        // columns from c0 to c1 - 1 see the key
        const int i0 = max(max(y - x_first, 0), a.T - rows);
        int i1 = a.T;
        if (a.window > 0 && y >= a.sinks) i1 = min(i1, y + a.window - x_first);
        const int c0 = max(min(i0, a.T) * a.G - pc.qt * kTile, 0);
        const int c1 = there ? min(max(i1, 0) * a.G - pc.qt * kTile, kTile) : 0;
        const bool masked = __any_sync(0xffffffffu, c0 > 0 || c1 < kTile);
        const int x = s & 3;
        ok = wait(&bars[kWSFull0 + x], (s >> 2) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ts = tmem + x * 128 + lane_off;
        float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
        uint32_t v[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, v[q]);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_reg_fence(v[q]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kWSEmpty0 + x]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t(&u)[32] = v[q];
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 l = lds128(vec_s + (32 * q + c) * 4);
            const float2 e0 = __ffma2_rn(u2f2(u[c], u[c + 1]), sc2, make_float2(l.x, l.y));
            const float2 e1 = __ffma2_rn(u2f2(u[c + 2], u[c + 3]), sc2, make_float2(l.z, l.w));
            float2 w0 = make_float2(exp2_approx(e0.x), exp2_approx(e0.y));
            float2 w1 = make_float2(exp2_approx(e1.x), exp2_approx(e1.y));
            if (masked) {
              const int k = 32 * q + c;
              w0.x = k >= c0 && k < c1 ? w0.x : 0.f;
              w0.y = k + 1 >= c0 && k + 1 < c1 ? w0.y : 0.f;
              w1.x = k + 2 >= c0 && k + 2 < c1 ? w1.x : 0.f;
              w1.y = k + 3 >= c0 && k + 3 < c1 ? w1.y : 0.f;
            }
            sum[(c >> 2) & 1] = __fadd2_rn(sum[(c >> 2) & 1], w0);
            sum[2 + ((c >> 2) & 1)] = __fadd2_rn(sum[2 + ((c >> 2) & 1)], w1);
          }
        }
        const float2 s01 = __fadd2_rn(sum[0], sum[1]), s23 = __fadd2_rn(sum[2], sum[3]);
        const float w = (s01.x + s01.y) + (s23.x + s23.y);
        if (key) {
          if (a.part) {
            a.part[(bg * a.n_qt + pc.qt) * a.slots + (own ? a.n_ct * kTile : 0) + r] = w;
          } else {
            float* to = own ? a.weights + bg * a.weight_rows + r : a.cart + bg * a.p + r;
            *to = a.accumulate && (!own || r < rows - a.T) ? *to + w : w;
          }
        }
        __syncwarp();
      }
      step += pc.n;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kWPieceEmpty0 + sl]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// --------------------------------------------------------------- finish ----
// A key per thread: its parts by column tile, in order.  Bound by the parts' reads:
// the column tiles that see a key tile are worked out once a block.
constexpr int kFinishThreads = 2 * kTile;

__global__ void __launch_bounds__(kFinishThreads)
    weigh_finish_kernel(const __grid_constant__ WeighArgs a) {
  // what column tile q0 + e sees of the block's key tiles
  __shared__ uint8_t sees[kFinishThreads];
  pdl_wait();
  const int tid = threadIdx.x, slot0 = blockIdx.x * kFinishThreads, slot = slot0 + tid;
  const int g = blockIdx.y, b = blockIdx.z;
  const int rows = max(held_rows(a.pt, b), 0);
  const int first = slot0 / kTile;  // key tiles: the cartridge's, then the rows'
  const bool own = slot >= a.n_ct * kTile;
  const int r = own ? slot - a.n_ct * kTile : slot;
  const bool there = r < (own ? rows : a.p);
  const long long bg = static_cast<long long>(b) * a.Hkv + g;
  const int mine = 1 << (slot / kTile - first);
  float w = 0.f;
  for (int q0 = 0; q0 < a.n_qt; q0 += kFinishThreads) {
    const int n = min(a.n_qt - q0, kFinishThreads);
    __syncthreads();
    if (tid < n) {
      const Tiles tl = column_tiles(a, rows, q0 + tid);
      int bits = 0;
      for (int k = 0; k < kFinishThreads / kTile; ++k) {
        const int t = first + k;
        if (tl.n > 0 && tl.has(t >= a.n_ct, t >= a.n_ct ? t - a.n_ct : t)) bits |= 1 << k;
      }
      sees[tid] = static_cast<uint8_t>(bits);
    }
    __syncthreads();
    if (!there) continue;
    const float* part = a.part + (bg * a.n_qt + q0) * a.slots + slot;
#pragma unroll 8
    for (int e = 0; e < n; ++e)
      if (sees[e] & mine) w += __ldcg(part + static_cast<long long>(e) * a.slots);
  }
  if (!there) return;
  float* to = own ? a.weights + bg * a.weight_rows + r : a.cart + bg * a.p + r;
  *to = a.accumulate && (!own || r < rows - a.T) ? *to + w : w;
}

struct WeighWs {
  size_t terms, nlse2, starts, part, total;
  long long term_elems;
  int n_qt, n_ct, slots;
  bool parts;
};
WeighWs weigh_ws(int B, int T, int Hq, int Hkv, int d, int p, int cap, bool window) {
  WeighWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~static_cast<size_t>(255);
    return o;
  };
  w.n_qt = static_cast<int>((static_cast<long long>(T) * (Hq / Hkv) + kTile - 1) / kTile);
  w.n_ct = (p + kTile - 1) / kTile;
  w.slots = (w.n_ct + (cap + kTile - 1) / kTile) * kTile;
  w.parts = w.n_qt > 1 || window;
  const size_t columns = static_cast<size_t>(B) * Hkv * w.n_qt * kTile;
  w.term_elems = static_cast<long long>(columns) * d;
  w.terms = take(kTerms * columns * d * 2);
  w.nlse2 = take(columns * 4);
  w.starts = take((static_cast<size_t>(B) + 1) * 8);
  // (taken whether or not this call needs parts: the size is asked for without
  // the window)
  w.part = take(static_cast<size_t>(B) * Hkv * w.n_qt * w.slots * 4);
  w.total = off;
  return w;
}

int check_weigh(int B, int T, int window, int sinks, int Hq, int Hkv, int d, int p, float scale,
                double theta, int n_pages, int page_rows, int max_pages) {
  int rc = check_tables(B, max_pages, n_pages, page_rows);
  if (rc) return rc;
  if (T < 1 || T >= (1 << 24) || static_cast<long long>(B) * T > 0x3fffffff || Hq < 1 || Hkv < 1 ||
      Hkv > 65535 || Hq % Hkv != 0 || Hq / Hkv > 8 || (d != 64 && d != 128) || p < 0 ||
      window < 0 || sinks < 0)
    return CART_ERR_GEOMETRY;
  const long long tiles = (static_cast<long long>(T) * (Hq / Hkv) + kTile - 1) / kTile;
  if (tiles * kTile > 0x7fffffffll / Hkv / B) return CART_ERR_GEOMETRY;
  if (!std::isfinite(scale) || !(scale > 0.f) || !(theta > 0.0) || !std::isfinite(theta))
    return CART_ERR_GEOMETRY;
  if (static_cast<long long>(p) + static_cast<long long>(max_pages) * page_rows >= (1ll << 24))
    return CART_ERR_GEOMETRY;
  return CART_OK;
}

template <int D>
cudaError_t launch_weigh(const WeighArgs& a, const void* kc, const void* k_pages, const Turns& f,
                         cudaStream_t st) {
  using L = WeighSmem<D>;
  cudaError_t e = set_smem_once<weigh_kernel<D>>(L::kAlloc);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms < 1) return cudaErrorInvalidValue;
  // [blocks, rows, heads, d] as (d, heads, rows, blocks), rows by the box
  auto rows_map = [&](CUtensorMap* m, const void* base, uint64_t blocks, uint64_t rows,
                      uint64_t heads, uint32_t box_rows) {
    const uint64_t dims[4] = {D, heads, rows, blocks};
    const uint64_t strides[3] = {D * 2, heads * D * 2, rows * heads * D * 2};
    const uint32_t box[4] = {64, 1, box_rows, 1};
    return encode_bf16_map4(m, base, dims, strides, box);
  };
  WeighMaps maps;
  const uint64_t columns = static_cast<uint64_t>(a.B) * a.Hkv * a.n_qt * kTile;
  for (int s = 0; s < kTerms; ++s)
    if (!rows_map(&maps.q[s], a.terms + s * a.term_elems, 1, columns, 1, kTile))
      return cudaErrorInvalidValue;
  const uint32_t page_rows = 1u << a.pt.page_log2;
  if (!rows_map(&maps.kp, k_pages, a.pt.n_pages, page_rows, a.Hkv, page_rows))
    return cudaErrorInvalidValue;
  maps.kc = maps.kp;  // (never loaded where there is no cartridge tile)
  if (a.p > 0 && !rows_map(&maps.kc, kc, 1, a.p, a.Hkv, kTile)) return cudaErrorInvalidValue;
  const int groups = (a.T + kPrepQueries - 1) / kPrepQueries;
  weigh_prep_kernel<D><<<1 + a.B * groups, kPrepThreads, 0, st>>>(a, f);
  e = cudaGetLastError();
  // no more CTAs than key tiles a batch can have
  const long long most = static_cast<long long>(a.B) * a.Hkv * a.n_qt * (a.slots / kTile);
  if (e == cudaSuccess)
    e = launch_dependent(weigh_kernel<D>,
                         dim3(static_cast<unsigned>(std::min<long long>(sms, most))),
                         dim3(kWeighThreads), L::kAlloc, st, maps, a);
  if (e == cudaSuccess && a.part)
    e = launch_dependent(weigh_finish_kernel, dim3((a.slots + kFinishThreads - 1) / kFinishThreads, a.Hkv, a.B),
                         dim3(kFinishThreads), 0,
                         st, a);
  return e;
}

}  // namespace
}  // namespace cart

using namespace cart;

extern "C" {

size_t cart_attn_weights_workspace_size(int B, int queries, int Hq, int Hkv, int d, int p,
                                        int page_rows, int max_pages) {
  if (check_weigh(B, queries, 0, 0, Hq, Hkv, d, p, 1.f, 1.0, 1, page_rows, max_pages)) return 0;
  return weigh_ws(B, queries, Hq, Hkv, d, p, max_pages * page_rows, true).total;
}

int cart_attn_weights(int B, int queries, int window, int sinks, int Hq, int Hkv, int d, int p,
                      float scale, double rope_theta, const void* q, const float* lse,
                      const void* kc, const void* k_pages, int n_pages, int page_rows,
                      const int* table, int max_pages, const int* lens, const int* pos,
                      int accumulate, float* weights, int weight_rows, float* cart,
                      void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_weigh(B, queries, window, sinks, Hq, Hkv, d, p, scale, rope_theta, n_pages,
                       page_rows, max_pages);
  if (rc) return rc;
  if (weight_rows < max_pages * page_rows || (accumulate != 0 && accumulate != 1))
    return CART_ERR_GEOMETRY;
  if (!aligned_to(q, 16) || !aligned_to(lse, 4) || !aligned_to(k_pages, 16) ||
      !aligned_to(weights, 16) || (p > 0 && (!aligned_to(kc, 16) || !aligned_to(cart, 16))) ||
      !aligned_to(table, 4) || !aligned_to(lens, 4) || (pos && !aligned_to(pos, 4)))
    return CART_ERR_POINTER;
  const WeighWs w =
      weigh_ws(B, queries, Hq, Hkv, d, p, max_pages * page_rows, window > 0);
  if (!aligned_to(workspace, 16) || workspace_bytes < w.total) return CART_ERR_WORKSPACE;
  rc = check_device();
  if (rc) return rc;
  char* ws = static_cast<char*>(workspace);
  WeighArgs a{};
  a.pt = PageTable{table, lens, max_pages, n_pages, page_log2_of(page_rows)};
  a.B = B;
  a.T = queries;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.p = p;
  a.window = std::min(window, kMostPlaces);
  a.sinks = std::min(sinks, kMostPlaces);
  a.accumulate = accumulate;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.pos = pos;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lse = lse;
  a.weights = weights;
  a.cart = cart;
  a.weight_rows = weight_rows;
  a.n_qt = w.n_qt;
  a.terms = reinterpret_cast<__nv_bfloat16*>(ws + w.terms);
  a.term_elems = w.term_elems;
  a.nlse2 = reinterpret_cast<float*>(ws + w.nlse2);
  a.starts = reinterpret_cast<long long*>(ws + w.starts);
  a.part = w.parts ? reinterpret_cast<float*>(ws + w.part) : nullptr;
  a.n_ct = w.n_ct;
  a.slots = w.slots;
  a.status = device_status_ptr();
  const RopeFreqs f = make_rope_freqs(d, rope_theta);
  Turns turns{};
  for (int j = 0; j < d / 2; ++j) turns.t[j] = f.turns[j];
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope tr("attn_weights", st);
  const cudaError_t e = d == 128 ? launch_weigh<128>(a, kc, k_pages, turns, st)
                                 : launch_weigh<64>(a, kc, k_pages, turns, st);
  return e == cudaSuccess ? CART_OK : CART_ERR_CUDA;
}

}  // extern "C"
