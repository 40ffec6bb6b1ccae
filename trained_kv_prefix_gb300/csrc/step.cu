// step.cu -- one new token per conversation over the shared cartridge and paged
// private rows, with the attention weights that the rows get added up
// (cart_attn_decode_paged).
//
// Three kernels, chained by programmatic dependent launch; the first two run at
// once, one CTA of each per SM:
//   cart    the B * G stacked query rows of each kv head against the cartridge,
//           as tcgen05 products: 128 rows and 64 keys at a time, Q resident as
//           two bf16 terms, S and O in TMEM.  All (kv head, row tile, key tile)
//           triples are cut into equal runs, one per CTA.
//   rows    the private rows, bound by HBM: 16 rows of up to four heads by one
//           box each for keys and values and 64 dims, three stages of up to 16 KB
//           of both per CTA, a warp per head and 16 rows: m16n8k16 products with
//           the query's terms in the rows of A that a group of heads leaves free,
//           and V^T as A of the second product, whose B has the layout that the
//           first one leaves.  The warp that comes to the new token's row
//           writes its head's rotated key and value to it and to the stage.  All
//           conversations' rows, one after the other, are cut into equal runs.
//   finish  joins a (conversation, kv head)'s parts by their log-sum-exps, and
//           adds exp2(logit - log-sum-exp) of the group's heads to each row.
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
// largest shared part of an SM's first-level cache: two kernels share one there,
// which fits only what the first of them was given.
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
  // ---- cart: row tiles, key tiles, tiles per CTA, most parts of a segment
  int row_tiles, key_tiles, cart_chunk, cart_parts;
  float *cart_o, *cart_lse;  // [Hkv * row_tiles, cart_parts, d / 4, 128] float4; [.., 128]
  // ---- rows: heads of a unit (of which a conversation has `units`), 16-row
  // groups that its warps take side by side, and of a stage, CTAs
  int heads, units, subs, stage_groups, row_ctas;
  int finish_heads;          // heads of a block of the last kernel: `heads` or 1
  long long* starts;         // [B + 1]: chunks of a unit before each conversation's
  float *row_o, *row_lse;    // [slots, turns * subs, heads, G, d], [.., G]
  int cap;                   // most private rows
  float* logits;             // [B, Hkv, G, cap], log2 domain, by the order of groups seen
};

struct Turns {
  float2 t[kMaxHeadDim / 2];
};

// The step of conversation b: the row of its new token (-1: idle, or the row
// has no page), that row's page; the rows it sees: those below `low` and from
// `high` to `row`, in n groups of 16: those below g_low and from g_high on.
struct StepOf {
  int row, page, low, high, g_low, g_high, n;
  bool lost;  // not idle, but without a page
  __device__ __forceinline__ int group(int i) const { return i < g_low ? i : i - g_low + g_high; }
  __device__ __forceinline__ bool sees(int r) const { return r <= row && (r < low || r >= high); }
};
__device__ __forceinline__ StepOf step_of(const StepArgs& a, int b) {
  StepOf s;
  const int len = held_rows(a.pt, b);
  s.page = len < 0 ? -1 : page_of(a.pt, b, len);
  s.lost = len >= 0 && s.page < 0;
  s.row = s.page < 0 ? -1 : len;
  s.high = a.window > 0 ? max(s.row - a.window + 1, 0) : 0;
  s.low = min(max(a.sinks - a.p, 0), s.high);
  s.g_high = s.high >> 4;
  s.g_low = min((s.low + 15) >> 4, s.g_high);
  s.n = s.row < 0 ? 0 : s.g_low + (s.row >> 4) + 1 - s.g_high;
  return s;
}
__device__ __forceinline__ int position_of(const StepArgs& a, int b, int row) {
  return min(max(a.pos ? __ldg(a.pos + b) : a.p + row, 0), (1 << 24) - 1);
}

// ----------------------------------------------------------------- cart ----
constexpr int kCartThreads = 192;  // four softmax warps, TMA warp, MMA warp
constexpr int kCartKeys = 64;      // keys of a tile

template <int D>
struct CartSmem {
  static constexpr int kQBytes = kTile * D * 2, kKBytes = kCartKeys * D * 2;
  static constexpr int kQ = 0;                 // two terms
  static constexpr int kK = kQ + 2 * kQBytes;  // two slots
  static constexpr int kV = kK + 2 * kKBytes;
  static constexpr int kBytes = kV + kKBytes;
  static constexpr int kAlloc = kBytes + 1024;  // slack for 1024-byte alignment
};

enum CartBar {
  kCKFull0 = 0,
  kCKEmpty0 = kCKFull0 + 2,
  kCVFull = kCKEmpty0 + 2,
  kCSFull0,                   // S of buffer x is in TMEM
  kCPFull0 = kCSFull0 + 2,    // its weights are (128 arrivals); by buffer, since those
                              // of the next tile may come before these are waited for
  kCPvDone = kCPFull0 + 2,    // O has them, and V has been read
  kCODone,                    // O has those of the piece's last tile (waits for this one
                              // may come two tiles after the last for the one before)
  kCDrain,
  kCBars
};

struct CartMaps {
  CUtensorMap k, v;
};

// (96 registers, and 104 of the rows' kernel: a quarter of an SM holds two of
// these warps and three of those)
template <int D>
__global__ void __maxnreg__(96)
    step_cart_kernel(const __grid_constant__ CartMaps maps, const __grid_constant__ StepArgs a,
                     const __grid_constant__ Turns f) {
  using L = CartSmem<D>;
  constexpr int HALF = D / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bars[kCBars];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, first_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t abort_s = smem_u32(&abort_flag);
  pdl_release();  // (the rows run beside this kernel)
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < kCBars; ++s)
      mbar_init(&bars[s], s == kCPFull0 || s == kCPFull0 + 1 ? 128 : 1);
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot, tO = tmem, tS = tmem + 128;
  const int total = a.Hkv * a.row_tiles * a.key_tiles;
  const int lo = min(blockIdx.x * a.cart_chunk, total), hi = min(lo + a.cart_chunk, total);
  const int R = a.B * a.G;
  int step = 0, pieces = 0;  // tiles walked, and pieces that had any, in every role
  bool ok = true;
  for (int u = lo; u < hi;) {
    const int seg = u / a.key_tiles, t0 = u - seg * a.key_tiles;
    const int t1 = min(t0 + hi - u, a.key_tiles);
    const int g = seg / a.row_tiles, row0 = (seg - g * a.row_tiles) * kTile;
    // ---- the tile's queries, rotated, as two terms; what they see
    if (threadIdx.x == 0) first_s = 0x7fffffff;
    __syncthreads();
    const int row = threadIdx.x, R0 = row0 + row;
    int first = 0x7fffffff;  // first key in the row's window
    if (row < kTile) {
      const uint32_t qs = smem_u32(smem + L::kQ);
      const bool inside = R0 < R;
      const int b = inside ? R0 / a.G : 0;
      StepOf s{};
      s.row = -1;
      if (inside) s = step_of(a, b);
      if (s.row >= 0) {
        first = a.window > 0 ? a.p + s.row - a.window + 1 : 0;
        const int pos = position_of(a, b, s.row);
        const __nv_bfloat16* x =
            a.q + (static_cast<long long>(b) * a.Hq + g * a.G + R0 % a.G) * D;
#pragma unroll
        for (int c = 0; c < HALF / 8; ++c) {  // pairs 8c .. 8c + 7
          const uint4 l4 = __ldg(reinterpret_cast<const uint4*>(x + 8 * c));
          const uint4 h4 = __ldg(reinterpret_cast<const uint4*>(x + HALF + 8 * c));
          const uint32_t pl[4] = {l4.x, l4.y, l4.z, l4.w}, ph[4] = {h4.x, h4.y, h4.z, h4.w};
          uint32_t yl[2][4], yh[2][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 fl = bf16x2_to_float2(pl[k]), fh = bf16x2_to_float2(ph[k]);
            float2 v, w;
            rope_pair(fl.x, fh.x, rope_cs_turns_fast(f.t[8 * c + 2 * k], pos), v.x, w.x);
            rope_pair(fl.y, fh.y, rope_cs_turns_fast(f.t[8 * c + 2 * k + 1], pos), v.y, w.y);
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
          const uint32_t o0 = sw128_offset(row, c);
          const uint32_t o1 = D == 128 ? 16384u + sw128_offset(row, c) : sw128_offset(row, c + 4);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            sts_u4(qs + m * L::kQBytes + o0, make_uint4(yl[m][0], yl[m][1], yl[m][2], yl[m][3]));
            sts_u4(qs + m * L::kQBytes + o1, make_uint4(yh[m][0], yh[m][1], yh[m][2], yh[m][3]));
          }
        }
      }
      fence_proxy_async_smem();
      if (a.window > 0) {
        const int w = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) atomicMin(&first_s, w);
      }
    }
    __syncthreads();
    // tiles that some row sees
    const int low = a.window > 0 ? first_s : 0;
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
          if (s >= 2)
            ok = mbar_wait(&bars[kCKEmpty0 + x], ((s >> 1) - 1) & 1, abort_s, a.status,
                           kDevErrTimeoutTma);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars[kCKFull0 + x], L::kKBytes);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(smem + L::kK + x * L::kKBytes + h * 8192, &maps.k, &bars[kCKFull0 + x],
                        h * 64, g, t * kCartKeys, 0);
          if (s >= 1)
            ok = mbar_wait(&bars[kCPvDone], (s - 1) & 1, abort_s, a.status, kDevErrTimeoutTma);
          if (!ok) {
            mbar_wait(&bars[kCKFull0 + x], (s >> 1) & 1, 0u, nullptr, 0);
            break;
          }
          mbar_arrive_expect_tx(&bars[kCVFull], L::kKBytes);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(smem + L::kV + h * 8192, &maps.v, &bars[kCVFull], h * 64, g,
                        t * kCartKeys, 0);
          ++s;
        }
        // (whatever went wrong: the last copies land before the CTA ends)
        if (s > step) {
          mbar_wait(&bars[kCKFull0 + ((s - 1) & 1)], ((s - 1) >> 1) & 1, 0u, nullptr, 0);
          if (s >= 2) mbar_wait(&bars[kCKFull0 + (s & 1)], ((s - 2) >> 1) & 1, 0u, nullptr, 0);
          mbar_wait(&bars[kCVFull], (s - 1) & 1, 0u, nullptr, 0);
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
      const uint64_t dV = sdesc_sw128(smem_u32(smem + L::kV), 8192u, 1024u);
      auto issue_s = [&](int s) {
        const uint64_t dk = desc_add(dK, (s & 1) * L::kKBytes);
#pragma unroll
        for (int m = 1; m >= 0; --m)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_bf16_ss_w(tS + (s & 1) * kCartKeys,
                           desc_add(dQ, m * L::kQBytes + (k >> 2) * 16384 + (k & 3) * 32),
                           desc_add(dk, (k >> 2) * 8192 + (k & 3) * 32), idS,
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
        ok = wait(&bars[kCVFull], s & 1) && wait(&bars[kCPFull0 + (s & 1)], (s >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kCartKeys / 16; ++k)
          umma_bf16_ts_w(tO, tS + (s & 1) * kCartKeys + k * 8, desc_add(dV, k * 2048), idPV,
                         t > 0 || k > 0 ? 1u : 0u);
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
        const uint32_t ts = tS + (s & 1) * kCartKeys + lane_off;
        // the row sees the keys up to `end` that are sinks or in its window
        const int k0 = t * kCartKeys;
        const int end = first == 0x7fffffff ? 0 : min(a.p - k0, kCartKeys);
        const int from = first > k0 ? min(first - k0, kCartKeys) : 0;
        const int sink = min(max(a.sinks - k0, 0), kCartKeys);
        const bool cut = __any_sync(0xffffffffu, end < kCartKeys || from > sink);
        // (S is read twice, half a tile at a time, to spare registers)
        auto load = [&](int half, uint32_t (&r)[32]) {
          tmem_ld32(ts + 32 * half, r);
          tmem_ld_wait();
          tmem_reg_fence(r);
          if (cut) {
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int k = 32 * half + c;
              if (k >= end || (k < from && k >= sink)) r[c] = __float_as_uint(-INFINITY);
            }
          }
        };
        float top = -INFINITY;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[32];
          load(half, r);
          float mx[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            mx[q] = __uint_as_float(r[16 * q]);
#pragma unroll
            for (int c = 1; c < 15; c += 2)
              mx[q] = fmax3(mx[q], __uint_as_float(r[16 * q + c]), __uint_as_float(r[16 * q + c + 1]));
            mx[q] = fmaxf(mx[q], __uint_as_float(r[16 * q + 15]));
          }
          top = fmax3(top, mx[0], mx[1]);
        }
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
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[32], pk[16];
          load(half, r);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 x = __ffma2_rn(u2f2(r[2 * c], r[2 * c + 1]), sc2, nm2);
            const float2 w = make_float2(exp2_approx(x.x), exp2_approx(x.y));
            sum[c & 1] = __fadd2_rn(sum[c & 1], w);
            pk[c] = pack_bf16x2(w.x, w.y);
          }
          tmem_st16(ts + 16 * half, pk);  // (over columns that have been read)
        }
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
          ok = wait(&bars[kCVFull], s & 1, kDevErrTimeoutSoftmax);
          if (!ok) break;
          const uint32_t vs = smem_u32(smem + L::kV);
          for (int e = row; e < (z1 - z0) * (D / 8); e += 128) {
            const int j = z0 + e / (D / 8), c = e % (D / 8);
            sts_u4(vs + (c >> 3) * 8192 + j * 128 + (c & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars[kCPFull0 + (s & 1)]);
        ++i;
      }
      // ---- the piece's part: column blocks of four by row
      const int part = blockIdx.x - seg * a.key_tiles / a.cart_chunk;
      const long long slot = static_cast<long long>(seg) * a.cart_parts + part;
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
          if (R0 < R)
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
    u += t1 - t0;
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
}

// ----------------------------------------------------------------- rows ----
constexpr int kRowTurns = 2;     // groups of four warps, which take a piece's chunks in turn
constexpr int kRowWarps = 4 * kRowTurns;
constexpr int kRowThreads = 32 * kRowWarps + 32;  // and the producer
constexpr int kRowStages = 3;
constexpr int kRowHeads = 4;     // most heads of a unit
constexpr int kRowGroups = 8;    // most 16-row groups of a stage

// What a stage holds: groups of 16 rows of conversation b and the unit's heads
// from h0 on; v0 the first's number among those seen, times 16; the rows of each
// that are there and seen; chunks of the piece before and after it, the slot of
// the piece's part; the token's position; groups; the new row's number among
// the stage's (-1: not here) and its place in the pool.
struct StageInfo {
  int b, h0, v0, before, after, slot, pos, groups, fresh;
  long long at;
  unsigned short bits[kRowGroups];
};

template <int D>
struct RowSmem {
  static constexpr int kHalfBytes = 16 * kRowHeads * 256;  // keys, or values
  static constexpr int kStage = 2 * kHalfBytes;
  static constexpr int kAlloc = kRowStages * kStage + 1024;  // slack for alignment
};

struct RowMaps {
  CUtensorMap k, v;  // (d, page_rows, Hkv, pages), box 64 x 16 x heads x 1
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Chunks (stages) of one unit of a conversation that sees n groups.
__device__ __forceinline__ int chunks_of(const StepArgs& a, int n) {
  return (n + a.stage_groups - 1) / a.stage_groups;
}

// The new token's rotated key and its value, one head's, by a warp: to its row
// of the pool, and to row r of the staged group, where what the pool held before
// has landed.
template <int D>
__device__ __forceinline__ void write_row(const StepArgs& a, const Turns& f, int b, int g, int pos,
                                          long long at, uint32_t ks, uint32_t vs, int half_bytes,
                                          int r) {
  constexpr int HALF = D / 2;
  const int lane = threadIdx.x & 31;
  const long long from = (static_cast<long long>(b) * a.Hkv + g) * D, to = at + g * D;
  auto staged = [&](int j) {  // place of element j
    return (j >> 6) * half_bytes + r * 128 + ((((j & 63) >> 3) ^ (r & 7)) << 4) + (j & 7) * 2;
  };
#pragma unroll
  for (int e = 0; e < HALF / 32; ++e) {
    const int j = lane + 32 * e;
    float y0, y1;
    rope_pair(__bfloat162float(a.k_new[from + j]), __bfloat162float(a.k_new[from + j + HALF]),
              rope_cs_turns(f.t[j], pos), y0, y1);
    const __nv_bfloat16 z0 = __float2bfloat16_rn(y0), z1 = __float2bfloat16_rn(y1);
    a.k_pages[to + j] = z0;
    a.k_pages[to + j + HALF] = z1;
    sts_u16(ks + staged(j), __bfloat16_as_ushort(z0));
    sts_u16(ks + staged(j + HALF), __bfloat16_as_ushort(z1));
  }
  if (lane < D / 8) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.v_new + from + lane * 8));
    *reinterpret_cast<uint4*>(a.v_pages + to + lane * 8) = v;
    sts_u4(vs + staged(lane * 8), v);
  }
  __syncwarp();
}

// kWide: groups of more than four query heads.  The first product's A has the
// queries' first terms in rows 0 .. G - 1 and their second ones in rows 8 ..;
// the third ones in rows 4 .. where the group leaves those free, else they are
// a product of their own.
template <int D, bool kWide>
__global__ void __maxnreg__(104)
    step_rows_kernel(const __grid_constant__ RowMaps maps, const __grid_constant__ StepArgs a,
                     const __grid_constant__ Turns f) {
  using L = RowSmem<D>;
  constexpr int KS = D / 16;  // steps of 16 dims
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kRowStages], empty[kRowStages];
  __shared__ StageInfo info[kRowStages];
  __shared__ long long scan[kRowThreads / 32];
  __shared__ int run_b, abort_flag;
  __shared__ long long run_off;
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t abort_s = smem_u32(&abort_flag);
  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < kRowStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kRowWarps);
    }
    fence_mbar_init();
  }
  // ---- the chunks of all conversations, and this CTA's run of them
  const int per = (a.B + kRowThreads - 1) / kRowThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const StepOf s = step_of(a, b);
    if (s.lost && blockIdx.x == 0) atomicOr(a.status, kDevErrNoPage);
    mine += static_cast<long long>(chunks_of(a, s.n)) * a.units;
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  long long total = 0, start = x - mine;
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) {
    start += w < warp ? scan[w] : 0;
    total += scan[w];
  }
  const long long chunk = (total + a.row_ctas - 1) / a.row_ctas;
  const long long lo = min(blockIdx.x * chunk, total), hi = min(lo + chunk, total);
  if (lo < hi && start <= lo && lo < start + mine) {  // (one thread)
    long long at = start;
    int b = b0;
    for (;; ++b) {
      const long long n = static_cast<long long>(chunks_of(a, step_of(a, b).n)) * a.units;
      if (lo < at + n) break;
      at += n;
    }
    run_b = b;
    run_off = lo - at;
  }
  if (blockIdx.x == 0) {  // for the last kernel
    long long at = start;
    for (int b = b0; b < b1; ++b) {
      a.starts[b] = at;
      at += static_cast<long long>(chunks_of(a, step_of(a, b).n)) * a.units;
    }
    if (tid == 0) a.starts[a.B] = total;
  }
  __syncthreads();
  const int n_chunks = static_cast<int>(hi - lo);
  constexpr int head_bytes = 2048;
  const int half_bytes = a.heads * head_bytes;  // 16 rows of 64 dims
  const int group_bytes = (D / 64) * half_bytes;

  if (warp == kRowWarps) {
    // ------------------------------------------------------------ producer --
    int b = run_b, n = 0;  // chunks handed on
    bool ok = n_chunks > 0;
    int unit = 0, c0 = 0;
    StepOf s{};
    if (ok) {
      s = step_of(a, b);
      const int per_unit = chunks_of(a, s.n);
      unit = static_cast<int>(run_off / per_unit);
      c0 = static_cast<int>(run_off - static_cast<long long>(unit) * per_unit);
    }
    while (ok && n < n_chunks) {
      const int all = chunks_of(a, s.n);
      if (all == 0) {  // idle
        s = step_of(a, ++b);
        continue;
      }
      const int pos = position_of(a, b, s.row), h0 = unit * a.heads;
      const int c1 = min(all, c0 + n_chunks - n);
      // the next conversation's, before they are needed
      const StepOf next = unit + 1 == a.units && b + 1 < a.B ? step_of(a, b + 1) : s;
      // the piece's slot: the run's first piece, its last one, or a whole unit
      const bool opens = n == 0 && c0 > 0, closes = c1 < all;
      const int slot = opens || (closes && n == 0) ? 2 * blockIdx.x
                       : closes                    ? 2 * blockIdx.x + 1
                                                   : 2 * a.row_ctas + b * a.units + unit;
      const int* pages = a.pt.table + static_cast<long long>(b) * a.pt.max_pages;
      const int mask = (1 << a.pt.page_log2) - 1;
      // a chunk's groups, a lane each: its first row, and that row's page
      auto row_of = [&](int c) {
        const int i = c * a.stage_groups + lane;
        return lane < a.stage_groups && i < s.n ? s.group(i) * 16 : -1;
      };
      auto look_up = [&](int r) { return r < 0 ? -1 : __ldg(pages + (r >> a.pt.page_log2)); };
      int row = row_of(c0), page = look_up(row);
      for (int c = c0; c < c1; ++c, ++n) {
        const int st = n % kRowStages;
        const int row_next = c + 1 < c1 ? row_of(c + 1) : -1, page_next = look_up(row_next);
        const bool there = row >= 0 && is_page(page, a.pt.n_pages);
        unsigned bits = 0;
        if (there) {
          bits = 0xffffu;
          if (row + 15 > s.row || (row + 15 >= s.low && row < s.high)) {
            bits = 0;
            for (int i = 0; i < 16; ++i) bits |= static_cast<unsigned>(s.sees(row + i)) << i;
          }
        }
        if (n >= kRowStages) {
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], (n / kRowStages - 1) & 1, abort_s,
                                                 a.status, kDevErrTimeoutTma));
          if (!ok) break;
        }
        const unsigned groups = __ballot_sync(0xffffffffu, there);
        StageInfo& o = info[st];
        if (lane < kRowGroups) o.bits[lane] = static_cast<unsigned short>(bits);
        if (lane == 0) {
          o.b = b;
          o.h0 = h0;
          o.v0 = c * a.stage_groups * 16;
          o.before = c - c0;
          o.after = c1 - 1 - c;
          o.slot = slot;
          o.pos = pos;
          o.groups = min(a.stage_groups, s.n - c * a.stage_groups);
          o.fresh = c + 1 < all ? -1 : (s.n - 1 - c * a.stage_groups) * 16 + (s.row & 15);
          o.at = ((static_cast<long long>(s.page) << a.pt.page_log2) + (s.row & mask)) *
                 a.Hkv * D;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[st], 2 * __popc(groups) * group_bytes);
        __syncwarp();
        if (there) {
          uint8_t* const ks = smem + st * L::kStage + lane * group_bytes;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            tma_load_4d(ks + h * half_bytes, &maps.k, &full[st], h * 64, row & mask, h0, page);
            tma_load_4d(ks + L::kHalfBytes + h * half_bytes, &maps.v, &full[st], h * 64, row & mask,
                        h0, page);
          }
        }
        __syncwarp();
        row = row_next;
        page = page_next;
      }
      c0 = 0;
      if (++unit == a.units) {
        unit = 0;
        ++b;
        s = next;
      }
    }
    pdl_release();
    if (lane == 0)  // the last copies land before the CTA ends
      for (int i = max(n - kRowStages, 0); i < n; ++i)
        mbar_wait(&full[i % kRowStages], (i / kRowStages) & 1, 0u, nullptr, 0);
    __syncwarp();
  } else {
    // --------------------------------------------------------------- heads --
    const int q8 = lane >> 2, t4 = lane & 3;  // query row, pair of columns
    const int turn = warp >> 2, h = (warp & 3) % a.heads;
    const int sub = (warp & 3) / a.heads;  // (idle beyond the last group)
    bool ok = true;
    float m = -INFINITY, l = 0.f;
    float o[D / 16][4];  // O^T: dims 16i + q8 (+ 8), queries 2 t4 (+ 1)
    // the queries' terms as A: rows 0-7 (first terms, and third in rows 4-7),
    // rows 8-15 (second ones)
    uint32_t qa[KS][2], qb[KS][2], qc[kWide ? KS : 1][2];
    // chunks of 16 bytes of a row's 64 dims lie by the row's last three bits
    const int krow = (lane & 7) + (lane >> 4) * 8, kcol = (lane >> 3) & 1;
    for (int n = 0; n < n_chunks && ok; ++n) {
      const int st = n % kRowStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (n / kRowStages) & 1, abort_s, a.status,
                                             kDevErrTimeoutSoftmax));
      if (!ok) break;
      const StageInfo& in = info[st];
      const int h0 = vld(in.h0);
      const int before = vld(in.before);
      const bool works = before % kRowTurns == turn && h0 + h < a.Hkv && sub < a.subs;
      if (works) {
        const int g = h0 + h, b = vld(in.b);
        if (before < kRowTurns) {  // ---- the first chunk of a piece: its queries
          const int pos = vld(in.pos);
          const __nv_bfloat16* x = a.q + (static_cast<long long>(b) * a.Hq + g * a.G) * D;
          const int third = q8 - 4;  // the query whose third term the row holds (not kWide)
          const bool has = q8 < a.G, more = !kWide && third >= 0 && third < a.G;
          const uint32_t* xq = reinterpret_cast<const uint32_t*>(x + (has ? q8 : more ? third : 0) * D);
          uint32_t raw[KS][2];
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) raw[k][e] = has || more ? __ldg(xq + 8 * k + 4 * e + t4) : 0u;
#pragma unroll
          for (int k = 0; k < KS / 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = 16 * k + 8 * e + 2 * t4;
              const float2 lo2 = bf16x2_to_float2(raw[k][e]), hi2 = bf16x2_to_float2(raw[k + KS / 2][e]);
              float2 y, z;
              rope_pair(lo2.x, hi2.x, rope_cs_turns(f.t[j], pos), y.x, z.x);
              rope_pair(lo2.y, hi2.y, rope_cs_turns(f.t[j + 1], pos), y.y, z.y);
              uint32_t ty[3], tz[3];
#pragma unroll
              for (int s = 0; s < 3; ++s) {
                ty[s] = pack_bf16x2(y.x, y.y);
                tz[s] = pack_bf16x2(z.x, z.y);
                const float2 dy = bf16x2_to_float2(ty[s]), dz = bf16x2_to_float2(tz[s]);
                y.x -= dy.x;
                y.y -= dy.y;
                z.x -= dz.x;
                z.y -= dz.y;
              }
              qa[k][e] = more ? ty[2] : ty[0];
              qa[k + KS / 2][e] = more ? tz[2] : tz[0];
              qb[k][e] = more ? 0u : ty[1];
              qb[k + KS / 2][e] = more ? 0u : tz[1];
              if (kWide) {
                qc[k][e] = ty[2];
                qc[k + KS / 2][e] = tz[2];
              }
            }
          m = -INFINITY;
          l = 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        }
        const int groups = vld(in.groups), fresh = vld(in.fresh);
        float* const lg = a.logits + ((static_cast<long long>(b) * a.Hkv + g) * a.G + q8) * a.cap +
                          vld(in.v0) + 2 * t4;
        const uint32_t ks = smem_u32(smem + st * L::kStage) + h * head_bytes + krow * 128;
        bool cleared = false;
        for (int i = sub; i < groups; i += a.subs) {
          const unsigned bits = *reinterpret_cast<const volatile unsigned short*>(&in.bits[i]);
          const uint32_t kg = ks + i * group_bytes, vg = kg + L::kHalfBytes;
          float x4[4] = {0.f, 0.f, 0.f, 0.f};  // query q8, keys 2 t4, + 1, + 8, + 9
          if (bits) {  // (uniform over the warp)
            if (fresh >> 4 == i) {
              write_row<D>(a, f, b, g, vld(in.pos), *const_cast<const volatile long long*>(&in.at),
                           kg - krow * 128, vg - krow * 128, half_bytes, fresh & 15);
              cleared = true;
            }
            // ---- S [query terms, 16 keys], even and odd steps apart (the
            // products of one chain wait for one another)
            float s0[2][4], s1[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) s0[0][e] = s0[1][e] = s1[0][e] = s1[1][e] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t kb[4];
              ldsm_x4(kg + (k >> 2) * half_bytes +
                          ((((2 * (k & 3) + kcol) ^ (lane & 7))) << 4), kb);
              mma_bf16_16816(s0[k & 1], qa[k][0], qb[k][0], qa[k][1], qb[k][1], kb[0], kb[1]);
              mma_bf16_16816(s1[k & 1], qa[k][0], qb[k][0], qa[k][1], qb[k][1], kb[2], kb[3]);
              if (kWide) {
                mma_bf16_16816(s0[k & 1], qc[k][0], 0u, qc[k][1], 0u, kb[0], kb[1]);
                mma_bf16_16816(s1[k & 1], qc[k][0], 0u, qc[k][1], 0u, kb[2], kb[3]);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s0[0][e] += s0[1][e];
              s1[0][e] += s1[1][e];
            }
            x4[0] = s0[0][0] + s0[0][2];
            x4[1] = s0[0][1] + s0[0][3];
            x4[2] = s1[0][0] + s1[0][2];
            x4[3] = s1[0][1] + s1[0][3];
            if (!kWide) {  // (rows 4-7 hold third terms)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x4[e] += __shfl_xor_sync(0xffffffffu, e < 2 ? s0[0][e] : s1[0][e - 2], 16);
            }
          }
          const bool live = q8 < a.G;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 2 * t4 + (e & 1) + 8 * (e >> 1);
            x4[e] = live && (bits >> key & 1) ? x4[e] * a.scale_log2 : -INFINITY;
          }
          if (a.logits && live) {
            *reinterpret_cast<float2*>(lg + i * 16) = make_float2(x4[0], x4[1]);
            *reinterpret_cast<float2*>(lg + i * 16 + 8) = make_float2(x4[2], x4[3]);
          }
          if (!bits) continue;
          float top = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          float alpha = 1.f;
          if (top > m + 8.f) {  // (the maximum is renewed where it grows by more than 8)
            alpha = exp2_approx(m - top);
            m = top;
          }
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
            l *= alpha;
            const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * t4);
            const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * t4 + 4);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[j][0] *= a0;
              o[j][1] *= a1;
              o[j][2] *= a0;
              o[j][3] *= a1;
            }
          }
          const float mr = m == -INFINITY ? 0.f : m;
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) e4[e] = exp2_approx(x4[e] - mr);
          l += (e4[0] + e4[1]) + (e4[2] + e4[3]);
          if (bits != 0xffffu) {
            // values of rows that are not seen may be anything, and 0 times them
            // need not be 0
            if (!(bits >> (lane & 15) & 1)) {
              const uint32_t at = vg + ((lane & 15) - krow) * 128 + (lane >> 4) * 64;
#pragma unroll
              for (int k = 0; k < D / 64; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  sts_u4(at + k * half_bytes + e * 16, make_uint4(0u, 0u, 0u, 0u));
            }
            cleared = true;
            __syncwarp();
          }
          // ---- O^T += V^T P^T: P^T as B has the layout of S
          const uint32_t p0 = pack_bf16x2(e4[0], e4[1]), p1 = pack_bf16x2(e4[2], e4[3]);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t vt[4];
            ldsm_x4_t(vg + (j >> 2) * half_bytes + (((2 * (j & 3) + kcol) ^ (lane & 7)) << 4), vt);
            mma_bf16_16816(o[j], vt[0], vt[1], vt[2], vt[3], p0, p1);
          }
        }
        if (cleared) fence_proxy_async_smem();  // before a later load of what was written
        if (vld(in.after) < kRowTurns) {  // ---- the last chunk of the piece: its part
          float sum = l;
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          const bool any = sum > 0.f || sum != sum;
          const float inv = any ? 1.f / sum : 0.f;
          const float i0 = __shfl_sync(0xffffffffu, inv, 8 * t4);
          const float i1 = __shfl_sync(0xffffffffu, inv, 8 * t4 + 4);
          const long long part =
              ((static_cast<long long>(vld(in.slot)) * kRowTurns + turn) * a.subs + sub) * a.heads + h;
          if (t4 == 0 && q8 < a.G) a.row_lse[part * a.G + q8] = any ? m + __log2f(sum) : -INFINITY;
          float* out = a.row_o + part * a.G * D;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int q = 2 * t4 + e;
            const float iq = e ? i1 : i0;
            if (q < a.G)
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                out[q * D + 16 * j + q8] = iq == 0.f ? 0.f : o[j][e] * iq;
                out[q * D + 16 * j + q8 + 8] = iq == 0.f ? 0.f : o[j][2 + e] * iq;
              }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
  }
  // the last kernel waits for this one alone: it has waited for the cartridge's
  pdl_wait();
}

// --------------------------------------------------------------- finish ----
constexpr int kFinishThreads = 512;
constexpr int kFinishParts = 32;                      // parts joined at a time
constexpr int kFinishHeads = kRowHeads * kMaxGroup;   // most query heads of a block

// Blocks (., heads, conversation), the heads a unit's or one: the parts' common
// log-sum-exp, a warp per query head; then the first block the output, some
// threads per column of four, the parts' weights and places settled before; the
// others the rows' weights.
template <int D>
__global__ void __launch_bounds__(kFinishThreads, 2)
    step_finish_kernel(const __grid_constant__ StepArgs a) {
  __shared__ float total[kFinishHeads];
  __shared__ float4 acc[kFinishThreads];
  __shared__ float weight[kFinishHeads][kFinishParts];
  __shared__ const float4* place[kFinishHeads][kFinishParts];
  pdl_wait();
  const int g0 = blockIdx.y * a.finish_heads, b = blockIdx.z;
  const int heads = min(a.finish_heads, a.Hkv - g0), nq = heads * a.G;  // query heads
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long start = __ldcg(a.starts + b), chunks = __ldcg(a.starts + a.B);
  const StepOf s = step_of(a, b);
  __nv_bfloat16* out = a.o + (static_cast<long long>(b) * a.Hq + g0 * a.G) * D;
  if (s.row < 0) {
    if (blockIdx.x == 0)
      for (int e = tid; e < nq * D; e += kFinishThreads) out[e] = __float2bfloat16_rn(0.f);
    return;
  }
  const int first = (static_cast<int>(blockIdx.x) - 1) * kFinishThreads;  // rows' blocks
  if (first >= s.n * 16) return;
  // ---- the parts of the private rows: those of the runs that hold the unit
  const int unit = g0 / a.heads, all = chunks_of(a, s.n), per = kRowTurns * a.subs;
  const long long chunk = (chunks + a.row_ctas - 1) / a.row_ctas;
  const long long u0 = start + static_cast<long long>(unit) * all, u1 = u0 + all;
  const int c0 = static_cast<int>(u0 / chunk), c1 = static_cast<int>((u1 - 1) / chunk);
  const int n_row = (c1 - c0 + 1) * per;
  auto row_part = [&](int q, int i) -> long long {  // its row, or -1
    const int c = c0 + i / per, k = i % per;
    // (warps whose turn is beyond the piece's chunks had none)
    if (k / a.subs >= min(u1, (c + 1) * chunk) - max(u0, c * chunk)) return -1;
    const long long slot = c0 == c1 ? 2 * a.row_ctas + static_cast<long long>(b) * a.units + unit
                           : c > c0 || u0 == c0 * chunk ? 2 * c
                                                        : 2 * c + 1;
    return ((slot * per + k) * a.heads + g0 - unit * a.heads) * a.G + q;
  };
  // ---- and of the cartridge, by the tile that holds the query's row
  auto cart_row = [&](int q) { return b * a.G + q % a.G; };
  auto cart_seg = [&](int q) { return (g0 + q / a.G) * a.row_tiles + cart_row(q) / kTile; };
  auto parts_of = [&](int q) {
    if (a.key_tiles == 0) return n_row;
    const int u = cart_seg(q) * a.key_tiles;
    return n_row + (u + a.key_tiles - 1) / a.cart_chunk - u / a.cart_chunk + 1;
  };
  auto lse_of = [&](int q, int i) {
    if (i >= n_row)
      return __ldcg(a.cart_lse +
                    (static_cast<long long>(cart_seg(q)) * a.cart_parts + i - n_row) * kTile +
                    cart_row(q) % kTile);
    const long long part = row_part(q, i);
    return part < 0 ? -INFINITY : __ldcg(a.row_lse + part);
  };
  for (int q = warp; q < nq; q += kFinishThreads / 32) {
    const int n = parts_of(q);
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < n; i += 32) {
      const float x = lse_of(q, i), top = fmaxf(m, x);
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
    if (lane == 0) total[q] = l == 0.f ? INFINITY : m + __log2f(l);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    int most = 0;
    for (int q = 0; q < nq; ++q) most = max(most, parts_of(q));
    const int cols = nq * (D / 4), each = max(kFinishThreads / cols, 1);
    const int turn = tid / cols;  // (below `each`, or idle; 0 where there are more columns)
    for (int col0 = 0; col0 < cols; col0 += kFinishThreads) {
      const int col = col0 + (each > 1 ? tid % cols : tid);
      const int q = col / (D / 4), j = col % (D / 4);
      const bool mine = turn < each && col < cols;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = 0; i0 < most; i0 += kFinishParts) {
        if (col0 == 0 || most > kFinishParts) {  // (else it is there already)
          __syncthreads();
          for (int e = tid; e < nq * kFinishParts; e += kFinishThreads) {
            const int qq = e / kFinishParts, k = e % kFinishParts, i = i0 + k;
            if (i >= parts_of(qq)) continue;
            weight[qq][k] = exp2_approx(lse_of(qq, i) - total[qq]);
            place[qq][k] = reinterpret_cast<const float4*>(
                i < n_row ? a.row_o + max(row_part(qq, i), 0ll) * D
                          : a.cart_o + ((static_cast<long long>(cart_seg(qq)) * a.cart_parts + i -
                                         n_row) * (D / 4) * kTile + cart_row(qq) % kTile) * 4);
          }
          __syncthreads();
        }
        if (mine) {
          const int n = min(parts_of(q) - i0, kFinishParts);
#pragma unroll 8
          for (int k = turn; k < n; k += each) {
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
      if (mine && turn == 0)
        *reinterpret_cast<uint2*>(out + q * D + 4 * j) =
            make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    }
    return;
  }
  const long long bg = static_cast<long long>(b) * a.Hkv + g0;
  const int step = (gridDim.x - 1) * kFinishThreads;
  for (int v = first + tid; v < s.n * 16; v += step) {
    const int r = s.group(v >> 4) * 16 + (v & 15);
    if (!s.sees(r)) continue;
    for (int h = 0; h < heads; ++h) {
      const float* lg = a.logits + (bg + h) * a.G * a.cap + v;
      float* w = a.weights + (bg + h) * a.weight_rows + r;
      const float old = r < s.row ? *w : 0.f;
      float x = 0.f;
#pragma unroll 4
      for (int hh = 0; hh < a.G; ++hh)
        x += exp2_approx(__ldcg(lg + static_cast<long long>(hh) * a.cap) - total[h * a.G + hh]);
      *w = old + x;
    }
  }
}

struct StepWs {
  size_t cart_o, cart_lse, row_o, row_lse, starts, logits, total;
  int row_tiles, key_tiles, cart_chunk, cart_parts, cart_ctas;
  int heads, units, subs, stage_groups, row_ctas;
};
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
  const int tiles = Hkv * w.row_tiles * w.key_tiles;
  if (tiles > 0) {
    w.cart_chunk = (tiles + sms - 1) / sms;
    w.cart_ctas = (tiles + w.cart_chunk - 1) / w.cart_chunk;
    w.cart_parts = (w.key_tiles + w.cart_chunk - 1) / w.cart_chunk + 1;
  }
  w.units = (Hkv + kRowHeads - 1) / kRowHeads;
  w.heads = (Hkv + w.units - 1) / w.units;
  w.units = (Hkv + w.heads - 1) / w.heads;
  w.subs = kRowHeads / w.heads;
  w.stage_groups = w.subs * (d == 64 ? 2 : 1);
  // one CTA per SM beside the cartridge's, two without
  w.row_ctas = p > 0 ? sms : 2 * sms;
  const size_t segments = static_cast<size_t>(Hkv) * w.row_tiles;
  w.cart_o = take(segments * w.cart_parts * kTile * d * 4);
  w.cart_lse = take(segments * w.cart_parts * kTile * 4);
  const size_t parts =
      (2 * static_cast<size_t>(w.row_ctas) + static_cast<size_t>(B) * w.units) * kRowTurns *
      w.subs * w.heads;
  w.row_o = take(parts * G * d * 4);
  w.row_lse = take(parts * G * 4);
  w.starts = take((static_cast<size_t>(B) + 1) * 8);
  w.logits = take(weights ? static_cast<size_t>(B) * Hq * cap * 4 : 0);
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
  cudaError_t e = cudaSuccess;
  if (w.cart_ctas > 0) {
    e = set_shared_once<step_cart_kernel<D>>(C::kAlloc);
    if (e != cudaSuccess) return e;
    const uint64_t dims[4] = {D, static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.p), 1};
    const uint64_t row = static_cast<uint64_t>(a.Hkv) * D * 2;
    const uint64_t strides[3] = {D * 2, row, row * a.p};
    const uint32_t box[4] = {64, 1, kCartKeys, 1};
    CartMaps maps;
    if (!encode_bf16_map4(&maps.k, a.kc, dims, strides, box) ||
        !encode_bf16_map4(&maps.v, a.vc, dims, strides, box))
      return cudaErrorInvalidValue;
    step_cart_kernel<D><<<w.cart_ctas, kCartThreads, C::kAlloc, st>>>(maps, a, f);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const uint64_t page_rows = 1ull << a.pt.page_log2, row = static_cast<uint64_t>(a.Hkv) * D * 2;
  const uint64_t dims[4] = {D, page_rows, static_cast<uint64_t>(a.Hkv),
                            static_cast<uint64_t>(a.pt.n_pages)};
  const uint64_t strides[3] = {row, D * 2, row * page_rows};
  const uint32_t box[4] = {64, 16, static_cast<uint32_t>(a.heads), 1};
  RowMaps maps;
  if (!encode_bf16_map4(&maps.k, a.k_pages, dims, strides, box) ||
      !encode_bf16_map4(&maps.v, a.v_pages, dims, strides, box))
    return cudaErrorInvalidValue;
  const bool wide = a.G > 4;
  e = wide ? set_shared_once<step_rows_kernel<D, true>>(L::kAlloc)
           : set_shared_once<step_rows_kernel<D, false>>(L::kAlloc);
  if (e != cudaSuccess) return e;
  auto* rows = wide ? step_rows_kernel<D, true> : step_rows_kernel<D, false>;
  if (w.cart_ctas > 0) {
    e = launch_dependent(rows, dim3(w.row_ctas), dim3(kRowThreads), L::kAlloc, st, maps, a, f);
  } else {
    rows<<<w.row_ctas, kRowThreads, L::kAlloc, st>>>(maps, a, f);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  // blocks of the last kernel: a unit's heads each where that leaves enough of
  // them, else one; and for the weights' rows as many as the GPU takes at once, at
  // most one for every 512 rows that a table can name
  StepArgs last = a;
  last.finish_heads = a.B * a.units >= sm_count() ? a.heads : 1;
  const int across = (a.Hkv + last.finish_heads - 1) / last.finish_heads;
  int blocks = 1;
  if (a.weights)
    blocks += std::max(1, std::min((a.cap + kFinishThreads - 1) / kFinishThreads,
                                   4 * sm_count() / std::max(1, a.B * across)));
  return launch_dependent(step_finish_kernel<D>, dim3(blocks, across, a.B), dim3(kFinishThreads), 0,
                          st, last);
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
  a.cart_chunk = w.cart_chunk;
  a.cart_parts = w.cart_parts;
  a.cart_o = reinterpret_cast<float*>(ws + w.cart_o);
  a.cart_lse = reinterpret_cast<float*>(ws + w.cart_lse);
  a.heads = w.heads;
  a.units = w.units;
  a.subs = w.subs;
  a.stage_groups = w.stage_groups;
  a.row_ctas = w.row_ctas;
  a.starts = reinterpret_cast<long long*>(ws + w.starts);
  a.row_o = reinterpret_cast<float*>(ws + w.row_o);
  a.row_lse = reinterpret_cast<float*>(ws + w.row_lse);
  a.cap = max_pages * page_rows;
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
