// weights.cu -- the attention weight that each key gets from a conversation's
// last queries, by the log-sum-exps that their attention came with
// (cart_attn_weights).
//
// With q~ = R(position) q and the cache's keys k~, the weight of key j is the
// sum over the queries i that see it and the heads of its group of
// exp(scale * q~_i . k~_j - lse_i): no maximum, no sum to wait for.  One query
// head's rows are turned into two bf16 terms whose sum is q~ to 2^-16, so that
// the f32 weights are good to about 1e-5.
//   prep   q~ in two terms, [B, Hkv, T * G, d] each, and -lse * log2(e)
//          [B, Hkv, T * G] (row i * G + hh);
//   weigh  a key per warp, over all of its queries.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cart {
namespace {

struct WeighArgs {
  PageTable pt;
  int B, T, Hq, Hkv, G, p, window, sinks, accumulate;
  float scale_log2;
  const int* pos;  // null: p + lens - T
  const __nv_bfloat16 *q, *kc, *k_pages;
  const float* lse;  // [B, Hq, T]
  float *weights, *cart;
  int weight_rows;
  __nv_bfloat16 *q_hi, *q_lo;
  float* nlse2;
};

struct Turns {
  float2 t[kMaxHeadDim / 2];
};

// Block: a query of a conversation.
template <int D>
__global__ void __launch_bounds__(128)
    weigh_prep_kernel(const __grid_constant__ WeighArgs a, const __grid_constant__ Turns f) {
  constexpr int HALF = D / 2;
  __shared__ float2 cs[HALF];
  pdl_release();
  const int i = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int len = held_rows(a.pt, b);
  if (len < 0 || len - a.T + i < 0) return;  // no such query
  const long long at = a.pos ? static_cast<long long>(__ldg(a.pos + b)) + i
                             : static_cast<long long>(a.p) + len - a.T + i;
  const int pos = static_cast<int>(min(max(at, 0ll), (1ll << 24) - 1));
  if (tid < HALF) cs[tid] = rope_cs_turns(f.t[tid], pos);
  __syncthreads();
  const __nv_bfloat16* x = a.q + (static_cast<long long>(b) * a.T + i) * a.Hq * D;
  for (int e = tid; e < a.Hq * HALF; e += 128) {
    const int h = e / HALF, j = e % HALF;
    float y[2];
    rope_pair(__bfloat162float(x[h * D + j]), __bfloat162float(x[h * D + j + HALF]), cs[j], y[0],
              y[1]);
    const long long row =
        (static_cast<long long>(b) * a.Hkv + h / a.G) * a.T * a.G + i * a.G + h % a.G;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const __nv_bfloat16 hi = __float2bfloat16_rn(y[s]);
      a.q_hi[row * D + j + s * HALF] = hi;
      a.q_lo[row * D + j + s * HALF] = __float2bfloat16_rn(y[s] - __bfloat162float(hi));
    }
    if (j == 0)
      a.nlse2[row] = -1.4426950408889634f * __ldg(a.lse + (static_cast<long long>(b) * a.Hq + h) * a.T + i);
  }
}

template <int D>
__global__ void __launch_bounds__(128) weigh_kernel(const __grid_constant__ WeighArgs a) {
  constexpr int E = D / 32;
  pdl_wait();
  const int g = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = held_rows(a.pt, b);
  const int rows = max(len, 0);
  const long long bg = static_cast<long long>(b) * a.Hkv + g;
  for (int place = blockIdx.x * 4 + warp; place < a.p + rows; place += gridDim.x * 4) {
    const int r = place - a.p;  // private row, or below 0
    const int page = r < 0 ? 0 : page_of(a.pt, b, r);
    float sum = 0.f;
    if (page >= 0) {
      const long long row = r < 0 ? place
                                  : (static_cast<long long>(page) << a.pt.page_log2) +
                                        (r & ((1 << a.pt.page_log2) - 1));
      const __nv_bfloat16* kp = (r < 0 ? a.kc : a.k_pages) + (row * a.Hkv + g) * D + lane * E;
      float k[E];
#pragma unroll
      for (int e = 0; e < E; ++e) k[e] = __bfloat162float(kp[e]);
      // queries at places p + len - T + i that see it
      int i0 = max(max(a.T - rows, r - (len - a.T)), 0), i1 = a.T;
      if (a.window > 0 && place >= a.sinks)
        i1 = min(static_cast<long long>(i1),
                 static_cast<long long>(place) + a.window - (a.p + len - a.T));
      for (int c = i0 * a.G; c < i1 * a.G; ++c) {
        const long long at = (bg * a.T * a.G + c) * D + lane * E;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
          x = fmaf(__bfloat162float(a.q_hi[at + e]) + __bfloat162float(a.q_lo[at + e]), k[e], x);
#pragma unroll
        for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        sum += exp2_approx(fmaf(x, a.scale_log2, a.nlse2[bg * a.T * a.G + c]));
      }
    }
    if (lane == 0) {
      float* w = r < 0 ? a.cart + bg * a.p + place : a.weights + bg * a.weight_rows + r;
      *w = a.accumulate && (r < 0 || r < len - a.T) ? *w + sum : sum;
    }
  }
}

struct WeighWs {
  size_t hi, lo, nlse2, total;
};
WeighWs weigh_ws(int B, int T, int Hq, int d) {
  WeighWs w{};
  const size_t rows = static_cast<size_t>(B) * T * Hq;
  w.hi = 0;
  w.lo = (rows * d * 2 + 255) & ~static_cast<size_t>(255);
  w.nlse2 = 2 * w.lo;
  w.total = w.nlse2 + ((rows * 4 + 255) & ~static_cast<size_t>(255));
  return w;
}

int check_weigh(int B, int T, int window, int sinks, int Hq, int Hkv, int d, int p, float scale,
                double theta, int n_pages, int page_rows, int max_pages) {
  int rc = check_tables(B, max_pages, n_pages, page_rows);
  if (rc) return rc;
  if (T < 1 || T >= (1 << 24) || Hq < 1 || Hkv < 1 || Hkv > 65535 || Hq % Hkv != 0 ||
      Hq / Hkv > 8 || (d != 64 && d != 128) || p < 0 || window < 0 || sinks < 0)
    return CART_ERR_GEOMETRY;
  if (!std::isfinite(scale) || !(scale > 0.f) || !(theta > 0.0) || !std::isfinite(theta))
    return CART_ERR_GEOMETRY;
  if (static_cast<long long>(p) + static_cast<long long>(max_pages) * page_rows >= (1ll << 24))
    return CART_ERR_GEOMETRY;
  return CART_OK;
}

template <int D>
cudaError_t launch_weigh(const WeighArgs& a, const Turns& f, cudaStream_t st) {
  weigh_prep_kernel<D><<<dim3(a.T, a.B), 128, 0, st>>>(a, f);
  cudaError_t e = cudaGetLastError();
  const int places = a.p + (a.pt.max_pages << a.pt.page_log2);
  if (e == cudaSuccess)
    e = launch_dependent(weigh_kernel<D>, dim3(places < 4096 ? (places + 3) / 4 : 1024, a.Hkv, a.B),
                         dim3(128), 0, st, a);
  return e;
}

}  // namespace
}  // namespace cart

using namespace cart;

extern "C" {

size_t cart_attn_weights_workspace_size(int B, int queries, int Hq, int Hkv, int d, int p,
                                        int page_rows, int max_pages) {
  if (check_weigh(B, queries, 0, 0, Hq, Hkv, d, p, 1.f, 1.0, 1, page_rows, max_pages)) return 0;
  return weigh_ws(B, queries, Hq, d).total;
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
  const WeighWs w = weigh_ws(B, queries, Hq, d);
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
  a.window = window;
  a.sinks = sinks;
  a.accumulate = accumulate;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.pos = pos;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.kc = static_cast<const __nv_bfloat16*>(kc);
  a.k_pages = static_cast<const __nv_bfloat16*>(k_pages);
  a.lse = lse;
  a.weights = weights;
  a.cart = cart;
  a.weight_rows = weight_rows;
  a.q_hi = reinterpret_cast<__nv_bfloat16*>(ws + w.hi);
  a.q_lo = reinterpret_cast<__nv_bfloat16*>(ws + w.lo);
  a.nlse2 = reinterpret_cast<float*>(ws + w.nlse2);
  const RopeFreqs f = make_rope_freqs(d, rope_theta);
  Turns turns{};
  for (int j = 0; j < d / 2; ++j) turns.t[j] = f.turns[j];
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope tr("attn_weights", st);
  const cudaError_t e =
      d == 128 ? launch_weigh<128>(a, turns, st) : launch_weigh<64>(a, turns, st);
  return e == cudaSuccess ? CART_OK : CART_ERR_CUDA;
}

}  // extern "C"
