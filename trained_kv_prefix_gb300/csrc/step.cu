// step.cu -- one new token per conversation over the shared cartridge and paged
// private rows, with the attention weights that the rows get added up
// (cart_attn_decode_paged).
//
// Two kernels, chained by programmatic dependent launch:
//   attend  a run of keys of one (conversation, kv head) per block: the group's
//           queries rotated at the conversation's position, the new token's
//           rotated key and its value written to its row by the block whose run
//           holds it, softmax over the run with a running maximum; leaves a
//           normalised partial output and its log2 log-sum-exp, and the logits
//           of private rows where weights are kept;
//   finish  joins a (conversation, kv head)'s runs by their log-sum-exps, and
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

constexpr int kMaxGroup = 8;  // query heads of a kv head
constexpr int kRun = 256;     // keys per block
constexpr int kStepThreads = 128;

struct StepArgs {
  PageTable pt;
  int B, Hq, Hkv, G, p, window, sinks;
  float scale_log2;
  const int* pos;  // null: p + lens
  const __nv_bfloat16 *q, *k_new, *v_new, *kc, *vc;
  __nv_bfloat16 *k_pages, *v_pages, *o;
  float* weights;  // [B, Hkv, weight_rows], or null
  int weight_rows;
  int cart_runs, runs, cap;  // runs of the cartridge, of all keys; most private rows
  float *part, *lse;         // [B, Hkv, runs, G, d], [B, Hkv, runs, G]
  float* logits;             // [B, Hkv, cap, G], log2 domain
  uint32_t* status;
};

struct Turns {
  float2 t[kMaxHeadDim / 2];
};

// The step of conversation b: the row of its new token (-1: idle, or the row
// has no page), that row's page, its rotary position.
struct StepOf {
  int row, page, pos;
  bool lost;  // not idle, but without a page
};
__device__ __forceinline__ StepOf step_of(const StepArgs& a, int b) {
  StepOf s;
  const int len = held_rows(a.pt, b);
  s.page = len < 0 ? -1 : page_of(a.pt, b, len);
  s.lost = len >= 0 && s.page < 0;
  s.row = s.page < 0 ? -1 : len;
  const int pos = a.pos ? __ldg(a.pos + b) : a.p + len;
  s.pos = min(max(pos, 0), (1 << 24) - 1);
  return s;
}
// Whether the token at private row `row` sees the key at a place.
__device__ __forceinline__ bool sees(const StepArgs& a, int row, int place) {
  return a.window <= 0 || place > a.p + row - a.window || place < a.sinks;
}

template <int D>
__global__ void __launch_bounds__(kStepThreads)
    step_attend_kernel(const __grid_constant__ StepArgs a, const __grid_constant__ Turns f) {
  constexpr int E = D / 32, HALF = D / 2;  // dims per lane
  __shared__ float2 cs[HALF];
  __shared__ float q_s[kMaxGroup][D];
  __shared__ float o_s[kStepThreads / 32][kMaxGroup][D];
  __shared__ float m_s[kStepThreads / 32][kMaxGroup], l_s[kStepThreads / 32][kMaxGroup];
  const int run = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_release();
  const StepOf s = step_of(a, b);
  if (s.lost && run == 0 && g == 0 && tid == 0) atomicOr(a.status, kDevErrNoPage);
  if (s.row < 0) return;
  const bool cart = run < a.cart_runs;
  const int k0 = (cart ? run : run - a.cart_runs) * kRun;
  const int k1 = min(k0 + kRun, cart ? a.p : s.row + 1);
  if (k0 >= k1) return;
  if (tid < HALF) cs[tid] = rope_cs_turns(f.t[tid], s.pos);
  __syncthreads();
  for (int e = tid; e < a.G * HALF; e += kStepThreads) {
    const int h = e / HALF, j = e % HALF;
    const __nv_bfloat16* x = a.q + (static_cast<long long>(b) * a.Hq + g * a.G + h) * D;
    rope_pair(__bfloat162float(x[j]), __bfloat162float(x[j + HALF]), cs[j], q_s[h][j],
              q_s[h][j + HALF]);
  }
  if (!cart && s.row < k1 && s.row >= k0) {  // the new row
    const long long at = (static_cast<long long>(s.page) << a.pt.page_log2) +
                         (s.row & ((1 << a.pt.page_log2) - 1));
    const long long to = (at * a.Hkv + g) * D, from = (static_cast<long long>(b) * a.Hkv + g) * D;
    for (int j = tid; j < HALF; j += kStepThreads) {
      float lo, hi;
      rope_pair(__bfloat162float(a.k_new[from + j]), __bfloat162float(a.k_new[from + j + HALF]),
                cs[j], lo, hi);
      a.k_pages[to + j] = __float2bfloat16_rn(lo);
      a.k_pages[to + j + HALF] = __float2bfloat16_rn(hi);
    }
    for (int j = tid; j < D; j += kStepThreads) a.v_pages[to + j] = a.v_new[from + j];
  }
  __syncthreads();  // (the block reads its own row back below)
  float q[kMaxGroup][E], o[kMaxGroup][E], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[h][e] = h < a.G ? q_s[h][lane * E + e] : 0.f;
      o[h][e] = 0.f;
    }
  }
  for (int k = k0 + warp; k < k1; k += kStepThreads / 32) {
    const int page = cart ? 0 : page_of(a.pt, b, k);
    const bool seen = page >= 0 && sees(a, s.row, cart ? k : a.p + k);
    float* lg = a.logits && !cart
                    ? a.logits + ((static_cast<long long>(b) * a.Hkv + g) * a.cap + k) * a.G
                    : nullptr;
    if (!seen) {
      if (lg && lane < a.G) lg[lane] = -INFINITY;
      continue;
    }
    const long long row = cart ? k
                               : (static_cast<long long>(page) << a.pt.page_log2) +
                                     (k & ((1 << a.pt.page_log2) - 1));
    const long long at = (row * a.Hkv + g) * D + lane * E;
    const __nv_bfloat16* kp = (cart ? a.kc : a.k_pages) + at;
    const __nv_bfloat16* vp = (cart ? a.vc : a.v_pages) + at;
    float kx[E], vx[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      kx[e] = __bfloat162float(kp[e]);
      vx[e] = __bfloat162float(vp[e]);
    }
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h) {
      if (h >= a.G) break;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x = fmaf(q[h][e], kx[e], x);
#pragma unroll
      for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      x *= a.scale_log2;
      if (lg && lane == h) lg[h] = x;
      const float top = fmaxf(m[h], x);
      const bool none = top == -INFINITY && x == x;  // no logit above -inf yet: weight 0
      const float r = none ? 1.f : exp2_approx(m[h] - top), w = none ? 0.f : exp2_approx(x - top);
      m[h] = top;
      l[h] = l[h] * r + w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[h][e] = none ? 0.f : fmaf(w, vx[e], o[h][e] * r);
    }
  }
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h) {
    if (h >= a.G) break;
#pragma unroll
    for (int e = 0; e < E; ++e) o_s[warp][h][lane * E + e] = o[h][e];
    if (lane == 0) m_s[warp][h] = m[h], l_s[warp][h] = l[h];
  }
  __syncthreads();
  const long long slot = ((static_cast<long long>(b) * a.Hkv + g) * a.runs + run) * a.G;
  for (int e = tid; e < a.G * D; e += kStepThreads) {
    const int h = e / D, j = e % D;
    float top = -INFINITY, sum = 0.f, x = 0.f;
    for (int w = 0; w < kStepThreads / 32; ++w) top = fmaxf(top, m_s[w][h]);
    for (int w = 0; w < kStepThreads / 32; ++w) {
      const float r = top == -INFINITY ? 0.f : exp2_approx(m_s[w][h] - top);
      sum += l_s[w][h] * r;
      x += o_s[w][h][j] * r;
    }
    a.part[slot * D + e] = sum > 0.f || sum != sum ? x / sum : 0.f;
    if (j == 0) a.lse[slot + h] = sum > 0.f || sum != sum ? top + log2f(sum) : -INFINITY;
  }
}

template <int D>
__global__ void __launch_bounds__(kStepThreads)
    step_finish_kernel(const __grid_constant__ StepArgs a) {
  __shared__ float total[kMaxGroup];
  pdl_wait();
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  __nv_bfloat16* out = a.o + (static_cast<long long>(b) * a.Hq + g * a.G) * D;
  const StepOf s = step_of(a, b);
  if (s.row < 0) {
    for (int e = tid; e < a.G * D; e += kStepThreads) out[e] = __float2bfloat16_rn(0.f);
    return;
  }
  const int runs = a.cart_runs + s.row / kRun + 1;
  const long long slot = (static_cast<long long>(b) * a.Hkv + g) * a.runs * a.G;
  for (int e = tid; e < a.G * D; e += kStepThreads) {
    const int h = e / D;
    float top = -INFINITY, sum = 0.f, x = 0.f;
    for (int r = 0; r < runs; ++r) top = fmaxf(top, a.lse[slot + r * a.G + h]);
    for (int r = 0; r < runs; ++r) {
      const float w = top == -INFINITY ? 0.f : exp2_approx(a.lse[slot + r * a.G + h] - top);
      sum += w;
      x += w == 0.f ? 0.f : w * a.part[(slot + r * a.G) * D + e];
    }
    out[e] = __float2bfloat16_rn(sum > 0.f || sum != sum ? x / sum : 0.f);
    if (e % D == 0) total[h] = sum > 0.f || sum != sum ? top + log2f(sum) : INFINITY;
  }
  if (!a.weights) return;
  __syncthreads();
  float* w = a.weights + (static_cast<long long>(b) * a.Hkv + g) * a.weight_rows;
  const float* lg = a.logits + (static_cast<long long>(b) * a.Hkv + g) * a.cap * a.G;
  for (int r = tid; r <= s.row; r += kStepThreads) {
    float x = 0.f;
    for (int h = 0; h < a.G; ++h) x += exp2_approx(lg[static_cast<long long>(r) * a.G + h] - total[h]);
    w[r] = r < s.row ? w[r] + x : x;
  }
}

struct StepWs {
  size_t part, lse, logits, total;
  int cart_runs, runs, cap;
};
StepWs step_ws(int B, int Hq, int d, int p, int cap, bool weights) {
  StepWs w{};
  size_t off = 0;
  auto take = [&](size_t floats) {
    const size_t o = off;
    off += (floats * 4 + 255) & ~static_cast<size_t>(255);
    return o;
  };
  w.cap = cap;
  w.cart_runs = (p + kRun - 1) / kRun;
  w.runs = w.cart_runs + (cap + kRun - 1) / kRun;
  w.part = take(static_cast<size_t>(B) * Hq * w.runs * d);
  w.lse = take(static_cast<size_t>(B) * Hq * w.runs);
  w.logits = weights ? take(static_cast<size_t>(B) * Hq * cap) : 0;
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
  return CART_OK;
}

template <int D>
cudaError_t launch_step(const StepArgs& a, const Turns& f, cudaStream_t st) {
  step_attend_kernel<D><<<dim3(a.runs, a.Hkv, a.B), kStepThreads, 0, st>>>(a, f);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = launch_dependent(step_finish_kernel<D>, dim3(a.Hkv, a.B), dim3(kStepThreads), 0, st, a);
  return e;
}

}  // namespace
}  // namespace cart

using namespace cart;

extern "C" {

size_t cart_attn_decode_paged_workspace_size(int B, int Hq, int Hkv, int d, int p, int page_rows,
                                             int max_pages, int weights) {
  if (check_step(B, 0, 0, Hq, Hkv, d, p, 1.f, 1.0, 1, page_rows, max_pages)) return 0;
  return step_ws(B, Hq, d, p, max_pages * page_rows, weights != 0).total;
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
  const StepWs w = step_ws(B, Hq, d, p, max_pages * page_rows, weights != nullptr);
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
  a.window = window;
  a.sinks = sinks;
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
  a.cart_runs = w.cart_runs;
  a.runs = w.runs;
  a.cap = w.cap;
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.lse = reinterpret_cast<float*>(ws + w.lse);
  a.logits = weights ? reinterpret_cast<float*>(ws + w.logits) : nullptr;
  a.status = device_status_ptr();
  const RopeFreqs f = make_rope_freqs(d, rope_theta);
  Turns turns{};
  for (int j = 0; j < d / 2; ++j) turns.t[j] = f.turns[j];
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope tr("decode_paged", st);
  const cudaError_t e = d == 128 ? launch_step<128>(a, turns, st) : launch_step<64>(a, turns, st);
  return e == cudaSuccess ? CART_OK : CART_ERR_CUDA;
}

}  // extern "C"
