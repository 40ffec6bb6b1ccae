// tree.cu -- attention of a tree of drafted tokens per conversation over the
// shared cartridge, the conversation's paged rows and each token's ancestors
// (cart_attn_decode_tree).
//
// Two kernels:
//   prep    one block per (conversation, node): the tree's ancestor sets, the
//           node's queries rotated into the workspace, its rotated key and
//           value written to its page row, its output set to 0 if unused.
//   attend  one block per (node, query head).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cart {
namespace {

struct TreeArgs {
  PageTable pt;
  int B, nodes, Hq, Hkv, p, window;
  float scale_log2;
  const __nv_bfloat16 *q, *k_new, *v_new, *kc, *vc;
  __nv_bfloat16 *k_pages, *v_pages, *o;
  const int* parents;
  __nv_bfloat16* qr;        // [B, nodes, Hq, d] rotated queries
  unsigned long long* anc;  // [B, nodes] ancestor sets (0: unused)
  uint32_t* status;
};

struct Turns {
  float2 t[kMaxHeadDim / 2];
};

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
  __shared__ TreeSmem tree;
  const int t = blockIdx.x, b = blockIdx.y;
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
  if (threadIdx.x == 0) a.anc[bt] = anc;
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
template <int D>
__global__ void __launch_bounds__(128) tree_attend_kernel(const TreeArgs a) {
  constexpr int E = D / 32;
  const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long bt = static_cast<long long>(b) * a.nodes + t;
  const unsigned long long anc = a.anc[bt];
  if (!anc) return;
  const int len = held_rows(a.pt, b), g = h / (a.Hq / a.Hkv);
  const int pos = a.p + len + __popcll(anc) - 1;
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.qr[(bt * a.Hq + h) * D + lane * E + e]) * a.scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  auto key = [&](const __nv_bfloat16* k, const __nv_bfloat16* v) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(k[lane * E + e]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s), al = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * al + w;
#pragma unroll
    for (int e = 0; e < E; ++e)
      acc[e] = acc[e] * al + w * __bfloat162float(v[lane * E + e]);
  };
  for (int j = lo + warp; j < a.p; j += 4) {
    const long long r = (static_cast<long long>(j) * a.Hkv + g) * D;
    key(a.kc + r, a.vc + r);
  }
  auto paged = [&](int r) {
    const int page = page_of(a.pt, b, r);
    if (page < 0) return;
    const long long x = (((static_cast<long long>(page) << a.pt.page_log2) +
                          (r & ((1 << a.pt.page_log2) - 1))) * a.Hkv + g) * D;
    key(a.k_pages + x, a.v_pages + x);
  };
  for (int r = max(0, lo - a.p) + warp; r < len; r += 4) paged(r);
  for (int n = warp; n < a.nodes; n += 4)
    if (anc >> n & 1) {
      const unsigned long long theirs = a.anc[bt - t + n];
      if (a.p + len + __popcll(theirs) - 1 >= lo) paged(len + n);
    }
  __shared__ float sm[4], sl[4], sa[4][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sa[warp][lane * E + e] = acc[e];
  __syncthreads();
  const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  for (int c = threadIdx.x; c < D; c += 128) {
    float num = 0.f, den = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float f = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - top);
      num += f * sa[w][c];
      den += f * sl[w];
    }
    a.o[(bt * a.Hq + h) * D + c] = __float2bfloat16_rn(num / den);
  }
}

// ------------------------------------------------------------- workspace ----
struct TreeWs {
  size_t qr, anc, total;
};

TreeWs tree_ws(int B, int nodes, int Hq, int d) {
  TreeWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~static_cast<size_t>(255);
    return o;
  };
  const size_t n = static_cast<size_t>(B) * nodes;
  w.qr = take(n * Hq * d * 2);
  w.anc = take(n * 8);
  w.total = off;
  return w;
}

int page_log2_of(int page_rows) {
  for (int l = 4; l <= 7; ++l)
    if (page_rows == 1 << l) return l;
  return -1;
}

int check_tree(int B, int nodes, int Hq, int Hkv, int d, int p, int page_rows, int max_pages) {
  if (B < 1 || nodes < 1 || nodes > kMaxNodes || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || p < 0 ||
      max_pages < 1 || page_log2_of(page_rows) < 0)
    return CART_ERR_GEOMETRY;
  const int G = Hq / Hkv;
  if ((G != 1 && G != 2 && G != 4 && G != 8) || Hq > 65535) return CART_ERR_GEOMETRY;
  if (d != 64 && d != 128) return CART_ERR_GEOMETRY;
  if (static_cast<long long>(B) * nodes > 65535) return CART_ERR_GEOMETRY;
  // positions must be exact in f32 (the rotation reduces its angles there)
  if (static_cast<long long>(max_pages) * page_rows + p + kMaxNodes >= (1ll << 24))
    return CART_ERR_GEOMETRY;
  return CART_OK;
}

bool al(const void* p, unsigned bytes) {
  return p && (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

template <int D>
cudaError_t launch_tree(const TreeArgs& a, const RopeFreqs& f, cudaStream_t st) {
  Turns turns;
  for (int j = 0; j < kMaxHeadDim / 2; ++j) turns.t[j] = f.turns[j];
  tree_prep_kernel<D><<<dim3(a.nodes, a.B), 256, 0, st>>>(a, turns);
  tree_attend_kernel<D><<<dim3(a.Hq, a.nodes, a.B), 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace cart

using namespace cart;

extern "C" {

size_t cart_attn_decode_tree_workspace_size(int B, int nodes, int Hq, int Hkv, int d, int p,
                                            int page_rows, int max_pages) {
  if (check_tree(B, nodes, Hq, Hkv, d, p, page_rows, max_pages)) return 0;
  return tree_ws(B, nodes, Hq, d).total;
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
    if (!al(ptr, 16)) return CART_ERR_POINTER;
  if (p > 0 && (!al(kc, 16) || !al(vc, 16))) return CART_ERR_POINTER;
  if (!al(table, 4) || !al(lens, 4) || (parents && !al(parents, 4))) return CART_ERR_POINTER;
  const TreeWs w = tree_ws(B, nodes, Hq, d);
  if (!al(workspace, 16) || workspace_bytes < w.total) return CART_ERR_WORKSPACE;
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
  a.anc = reinterpret_cast<unsigned long long*>(ws + w.anc);
  a.status = device_status_ptr();
  if (!a.status) return CART_ERR_CUDA;
  const RopeFreqs f = make_rope_freqs(d, rope_theta);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope tr("decode_tree", st);
  const cudaError_t e = d == 128 ? launch_tree<128>(a, f, st) : launch_tree<64>(a, f, st);
  return e == cudaSuccess ? CART_OK : CART_ERR_CUDA;
}

}  // extern "C"
