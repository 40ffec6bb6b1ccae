// rows.cu -- operators on the rows of paged private caches (cartattn.h, "A
// paged cache held to a budget of rows"): append a prompt's rows, evict rows of
// little weight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cart {
namespace {

struct Turns {
  float2 t[kMaxHeadDim / 2];
};

// --------------------------------------------------------------- append ----
struct AppendArgs {
  PageTable pt;
  int B, n, total, Hkv, d, p;
  const int* cu;   // packed: [B + 1]; null: sequences of n tokens
  const int* pos;  // null: p + lens
  const __nv_bfloat16 *k, *v;
  __nv_bfloat16 *k_pages, *v_pages;
  uint32_t* status;
};

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 4;  // tokens per block

// Segment of token t: the last b with cu[b] <= t (0 if none).
__device__ __forceinline__ int segment_of(const int* cu, int B, int t) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Four tokens of the token axis per block: their page rows and angles first,
// then 16-byte pieces, a key's with those d/2 further on.  Bound by HBM: 48
// prompts of up to 2000 tokens of 8 x 128 take 73 us, at 85% of a copy's rate.  Many
// small blocks carry it (32 registers, eight blocks an SM): with pieces asked for
// before their places are known 88 us, keys and values in blocks of their own 85,
// two tokens a block 112, eight 71 (but 27 tokens 7.5 us against 6.2).
__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ Turns f) {
  __shared__ float2 cs[kAppendTokens][kMaxHeadDim / 2];
  __shared__ long long at_s[kAppendTokens];  // row of the pool, -1: dropped
  __shared__ int pos_s[kAppendTokens];
  const int tid = threadIdx.x, half = a.d / 2;
  const int t0 = blockIdx.x * kAppendTokens, nt = min(kAppendTokens, a.total - t0);
  if (tid < nt) {
    const int t = t0 + tid;
    int b, i;
    bool ok = true;
    if (a.cu) {
      b = segment_of(a.cu, a.B, t);
      i = t - __ldg(a.cu + b);
      ok = i >= 0 && t < __ldg(a.cu + b + 1);
      if (!ok) atomicOr(a.status, kDevErrSegments);
    } else {
      b = t / a.n;
      i = t % a.n;
    }
    const int len = ok ? __ldg(a.pt.lens + b) : -1;
    // (below 2^25: both are below 2^24 where the row can have a page)
    const long long r = static_cast<long long>(len) + i;
    const int page = len >= 0 && r < (a.pt.max_pages << a.pt.page_log2)
                         ? page_of(a.pt, b, static_cast<int>(r))
                         : -1;
    if (len >= 0 && page < 0) atomicOr(a.status, kDevErrNoPage);
    at_s[tid] = page < 0 ? -1
                         : (static_cast<long long>(page) << a.pt.page_log2) +
                               (r & ((1 << a.pt.page_log2) - 1));
    const long long first = a.pos ? __ldg(a.pos + b) : static_cast<long long>(a.p) + len;
    pos_s[tid] = static_cast<int>(min(max(first + i, 0ll), (1ll << 24) - 1));
  }
  __syncthreads();
  for (int e = tid; e < nt * half; e += kAppendThreads) {
    const int t = e / half, j = e % half;
    cs[t][j] = rope_cs_turns(f.t[j], pos_s[t]);
  }
  __syncthreads();
  const int row = a.Hkv * a.d;  // elements of a row
  // keys: pairs of 8 values
  const int per_head = half / 8, per_tok = a.Hkv * per_head;
  for (int e = tid; e < nt * per_tok; e += kAppendThreads) {
    const int t = e / per_tok, c = e % per_tok, h = c / per_head, j0 = c % per_head * 8;
    if (at_s[t] < 0) continue;
    const __nv_bfloat16* x = a.k + static_cast<long long>(t0 + t) * row + h * a.d + j0;
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(x));
    const uint4 hi = __ldg(reinterpret_cast<const uint4*>(x + half));
    const uint32_t pl[4] = {lo.x, lo.y, lo.z, lo.w}, ph[4] = {hi.x, hi.y, hi.z, hi.w};
    uint32_t yl[4], yh[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 fl = bf16x2_to_float2(pl[k]), fh = bf16x2_to_float2(ph[k]);
      float2 u, w;
      rope_pair(fl.x, fh.x, cs[t][j0 + 2 * k], u.x, w.x);
      rope_pair(fl.y, fh.y, cs[t][j0 + 2 * k + 1], u.y, w.y);
      yl[k] = pack_bf16x2(u.x, u.y);
      yh[k] = pack_bf16x2(w.x, w.y);
    }
    __nv_bfloat16* y = a.k_pages + at_s[t] * row + h * a.d + j0;
    *reinterpret_cast<uint4*>(y) = make_uint4(yl[0], yl[1], yl[2], yl[3]);
    *reinterpret_cast<uint4*>(y + half) = make_uint4(yh[0], yh[1], yh[2], yh[3]);
  }
  const int v_tok = row / 8;
  for (int e = tid; e < nt * v_tok; e += kAppendThreads) {
    const int t = e / v_tok, c = e % v_tok * 8;
    if (at_s[t] < 0) continue;
    *reinterpret_cast<uint4*>(a.v_pages + at_s[t] * row + c) =
        __ldg(reinterpret_cast<const uint4*>(a.v + static_cast<long long>(t0 + t) * row + c));
  }
}

// ---------------------------------------------------------------- evict ----
// Conversations that hold more than keep[b] rows give up all but that many, in
// every layer and kv head on their own: the rows below `first`, the last
// `recent` ones, and of those between the ones of most weight, ties to the
// lower row.  Three launches: a plan (pages that are needed, and given back),
// the moves, and the new tables and lengths.
struct EvictArgs {
  PageTable pt;  // (as it was before the call, until the last launch)
  int B, layers, Hkv, first, recent, weight_rows;
  int *table, *lens, *refs, *done;
  const int* keep;
  float* weights;  // [layers, B, Hkv, weight_rows], or null
  // workspace: free pages per CTA of the plan; shared pages that a conversation
  // needs replaced (kIdle: nothing to evict, kTorn: a page of its rows is not
  // there); such pages before it; whether it is evicted; free pages; the new
  // pages of its rows [B, max_pages]
  int *head, *need, *base, *go, *free, *to;
  char *k, *v;
  long long layer_bytes, page_bytes;
  int row_bytes, piece;  // bytes of a row and of one head's part of it
};
enum { kIdle = -2, kTorn = -1, kSwap = -2 };  // kSwap: an entry of `to` for a shared page

struct EvictWs {
  size_t need, base, go, free, to, total;
};
EvictWs evict_ws(int B, int max_pages, int n_pages) {
  EvictWs w{};
  size_t off = 256;  // (the head)
  auto take = [&](size_t ints) {
    const size_t o = off;
    off += (ints * 4 + 255) & ~static_cast<size_t>(255);
    return o;
  };
  w.need = take(B);
  w.base = take(B);
  w.go = take(B);
  w.free = take(n_pages);
  w.to = take(static_cast<size_t>(B) * max_pages);
  w.total = off;
  return w;
}

// What conversation b is to come down to: rows held and kept (len <= keep: it
// is left as it is), the first row that may change.
struct Budget {
  int len, keep, first;
};
__device__ __forceinline__ Budget budget_of(const EvictArgs& a, int b) {
  Budget q;
  q.len = held_rows(a.pt, b);
  q.keep = __ldg(a.keep + b);
  if (q.keep < 0 || q.len <= q.keep) q.keep = q.len;
  q.first = min(a.first, q.keep);
  return q;
}
__device__ __forceinline__ int pages_for(const EvictArgs& a, int rows) {
  return (rows + (1 << a.pt.page_log2) - 1) >> a.pt.page_log2;
}

// Bound by latency, as the plan of cart_pages_reserve, whose shape it has: 9 to 12
// us alone.
__global__ void __cluster_dims__(kMetaCtas, 1, 1) __launch_bounds__(kMetaThreads)
    evict_plan_kernel(const __grid_constant__ EvictArgs a) {
  pdl_release();
  __shared__ int sums[33];
  const int rank = cluster_rank(), lane = threadIdx.x & 31;
  const int gw = rank * (kMetaThreads / 32) + (threadIdx.x >> 5);
  // ---- pages of the rows that stay and change, shared with others
  for (int b = gw; b < a.B; b += kMetaWarps) {
    const Budget q = budget_of(a, b);
    int n = kIdle;
    if (q.len > q.keep) {
      const int* row = a.pt.table + static_cast<long long>(b) * a.pt.max_pages;
      int* to = a.to + static_cast<long long>(b) * a.pt.max_pages;
      const int held = pages_for(a, q.len), end = pages_for(a, q.keep);
      const int from = q.first < q.keep ? q.first >> a.pt.page_log2 : end;  // (see kSwap)
      bool torn = false;
      n = 0;
      for (int k0 = 0; k0 < held; k0 += 32) {
        const int k = k0 + lane;
        const int page = k < held ? __ldg(row + k) : 0;
        const bool there = is_page(page, a.pt.n_pages);
        torn |= k < held && !there;
        const bool swap = there && k >= from && k < end && __ldcg(a.refs + page) > 1;
        if (k < end) to[k] = swap ? kSwap : page;
        n += __popc(__ballot_sync(0xffffffffu, swap));
      }
      if (__any_sync(0xffffffffu, torn)) n = kTorn;
    }
    if (lane == 0) a.need[b] = n;
  }
  const int part = (a.pt.n_pages + kMetaCtas - 1) / kMetaCtas;
  const int lo = rank * part, hi = min(lo + part, a.pt.n_pages);
  int mine = 0, n_part = 0;
  for (int i = lo + threadIdx.x; i < hi; i += kMetaThreads) mine += __ldcg(a.refs + i) <= 0;
  block_scan(mine, sums, &n_part);
  if (threadIdx.x == 0) a.head[rank] = n_part;
  cluster_sync();
  // ---- free pages in order (every CTA its part), and over conversations the
  // running need (CTA 0)
  int before = 0, n_free = 0;
  for (int r = 0; r < kMetaCtas; ++r) {
    const int n = __ldcg(a.head + r);
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
    long long run = 0;  // saturates above any pool
    for (int b0 = 0; b0 < a.B; b0 += kMetaThreads) {
      const int b = b0 + threadIdx.x;
      int n;
      const int at = block_scan(b < a.B ? max(__ldcg(a.need + b), 0) : 0, sums, &n);
      if (b < a.B) a.base[b] = static_cast<int>(min(run + at, 0x40000000ll));
      run += n;
    }
  }
  cluster_sync();
  // ---- the new pages; counts of those left and given back
  for (int b = gw; b < a.B; b += kMetaWarps) {
    const Budget q = budget_of(a, b);
    const int n = __ldcg(a.need + b), base = __ldcg(a.base + b);
    const bool go = n >= 0 && (n == 0 || base + n <= n_free);
    if (lane == 0) a.go[b] = go;
    if (!go) continue;
    const int* row = a.pt.table + static_cast<long long>(b) * a.pt.max_pages;
    int* to = a.to + static_cast<long long>(b) * a.pt.max_pages;
    const int end = pages_for(a, q.keep);
    int taken = 0;
    for (int k0 = 0; k0 < a.pt.max_pages; k0 += 32) {
      const int k = k0 + lane;
      const int page = k < a.pt.max_pages ? __ldg(row + k) : -1;
      const bool there = is_page(page, a.pt.n_pages), swap = k < end && __ldcg(to + k) == kSwap;
      const unsigned m = __ballot_sync(0xffffffffu, swap);
      if (swap) {
        const int now = __ldcg(a.free + base + taken + __popc(m & ((1u << lane) - 1)));
        a.refs[now] = 1;
        to[k] = now;
      }
      if (there && (swap || k >= end)) atomicSub(a.refs + page, 1);
      taken += __popc(m);
    }
  }
}

// Weights as unsigned numbers of the same order: -0 as 0, NaN above all.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// T threads a block.  The weights of the rows between, while the least of those
// that stay is looked for; then a list of rows that stay.
template <int T>
struct MoveShared {
  static constexpr int kRows = 6 * T, kKeys = (T == 256 ? 6 : 7) * kRows;
  static constexpr int kLoads = 512 / T;  // 16-byte pieces of K, and of V, a thread and turn
  union {
    uint32_t keys[kKeys];
    struct {
      long long src[kRows], dst[kRows];  // (dst < 0: stays where it is)
      int row[kRows];
      float weight[kRows];
    } list;
  };
  uint32_t hist[256], sums[T / 32], pick[2];
};

// Inclusive prefix sum of v over the block, and the sum.  Every thread calls it.
template <int T>
__device__ __forceinline__ uint2 move_scan(uint32_t v, uint32_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // sums may still be read from an earlier call
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) {
    before += w < warp ? sums[w] : 0;
    all += sums[w];
  }
  return make_uint2(before + x, all);
}

// Block (layer, conversation, kv head): the weight of the last row that stays
// by a search over its 32 bits, eight at a time from the top (a histogram of
// the rows that agree so far), then the rows in order: a list of those that
// stay, 4 T rows looked at a time, then its moves.  Row i of those that stay is
// never before place i, so a row may be written once all up to it have been
// read, whatever is read later: a turn's rows are asked for before those of the
// turn before are written.  Bound by HBM where there are many blocks: 16 layers of
// 64 conversations and 8 kv heads from up to 1100 rows to 512 take 330 us, as long
// as a copy of the 2.2 GB that moves; by latency where there are few.  (The bounds'
// second part is left open for 256 threads: a 1 there costs 10%.)
template <int T>
__global__ void __launch_bounds__(T, T == 512 ? 2 : 0)
    evict_move_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) char move_smem[];
  MoveShared<T>& sh = *reinterpret_cast<MoveShared<T>*>(move_smem);
  constexpr int kLoads = MoveShared<T>::kLoads;
  uint32_t* const sums = sh.sums;
  const int g = blockIdx.x % a.Hkv, lb = blockIdx.x / a.Hkv;
  const int b = lb % a.B, layer = lb / a.B, tid = threadIdx.x;
  const Budget q = budget_of(a, b);
  float* w = a.weights ? a.weights + (static_cast<long long>(lb) * a.Hkv + g) * a.weight_rows
                       : nullptr;
  const int last = w ? min(a.recent, q.keep - q.first) : q.keep - q.first;
  const int m0 = q.first, m1 = q.len - last;        // the rows between
  const int stay = q.keep - q.first - last;         // and how many of them stay
  // the weights of four rows (r a multiple of 4)
  const bool wide = (a.weight_rows & 3) == 0;
  auto weights_at = [&](int r) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!w || r >= q.len) return x;
    if (wide) return *reinterpret_cast<const float4*>(w + r);
    x.x = w[r];
    if (r + 1 < q.len) x.y = w[r + 1];
    if (r + 2 < q.len) x.z = w[r + 2];
    if (r + 3 < q.len) x.w = w[r + 3];
    return x;
  };
  uint32_t cut = 0xffffffffu, ties = 0;  // rows of a higher key stay, and so many of this key
  bool any = false;
  // (needs nothing of the plan, which writes nothing that it reads, and runs beside it)
  if (stay > 0 && q.len > q.keep) {
    any = true;
    const bool cached = m1 - m0 <= MoveShared<T>::kKeys;
    uint32_t left = stay, prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) sh.hist[tid] = 0;
      __syncthreads();
      const uint32_t above = shift == 24 ? 0 : 0xffffffffu << (shift + 8);
      auto count = [&](uint32_t key) {
        if ((key & above) == prefix) atomicAdd(sh.hist + (key >> shift & 255), 1);
      };
      if (shift == 24 || !cached) {
#pragma unroll 2
        for (int i = (m0 & ~3) + 4 * tid; i < m1; i += 4 * T) {
          const float4 x = weights_at(i);
          const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (i + u < m0 || i + u >= m1) continue;
            const uint32_t key = weight_key(y[u]);
            if (cached) sh.keys[i + u - m0] = key;
            count(key);
          }
        }
      } else {
        for (int i = tid; i < m1 - m0; i += T) count(sh.keys[i]);
      }
      __syncthreads();
      const uint32_t mine = tid < 256 ? sh.hist[255 - tid] : 0;
      const uint32_t upto = move_scan<T>(mine, sums).x;
      if (upto >= left && upto - mine < left) {
        sh.pick[0] = 255 - tid;
        sh.pick[1] = left - (upto - mine);
      }
      __syncthreads();
      prefix |= sh.pick[0] << shift;
      left = sh.pick[1];
    }
    cut = prefix;
    ties = left;
  }
  pdl_wait();
  pdl_release();
  if (!__ldcg(a.go + b)) return;
  const int* from_row = a.pt.table + static_cast<long long>(b) * a.pt.max_pages;
  const int* to_row = a.to + static_cast<long long>(b) * a.pt.max_pages;
  const int mask = (1 << a.pt.page_log2) - 1;
  char* const kp = a.k + layer * a.layer_bytes + static_cast<long long>(g) * a.piece;
  char* const vp = a.v + layer * a.layer_bytes + static_cast<long long>(g) * a.piece;
  const int per = a.piece / 16;
  // rows that stay so far, and of them those of key `cut` (all of that key)
  uint32_t above = 0, equal = 0;
  // (the pages of the rows before are as they were)
  const int begin = q.first & ~mask;
  above = begin;
  auto& list = sh.list;
  float4 ahead = weights_at(begin + 4 * tid);
  for (int r0 = begin; r0 < q.len;) {
    const int base = static_cast<int>(above + min(equal, ties));  // the list's first place
    int n = 0;
    for (; r0 < q.len && n + 4 * T <= MoveShared<T>::kRows; r0 += 4 * T) {
      const int r = r0 + 4 * tid;
      const float x[4] = {ahead.x, ahead.y, ahead.z, ahead.w};
      ahead = weights_at(r + 4 * T);
      uint32_t more = 0, same = 0;  // by row
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (r + u >= q.len) continue;
        if (r + u < m0 || r + u >= m1) {
          more |= 1u << u;
        } else if (any) {
          const uint32_t key = weight_key(x[u]);
          more |= static_cast<uint32_t>(key > cut) << u;
          same |= static_cast<uint32_t>(key == cut) << u;
        }
      }
      // both counts in one scan: at most 4 T of each
      const uint32_t mine = __popc(more) | __popc(same) << 16;
      const uint2 s = move_scan<T>(mine, sums);
      uint32_t more_to = above + ((s.x - mine) & 0xffff), same_to = equal + ((s.x - mine) >> 16);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool is_more = more >> u & 1, is_same = same >> u & 1;
        more_to += is_more;
        same_to += is_same;
        if (is_more || (is_same && same_to <= ties)) {
          const int i = static_cast<int>(more_to + min(same_to, ties)) - 1 - base;
          list.row[i] = r + u;
          list.weight[i] = x[u];
        }
      }
      above += s.y & 0xffff;
      equal += s.y >> 16;
      n = static_cast<int>(above + min(equal, ties)) - base;
    }
    __syncthreads();
    for (int i = tid; i < n; i += T) {
      const int r = list.row[i], z = base + i;
      const int page = __ldg(from_row + (r >> a.pt.page_log2));
      const int now = __ldcg(to_row + (z >> a.pt.page_log2));
      const bool moves = z != r || now != page;
      list.src[i] = page * a.page_bytes + static_cast<long long>(r & mask) * a.row_bytes;
      list.dst[i] =
          moves ? now * a.page_bytes + static_cast<long long>(z & mask) * a.row_bytes : -1;
      if (w) w[z] = list.weight[i];
    }
    __syncthreads();
    // ---- the moves, a turn's loads ahead of the stores of the turn before
    uint4 rk[2][kLoads], rv[2][kLoads];
    long long to[2][kLoads];
    int i = tid / per, c = tid - i * per;  // (of the next piece)
    const int di = T / per, dc = T - di * per;
    auto load = [&](int x) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        to[x][u] = i < n ? list.dst[i] : -1;
        if (to[x][u] >= 0) {
          const long long at = list.src[i] + c * 16;
          to[x][u] += c * 16;
          rk[x][u] = __ldcg(reinterpret_cast<const uint4*>(kp + at));
          rv[x][u] = __ldcg(reinterpret_cast<const uint4*>(vp + at));
        }
        i += di;
        c += dc;
        if (c >= per) {
          c -= per;
          ++i;
        }
      }
    };
    auto store = [&](int x) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        if (to[x][u] >= 0) {
          *reinterpret_cast<uint4*>(kp + to[x][u]) = rk[x][u];
          *reinterpret_cast<uint4*>(vp + to[x][u]) = rv[x][u];
        }
    };
    const int turns = (n * per + T * kLoads - 1) / (T * kLoads);
    load(0);
    for (int t = 0; t < turns; t += 2) {
      load(1);
      __syncthreads();  // turn t - 1 has been read by all
      store(0);
      load(0);
      __syncthreads();
      store(1);
    }
    __syncthreads();  // the list is free again
  }
}

template <int T>
cudaError_t launch_moves(unsigned blocks, cudaStream_t st, const EvictArgs& a) {
  constexpr int bytes = sizeof(MoveShared<T>);
  const cudaError_t e = set_smem_once<evict_move_kernel<T>>(bytes);
  return e == cudaSuccess
             ? launch_dependent(evict_move_kernel<T>, dim3(blocks), dim3(T), bytes, st, a)
             : e;
}

// The new tables, lengths and `done` (written behind the last read of keep, whose
// place it may have), a warp per conversation.
__global__ void __launch_bounds__(256) evict_tables_kernel(const __grid_constant__ EvictArgs a) {
  pdl_wait();
  const int b = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= a.B) return;
  const bool go = __ldcg(a.go + b);
  const int keep = __ldcg(a.keep + b), end = pages_for(a, keep);
  __syncwarp();
  if (lane == 0) a.done[b] = go || __ldcg(a.need + b) == kIdle;
  if (!go) return;
  int* row = a.table + static_cast<long long>(b) * a.pt.max_pages;
  const int* to = a.to + static_cast<long long>(b) * a.pt.max_pages;
  for (int k = lane; k < a.pt.max_pages; k += 32) row[k] = k < end ? __ldcg(to + k) : -1;
  if (lane == 0) a.lens[b] = keep;
}

}  // namespace
}  // namespace cart

using namespace cart;

extern "C" {

int cart_pages_append(int B, int n, int total, const int* cu_seqlens, int Hkv, int d, int p,
                      double rope_theta, const void* k, const void* v, void* k_pages,
                      void* v_pages, int n_pages, int page_rows, const int* table, int max_pages,
                      const int* lens, const int* pos, void* stream) {
  int rc = check_tables(B, max_pages, n_pages, page_rows);
  if (!rc) rc = check_pool(1, Hkv, d, CART_BF16, k_pages, v_pages);
  if (rc) return rc;
  if (d != 64 && d != 128) return CART_ERR_GEOMETRY;
  if (p < 0 || static_cast<long long>(p) + static_cast<long long>(max_pages) * page_rows >=
                   (1ll << 24))
    return CART_ERR_GEOMETRY;
  if (!(rope_theta > 0.0) || !std::isfinite(rope_theta)) return CART_ERR_GEOMETRY;
  if (total < 1 || (!cu_seqlens && (n < 1 || static_cast<long long>(B) * n != total)))
    return CART_ERR_GEOMETRY;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(table, 4) || !aligned_to(lens, 4) ||
      (cu_seqlens && !aligned_to(cu_seqlens, 4)) || (pos && !aligned_to(pos, 4)))
    return CART_ERR_POINTER;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AppendArgs a{};
  a.pt = PageTable{table, lens, max_pages, n_pages, page_log2_of(page_rows)};
  a.B = B;
  a.n = n;
  a.total = total;
  a.Hkv = Hkv;
  a.d = d;
  a.p = p;
  a.cu = cu_seqlens;
  a.pos = pos;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  a.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  a.status = device_status_ptr();
  const RopeFreqs f = make_rope_freqs(d, rope_theta);
  Turns turns{};
  for (int j = 0; j < d / 2; ++j) turns.t[j] = f.turns[j];
  TraceScope tr("pages_append", st);
  append_kernel<<<(total + kAppendTokens - 1) / kAppendTokens, kAppendThreads, 0, st>>>(a, turns);
  return cudaGetLastError() == cudaSuccess ? CART_OK : CART_ERR_CUDA;
}

size_t cart_pages_evict_workspace_size(int B, int max_pages, int n_pages) {
  if (check_tables(B, max_pages, n_pages, 16)) return 0;
  return evict_ws(B, max_pages, n_pages).total;
}

int cart_pages_evict(int B, int layers, int Hkv, int d, cart_dtype dtype, void* k_pages,
                     void* v_pages, int n_pages, int page_rows, int* table, int max_pages,
                     int* lens, int* refs, float* weights, int weight_rows, const int* keep,
                     int first, int recent, int* done, void* workspace, size_t workspace_bytes,
                     void* stream) {
  int rc = check_tables(B, max_pages, n_pages, page_rows);
  if (!rc) rc = check_pool(layers, Hkv, d, dtype, k_pages, v_pages);
  if (rc) return rc;
  const int piece = d * (dtype == CART_BF16 ? 2 : 4);
  if (piece % 16 != 0 || first < 0 || recent < 0) return CART_ERR_GEOMETRY;
  if (weights && weight_rows < max_pages * page_rows) return CART_ERR_GEOMETRY;
  const long long blocks = static_cast<long long>(layers) * B;
  if (blocks > 0x7fffffff / Hkv) return CART_ERR_GEOMETRY;
  if (!aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(refs, 4) ||
      !aligned_to(keep, 4) || !aligned_to(done, 4) || (weights && !aligned_to(weights, 16)))
    return CART_ERR_POINTER;
  const EvictWs w = evict_ws(B, max_pages, n_pages);
  if (!aligned_to(workspace, 16) || workspace_bytes < w.total) return CART_ERR_WORKSPACE;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  EvictArgs a{};
  a.pt = PageTable{table, lens, max_pages, n_pages, page_log2_of(page_rows)};
  a.B = B;
  a.layers = layers;
  a.Hkv = Hkv;
  a.first = first;
  a.recent = recent;
  a.weight_rows = weight_rows;
  a.table = table;
  a.lens = lens;
  a.refs = refs;
  a.done = done;
  a.keep = keep;
  a.weights = weights;
  a.head = reinterpret_cast<int*>(ws);
  a.need = reinterpret_cast<int*>(ws + w.need);
  a.base = reinterpret_cast<int*>(ws + w.base);
  a.go = reinterpret_cast<int*>(ws + w.go);
  a.free = reinterpret_cast<int*>(ws + w.free);
  a.to = reinterpret_cast<int*>(ws + w.to);
  a.k = static_cast<char*>(k_pages);
  a.v = static_cast<char*>(v_pages);
  a.piece = piece;
  a.row_bytes = Hkv * piece;
  a.page_bytes = static_cast<long long>(a.row_bytes) * page_rows;
  a.layer_bytes = a.page_bytes * n_pages;
  TraceScope tr("pages_evict", st);
  evict_plan_kernel<<<kMetaCtas, kMetaThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    // Blocks that the SMs take two at a time have more threads: 153 us against 175
    // with 192 blocks and up to 20000 rows (16.4 against 15.7 with 12 of 200); with
    // 8192 blocks and 1100 rows 370 against 334.
    e = blocks * Hkv <= 2 * sm_count()
            ? launch_moves<512>(static_cast<unsigned>(blocks * Hkv), st, a)
            : launch_moves<256>(static_cast<unsigned>(blocks * Hkv), st, a);
  if (e == cudaSuccess)
    e = launch_dependent(evict_tables_kernel, dim3((B + 7) / 8), dim3(256), 0, st, a);
  return e == cudaSuccess ? CART_OK : CART_ERR_CUDA;
}

}  // extern "C"
