// Page selection for the sparse decode: one key per cache page, a score of every page for every query
// token, and the pages with the largest scores.
#pragma once

#include "cache8.cuh"
#include "common.cuh"

namespace mla {
namespace pages {

// Pages of a sequence that token t of s_q sees, given its length: those with a position below
// L - s_q + t + 1.
__device__ __forceinline__ int visible_pages(int L, int s_q, int t) {
  const int vis = L - s_q + t + 1;
  return vis > 0 ? (vis - 1) / 64 + 1 : 0;
}

// =============================================================================================
// Page keys: key_p = mean over the page's rows j < L of [c_j ; k_r,j], summed in fp32 and rounded once.
// The key is made from the rows as they stand, not updated from its old value: a position that was
// rewritten (a rejected draft token) leaves nothing behind, and the result does not depend on the
// order of the calls. One block per page that holds one of the s_q newest positions; bound by
// reading those rows. Thread (g, q) sums piece q (V columns) of rows g, g + G, ..., four rows' loads at a
// time and as they lie in memory, so that two blocks share an SM; the G partial sums are added in order.
// 420 pages of 64 rows of 1152 bytes: 9.2 us (18.8 us with one block an SM); 64 pages: 4.7 us, latency.
// =============================================================================================
// Rows of a cache in storage type (latent rows in T) or in 8 bits (codes and one scale per row).
template <typename T>
struct CacheView {
  const T* latent;
  int64_t latent_stride;
  const uint8_t* codes;
  int64_t code_stride;
  const float* scales;
  const T* rope;
  int64_t rope_stride;
  int num_pages;
};

// V values of a row as they lie in memory: 16 bytes of T, or one value (V = 1), or V codes; and as fp32.
template <typename T, int V>
__device__ __forceinline__ uint4 load_raw(const T* p) {
  if constexpr (V == 1) {
    return make_uint4(__float_as_uint(ld(p)), 0u, 0u, 0u);
  } else {
    return *reinterpret_cast<const uint4*>(p);
  }
}
template <int V>
__device__ __forceinline__ uint4 load_raw_codes(const uint8_t* p) {
  static_assert(V == 4 || V == 8, "codes are read four or eight at a time");
  if constexpr (V == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_uint4(v.x, v.y, 0u, 0u);
  } else {
    return make_uint4(*reinterpret_cast<const uint32_t*>(p), 0u, 0u, 0u);
  }
}
template <typename T, int V>
__device__ __forceinline__ void add_raw(const uint4& v, float (&acc)[V]) {
  if constexpr (V == 1) {
    acc[0] += __uint_as_float(v.x);
  } else {
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] += ld(e + k);
  }
}
template <int V>
__device__ __forceinline__ void add_raw_codes(const uint4& v, float sc, float (&acc)[V]) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    const float2 x = cache8::e4m3x2_values(w[k >> 2] >> (16 * ((k >> 1) & 1)) & 0xffffu);
    acc[k] += x.x * sc;
    acc[k + 1] += x.y * sc;
  }
}

constexpr int kKeyGroups = 8;
constexpr int kKeyThreads = 640;   // most threads of a block

// V: columns per piece (16 bytes of T, or 1 when a width is not a multiple of that); kCodes: 8-bit rows.
template <typename T, int V, bool kCodes>
__global__ void __launch_bounds__(kKeyThreads, 2)
page_keys_kernel(CacheView<T> cache, const int32_t* block_table, int max_pages,
                                 const int32_t* seqlens, int s_q, int per_seq, int d_c, int d_r,
                                 T* keys, int64_t key_stride) {
  extern __shared__ __align__(16) float part[];   // [kKeyGroups][W]
  grid_dependency_wait();
  allow_dependents();
  const int b = blockIdx.x / per_seq, i = blockIdx.x % per_seq;
  const int L = seqlens[b];
  if (L <= 0) return;
  const int page0 = max(0, L - s_q) / 64, last = (L - 1) / 64;
  const int p = page0 + i;
  if (p > last) return;
  if (p >= max_pages) {
    if (threadIdx.x == 0) report(MLA_ERR_DEVICE_CHECK);
    return;
  }
  const int page = block_table[(int64_t)b * max_pages + p];
  if (page < 0 || page >= cache.num_pages) {
    if (threadIdx.x == 0) report(MLA_ERR_DEVICE_CHECK);
    return;
  }
  const int n = min(64, L - p * 64);
  const int W = d_c + d_r, Q = W / V, qc = d_c / V;
  for (int it = threadIdx.x; it < Q * kKeyGroups; it += blockDim.x) {
    const int q = it % Q, g = it / Q;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    constexpr int kBatch = 4;   // rows loaded before the first is added
#pragma unroll 1
    for (int r0 = g; r0 < n; r0 += kBatch * kKeyGroups) {
      uint4 raw[kBatch];
      float sc[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int r = r0 + u * kKeyGroups;
        const int64_t row = (int64_t)page * 64 + r;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        sc[u] = 0.f;
        if (r >= n) continue;
        if (q >= qc) {
          raw[u] = load_raw<T, V>(cache.rope + row * cache.rope_stride + (q - qc) * V);
        } else if constexpr (kCodes) {
          raw[u] = load_raw_codes<V>(cache.codes + row * cache.code_stride + q * V);
          sc[u] = cache.scales[row];
        } else {
          raw[u] = load_raw<T, V>(cache.latent + row * cache.latent_stride + q * V);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if constexpr (kCodes) {
          if (q < qc) add_raw_codes<V>(raw[u], sc[u], acc);
          else add_raw<T, V>(raw[u], acc);
        } else {
          add_raw<T, V>(raw[u], acc);
        }
      }
    }
    if constexpr (V == 1) {
      part[g * W + q] = acc[0];
    } else {   // (W is a multiple of V here: 16-byte stores)
#pragma unroll
      for (int k = 0; k < V; k += 4)
        *reinterpret_cast<float4*>(part + g * W + q * V + k) = make_float4(acc[k], acc[k + 1], acc[k + 2], acc[k + 3]);
    }
  }
  __syncthreads();
  T* dst = keys + (int64_t)page * key_stride;
  const float fn = (float)n;
  for (int c = threadIdx.x; c < W; c += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kKeyGroups; ++g) s += part[g * W + c];
    st(dst + c, s / fn);
  }
}

// =============================================================================================
// Page scores on CUDA cores, for fp32 and for shapes the tensor-core kernel does not take:
//   u[v, h, p] = sm_scale q[v, h, :] · key_p       over the pages p that token v sees
//   score[v, p] = sum_h exp(u[v, h, p] - logsumexp_p u[v, h, :])
// in three launches: u into the workspace, the log-sum-exp of each (token, head), the sums over heads.
// =============================================================================================
constexpr int kScoreHeads = 8;    // one warp each
constexpr int kScorePages = 32;   // one lane each

struct ScoreArgs {
  const int32_t* block_table;
  int max_pages, num_pages;
  const int32_t* seqlens;
  int s_q, H, W;
  float sm_scale;
  float* u;     // [tokens, H, max_pages]
  float* lse;   // [tokens, H]
  float* scores;   // [tokens, max_pages]
};

__device__ __forceinline__ int token_pages(const ScoreArgs& A, int v, bool may_report) {
  const int n = visible_pages(A.seqlens[v / A.s_q], A.s_q, v % A.s_q);
  if (n > A.max_pages && may_report) report(MLA_ERR_DEVICE_CHECK);
  return min(n, A.max_pages);
}

template <typename T>
__global__ void __launch_bounds__(32 * kScoreHeads)
score_products_kernel(ScoreArgs A, const T* q, const T* keys, int64_t key_stride) {
  extern __shared__ float sm[];
  const int v = blockIdx.x, p0 = blockIdx.y * kScorePages, h0 = blockIdx.z * kScoreHeads;
  const int n = token_pages(A, v, threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0);
  if (p0 >= n) return;
  const int W = A.W, WP = W + 1;   // padded key row: conflict-free column reads
  float* qs = sm;                  // [8][W]
  float* ks = sm + kScoreHeads * W;   // [32][WP]
  for (int i = threadIdx.x; i < kScoreHeads * W; i += blockDim.x) {
    const int h = h0 + i / W;
    qs[i] = h < A.H ? ld(q + ((int64_t)v * A.H + h) * W + i % W) : 0.f;
  }
  const int32_t* table = A.block_table + (int64_t)(v / A.s_q) * A.max_pages;
  for (int i = threadIdx.x; i < kScorePages * W; i += blockDim.x) {
    const int r = i / W, d = i % W;
    float x = 0.f;
    if (p0 + r < n) {
      const int page = table[p0 + r];
      if (page >= 0 && page < A.num_pages) x = ld(keys + (int64_t)page * key_stride + d);
      else if (d == 0) report(MLA_ERR_DEVICE_CHECK);   // scored as an all-zero key
    }
    ks[r * WP + d] = x;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = h0 + warp;
  if (h >= A.H || p0 + lane >= n) return;
  float acc = 0.f;
  for (int d = 0; d < W; ++d) acc = fmaf(qs[warp * W + d], ks[lane * WP + d], acc);
  A.u[((int64_t)v * A.H + h) * A.max_pages + p0 + lane] = acc * A.sm_scale;
}

__global__ void __launch_bounds__(256) score_lse_kernel(ScoreArgs A) {
  __shared__ float red[32];
  const int64_t vh = blockIdx.x;
  const int n = token_pages(A, (int)(vh / A.H), false);
  const float* u = A.u + vh * A.max_pages;
  float m = -INFINITY;
  for (int p = threadIdx.x; p < n; p += blockDim.x) m = fmaxf(m, u[p]);
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) m = fmaxf(m, red[w]);
  float l = 0.f;
  for (int p = threadIdx.x; p < n; p += blockDim.x) l += expf(u[p] - m);
  l = block_sum(l, red);
  if (threadIdx.x == 0) A.lse[vh] = m + logf(l);
}

__global__ void __launch_bounds__(256) score_mass_kernel(ScoreArgs A) {
  const int v = blockIdx.x;
  const int n = token_pages(A, v, false);
  for (int p = blockIdx.y * blockDim.x + threadIdx.x; p < n; p += gridDim.y * blockDim.x) {
    float s = 0.f;
    for (int h = 0; h < A.H; ++h) {
      const int64_t vh = (int64_t)v * A.H + h;
      s += expf(A.u[vh * A.max_pages + p] - A.lse[vh]);
    }
    A.scores[(int64_t)v * A.max_pages + p] = s;
  }
}

// =============================================================================================
// Selection: the k pages of largest score among those a token sees, as an ascending list. The first
// n_first and the last n_recent visible pages are always in it; equal scores go to the lower page; a
// NaN ranks below every number. One block per token. The k-th largest rank is found digit by digit
// (four 8-bit digits of an order-preserving 32-bit rank, most significant first: a histogram of the
// ranks that match the digits found so far, then the digit at which the count from above reaches k),
// and one ordered pass writes the pages above it and the first of those equal to it. Counts are
// integers, so the result does not depend on the order of the shared-memory additions. 64 tokens of 64
// pages: 4.9 us; 512 tokens of up to 2048 pages: 11.7 us, a chain of four histograms and eight ordered steps.
// =============================================================================================
constexpr int kKeep = 8;   // ranks a thread holds in registers; a longer list is re-read

__device__ __forceinline__ uint32_t rank_of(float x) {
  if (x != x) return 0u;
  if (x == 0.f) x = 0.f;   // -0 ranks as +0
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads)
select_pages_kernel(const float* scores, int max_pages, const int32_t* seqlens, int s_q, int k,
                    int n_first, int n_recent, int32_t* list, int32_t* counts) {
  __shared__ int hist[256];
  __shared__ int s_digit, s_left;
  __shared__ int warp_gt[32], warp_eq[32];
  grid_dependency_wait();
  allow_dependents();
  const int v = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int n = visible_pages(seqlens[v / s_q], s_q, v % s_q);
  if (n > max_pages) {
    if (tid == 0) report(MLA_ERR_DEVICE_CHECK);
    n = max_pages;
  }
  int32_t* out = list + (int64_t)v * k;
  const int kept = min(k, n);
  if (tid == 0) counts[v] = kept;
  for (int i = kept + tid; i < k; i += kThreads) out[i] = -1;
  if (n <= k) {   // every visible page
    for (int i = tid; i < n; i += kThreads) out[i] = i;
    return;
  }
  const float* sc = scores + (int64_t)v * max_pages;
  auto rank_at = [&](int p) -> uint32_t {
    // the highest rank of a number is that of +inf: 0xff800000
    return (p < n_first || p >= n - n_recent) ? 0xffffffffu : rank_of(sc[p]);
  };
  uint32_t keep[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int p = i * kThreads + tid;
    keep[i] = p < n ? rank_at(p) : 0u;
  }
  uint32_t found = 0, mask = 0;   // the digits of the k-th largest rank so far
  int left = kept;                // how many of the ranks that match them are still to be taken
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (i * kThreads + tid < n && (keep[i] & mask) == found) atomicAdd(&hist[(keep[i] >> shift) & 255u], 1);
    for (int p = kKeep * kThreads + tid; p < n; p += kThreads) {
      const uint32_t r = rank_at(p);
      if ((r & mask) == found) atomicAdd(&hist[(r >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds digits 255 - 8 l downwards: ranks with a digit at or above each
      int c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = hist[255 - 8 * lane - j];
        sum += c[j];
      }
      int above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += x;
      }
      above -= sum;   // in the lanes before this one
      if (above < left && left <= above + sum) {
        int d = 0, a = above;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (a + c[j] < left && d == j) { a += c[j]; d = j + 1; }
        s_digit = 255 - 8 * lane - d;
        s_left = left - a;
      }
    }
    __syncthreads();
    found |= (uint32_t)s_digit << shift;
    mask |= 255u << shift;
    left = s_left;
  }
  // ordered pass: page p goes to (pages above it so far) + (equal ones so far, `left` of them at most)
  int gt0 = 0, eq0 = 0;
  for (int base = 0, i = 0; base < n; base += kThreads, ++i) {
    const int p = base + tid;
    uint32_t r = 0;
    if (i < kKeep) {
#pragma unroll
      for (int j = 0; j < kKeep; ++j)
        if (j == i) r = keep[j];
    } else if (p < n) {
      r = rank_at(p);
    }
    const bool gt = p < n && r > found, eq = p < n && r == found;
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) { warp_gt[warp] = __popc(mg); warp_eq[warp] = __popc(me); }
    __syncthreads();
    int g = gt0, e = eq0, tg = 0, te = 0;
#pragma unroll 8
    for (int w = 0; w < kThreads / 32; ++w) {
      const int a = warp_gt[w], c = warp_eq[w];
      if (w < warp) { g += a; e += c; }
      tg += a;
      te += c;
    }
    g += __popc(mg & ((1u << lane) - 1u));
    e += __popc(me & ((1u << lane) - 1u));
    if (gt || (eq && e < left)) out[g + min(e, left)] = p;
    gt0 += tg;
    eq0 += te;
    __syncthreads();
  }
}

}  // namespace pages
}  // namespace mla
