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
// order of the calls. L is the sequence's length, all new tokens included: the key of a page that several of them
// share is one for all, and holds rows that the earlier ones do not see. One block per page that holds one of the s_q newest positions; bound by
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
// floats from one group's sums to the next
__host__ __device__ constexpr int key_part_width(int W) { return (W + 3) / 4 * 4; }
constexpr int kKeyThreads = 640;   // most threads of a block

// V, VR: columns per piece of the latent row (16 bytes of T, or 1 when a width is not a multiple of that) and of the
// key; kCodes: 8-bit rows, whose latent width is a multiple of 16 and whose key may have any even one.
template <typename T, int V, int VR, bool kCodes>
__global__ void __launch_bounds__(kKeyThreads, 2)
page_keys_kernel(CacheView<T> cache, const int32_t* block_table, int max_pages,
                                 const int32_t* seqlens, int s_q, int per_seq, int d_c, int d_r,
                                 T* keys, int64_t key_stride) {
  extern __shared__ __align__(16) float part[];   // [kKeyGroups][WP]
  grid_dependency_wait();
  allow_dependents();
  const int b = blockIdx.x / per_seq, i = blockIdx.x % per_seq;
  const int L = seqlens[b];
  if (L <= 0) return;
  const int page0 = max(0, L - s_q) / 64, last = (L - 1) / 64;
  // a sequence longer than its table row is reported by its first block: the grid has none for pages past the row
  if (i == 0 && last >= max_pages && threadIdx.x == 0) report(MLA_ERR_DEVICE_CHECK);
  const int p = page0 + i;
  if (p > last || p >= max_pages) return;
  const int page = block_table[(int64_t)b * max_pages + p];
  if (page < 0 || page >= cache.num_pages) {
    if (threadIdx.x == 0) report(MLA_ERR_DEVICE_CHECK);
    return;
  }
  const int n = min(64, L - p * 64);
  const int W = d_c + d_r, qc = d_c / V, Q = qc + d_r / VR, WP = key_part_width(W);
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
          raw[u] = load_raw<T, VR>(cache.rope + row * cache.rope_stride + (q - qc) * VR);
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
          else if constexpr (VR == 1) acc[0] += __uint_as_float(raw[u].x);
          else add_raw<T, V>(raw[u], acc);
        } else {
          add_raw<T, V>(raw[u], acc);
        }
      }
    }
    float* dst = part + g * WP;
    if (V == 1 || (VR == 1 && q >= qc)) {
      dst[V == 1 ? q : d_c + (q - qc)] = acc[0];
    } else {   // (16-byte stores: WP and, for VR = V, d_c are multiples of 4)
#pragma unroll
      for (int k = 0; k + 3 < V; k += 4)
        *reinterpret_cast<float4*>(dst + q * V + k) = make_float4(acc[k], acc[k + 1], acc[k + 2], acc[k + 3]);
    }
  }
  __syncthreads();
  T* dst = keys + (int64_t)page * key_stride;
  const float fn = (float)n;
  for (int c = threadIdx.x; c < W; c += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kKeyGroups; ++g) s += part[g * WP + c];
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
// NaN ranks below every number. One block per token. The rank of the last page taken is found digit by digit
// (the 9, 8, 8 and 7 bits of an order-preserving 32-bit rank, most significant first: a histogram of the
// ranks that match the digits found so far, then the digit at which the count from above reaches what
// is left to take), and no further than to a digit all of whose ranks are taken: with scores that
// differ two digits, the exponent and eight more bits, mostly are enough. One ordered pass then writes the
// pages above it and the first of those equal to it. Counts are integers, so the result does not depend on the
// order of the shared-memory additions. A chain of latencies: 64 tokens of 64 pages 3.4 us back to back; 512 tokens of
// 2048 pages 11.0 us, 16 of 8192 10.8 us (13.2 and 23.3 us with four digits always and a block-wide step for every
// 256 or 1024 pages).
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
  constexpr int kBins = 512, kWarps = kThreads / 32, kEntries = kKeep * kWarps;
  __shared__ int hist[kBins];
  __shared__ int s_digit, s_left, s_all;
  __shared__ int before[kEntries + 1];   // (above | equal << 16) of the warps' pages in order, then their sums
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
  // bin b lies where the lane that sums bins b, b + 1, ... of a run of 16 reads without bank conflicts
  constexpr int kPerLane = kBins / 32;
  auto bin = [&](uint32_t b) { return (b % kPerLane) * 32 + b / kPerLane; };
  const int groups = min(kKeep, (n + kThreads - 1) / kThreads);   // of the pages held in registers
  // the pages always kept are not ranked (fewer than n, as k is)
  auto forced = [&](int p) { return p < n_first || p >= n - n_recent; };
  uint32_t keep[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int p = i * kThreads + tid;
    keep[i] = p < n && !forced(p) ? rank_of(sc[p]) : 0u;
  }
  uint32_t found = 0, mask = 0;              // the digits found so far
  int left = kept - n_first - n_recent;      // how many of the ranks that match them are still to be taken
  bool all = left == 0;                      // every rank >= found is taken (none: found is above every rank)
  if (all) found = 0xffffffffu;
  for (int shift = 23, width = 9; !all && shift >= 0;) {
    const uint32_t digit = (1u << width) - 1u;
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      if (i >= groups) break;
      const int p = i * kThreads + tid;
      if (p < n && !forced(p) && (keep[i] & mask) == found) atomicAdd(&hist[bin((keep[i] >> shift) & digit)], 1);
    }
    for (int p = kKeep * kThreads + tid; p < n; p += kThreads) {
      if (forced(p)) continue;
      const uint32_t r = rank_of(sc[p]);
      if ((r & mask) == found) atomicAdd(&hist[bin((r >> shift) & digit)], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds digits 511 - 16 l downwards: ranks with a digit at or above each
      int c[kPerLane], sum = 0;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        c[j] = hist[bin(kBins - 1 - kPerLane * lane - j)];
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
        int d = 0, a = above, at = c[0];
#pragma unroll
        for (int j = 0; j < kPerLane; ++j)
          if (d == j) {
            at = c[j];
            if (a + c[j] < left) { a += c[j]; d = j + 1; }
          }
        s_digit = kBins - 1 - kPerLane * lane - d;
        s_left = left - a;
        s_all = left - a == at;
      }
    }
    __syncthreads();
    found |= (uint32_t)s_digit << shift;
    mask |= digit << shift;
    left = s_left;
    all = s_all != 0;
    width = shift >= 15 ? 8 : 7;
    shift = shift == 23 ? 15 : shift == 15 ? 7 : shift == 7 ? 0 : -1;
  }
  // in order: page p goes to (pages above found so far) + (equal ones so far, `left` of them at most)
  auto above = [&](int p, uint32_t r) { return p < n && (forced(p) || (all ? r >= found && left > 0 : r > found)); };
  auto equal = [&](int p, uint32_t r) { return p < n && !all && !forced(p) && r == found; };
  auto place = [&](int p, bool gt, bool eq, uint32_t mg, uint32_t me, int g, int e) {
    g += __popc(mg & ((1u << lane) - 1u));
    e += __popc(me & ((1u << lane) - 1u));
    if (gt || (eq && e < left)) out[g + min(e, all ? 0 : left)] = p;
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {   // the pages held in registers: counts of every warp's 32 first
    if (i >= groups) break;
    const int p = i * kThreads + tid;
    const uint32_t mg = __ballot_sync(0xffffffffu, above(p, keep[i])), me = __ballot_sync(0xffffffffu, equal(p, keep[i]));
    if (lane == 0) before[i * kWarps + warp] = __popc(mg) | (__popc(me) << 16);
  }
  __syncthreads();
  if (warp == 0) {
    constexpr int kPer = kEntries / 32;
    int c[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      c[j] = kPer * lane + j < groups * kWarps ? before[kPer * lane + j] : 0;
      sum += c[j];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    int at = incl - sum;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      before[kPer * lane + j] = at;
      at += c[j];
    }
    if (lane == 31) before[kEntries] = at;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    if (i >= groups) break;
    const int p = i * kThreads + tid;
    const bool gt = above(p, keep[i]), eq = equal(p, keep[i]);
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    const int at = before[i * kWarps + warp];
    place(p, gt, eq, mg, me, at & 0xffff, at >> 16);
  }
  int gt0 = before[kEntries] & 0xffff, eq0 = before[kEntries] >> 16;
  for (int base = kKeep * kThreads; base < n; base += kThreads) {   // a longer list, 32 pages a warp at a time
    const int p = base + tid;
    const uint32_t r = p < n && !forced(p) ? rank_of(sc[p]) : 0u;
    const bool gt = above(p, r), eq = equal(p, r);
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) { warp_gt[warp] = __popc(mg); warp_eq[warp] = __popc(me); }
    __syncthreads();
    int g = gt0, e = eq0, tg = 0, te = 0;
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) {
      const int a = warp_gt[w], c = warp_eq[w];
      if (w < warp) { g += a; e += c; }
      tg += a;
      te += c;
    }
    place(p, gt, eq, mg, me, g, e);
    gt0 += tg;
    eq0 += te;
    __syncthreads();
  }
}

}  // namespace pages
}  // namespace mla
