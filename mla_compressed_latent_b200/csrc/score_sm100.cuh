// Page scores on the sm_100a tensor cores.
//
//   u[h, p] = sm_scale q[h, :] · key_p          score[p] = sum_h exp(u[h, p] - logsumexp_p u[h, :])
//
// for every token v, over the pages p it sees. The softmax runs over the pages of one head and the sum over
// the heads of one page, so a token needs all of u before it can write anything. u never leaves the
// SM: the 128 heads are the M rows of the product and pages its N columns, and an accumulator of 128
// lanes x 512 columns is exactly the tensor memory of one SM. A cluster of 1 to 8 CTAs takes one
// token, up to 512 pages each. A CTA puts e = exp(u - its head's maximum) in u's place, the CTAs swap each
// head's maximum and sum through distributed shared memory, and e times one factor a head is then summed
// over the heads: each exponential is computed once.
// Bound: q (128 rows) and the keys, read once per token (keys of one sequence come from L2 after the first
// token); 2 · 128 · (d_c + d_r) operations a page.
//
// Warps 0-7 gather the keys (a page's key lies wherever the block table says, so rows are fetched 16 bytes a
// thread with asynchronous copies into 128-byte swizzled stages of 128 pages x 64 columns), then turn
// the accumulator into masses; warp 8 loads q by TMA and issues the products. The column chunks are the
// outer loop and the page tiles the inner one: all tiles' accumulators live at once, so only the chunk of q
// at hand has to be in shared memory. 8 sequences of 16K-128K positions, 2 tokens each (6 CTAs a token; from
// the start of the longest's): page table 3.4 us, keys gathered 13.5 (27 stages, 16 KB in 0.35 us whatever is in
// flight), products done 14.6, exponentials 16.6, exchanged 17.7, summed 20.4; 33 us with q resident and
// clusters of powers of two, 23 us with every exponential computed twice and eight stages ahead. 64 sequences of
// 4096 positions, a token each: 9.2 us (10.7 with three chunks of q), latency.
#pragma once

#include "common.cuh"
#include "gemm_sm100.cuh"
#include "pages.cuh"
#include "ptx_sm100.cuh"
#include "tmap.cuh"

namespace mla {
namespace score {

constexpr int kH = 128;               // accumulator rows: heads, padded
constexpr int kTile = 128;            // pages per product
constexpr int kMaxPages = 512;        // pages per CTA: the accumulator's columns
constexpr int kMaxChunks = 9;         // 64-column chunks of a row of up to 576 values
// Key stages and chunks of q in shared memory. Six of each: the copies' issue bounds the gather, not what is in
// flight (two to eight stages ahead bring a long context's keys in the same time, but what is handed over late
// delays the products), and with one tile of pages the query is the larger part of what a CTA loads. For
// many tokens of at most one tile, three of each, so that two CTAs share an SM and one's latencies hide the
// other's (336 tokens of 11-18 pages: 33 us with one CTA, 21 us with two).
constexpr int kStagesOne = 6, kStagesTwo = 3;
constexpr int kStageBytes = kTile * 128;
constexpr int kQChunkBytes = kH * 128;
constexpr int kWorkers = 256;         // threads of warps 0-7
constexpr int kThreads = kWorkers + 32;
constexpr int kMaxCluster = 8;
template <int kStages>
struct Layout {
  static constexpr int kAhead = kStages > 3 ? 3 : 2;   // stages a thread's copies run ahead of what it has handed over
  static constexpr int kQSlots = kStages;
  static constexpr int kOffRing = kQSlots * kQChunkBytes;
  static constexpr int kClusters = kStages == kStagesTwo ? 1 : kMaxCluster;
  static constexpr int kTmemCols = kStages == kStagesTwo ? kTile : kMaxPages;
  static_assert(4 * kMaxPages * 4 <= kOffRing, "the column sums fit the query's place");
  static constexpr int kOffStats = kOffRing + kStages * kStageBytes;   // float2 [cluster][2][kH]
  static constexpr int kOffBar = kOffStats + kClusters * 2 * kH * 8;
  static constexpr int FULL = 0, EMPTY = FULL + kStages, Q_FULL = EMPTY + kStages, Q_EMPTY = Q_FULL + kQSlots,
                       DONE = Q_EMPTY + kQSlots, NUM_BARS = DONE + 1;
  static constexpr int kOffSlot = kOffBar + NUM_BARS * 8;
  static constexpr int kSmemBytes = kOffSlot + 16 + 1024;   // + alignment slack of the dynamic base
};
static_assert(Layout<kStagesOne>::kSmemBytes <= 232448, "shared memory budget");
static_assert(2 * (Layout<kStagesTwo>::kSmemBytes + 1024) <= 233472, "two CTAs to an SM");

constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(kH, kTile, false);

struct Params {
  const __nv_bfloat16* keys;
  int64_t key_stride;
  const int32_t* block_table;
  int max_pages, num_pages;
  const int32_t* seqlens;
  int s_q, H, W;
  float scale_log2;
  float* scores;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  const uint32_t n = live ? 16u : 0u;   // 0: the 16 bytes are zeros and src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory"); }

template <int kStages>
__global__ void __launch_bounds__(kThreads, kStages == kStagesTwo ? 2 : 1)
score_kernel(const __grid_constant__ CUtensorMap tm_q, const Params p) {
  using La = Layout<kStages>;
  constexpr int FULL = La::FULL, EMPTY = La::EMPTY, Q_FULL = La::Q_FULL, Q_EMPTY = La::Q_EMPTY, DONE = La::DONE;
  constexpr int kOffBar = La::kOffBar, kOffSlot = La::kOffSlot, kOffStats = La::kOffStats, kAhead = La::kAhead;
  constexpr int kTiles = La::kTmemCols / kTile;   // most tiles of a CTA
  constexpr int kQSlots = La::kQSlots, kOffRing = La::kOffRing;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int v = (int)ptx::cluster_id_x();
  const int csize = (int)(gridDim.x / ptx::num_clusters_x());
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * (uint32_t)i; };
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + kOffSlot + 8);

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) { ptx::mbar_init(bar(FULL + i), kWorkers / 32); ptx::mbar_init(bar(EMPTY + i), 1); }
    for (int i = 0; i < kQSlots; ++i) { ptx::mbar_init(bar(Q_FULL + i), 1); ptx::mbar_init(bar(Q_EMPTY + i), 1); }
    ptx::mbar_init(bar(DONE), 1);
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tm_q);
  }
  if (warp == 8) { ptx::tmem_alloc(base + kOffSlot, La::kTmemCols); ptx::tmem_relinquish(); }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_arrive();   // waited for before the first store into another CTA: by then it has started
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + kOffSlot);
  grid_dependency_wait();
  allow_dependents();

  // this CTA's pages: [p0, p0 + n) of the token's
  const int seq = v / p.s_q;
  int n_all = pages::visible_pages(p.seqlens[seq], p.s_q, v % p.s_q);
  if (n_all > p.max_pages) {
    if (tid == 0 && rank == 0) report(MLA_ERR_DEVICE_CHECK);
    n_all = p.max_pages;
  }
  const int per = ((n_all + csize - 1) / csize + 31) / 32 * 32;
  const int p0 = min(n_all, (int)rank * per), n = min(n_all - p0, per);
  const int tiles = (n + kTile - 1) / kTile, chunks = (p.W + 63) / 64, total = tiles * chunks;
  float2* stats = reinterpret_cast<float2*>(gbase + kOffStats);

  if (warp < 8) {
    // ---- gather: rows r0 + 32 u of each tile, one 16-byte piece of the chunk's 128 bytes
    constexpr int kU = kTile / 32;
    const int r0 = tid >> 3, piece = tid & 7;
    const uint32_t dst0 = base + kOffRing + (uint32_t)r0 * 128u + (((uint32_t)piece ^ ((uint32_t)r0 & 7u)) << 4);
    const int32_t* table = p.block_table + (int64_t)seq * p.max_pages + p0;
    int pg[kTiles][kU];   // the pages of this thread's rows, tile by tile; -1: zeros
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int row = t * kTile + r0 + 32 * u;
        pg[t][u] = row < n ? table[row] : -1;
      }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (pg[t][u] < 0 || pg[t][u] >= p.num_pages) {
          if (t * kTile + r0 + 32 * u < n) report(MLA_ERR_DEVICE_CHECK);
          pg[t][u] = -1;
        }
    bool live = true;
    for (int i = 0, kc = 0, tile = 0; i < total + kAhead; ++i) {
      if (i < total && live) {
        const int s = i % kStages;
        if (i >= kStages) live = __all_sync(0xffffffffu, gemm::wait(bar(EMPTY + s), ((i / kStages) & 1u) ^ 1u, abort));
        if (live) {
          const int col = kc * 64 + piece * 8;
          const bool in = col < p.W;
          const uint32_t dst = dst0 + (uint32_t)s * kStageBytes;
          const __nv_bfloat16* k0 = p.keys + (in ? col : 0);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            if (t != tile) continue;
#pragma unroll
            for (int u = 0; u < kU; ++u)
              cp_async16(dst + u * 32 * 128, k0 + (int64_t)max(pg[t][u], 0) * p.key_stride, in && pg[t][u] >= 0);
          }
        }
        if (++tile == tiles) { tile = 0; ++kc; }
      }
      cp_async_commit();
      if (i >= kAhead && live) {   // this warp's copies of stage i - kAhead have landed: hand it over
        cp_async_wait<kAhead>();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(FULL + (i - kAhead) % kStages));
      }
    }
    cp_async_wait<0>();
    if (!live) *abort = 1;
    // ---- per head (= lane of the accumulator): maximum and sum of exponentials over this CTA's pages; warps
    // 0-3 take the first half of each tile, 4-7 the second
    __syncwarp();
    const int q4 = warp & 3, half = warp >> 2, head = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const bool ok = __all_sync(0xffffffffu, gemm::wait(bar(DONE), 0, abort));
    ptx::tc_fence_after();
    const float s2 = p.scale_log2;
    // the maximum first, so that the exponentials, which go back into the accumulator's place, share one
    // reference and are never computed again (the exponential unit is what these passes are bound by)
    auto load = [&](int t, uint32_t (&r0v)[32], uint32_t (&r1v)[32]) {   // 64 pages; those past the end at -inf
      const int c = half * (kTile / 2), valid = n - t * kTile - c;
      ptx::tmem_ld32(tmem + lane_off + (uint32_t)(t * kTile + c), r0v);
      ptx::tmem_ld32(tmem + lane_off + (uint32_t)(t * kTile + c + 32), r1v);
      ptx::tmem_wait_ld_regs(r0v);
      ptx::tmem_wait_ld_regs(r1v);
      if (valid < 64) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (j >= valid) r0v[j] = 0xff800000u;
          if (32 + j >= valid) r1v[j] = 0xff800000u;
        }
      }
    };
    const int mine = ok ? max(0, (n - half * (kTile / 2) + kTile - 1) / kTile) : 0;   // tiles this half has pages of
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, sm[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int t = 0; t < mine; ++t) {
      uint32_t r0v[32], r1v[32];
      load(t, r0v, r1v);
#pragma unroll
      for (int j = 0; j < 32; ++j)
        mx[j & 3] = fmaxf(mx[j & 3], fmaxf(__uint_as_float(r0v[j]), __uint_as_float(r1v[j])));
    }
    // (nothing but -inf here: exponents against 0, so that they are masses of 0 and the sum is 0, or NaN)
    const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), off = m == -INFINITY ? 0.f : -m * s2;
#pragma unroll 1
    for (int t = 0; t < mine; ++t) {
      uint32_t r0v[32], r1v[32];
      load(t, r0v, r1v);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float e0 = ptx::ex2_approx(fmaf(__uint_as_float(r0v[j]), s2, off));
        const float e1 = ptx::ex2_approx(fmaf(__uint_as_float(r1v[j]), s2, off));
        sm[j & 3] += e0;
        sm[(j + 2) & 3] += e1;
        r0v[j] = __float_as_uint(e0);
        r1v[j] = __float_as_uint(e1);
      }
      ptx::tmem_st32(tmem + lane_off + (uint32_t)(t * kTile + half * (kTile / 2)), r0v);
      ptx::tmem_st32(tmem + lane_off + (uint32_t)(t * kTile + half * (kTile / 2) + 32), r1v);
    }
    ptx::tmem_wait_st();
    const float l = (sm[0] + sm[1]) + (sm[2] + sm[3]);
    __syncwarp();
    ptx::cluster_wait();
    for (int r = 0; r < csize; ++r) {
      const uint32_t at = ptx::map_to_cta(base + kOffStats + (uint32_t)(((int)rank * 2 + half) * kH + head) * 8u, (uint32_t)r);
      ptx::st_cluster_f32(at, m);
      ptx::st_cluster_f32(at + 4u, l);
    }
  } else {
    // ---- q by TMA, chunk by chunk, and the products
    auto load_q = [&](int kc) {   // (lane 0; its slot is free)
      const int s = kc % kQSlots;
      const uint32_t dst = base + s * kQChunkBytes;
      ptx::mbar_arrive_expect_tx(bar(Q_FULL + s), kQChunkBytes);
      ptx::tma_load_2d(dst, &tm_q, kc * 64, v * p.H, bar(Q_FULL + s));
      ptx::tma_load_2d(dst + kQChunkBytes / 2, &tm_q, kc * 64, v * p.H + 64, bar(Q_FULL + s));
    };
    int loaded = 0;
    if (tiles > 0)
      for (; loaded < min(chunks, kQSlots - 1); ++loaded)
        if (lane == 0) load_q(loaded);
    __syncwarp();
    const uint64_t qd = ptx::smem_desc_sw128(base, 16, 1024), kd = ptx::smem_desc_sw128(base + kOffRing, 16, 1024);
    bool live = true;
    for (int i = 0, kc = 0, tile = 0; i < total && live; ++i) {
      const int s = i % kStages, qs = kc % kQSlots;
#ifdef MLA_TEST_HOOKS
      if (test_stall(1, i)) {
        live = __all_sync(0xffffffffu, gemm::wait(bar(DONE), 0, nullptr, kTestStallNs));
        if (!live) break;
      }
#endif
      if (tile == 0) {
        if (loaded < chunks) {   // the next chunk into the slot whose products were issued a chunk ago
          live = __all_sync(0xffffffffu, gemm::wait(bar(Q_EMPTY + loaded % kQSlots), ((loaded / kQSlots) & 1u) ^ 1u, abort));
          if (!live) break;
          if (lane == 0) load_q(loaded);
          ++loaded;
          __syncwarp();
        }
        live = __all_sync(0xffffffffu, gemm::wait(bar(Q_FULL + qs), (kc / kQSlots) & 1u, abort));
      }
      live = live && __all_sync(0xffffffffu, gemm::wait(bar(FULL + s), (i / kStages) & 1u, abort));
      if (live && ptx::elect_one()) {
        ptx::tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ptx::mma_ss(tmem + (uint32_t)(tile * kTile), qd + (uint64_t)(qs * (kQChunkBytes >> 4) + 2 * k),
                      kd + (uint64_t)(s * (kStageBytes >> 4) + 2 * k), kIdesc, (kc | k) ? 1u : 0u);
        ptx::mma_commit(bar(EMPTY + s));
        if (tile == tiles - 1) ptx::mma_commit(bar(Q_EMPTY + qs));
        if (i == total - 1) ptx::mma_commit(bar(DONE));
      }
      __syncwarp();
      if (++tile == tiles) { tile = 0; ++kc; }
    }
    if (total == 0 && lane == 0) ptx::mbar_arrive(bar(DONE));
    if (!live) {
      *abort = 1;
      if (ptx::elect_one()) ptx::mma_commit(bar(DONE));   // what was issued completes before the exit
      for (int kc = max(0, loaded - kQSlots); kc < loaded; ++kc) gemm::wait(bar(Q_FULL + kc % kQSlots), (kc / kQSlots) & 1u);   // and so do the loads
      gemm::wait(bar(DONE), 0);
    }
    __syncwarp();
    ptx::cluster_wait();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();   // every CTA's statistics are in place
  ptx::tc_fence_after();
  if (warp < 8 && !*abort) {
    const int q4 = warp & 3, half = warp >> 2, head = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const float s2 = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    for (int r = 0; r < 2 * csize; ++r) m = fmaxf(m, stats[r * kH + head].x);
    for (int r = 0; r < 2 * csize; ++r) {
      const float2 st = stats[r * kH + head];
      if (st.y != 0.f) l += st.y * ptx::ex2_approx((st.x - m) * s2);
    }
    // what this half's exponentials are to be multiplied by
    const float own = stats[((int)rank * 2 + half) * kH + head].x;
    const float f = head < p.H ? ptx::ex2_approx((own - m) * s2) / l : 0.f;
    // masses, summed over the warp's 32 heads: at each step a lane keeps half of its columns and
    // adds the other lane's values of them, so that of 64 columns lane j ends with 2 j and 2 j + 1
    float* colsum = reinterpret_cast<float*>(gbase);   // [4][kMaxPages], over the query (its products are done)
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
      const int c = half * (kTile / 2);
      if (t * kTile + c >= n) break;
      uint32_t r0v[32], r1v[32];
      ptx::tmem_ld32(tmem + lane_off + (uint32_t)(t * kTile + c), r0v);
      ptx::tmem_ld32(tmem + lane_off + (uint32_t)(t * kTile + c + 32), r1v);
      ptx::tmem_wait_ld_regs(r0v);
      ptx::tmem_wait_ld_regs(r1v);
      float a[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) {
        const float e = __uint_as_float(j < 32 ? r0v[j & 31] : r1v[j & 31]) * f;
        a[j] = head < p.H ? e : 0.f;   // (rows past the last head may hold anything)
      }
#pragma unroll
      for (int o = 32; o > 1; o >>= 1) {
        const bool up = (lane & (o >> 1)) != 0;
#pragma unroll
        for (int j = 0; j < o; ++j) {
          const float send = up ? a[j] : a[j + o], keep = up ? a[j + o] : a[j];
          a[j] = keep + __shfl_xor_sync(0xffffffffu, send, o >> 1);
        }
      }
      // lane j holds columns 2 j and 2 j + 1
      *reinterpret_cast<float2*>(&colsum[q4 * kMaxPages + t * kTile + c + 2 * lane]) = make_float2(a[0], a[1]);
    }
    ptx::tc_fence_before();
    ptx::named_bar_sync(1, kWorkers);
    float* out = p.scores + (int64_t)v * p.max_pages + p0;
    for (int i = tid; i < n; i += kWorkers)
      out[i] = (colsum[i] + colsum[kMaxPages + i]) + (colsum[2 * kMaxPages + i] + colsum[3 * kMaxPages + i]);
  }
  __syncthreads();
  if (warp == 8) {
    gemm::wait(bar(DONE), 0);   // (also where the workers gave up before the products were done)
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, La::kTmemCols);
  }
}

// ---- host ----------------------------------------------------------------------------------------
inline bool supported(const mla_dims_t* d, int32_t dtype, int64_t rows, int32_t max_pages) {
  const int W = d->d_c + d->d_r;
  return dtype == MLA_BF16 && d->H <= kH && W >= 64 && W <= 64 * kMaxChunks && W % 8 == 0 && max_pages <= kMaxCluster * kMaxPages &&
         rows * d->H <= INT32_MAX && rows * kMaxCluster <= INT32_MAX;
}

// Clusters of c CTAs that the device runs at once, asked once.
inline int resident_clusters(int c, int num_sms) {
  static int cached[64][kMaxCluster + 1] = {{0}};
  int dev = 0;
  cudaGetDevice(&dev);
  const bool known = dev >= 0 && dev < 64;
  if (known && cached[dev][c]) return cached[dev][c];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_sms / c * c));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<kStagesOne>::kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, score_kernel<kStagesOne>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = num_sms / c;
  }
  if (known) cached[dev][c] = n;
  return n;
}

inline int launch_score(const mla_dims_t* d, int32_t rows, int32_t s_q, const void* q_abs, const void* keys, int64_t key_stride,
                        int32_t num_pages, const int32_t* block_table, int32_t max_pages, const int32_t* seqlens,
                        float scale, float* scores, int num_sms, cudaStream_t st) {
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    if (cudaFuncSetAttribute(score_kernel<kStagesOne>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Layout<kStagesOne>::kSmemBytes) != cudaSuccess ||
        cudaFuncSetAttribute(score_kernel<kStagesTwo>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Layout<kStagesTwo>::kSmemBytes) != cudaSuccess)
      return MLA_ERR_CUDA;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  const int W = d->d_c + d->d_r;
  CUtensorMap tm_q;   // q_abs as [rows * H, W]: boxes of 64 heads x 64 columns
  if (!tmap::make_bf16_sw128(&tm_q, q_abs, W, (int64_t)rows * d->H, W, 64)) return MLA_ERR_INVALID_ARG;
  // as few CTAs a token as hold its pages, more while all tokens' clusters still run at once and a CTA has
  // half a tile
  int c = (max_pages + kMaxPages - 1) / kMaxPages;
  // (a cluster lies within one GPC: fewer than num_sms / c of them may run at once)
  while (c < kMaxCluster && rows <= resident_clusters(c + 1, num_sms) && max_pages > c * kTile / 2) ++c;
  Params prm{reinterpret_cast<const __nv_bfloat16*>(keys), key_stride, block_table, max_pages, num_pages, seqlens, s_q,
             d->H, W, scale * 1.4426950408889634f, scores};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * c));
  cfg.blockDim = dim3(kThreads);
  const bool many_short = rows > num_sms && max_pages <= kTile;
  cfg.dynamicSmemBytes = many_short ? Layout<kStagesTwo>::kSmemBytes : Layout<kStagesOne>::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, many_short ? score_kernel<kStagesTwo> : score_kernel<kStagesOne>, tm_q, prm);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace score
}  // namespace mla
