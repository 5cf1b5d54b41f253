// Projection of many tokens by pairs of SMs:  part[split, tok, m] = sum over the split's k of x[tok, k] W[k, m]
//
// With thousands of tokens the projection is bound by what L2 delivers to all SMs together (about 9 TB/s), so the
// tile is the one that moves the fewest bytes per product. A pair of CTAs shares one product of M = 256
// features and N = 256 tokens (each SM's tensor core reads both CTAs' shared memory): a CTA loads its own 128
// features and half of the tokens, and two such products side by side fill all 512 accumulator columns of
// both SMs: 256 features x 512 tokens a pair, 48 KB a CTA and K chunk of 64 where a CTA of its own loads 64 KB
// for the same products. 4096 tokens, C = 7168, 576 features (three K splits, 72 pairs): about 31 us, where tiles of 256 x
// 256 by single CTAs took 41 us, 384 x 128 49 us and 128 x 128 64 us; the products alone want 38,000 cycles (the
// last tile's 64 of 256 features cost a whole one), the 236 MB out of L2 26 us.
#pragma once

#include "common.cuh"
#include "gemm_sm100.cuh"
#include "ptx_sm100.cuh"
#include "tmap.cuh"

namespace mla {
namespace gemm_pair {

constexpr int kPairM = 256;            // features per pair
constexpr int kBlockN = 256;           // tokens per product
constexpr int kPairN = 2 * kBlockN;    // tokens per pair
constexpr int kBK = 64;
constexpr int kStages = 4;
constexpr int kABytes = kBK * 128 * 2;           // this CTA's 128 features: two boxes of 64 k-rows x 64 features
constexpr int kBBytes = (kBlockN / 2) * kBK * 2; // its half of a product's tokens: one box of 128 rows x 64 k
constexpr int kStageBytes = kABytes + 2 * kBBytes;
constexpr int kBarBytes = 1024;
constexpr int kSmemBytes = 1024 + kBarBytes + kStages * kStageBytes;
constexpr int kThreads = 256;          // warp 0 TMA producer, 1 MMA issuer (CTA 0), 2 TMEM; then all eight: epilogue
constexpr int kTmemCols = 512;
static_assert(kSmemBytes <= 232448 && kStageBytes % 1024 == 0, "shared memory");

struct Params {
  int M, n_tok;
  int chunks, chunks_per_split;
  float* part;     // [splits, n_tok, M]
};

// The paired forms (cta_group::2): one thread of CTA 0 issues; both CTAs hold their part at the same offsets.
__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(kTmemCols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kTmemCols) : "memory");
}
__device__ __forceinline__ void mma2_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum) : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(bar), "h"((uint16_t)3) : "memory");
}
// A tile into this CTA's shared memory, counted on a barrier of either CTA of the pair (a cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar_cluster) : "memory");
}

// Bounded wait for a phase that arrivals from either CTA complete; false on expiry (recorded) or abort.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const volatile int* abort,
                                     uint64_t limit_ns = gemm::kTimeoutNs) {
  uint64_t t0 = 0;
  for (uint32_t n = 0;; ++n) {
    if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
    if ((n & 15u) == 15u) {
      if (abort && *abort) return false;
      const uint64_t now = ptx::globaltimer();
      if (t0 == 0) t0 = now;
      else if (now - t0 > limit_ns) { report(MLA_ERR_TIMEOUT); return false; }
    }
  }
}

// Cluster (2 CTAs) x = m-tile of 256 features, y = block of 512 tokens, z = K split.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
pair_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int f0 = (int)(blockIdx.x >> 1) * kPairM + (int)rank * 128;   // this CTA's first feature
  const int tok0 = (int)blockIdx.y * kPairN;
  const int nblk = p.n_tok - tok0 > kBlockN ? 2 : 1;
  const int kc0 = (int)blockIdx.z * p.chunks_per_split;
  const int nk = max(0, min(p.chunks, kc0 + p.chunks_per_split) - kc0);
  const uint32_t full0 = base, empty0 = base + 8u * kStages, done = base + 16u * kStages, slot = done + 8u;
  const uint32_t abort_addr = done + 16u;
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + (abort_addr - base));
  const uint32_t begun_addr = abort_addr + 4u;   // K chunks this CTA's producer has begun
  volatile int* begun = reinterpret_cast<volatile int*>(gbase + (begun_addr - base));
  const uint32_t ring = base + kBarBytes;

  if (threadIdx.x == 0) {
    // full (CTA 0's): one arrival and the bytes of both CTAs; empty, done: one commit each
    for (int s = 0; s < kStages; ++s) { ptx::mbar_init(full0 + 8u * s, 1); ptx::mbar_init(empty0 + 8u * s, 1); }
    ptx::mbar_init(done, 1);
    *abort = 0;
    *begun = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tm_w);
    ptx::prefetch_tmap(&tm_x);
  }
  if (warp == 2) tmem_alloc2(slot);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // both CTAs' barriers are initialised
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + (slot - base));
  auto give_up = [&]() {   // in both CTAs
    *abort = 1;
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ptx::map_to_cta(abort_addr, rank ^ 1u)), "r"(1) : "memory");
  };

  const uint32_t full_cta0 = ptx::map_to_cta(full0, 0);
  const uint32_t pair_bytes = 2u * (uint32_t)(kABytes + nblk * kBBytes);
  auto begin_stage = [&](int i) {   // stage of chunk i: CTA 0 announces both CTAs' bytes; the weights
    const uint32_t s = (uint32_t)(i % kStages), st = ring + s * kStageBytes;
    if (rank == 0) ptx::mbar_arrive_expect_tx(full0 + 8u * s, pair_bytes);
    // (features past M read the fill value)
    tma_load_2d_pair(st, &tm_w, f0, (kc0 + i) * kBK, full_cta0 + 8u * s);
    tma_load_2d_pair(st + kABytes / 2, &tm_w, f0 + 64, (kc0 + i) * kBK, full_cta0 + 8u * s);
  };
  auto load_tokens = [&](int i) {   // (tokens past n_tok read zeros)
    const uint32_t s = (uint32_t)(i % kStages), st = ring + s * kStageBytes;
    for (int nb = 0; nb < nblk; ++nb)
      tma_load_2d_pair(st + kABytes + nb * kBBytes, &tm_x, (kc0 + i) * kBK,
                       tok0 + nb * kBlockN + (int)rank * (kBlockN / 2), full_cta0 + 8u * s);
  };
  // The first two stages' weights are not written by the kernel before this one (as in the projections for
  // fewer tokens); everything else waits for it.
  const int pre = min(nk, 2);
  if (warp == 0 && lane == 0)
    for (int i = 0; i < pre; ++i) begin_stage(i);
  grid_dependency_wait();
  allow_dependents();

  if (warp == 0 && lane == 0) {
    // ---- TMA producer
    int i = 0;
    for (; i < nk; ++i) {
      const uint32_t s = (uint32_t)(i % kStages);
      if (i >= pre) {
        if (!wait(empty0 + 8u * s, ((i / kStages) & 1u) ^ 1u, abort)) { give_up(); break; }
        begin_stage(i);
      }
      load_tokens(i);
    }
    *begun = i;
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- MMA issuer: four K = 16 steps a chunk and product, M = 256 (both CTAs' features), N = 256
    const uint32_t idesc = ptx::idesc_bf16_f32_ab(kPairM, kBlockN, true, false);
    bool live = true;
    for (int i = 0; i < nk && live; ++i) {
#ifdef MLA_TEST_HOOKS
      if (test_stall(1, i) && !(live = wait(done, 0, nullptr, kTestStallNs))) break;
#endif
      const uint32_t s = (uint32_t)(i % kStages), st = ring + s * kStageBytes;
      if (!wait(full0 + 8u * s, (i / kStages) & 1u, abort)) { live = false; break; }
      ptx::tc_fence_after();
      // A, MN-major: 8-row K groups 1024 B apart, the two 64-feature halves one box apart; a K step of 16
      // moves 2048 B. B, K-major: 8-token groups 1024 B apart; a K step moves 32 B inside the swizzle row.
      const uint64_t ad = ptx::smem_desc_sw128(st, kABytes / 2, 1024);
      for (int nb = 0; nb < nblk; ++nb) {
        const uint64_t bd = ptx::smem_desc_sw128(st + kABytes + nb * kBBytes, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma2_ss(tmem + (uint32_t)(nb * kBlockN), ad + (uint64_t)(k * (2048 >> 4)), bd + (uint64_t)(2 * k), idesc,
                  (i | k) ? 1u : 0u);
      }
      commit2(empty0 + 8u * s);
    }
    if (!live) give_up();
    commit2(done);
  }
  __syncwarp();
  // ---- epilogue: lane = feature, 32 tokens (accumulator columns) at a time through a 4 KB [token][feature] tile
  // of the ring (free: every product is done), stored as 16-byte pieces. Warps 4-7 take the first product's
  // tokens and warps 0-3 the second's; of a single product each set takes every other 32.
  {
    const bool ok = __all_sync(0xffffffffu, wait(done, 0, nullptr) && !*abort);
    ptx::tc_fence_after();
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    uint8_t* tile = gbase + kBarBytes + warp * 4096;
    const uint32_t tile_s = ring + (uint32_t)warp * 4096u;
    const int fw = f0 + (warp & 3) * 32;   // the warp's first feature
    const int set = warp >= 4 ? 0 : 1;
    const int c0 = nblk == 2 ? set * kBlockN : 32 * set, c1 = nblk == 2 ? c0 + kBlockN : kBlockN;
    if (ok && fw < p.M) {
      for (int c = c0; c < c1 && tok0 + c < p.n_tok; c += nblk == 2 ? 32 : 64) {
        uint32_t r[32];
        ptx::tmem_ld32(tmem + lane_off + (uint32_t)c, r);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) reinterpret_cast<float*>(tile)[k * 32 + lane] = nk > 0 ? __uint_as_float(r[k]) : 0.f;
        __syncwarp();
        const int kn = min(32, p.n_tok - tok0 - c);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = lane + 32 * u, t = i / 8, f = fw + (i % 8) * 4;
          if (t >= kn || f >= p.M) continue;
          const uint4 v = ptx::ld_shared_v4(tile_s + (uint32_t)i * 16u);
          *reinterpret_cast<uint4*>(p.part + ((int64_t)blockIdx.z * p.n_tok + tok0 + c + t) * p.M + f) = v;
        }
        __syncwarp();
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // both CTAs have read their accumulators, and nobody issues any more
  if (*abort) {   // (the same in both CTAs)
    // After a failure what was issued must still land before the CTAs may exit (otherwise the issuer waited for every
    // stage). A stage's barrier counts both CTAs' bytes and one producer may have begun up to kStages more chunks
    // than the other: what one has begun the other completes (the stage is free in both), and CTA 0, whose barriers
    // they are, waits for all of them.
    if (threadIdx.x == 0) {
      int other;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(other) : "r"(ptx::map_to_cta(begun_addr, rank ^ 1u)) : "memory");
      const int own = *begun, n = max(own, other);
      for (int i = own; i < n; ++i) { begin_stage(i); load_tokens(i); }
      if (rank == 0)
        for (int k = max(0, n - kStages); k < n; ++k) wait(full0 + 8u * (k % kStages), (k / kStages) & 1u, nullptr);
    }
    __syncwarp();
    ptx::cluster_sync();   // no load is in flight to either CTA
  }
  if (warp == 2) {
    wait(done, 0, nullptr);   // (the products are done, also where the epilogue gave up before the issuer ended them)
    ptx::tc_fence_after();
    __syncwarp();
    tmem_dealloc2(tmem);
  }
  ptx::cluster_sync();
}

// ---- host ----------------------------------------------------------------------------------------
// K splits: those that cost the fewest chunks' time (0.7 us). A tile costs kTileChunks more than its own (its start,
// its last stages and its stores), and a split what its sums cost to write and to read back: one for the
// latency of a slice in the finish and one per kSplitTokens tokens. (The whole append, C = 7168:
// 1024 tokens 25.3 us with 12 splits, 23.9 with 7; 8192 tokens 86 us with 1, 79 with 3. C = 2048: 4096 tokens 24.6
// us with 2, 22.1 with 3; 8192 tokens 37.8 us with 1, 43.6 with 3.)
constexpr int kTileChunks = 6, kSplitTokens = 1536, kMaxSplits = 24;
inline int plan_splits(int M, int K, int n_tok, int num_sms) {
  const int64_t tiles = (int64_t)((M + kPairM - 1) / kPairM) * ((n_tok + kPairN - 1) / kPairN);
  const int chunks = K / kBK, pairs = num_sms / 2;
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int ks = 1; ks <= std::min(chunks, kMaxSplits); ++ks) {
    const int per = (chunks + ks - 1) / ks;
    if ((chunks + per - 1) / per != ks) continue;   // (an empty split)
    const int64_t cost = (tiles * ks + pairs - 1) / pairs * (per + kTileChunks) + ks + (int64_t)ks * n_tok / kSplitTokens;
    if (cost < best_cost) { best_cost = cost; best = ks; }
  }
  return best;
}

// w [K, M], x [n_tok, K] bf16, K % 64 == 0, M % 8 == 0, all 16-byte aligned; part fp32 [splits, n_tok, M].
inline int run(const void* w, const void* x, int K, int M, int n_tok, int splits, float* part, cudaStream_t st) {
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  const bool known = dev >= 0 && dev < 64;
  if (!known || !attr_done[dev]) {
    if (cudaFuncSetAttribute(pair_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
      return MLA_ERR_CUDA;
    if (known) attr_done[dev] = true;
  }
  CUtensorMap tm_w, tm_x;
  if (!tmap::make_bf16_sw128(&tm_w, w, M, K, M, kBK) || !tmap::make_bf16_sw128(&tm_x, x, K, n_tok, K, kBlockN / 2))
    return MLA_ERR_INVALID_ARG;
  const int chunks = K / kBK;
  const Params prm{M, n_tok, chunks, (chunks + splits - 1) / splits, part};
  launch_pdl(pair_gemm_kernel, dim3(2 * ((M + kPairM - 1) / kPairM), (n_tok + kPairN - 1) / kPairN, splits), dim3(kThreads),
             kSmemBytes, st, tm_w, tm_x, prm);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace gemm_pair
}  // namespace mla
