// Absorbed decode over selected pages of an 8-bit latent cache, on the sm_100a tensor cores, straight
// from the stored codes.
//
//   S[h, j] = s_j (q_h · code_j) + q_r,h · k_r,j        O[h, :] = sum_j (P[h, j] s_j) code_j
//
// A row's scale s_j multiplies a column of S and a column of P, so no dequantised row is ever made
// and the cache's bytes cross the memory system once, at 644 a position where 16-bit rows take 1152.
// S is an E4M3 product of the codes as they lie in the cache (K-major). It wants E4M3 queries too, and
// four significant bits are too few, but two terms hold eight: q 2^t = q_hi + q_lo, the nearest E4M3
// value and the nearest to what is left. t brings the head's largest value to 128..256; the sum is
// the bf16 value itself down to a thousandth of that, and off by at most 2^-10 (2^-18 of the
// largest) below. An 8-bit product of K = 32 takes the time of a 16-bit one of K = 16, so the two terms cost
// what the 16-bit decode pays, with half the bytes to load and to keep in shared memory.
// O is an fp16 product: the output CTA's row warps widen the codes (every E4M3 value is an fp16 value)
// on their way into shared memory, and the weights w = P s are rounded to fp16's 11 bits. (An E4M3
// product there, with the weights in two terms, would read the codes MN-major; 8-bit MN-major operands
// ran at a third of the rate: 380 cycles for M = 128, N = 256, K = 32, against 128.)
//
// The frame is that of decode_sm100.cuh: a pair of CTAs per worker (the score CTA holds q_hi and q_lo in
// 256 TMEM columns and two score buffers of 64 + 64, the latents' products and the RoPE keys' apart
// because only the former are scaled; the output CTA holds O in 512), eight row warps in two sets on
// alternate tiles, P tiles handed over by bulk copies, lazy running maxima, ranges of tiles per pair and one
// merge of cut rows. The reference M of a row's exponentials includes the scales: e = 2^(x - M) with
// M >= max_j (x_j + E_j) - 14 and 2^E_j above the scale of row j, so that w = e s stays below 2^14 and the
// largest is 2^-3 or more: fp16 holds every weight that counts, whatever the scales are; l sums the same e, and
// O / l and M + log2 l need no correction. Rows of one tile mostly have scales of a size (RMSNorm), and the
// largest E then stands for all; a tile whose scales are further apart than 2^kNearLog2 takes each row's own.
//
// 64 rows of 40 pages (105 MB of codes, scales and keys, 46 GFLOP with the second term not counted): 67-70 us, where a
// dequantising pass and the 16-bit decode took 124 us and attended rows rounded to bf16. A tile takes about
// 1650 cycles at 1.55 GHz: its 36 S MMAs run at 43 cycles each beside the loads and the softmax (34
// alone), and the widening's 64 KB of stores share the output CTA's shared memory with the MMAs' reads. About
// 20 us of the call lie outside the tiles (the query 7, the last tiles' hand-over 5, the epilogue 4, the launch).
#pragma once

#include "cache8.cuh"
#include "decode_sm100.cuh"

namespace mla {
namespace sm100f8 {

using sm100::kDC;
using sm100::kDR;
using sm100::kGroup;
using sm100::kH;
using sm100::kRow;
using sm100::kThreads;
using sm100::kTile;
using sm100::wait_bar;
using sm100::wait_bar_warp;

constexpr int kBoxBytes = 64 * 128;                    // 64 rows x 128 bytes: 128 codes, or 64 bf16
constexpr int kCodeBoxes = kDC / 128;                  // 4
constexpr int kKStages = 4;                            // score CTA: whole tiles, four code boxes and one of RoPE keys
constexpr int kKStageBytes = (kCodeBoxes + 1) * kBoxBytes;   // 40960
constexpr int kScaleBytes = kTile * 4;                 // the tile's 64 scales
// Scales have a ring of their own, twice as deep: the softmax of tile i reads them after the products of
// tile i are done. Tile i + 8 is loaded once the products of tile i + 4 are, which waited for the
// scores of tile i + 2 to be read, and a set reads those after it has finished tile i.
constexpr int kScaleSlots = 2 * kKStages;
constexpr int kVStages = 2;                            // output CTA: tiles of fp16 values
constexpr int kVChunks = kDC / 64;                     // 8 chunks of 64 rows x 64 values
constexpr int kVStageBytes = kVChunks * kBoxBytes;     // 65536
constexpr int kQBoxes = 2 * (kDC / 64);                // the query's latent part: 16 boxes of 64 heads x 64 columns
constexpr int kSBufs = 2;
constexpr int kSCol0 = 256;                            // buffer b: latent products at 256 + 128 b, RoPE products 64 on
constexpr int kTmemCols = 512;
constexpr int kPSlots = 4, kStaging = 2;
constexpr int kPBytes = kH * kTile * 2;                // a P tile: fp16 weights
constexpr int kAlphaOff = kPBytes;
constexpr int kCopyBytes = kPBytes + kH * 4;
constexpr int kStgStride = kCopyBytes;
constexpr int kSlotStride = 17408;                     // a multiple of 1024 (the swizzle repeat)
// M moves when a tile would take a weight past 2^14; it then leaves room for 2^8 more
constexpr float kTopLog2 = 14.0f, kRoomLog2 = 8.0f;
constexpr int kNearLog2 = 8;
// E at least this (a row of zeros has no E): e is at most 2^(14 - kMinLog2), so that a sum of 2^20 of them stays a
// float. Scales lose bits of their weights only below 2^(kMinLog2 - 20).
constexpr int kMinLog2 = -92;
// 2^E is above the magnitude of a scale
__device__ __forceinline__ int scale_log2(uint32_t bits) { return max((int)((bits >> 23) & 255u) - 126, kMinLog2); }

constexpr int kOffK = 0;
constexpr int kOffQR = kKStages * kKStageBytes;                       // the query's RoPE part, two boxes
constexpr int kOffStaging = kOffQR + 2 * kBoxBytes;
constexpr int kOffScale = kOffStaging + kStaging * kStgStride;
// the query's latent boxes pass through the three tile stages that the row's first tile does not take (five
// boxes a stage) and one box of their own, so that this tile is loaded while the query is converted
constexpr int kOffQX = (kOffScale + kScaleSlots * kScaleBytes + 1023) / 1024 * 1024;
constexpr int kOffQTop = kOffQX + kBoxBytes;           // uint32 [2][128]: each set's largest query magnitude per row
constexpr int kRegion0 = kOffQTop + 2 * kH * 4;
constexpr int kBoxesPerStage = kCodeBoxes + 1;
__device__ __forceinline__ uint32_t q_box(uint32_t base, uint32_t first_tile, int i) {   // address of box i
  if (i == kQBoxes - 1) return base + kOffQX;
  return base + kOffK + (uint32_t)((first_tile + 1 + i / kBoxesPerStage) % kKStages) * kKStageBytes +
         (uint32_t)(i % kBoxesPerStage) * kBoxBytes;
}
constexpr int kOffV = 0;
constexpr int kOffPSlots = kVStages * kVStageBytes;
constexpr int kOffEpi = kOffPSlots + kPSlots * kSlotStride;
constexpr int kEpiWarpBytes = 2048;
constexpr int kRegion1 = kOffEpi + 8 * kEpiWarpBytes;
constexpr int kRegion = kRegion0 > kRegion1 ? kRegion0 : kRegion1;
constexpr int kOffStats = kRegion;                     // float [128], as in the 16-bit decode
constexpr int kOffBar = kOffStats + kH * 4;
enum Bar : int {
  K_FULL = 0, K_EMPTY = K_FULL + kKStages, S_FULL = K_EMPTY + kKStages, S_EMPTY = S_FULL + kSBufs,
  Q_LOADED = S_EMPTY + kSBufs, Q_FULL, P_EMPTY, P_WRITTEN = P_EMPTY + kPSlots, STG_FREE = P_WRITTEN + kStaging,
  STATS_EMPTY = STG_FREE + kStaging, DEC_FULL, V_FULL, V_EMPTY = V_FULL + kVStages, P_FULL = V_EMPTY + kVStages,
  P_LOCAL = P_FULL + kPSlots, STATS_FULL = P_LOCAL + kPSlots, MMA_END,   // [2], as in the 16-bit decode
  NUM_BARS = MMA_END + 2
};
constexpr int kOffTmemSlot = kOffBar + NUM_BARS * 8;
constexpr int kOffAbort = kOffTmemSlot + 8;
constexpr int kOffWork = kOffAbort + 8;
constexpr int kSmemUsed = kOffWork + 48;
constexpr int kSmemBytes = kSmemUsed + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kQBoxes - 1 <= (kKStages - 1) * kBoxesPerStage, "the query passes through the tile ring");
static_assert(kOffQR % 1024 == 0 && kOffPSlots % 1024 == 0 && kKStageBytes % 1024 == 0 && kSlotStride % 1024 == 0 &&
              kOffScale % 16 == 0 && kOffStaging % 16 == 0 && kOffBar % 8 == 0 && kOffWork % 8 == 0, "alignment");

constexpr uint32_t kIdescS = ptx::idesc_e4m3_f32(kH, kTile, false);   // q · codeᵀ (K-major B)
constexpr uint32_t kIdescR = ptx::idesc_bf16_f32(kH, kTile, false);   // q_r · k_rᵀ
constexpr uint32_t kIdescO = ptx::idesc_f16_f32(kH, 256, true);       // w · value (MN-major B)

struct Params {
  const int32_t* block_table;
  int max_pages, num_pages;
  const int32_t* seqlens;
  int rows;                    // tokens: row v attends page_list[v * k + i], i < counts[v]
  const int32_t* page_list;
  const int32_t* counts;
  int k, s_q;                  // rows per sequence
  const uint8_t* codes;
  int64_t code_stride;
  const float* scales;
  __nv_bfloat16* o_lat;        // [rows, 128, 512]
  float* lse;                  // [rows, 128]
  float* part_o;               // [2 * pairs, 128, 512]
  float* part_lse;             // [2 * pairs, 128]
  float sm_scale_log2;
  int merge_in_kernel;
};

// Two values as E4M3 pairs: hi = the nearest values, lo = the nearest to what is left of the fp16 values
// (of bf16 values below 2^8, fp16 keeps everything but what is under 2^-24; the difference is exact).
__device__ __forceinline__ void split_e4m3x2(float w0, float w1, uint32_t* hi, uint32_t* lo) {
  uint32_t h16, b16, d16;
  uint16_t h8, l8;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h16) : "f"(w1), "f"(w0));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h8) : "r"(h16));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b16) : "h"(h8));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d16) : "r"(h16), "r"(b16));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l8) : "r"(d16));
  *hi = h8;
  *lo = l8;
}

// Warp roles.  Score CTA: 0 TMA producer | 1, 2 S-MMA issuers of even and odd tiles (2 owns TMEM) | 3
// copier | 4-11 row warps. Output CTA: 0-3 rescale (1 also issues the O MMAs, 2 returns staging buffers) |
// 4-11 widening and epilogue.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
decode8_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_rope,
               const __grid_constant__ CUtensorMap tm_q, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t rank = ptx::cluster_ctarank();
  const int pair = (int)ptx::cluster_id_x();
  const int npairs = (int)ptx::num_clusters_x();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * (uint32_t)i; };
  const uint32_t abort_addr = base + kOffAbort;
  long long* work = reinterpret_cast<long long*>(gbase + kOffWork);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kKStages; ++i) { ptx::mbar_init(bar(K_FULL + i), 1); ptx::mbar_init(bar(K_EMPTY + i), 1); }
    for (int i = 0; i < kSBufs; ++i) { ptx::mbar_init(bar(S_FULL + i), 1); ptx::mbar_init(bar(S_EMPTY + i), kH); }
    ptx::mbar_init(bar(Q_LOADED), 1);
    ptx::mbar_init(bar(Q_FULL), kGroup);
    for (int i = 0; i < kPSlots; ++i) {
      ptx::mbar_init(bar(P_EMPTY + i), 1);
      ptx::mbar_init(bar(P_FULL + i), 1);
      ptx::mbar_init(bar(P_LOCAL + i), 128);
    }
    for (int i = 0; i < kStaging; ++i) { ptx::mbar_init(bar(P_WRITTEN + i), kH); ptx::mbar_init(bar(STG_FREE + i), 1); }
    ptx::mbar_init(bar(DEC_FULL), kH);
    ptx::mbar_init(bar(STATS_EMPTY), kGroup);
    for (int i = 0; i < kVStages; ++i) { ptx::mbar_init(bar(V_FULL + i), kGroup); ptx::mbar_init(bar(V_EMPTY + i), 1); }
    ptx::mbar_init(bar(STATS_FULL), kH);
    for (int i = 0; i < 2; ++i) ptx::mbar_init(bar(MMA_END + i), 1);
    *reinterpret_cast<volatile int*>(gbase + kOffAbort) = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tm_codes);
    ptx::prefetch_tmap(&tm_rope);
    ptx::prefetch_tmap(&tm_q);
  }
  if (warp == 2) {
    ptx::tmem_alloc(base + kOffTmemSlot, kTmemCols);
    ptx::tmem_relinquish();
  }
  grid_dependency_wait();   // nothing above touched global memory
  if (warp == 3) sm100::plan_range<true>(p.counts, p.rows, 1, p.k, pair, npairs, work);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();      // the peer's barriers are initialised before any remote arrive
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + kOffTmemSlot);
  sm100::SegIter<true> segs{work[0], work[1], work[2], (int)work[3]};
  int b, t_lo, t_hi, tiles_b;
  auto next = [&]() -> bool { return segs.next(p.counts, p.rows, p.k, b, t_lo, t_hi, tiles_b); };
  auto visible = [&](int v) -> int { return p.seqlens[v / p.s_q] - (p.s_q - 1 - v % p.s_q); };
  // positions of row v's listed pages laid end to end that it sees (every page but the last is full)
  auto vlen = [&](int v) -> int {
    const int n = sm100::item_tiles<true>(p.counts, v, p.k);
    if (n == 0) return 0;
    const long long left = (long long)visible(v) - (long long)p.page_list[(long long)v * p.k + n - 1] * kTile;
    return (n - 1) * kTile + (int)min(max(left, 0ll), (long long)kTile);
  };
  // pool page of row v's tile t; num_pages (off the maps: zeros) when the list or the table is bad there
  auto page_at = [&](int v, int t, bool may_report) -> int {
    const int32_t* list = p.page_list + (long long)v * p.k;
    const int seq = v / p.s_q, pg = list[t], before = t > 0 ? list[t - 1] : -1, vis = visible(v);
    int page = -1;
    if (pg >= 0 && pg > before && pg < p.max_pages && vis > 0 && pg <= (vis - 1) / kTile)
      page = p.block_table[(long long)seq * p.max_pages + pg];
    if (page < 0 || page >= p.num_pages) {
      if (may_report) report(MLA_ERR_DEVICE_CHECK);
      page = p.num_pages;
    }
    return page;
  };

  if (rank == 0) {
    // ============================== score CTA ==============================
    if (warp == 0) {
      // ---- TMA producer: the warp looks up the pages of 32 tiles at a time and waits as a whole; lane 0
      // issues the loads
      auto load_tile = [&](uint32_t i, int page) {   // tile i of this pair, into its (free) stage
        if (lane == 0) {
          const uint32_t s = i % kKStages, dst = base + kOffK + s * kKStageBytes;
          ptx::mbar_arrive_expect_tx(bar(K_FULL + s), kKStageBytes + kScaleBytes);
          // (an off-the-map page takes page 0's scales: its result is undefined, its reads are not)
          ptx::bulk_load(base + kOffScale + (i % kScaleSlots) * kScaleBytes,
                         p.scales + (size_t)(page < p.num_pages ? page : 0) * kTile, kScaleBytes, bar(K_FULL + s));
          for (int j = 0; j < kCodeBoxes; ++j)
            ptx::tma_load_2d(dst + j * kBoxBytes, &tm_codes, 128 * j, page * kTile, bar(K_FULL + s));
          ptx::tma_load_2d(dst + kCodeBoxes * kBoxBytes, &tm_rope, 0, page * kTile, bar(K_FULL + s));
        }
        __syncwarp();
      };
      uint32_t it = 0, seg = 0;
      bool ok = true, q_out = false;
      while (ok && next()) {
        int pages = t_lo + lane < t_hi ? page_at(b, t_lo + lane, true) : 0;
        // the row's query passes through the tile ring once every earlier tile's products are done
        for (uint32_t i = (it > (uint32_t)kKStages ? it - kKStages : 0); i < it && ok; ++i)
          ok = wait_bar_warp(bar(K_EMPTY + i % kKStages), (i / kKStages) & 1u, abort_addr, false);
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(bar(Q_LOADED), (kQBoxes + 2) * kBoxBytes);
          for (int i = 0; i < kQBoxes; ++i)
            ptx::tma_load_2d(q_box(base, it, i), &tm_q, 64 * (i >> 1), b * kH + 64 * (i & 1), bar(Q_LOADED));
          for (int i = 0; i < 2; ++i)
            ptx::tma_load_2d(base + kOffQR + i * kBoxBytes, &tm_q, kDC, b * kH + 64 * i, bar(Q_LOADED));
        }
        q_out = true;
        // meanwhile the first tile into its stage, and the next ones into L2 (a box a lane)
        load_tile(it, __shfl_sync(0xffffffffu, pages, 0));
        const int pre = min(t_hi - t_lo, kKStages);
        const int pre_page = __shfl_sync(0xffffffffu, pages, lane / kCodeBoxes);
        if (lane < pre * kCodeBoxes) ptx::tma_prefetch_2d(&tm_codes, 128 * (lane % kCodeBoxes), pre_page * kTile);
        __syncwarp();
        if (!(ok = wait_bar_warp(bar(Q_FULL), seg & 1u, abort_addr, false))) break;
        q_out = false;
        ++seg;
        for (int t = t_lo; t < t_hi; ++t, ++it) {
          const uint32_t s = it % kKStages;
          if (t > t_lo && ((t - t_lo) & 31) == 0) pages = t + lane < t_hi ? page_at(b, t + lane, true) : 0;
          const int page = __shfl_sync(0xffffffffu, pages, (t - t_lo) & 31);
          if (t == t_lo) continue;   // loaded above
          if (!(ok = wait_bar_warp(bar(K_EMPTY + s), ((it / kKStages) & 1u) ^ 1u, abort_addr, false))) break;
          load_tile(it, page);
        }
      }
      // loads still in flight must land before the CTA may exit
      if (lane == 0) {
        if (q_out) {   // given up between the query's loads and the first tile's count
          wait_bar(bar(Q_LOADED), seg & 1u, abort_addr, false, false);
          ++it;
        }
        for (uint32_t i = (it > (uint32_t)kKStages ? it - kKStages : 0); i < it; ++i)
          wait_bar(bar(K_FULL + i % kKStages), (i / kKStages) & 1u, abort_addr, false, false);
      }
    } else if (warp == 3) {
      if (lane == 0) {   // ---- copier: each finished staging buffer goes to the output CTA's slot
        const uint32_t slot_remote0 = ptx::map_to_cta(base + kOffPSlots, 1);
        uint32_t it = 0;
        bool ok = true;
        while (ok && next()) {
          for (int t = t_lo; t < t_hi; ++t, ++it) {
            const uint32_t stg = it % kStaging, slot = it % kPSlots;
            if (!(ok = wait_bar(bar(P_WRITTEN + stg), (it / kStaging) & 1u, abort_addr, false))) break;
            if (!(ok = wait_bar(bar(P_EMPTY + slot), ((it / kPSlots) & 1u) ^ 1u, abort_addr, true))) break;
            const uint32_t full = ptx::map_to_cta(bar(P_FULL + slot), 1);
            const uint32_t src = base + kOffStaging + stg * kStgStride, dst = slot_remote0 + slot * kSlotStride;
            ptx::mbar_arrive_expect_tx_remote(bar(P_FULL + slot), 1, kCopyBytes);
            ptx::bulk_copy_to_cta(dst, src, kCopyBytes, full);
          }
        }
        // before leaving: every copy has landed and every slot came back
        for (uint32_t i = (it > (uint32_t)kPSlots ? it - kPSlots : 0); i < it; ++i)
          wait_bar(bar(P_EMPTY + i % kPSlots), (i / kPSlots) & 1u, abort_addr, true, false);
        for (uint32_t i = (it > (uint32_t)kStaging ? it - kStaging : 0); i < it; ++i)
          wait_bar(bar(STG_FREE + i % kStaging), (i / kStaging) & 1u, abort_addr, true, false);
      }
    } else if (warp == 1 || warp == 2) {
      // ---- S-MMA issuers: the latents' 512 codes twice (q_hi, q_lo) in steps of 32, then the RoPE keys
      const uint32_t parity = warp == 1 ? 0u : 1u;
      const uint64_t k_desc = ptx::smem_desc_sw128(base + kOffK, 16, 1024);
      const uint64_t qr_desc = ptx::smem_desc_sw128(base + kOffQR, 16, 1024);
      uint32_t it = 0, seg = 0;
      bool ok = true;
      while (ok && next()) {
        if (!(ok = wait_bar_warp(bar(Q_FULL), seg & 1u, abort_addr, false))) break;
        ++seg;
        for (int t = t_lo; t < t_hi; ++t, ++it) {
          if ((it & 1u) != parity) continue;
          const uint32_t sb = it % kSBufs, s = it % kKStages;
#ifdef MLA_TEST_HOOKS
          if (test_stall(1, (int)it) && !(ok = sm100::stall_products(bar(MMA_END + parity), abort_addr))) break;
#endif
          if (!(ok = wait_bar_warp(bar(S_EMPTY + sb), ((it / kSBufs) & 1u) ^ 1u, abort_addr, false))) break;
          if (!(ok = wait_bar_warp(bar(K_FULL + s), (it / kKStages) & 1u, abort_addr, false))) break;
          if (ptx::elect_one()) {
            ptx::tc_fence_after();
            const uint32_t d = tmem + kSCol0 + 128u * sb;
            const uint64_t kd = k_desc + (uint64_t)(s * (kKStageBytes >> 4));
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int j = 0; j < kCodeBoxes; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  ptx::mma_ts_f8(d, tmem + 128u * part + 32u * j + 8u * k, kd + (uint64_t)(j * (kBoxBytes >> 4) + 2 * k), kIdescS,
                                 (part | j | k) ? 1u : 0u);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::mma_ss(d + 64u, qr_desc + 2 * k, kd + (uint64_t)(kCodeBoxes * (kBoxBytes >> 4) + 2 * k), kIdescR, k ? 1u : 0u);
            ptx::mma_commit(bar(K_EMPTY + s));
            ptx::mma_commit(bar(S_FULL + sb));
          }
          __syncwarp();
        }
      }
      sm100::end_products(bar(MMA_END + parity), abort_addr);
    } else if (warp >= 4) {
      // ---- row warps: thread = one head row; two sets of four warps on alternate tiles
      const int set = (warp - 4) >> 2;
      const int row = ((warp & 3) << 5) | lane;
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t stats_remote = ptx::map_to_cta(base + kOffStats, 1);
      float* dec = reinterpret_cast<float*>(gbase + kOffStats);   // [128]: M after the latest tile
      const float scale2 = p.sm_scale_log2;
      uint32_t it = 0, seg = 0;
      bool ok = true;
      // (a warp that has given up goes on to the next place where all of them meet, so that none waits there for it)
      while (next()) {
        const int L = vlen(b);
        // ---- the row's query: q 2^t as two E4M3 terms into TMEM. Each set takes half of its columns; the
        // row's largest value comes from both
        float q_unit = 0.f;   // 2^-t
        ok = ok && wait_bar_warp(bar(Q_LOADED), seg & 1u, abort_addr, false);
        uint32_t* q_top = reinterpret_cast<uint32_t*>(gbase + kOffQTop);
        const int r = row & 63, rh = row >> 6;
        if (ok) {
          uint32_t top = 0;   // the largest magnitude of the two halves of each word, as bf16 bits
#pragma unroll 1
          for (int cb = 4 * set; cb < 4 * set + 4; ++cb) {
            const uint32_t srow = q_box(base, it, 2 * cb + rh) + (uint32_t)r * 128u;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint4 x = ptx::ld_shared_v4(srow + ((uint32_t)(k ^ (r & 7)) << 4));
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
            }
          }
          q_top[set * kH + row] = max(top & 0xffffu, top >> 16);
        }
        ok = !ptx::named_bar_or(3, kGroup, !ok);   // all row warps meet here, and agree
        if (ok) {
          // largest value < 2^(e - 126): 2^t = 2^(134 - e) brings it below 2^8 (e at least 8, so that 2^t is
          // a float); an infinite or NaN query has no finite scores
          const int e = max((int)(max(q_top[row], q_top[kH + row]) >> 7), 8);
          const float up = __uint_as_float((uint32_t)(261 - e) << 23);
          q_unit = e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(e - 7) << 23);
#pragma unroll 1
          for (int cb = 4 * set; cb < 4 * set + 4; ++cb) {
            const uint32_t srow = q_box(base, it, 2 * cb + rh) + (uint32_t)r * 128u;
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint4 x = ptx::ld_shared_v4(srow + ((uint32_t)(k ^ (r & 7)) << 4));
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                uint32_t h0, l0, h1, l1;
                split_e4m3x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up, &h0, &l0);
                split_e4m3x2(__uint_as_float(w[j + 1] << 16) * up, __uint_as_float(w[j + 1] & 0xffff0000u) * up, &h1, &l1);
                hi[2 * k + j / 2] = __byte_perm(h0, h1, 0x5410);
                lo[2 * k + j / 2] = __byte_perm(l0, l1, 0x5410);
              }
            }
            ptx::tmem_st16(tmem + lane_off + 16u * cb, hi);
            ptx::tmem_st16(tmem + lane_off + 128u + 16u * cb, lo);
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          // the ring's next loads (async proxy) come after these generic reads of it
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(bar(Q_FULL));
        }
        float m_own = -INFINITY, l_own = 0.f;   // this set's reference and partial row sum
        for (int t = t_lo; t < t_hi; ++t, ++it) {
          if ((it & 1u) != (uint32_t)set || !ok) continue;
          const uint32_t sb = it % kSBufs, stg = it % kStaging;
          const uint32_t sc_addr = base + kOffScale + (it % kScaleSlots) * kScaleBytes;
          const bool stg_free = ptx::mbar_test_wait_cluster(bar(STG_FREE + stg), ((it / kStaging) & 1u) ^ 1u);
          // (the tile's scales landed with its rows, before its products)
          if (!wait_bar_warp(bar(S_FULL + sb), (it / kSBufs) & 1u, abort_addr, false)) { ok = false; continue; }
          const int valid = L - t * kTile;
          if (valid < kTile) {   // slots past the end weigh nothing, whatever the cache holds there
            for (int j = max(valid, 0) + lane; j < kTile; j += 32) ptx::st_shared_u32(sc_addr + 4u * j, 0u);
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
          int e_top = kMinLog2, e_low = kMinLog2;
          uint64_t x2[32];   // x of positions 2 i, 2 i + 1
          const uint64_t unit2 = ptx::pack_f32x2(q_unit, q_unit);
          ptx::tc_fence_after();
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t vc[32], vr[32];
            ptx::tmem_ld32(tmem + lane_off + kSCol0 + 128u * sb + 32u * half, vc);
            ptx::tmem_ld32(tmem + lane_off + kSCol0 + 128u * sb + 64u + 32u * half, vr);
            if (half == 0) {
              const int e0 = scale_log2(ptx::ld_shared_u32(sc_addr + 4u * lane));
              const int e1 = scale_log2(ptx::ld_shared_u32(sc_addr + 4u * (lane + 32)));
              e_top = __reduce_max_sync(0xffffffffu, max(e0, e1));
              // (slots past the end do not count)
              e_low = __reduce_min_sync(0xffffffffu, min(lane < valid ? e0 : e_top, lane + 32 < valid ? e1 : e_top));
            }
            ptx::tmem_wait_ld_regs(vc);
            ptx::tmem_wait_ld_regs(vr);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              uint64_t sa, sb2;
              ptx::ld_shared_v2u64(sc_addr + 4u * (32 * half + j), &sa, &sb2);
              x2[(32 * half + j) / 2] = ptx::fma_f32x2(ptx::pack_f32x2(__uint_as_float(vc[j]), __uint_as_float(vc[j + 1])),
                                                       ptx::mul_f32x2(sa, unit2),
                                                       ptx::pack_f32x2(__uint_as_float(vr[j]), __uint_as_float(vr[j + 1])));
              x2[(32 * half + j) / 2 + 1] =
                  ptx::fma_f32x2(ptx::pack_f32x2(__uint_as_float(vc[j + 2]), __uint_as_float(vc[j + 3])),
                                 ptx::mul_f32x2(sb2, unit2),
                                 ptx::pack_f32x2(__uint_as_float(vr[j + 2]), __uint_as_float(vr[j + 3])));
            }
          }
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar(S_EMPTY + sb));
          if (valid < kTile) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float x0, x1;
              ptx::unpack_f32x2(x2[i], &x0, &x1);
              x2[i] = ptx::pack_f32x2(2 * i < valid ? x0 : -INFINITY, 2 * i + 1 < valid ? x1 : -INFINITY);
            }
          }
          // the reference this tile needs: its weights below 2^kTopLog2
          float a4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, need;
          if (e_top - e_low <= kNearLog2) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float x0, x1;
              ptx::unpack_f32x2(x2[i], &x0, &x1);
              a4[i & 3] = fmaxf(a4[i & 3], fmaxf(x0, x1));
            }
            need = fmaf(fmaxf(fmaxf(a4[0], a4[1]), fmaxf(a4[2], a4[3])), scale2, (float)e_top - kTopLog2);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              uint64_t sc[2];
              ptx::ld_shared_v2u64(sc_addr + 8u * i, &sc[0], &sc[1]);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float x0, x1;
                ptx::unpack_f32x2(x2[i + j], &x0, &x1);
                a4[2 * j] = fmaxf(a4[2 * j], fmaf(x0, scale2, (float)scale_log2((uint32_t)sc[j])));
                a4[2 * j + 1] = fmaxf(a4[2 * j + 1], fmaf(x1, scale2, (float)scale_log2((uint32_t)(sc[j] >> 32))));
              }
            }
            need = fmaxf(fmaxf(a4[0], a4[1]), fmaxf(a4[2], a4[3])) - kTopLog2;
          }
          float m_prev = -INFINITY;
          if (t > t_lo) {
            if (!wait_bar_warp(bar(DEC_FULL), (it - 1) & 1u, abort_addr, true)) { ok = false; continue; }
            m_prev = dec[row];
          }
          float al = 1.f, m_new = m_prev;
          if (need > m_prev) {
            m_new = need + kRoomLog2;
            al = (m_prev == -INFINITY) ? 0.f : ptx::ex2_approx(m_prev - m_new);
          }
          dec[row] = m_new;
          ptx::mbar_arrive(bar(DEC_FULL));
          if (m_new != m_own) {   // (before any score above -inf the sum is zero, or NaN)
            if (m_own != -INFINITY) l_own *= ptx::ex2_approx(m_own - m_new);
            m_own = m_new;
          }
          // while every score so far is -inf (or NaN) the exponents are taken against 0
          const float m_ref = m_new == -INFINITY ? 0.f : m_new;
          // e, its sum, and w = e s, sixteen positions at a time
          uint32_t pk[32];
          uint64_t l2[2] = {0ull, 0ull};
          const uint64_t scale22 = ptx::pack_f32x2(scale2, scale2), neg_m2 = ptx::pack_f32x2(-m_ref, -m_ref);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint64_t e2[8], s2[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) ptx::ld_shared_v2u64(sc_addr + 4u * (16 * c + 2 * i), &s2[i], &s2[i + 1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x0, x1;
              ptx::unpack_f32x2(ptx::fma_f32x2(x2[8 * c + i], scale22, neg_m2), &x0, &x1);
              e2[i] = ptx::pack_f32x2(ptx::ex2_approx(x0), ptx::ex2_approx(x1));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              l2[i & 1] = ptx::add_f32x2(l2[i & 1], e2[i]);
              float w0, w1;
              ptx::unpack_f32x2(ptx::mul_f32x2(e2[i], s2[i]), &w0, &w1);
              pk[8 * c + i] = ptx::pack_f16x2(w0, w1);
            }
          }
          float ls[4];
          ptx::unpack_f32x2(l2[0], &ls[0], &ls[1]);
          ptx::unpack_f32x2(l2[1], &ls[2], &ls[3]);
          l_own += (ls[0] + ls[1]) + (ls[2] + ls[3]);
          if (!__all_sync(0xffffffffu, stg_free) &&
              !wait_bar_warp(bar(STG_FREE + stg), ((it / kStaging) & 1u) ^ 1u, abort_addr, true)) {
            ok = false;
            continue;
          }
          // the row into the K-major, 128-byte swizzled tile, and its rescale factor
          const uint32_t st0 = base + kOffStaging + stg * kStgStride;
          const uint32_t prow = st0 + (uint32_t)(row >> 3) * 1024u + (uint32_t)(row & 7) * 128u;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            ptx::st_shared_v4(prow + (((uint32_t)c ^ (uint32_t)(row & 7)) << 4), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
          reinterpret_cast<float*>(gbase + kOffStaging + stg * kStgStride + kAlphaOff)[row] = al;
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(bar(P_WRITTEN + stg));
        }
        // segment end: the two sets' sums at the reference after the segment's last tile
        float m_fin = -INFINITY;
        if (ok) {
          const uint32_t last = it - 1;
          if ((last & 1u) == (uint32_t)set) m_fin = m_own;
          else if (wait_bar_warp(bar(DEC_FULL), last & 1u, abort_addr, true)) m_fin = dec[row];
          else ok = false;
        }
        const float l_fin = (m_own == -INFINITY) ? l_own : l_own * ptx::ex2_approx(m_own - m_fin);
        if (ptx::named_bar_or(2, kGroup, !ok)) { ok = false; break; }
        if (set == 1) dec[row] = l_fin;
        ptx::named_bar_sync(2, kGroup);
        if (set == 0) {
          const float l = l_fin + dec[row];
          if (!wait_bar_warp(bar(STATS_EMPTY), (seg & 1u) ^ 1u, abort_addr, true)) ok = false;
          if (ok) {
            const bool partial = !(t_lo == 0 && t_hi == tiles_b);
            float* lse_dst = partial ? p.part_lse + ((size_t)pair * 2 + (seg > 0)) * kH : p.lse + (size_t)b * kH;
            lse_dst[row] = (m_fin + log2f(l)) * 0.69314718055994531f;
            ptx::st_cluster_f32(stats_remote + row * 4u, l != 0.f ? 1.f / l : 0.f);
            ptx::mbar_arrive_remote(bar(STATS_FULL), 1);
          }
        }
        ++seg;
      }
      if (set == 0 && seg > 0) wait_bar(bar(STATS_EMPTY), (seg - 1) & 1u, abort_addr, true, false);
    }
  } else {
    // ============================== output CTA ==============================
    if (warp < 4) {
      // ---- control warps: as a tile of weights lands, warp w rescales its 32 rows of O if their reference
      // moved; warp 2 hands the staging buffer back to the score CTA; warp 1 then issues O += w · value, K = 64
      // positions in steps of 16, N = 512 in 2 halves
      if (warp == 3) {   // (rows that list no page attend nothing: zeros and lse = -inf)
        for (int v = pair; v < p.rows; v += npairs) {
          if (sm100::item_tiles<true>(p.counts, v, p.k) > 0) continue;
          uint4* o = reinterpret_cast<uint4*>(p.o_lat + (size_t)v * kH * kDC);
          for (int i = lane; i < kH * kDC / 8; i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
          for (int i = lane; i < kH; i += 32) p.lse[(size_t)v * kH + i] = -INFINITY;
        }
        __syncwarp();
      }
      const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
      const uint64_t v_desc0 = ptx::smem_desc_sw128(base + kOffV, kBoxBytes, 1024);
      const uint64_t p_desc0 = ptx::smem_desc_sw128(base + kOffPSlots, 16, 1024);
      uint32_t it = 0;
      bool ok = true;
      while (ok && next()) {
        for (int t = t_lo; t < t_hi; ++t, ++it) {
          const uint32_t slot = it % kPSlots, s = it % kVStages;
          if (!(ok = wait_bar_warp(bar(P_FULL + slot), (it / kPSlots) & 1u, abort_addr, true))) break;
          if (warp == 2 && lane == 0) ptx::mbar_arrive_remote(bar(STG_FREE + it % kStaging), 0);
          const float al = reinterpret_cast<const float*>(gbase + kOffPSlots + slot * kSlotStride + kAlphaOff)[warp * 32 + lane];
          if (t > t_lo && __any_sync(0xffffffffu, al != 1.f)) {   // once the products of the tile before are done
            const uint32_t pt = it - 1;
            if (!(ok = wait_bar_warp(bar(P_EMPTY + pt % kPSlots), (pt / kPSlots) & 1u, abort_addr, false))) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kDC; c += 32) {
              uint32_t r[32];
              ptx::tmem_ld32(tmem + lane_off + c, r);
              ptx::tmem_wait_ld_regs(r);
#pragma unroll
              for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * al);
              ptx::tmem_st32(tmem + lane_off + c, r);
            }
            ptx::tmem_wait_st();
          }
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar(P_LOCAL + slot));
          if (warp != 1) continue;
#ifdef MLA_TEST_HOOKS
          if (test_stall(2, (int)it) && !(ok = sm100::stall_products(bar(MMA_END), abort_addr))) break;
#endif
          if (!(ok = wait_bar_warp(bar(V_FULL + s), (it / kVStages) & 1u, abort_addr, false))) break;
          if (!(ok = wait_bar_warp(bar(P_LOCAL + slot), (it / kPSlots) & 1u, abort_addr, false))) break;
          if (ptx::elect_one()) {
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_after();
            const uint64_t pd = p_desc0 + (uint64_t)(slot * (kSlotStride >> 4));
            const uint64_t vd = v_desc0 + (uint64_t)(s * (kVStageBytes >> 4));
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk) {
              const uint32_t acc = (t > t_lo || kk > 0) ? 1u : 0u;
              ptx::mma_ss(tmem, pd + 2 * kk, vd + 128 * kk, kIdescO, acc);
              ptx::mma_ss(tmem + 256, pd + 2 * kk, vd + 2048 + 128 * kk, kIdescO, acc);
            }
            ptx::mma_commit(bar(V_EMPTY + s));
            ptx::mma_commit_mc(bar(P_EMPTY + slot), (uint16_t)0x3);
          }
          __syncwarp();
        }
      }
      if (warp == 1) sm100::end_products(bar(MMA_END), abort_addr);
    } else {
      // ---- row warps: each tile's codes widened to fp16 on their way into shared memory, and the segment
      // epilogue.
      // Warp w takes latents [64 w', + 64) (w' = w - 4), eight rows at a time, 16 codes a thread: the loads
      // read whole 32-byte sectors and the stores of a warp spread over all banks. A tile's codes are
      // loaded into registers while the tile before it is widened, its page is looked up one tile
      // earlier still; the loads mostly hit L2, where the score CTA's reads have brought the rows.
      const int sub = (warp - 4) >> 2, qd = warp & 3;
      const int g = sub;                                  // epilogue: latent half g
      const int h = (qd << 5) | lane;
      const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
      const uint32_t col0 = 256u * g;
      float* stats = reinterpret_cast<float*>(gbase + kOffStats);
      uint32_t it = 0, seg = 0;
      bool ok = true;
      // the walk over this pair's tiles that runs ahead of the main one
      sm100::SegIter<true> ahead = segs;
      int ab = 0, at = 0, a_lo = 0, a_hi = 0, a_pages = 0;   // lane l: page of the l-th tile of the current 32
      auto next_page = [&]() -> int {   // pool page of the next tile of the walk; num_pages when it ends
        bool fresh = at < a_hi && ((at - a_lo) & 31) == 0;
        if (at == a_hi) {
          int all;
          if (!ahead.next(p.counts, p.rows, p.k, ab, a_lo, a_hi, all)) { a_hi = at; return p.num_pages; }
          at = a_lo;
          fresh = true;
        }
        if (fresh) a_pages = at + lane < a_hi ? page_at(ab, at + lane, false) : 0;   // (the score CTA reports)
        const int page = __shfl_sync(0xffffffffu, a_pages, (at - a_lo) & 31);
        ++at;
        return page;
      };
      const int w8 = warp - 4, lrow = lane >> 2;
      const uint32_t vdst = base + kOffV + (uint32_t)w8 * kBoxBytes + (uint32_t)lrow * 128u;
      const uint32_t vsw0 = (((uint32_t)(2 * (lane & 3))) ^ (uint32_t)lrow) << 4;
      const uint32_t vsw1 = (((uint32_t)(2 * (lane & 3) + 1)) ^ (uint32_t)lrow) << 4;
      const uint8_t* lane_codes = p.codes + (int64_t)lrow * p.code_stride + 64 * w8 + 16 * (lane & 3);
      uint4 cd[8];
      auto load_codes = [&](int page) {
        const uint8_t* src = lane_codes + (int64_t)(page < p.num_pages ? page : 0) * kTile * p.code_stride;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          cd[i] = page < p.num_pages ? *reinterpret_cast<const uint4*>(src + (int64_t)(8 * i) * p.code_stride)
                                     : make_uint4(0u, 0u, 0u, 0u);
      };
      load_codes(next_page());
      int page1 = next_page();
      while (next()) {
        const int L = vlen(b);
        for (int t = t_lo; t < t_hi; ++t, ++it) {
          if (!ok) continue;
          const uint32_t vs = it % kVStages;
          if (!wait_bar_warp(bar(V_EMPTY + vs), ((it / kVStages) & 1u) ^ 1u, abort_addr, false)) { ok = false; continue; }
          const int valid = L - t * kTile;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t f[8];
            const uint32_t q[4] = {cd[i].x, cd[i].y, cd[i].z, cd[i].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = ptx::e4m3x2_to_f16x2(q[k >> 1] >> (16 * (k & 1)));
            if (8 * i + lrow >= valid) {   // a slot past the end may hold NaN codes, and 0 * NaN = NaN
#pragma unroll
              for (int k = 0; k < 8; ++k) f[k] = 0u;
            }
            const uint32_t dst = vdst + vs * kVStageBytes + (uint32_t)i * 1024u;
            ptx::st_shared_v4(dst + vsw0, f[0], f[1], f[2], f[3]);
            ptx::st_shared_v4(dst + vsw1, f[4], f[5], f[6], f[7]);
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(bar(V_FULL + vs));
          load_codes(page1);
          page1 = next_page();
        }
        if (ok && !wait_bar_warp(bar(P_EMPTY + (it - 1) % kPSlots), ((it - 1) / kPSlots) & 1u, abort_addr, false)) ok = false;
        if (ok && !wait_bar_warp(bar(STATS_FULL), seg & 1u, abort_addr, true)) ok = false;
        if (ptx::named_bar_or(1, kGroup, !ok)) break;
        ptx::tc_fence_after();
        const float inv_l = stats[h];
        const bool partial = !(t_lo == 0 && t_hi == tiles_b);
        // 32 columns of the warp's 32 rows at a time through a 2 KB transpose buffer
        const uint32_t ebuf = base + kOffEpi + (uint32_t)(warp - 4) * kEpiWarpBytes;
        const uint32_t wrow = ebuf + (uint32_t)lane * 64u;
        const uint32_t sw = (uint32_t)(lane >> 1) & 3u;
        const int c4 = lane & 3, rsub = lane >> 2;
        const int row0 = qd * 32;
        auto flush = [&](char* dst0, size_t row_bytes) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 8 * i + rsub;
            const uint4 v = ptx::ld_shared_v4(ebuf + rr * 64u + (((uint32_t)c4 ^ (((uint32_t)rr >> 1) & 3u)) << 4));
            *reinterpret_cast<uint4*>(dst0 + (size_t)(row0 + rr) * row_bytes + c4 * 16) = v;
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int c = 0; c < kDC / 2; c += 32) {
          uint32_t r[32];
          ptx::tmem_ld32(tmem + lane_off + col0 + c, r);
          ptx::tmem_wait_ld();
          if (partial) {
            float* dst = p.part_o + ((size_t)pair * 2 + (seg > 0)) * kH * kDC + col0 + c;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int j = 16 * half + 4 * k;
                ptx::st_shared_v4(wrow + ((k ^ sw) << 4), __float_as_uint(__uint_as_float(r[j]) * inv_l),
                                  __float_as_uint(__uint_as_float(r[j + 1]) * inv_l),
                                  __float_as_uint(__uint_as_float(r[j + 2]) * inv_l),
                                  __float_as_uint(__uint_as_float(r[j + 3]) * inv_l));
              }
              flush(reinterpret_cast<char*>(dst + 16 * half), kDC * sizeof(float));
            }
          } else {
            __nv_bfloat16* dst = p.o_lat + (size_t)b * kH * kDC + col0 + c;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = 8 * k;
              ptx::st_shared_v4(wrow + ((k ^ sw) << 4),
                                ptx::pack_bf16x2(__uint_as_float(r[j]) * inv_l, __uint_as_float(r[j + 1]) * inv_l),
                                ptx::pack_bf16x2(__uint_as_float(r[j + 2]) * inv_l, __uint_as_float(r[j + 3]) * inv_l),
                                ptx::pack_bf16x2(__uint_as_float(r[j + 4]) * inv_l, __uint_as_float(r[j + 5]) * inv_l),
                                ptx::pack_bf16x2(__uint_as_float(r[j + 6]) * inv_l, __uint_as_float(r[j + 7]) * inv_l));
            }
            flush(reinterpret_cast<char*>(dst), kDC * sizeof(__nv_bfloat16));
          }
        }
        // (the next segment's first product overwrites O: it waits for these threads' next tile)
        ptx::tc_fence_before();
        ptx::mbar_arrive_remote(bar(STATS_EMPTY), 0);
        ++seg;
      }
    }
  }

  // teardown: TMEM back, then leave together so no remote access can target an exited CTA
  ptx::tc_fence_before();
  __syncthreads();
  if (!p.merge_in_kernel) allow_dependents();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  ptx::cluster_sync();
  if (p.merge_in_kernel) {
    // launched cooperatively: when a row was cut, one grid-wide barrier, then the merge
    if (work[4] > 0 && work[5] == 0) {
      cooperative_groups::this_grid().sync();
      sm100::merge_rows(p.counts, p.rows, p.k, sm100::active_groups<true>(npairs, work[4]), work[4],
                        reinterpret_cast<sm100::CutRows*>(gbase), (int)blockIdx.x, (int)gridDim.x, kThreads / 32, p.part_o, p.part_lse, p.o_lat, p.lse);
    }
    allow_dependents();
  }
}

// ---- host ----------------------------------------------------------------------------------------
inline int active_pairs(int num_sms) {
  static int cached[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  const bool known = dev >= 0 && dev < 64;
  if (known && cached[dev]) return cached[dev];
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * sm100::max_pairs(num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  if (cudaOccupancyMaxActiveClusters(&n, decode8_kernel, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = sm100::max_pairs(num_sms);
  }
  n = std::min(n, sm100::max_pairs(num_sms));
  if (known) cached[dev] = n;
  return n;
}

inline int launch_decode8(const mla_dims_t* d, int32_t rows, const void* q_abs, const mla_latent_cache_fp8_t* cache,
                          const int32_t* block_table, int32_t max_pages, const int32_t* seqlens, void* o_lat, float* lse,
                          void* workspace, size_t ws_bytes, int num_sms, cudaStream_t st, const sm100::PageLists& lists) {
  if (!workspace || ws_bytes < sm100::decode_workspace_bytes(d, MLA_BF16, rows, 1, num_sms)) return MLA_ERR_WORKSPACE;
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  const bool known = dev >= 0 && dev < 64;
  if (!known || !attr_done[dev]) {
    if (cudaFuncSetAttribute(decode8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
      return MLA_ERR_CUDA;
    if (known) attr_done[dev] = true;
  }
  CUtensorMap tm_codes, tm_rope, tm_q;
  const int64_t pool = (int64_t)cache->num_pages * kTile;
  if (!tmap::make_u8_sw128(&tm_codes, cache->codes, kDC, pool, cache->code_stride, kTile) ||
      !tmap::make_bf16_sw128(&tm_rope, cache->rope, kDR, pool, cache->rope_stride, kTile) ||
      !tmap::make_bf16_sw128(&tm_q, q_abs, kRow, (int64_t)rows * kH, kRow, 64))
    return MLA_ERR_INVALID_ARG;
  const int P = active_pairs(num_sms);
  Params prm;
  prm.block_table = block_table;
  prm.max_pages = max_pages;
  prm.num_pages = cache->num_pages;
  prm.seqlens = seqlens;
  prm.rows = rows;
  prm.page_list = lists.pages;
  prm.counts = lists.counts;
  prm.k = lists.k;
  prm.s_q = lists.s_q;
  prm.codes = cache->codes;
  prm.code_stride = cache->code_stride;
  prm.scales = cache->scales;
  prm.o_lat = reinterpret_cast<__nv_bfloat16*>(o_lat);
  prm.lse = lse;
  prm.part_o = reinterpret_cast<float*>(workspace);
  prm.part_lse = prm.part_o + (size_t)2 * sm100::max_pairs(num_sms) * kH * kDC;
  prm.sm_scale_log2 = d->sm_scale * 1.4426950408889634f;
  // one cooperative launch that merges cut rows itself; where the runtime refuses it, two launches
  static int coop_mode[64] = {0};   // 0 unknown, 1 cooperative + PDL, 2 cooperative, 3 two launches
  bool forced = false;
#ifdef MLA_TEST_HOOKS
  forced = sm100::g_test_two_launches;
#endif
  for (int mode = forced ? 3 : (known && coop_mode[dev] ? coop_mode[dev] : 1); mode <= 3; ++mode) {
    if (mode == 3) {
      prm.merge_in_kernel = 0;
      launch_pdl(decode8_kernel, dim3(2 * P), dim3(kThreads), kSmemBytes, st, tm_codes, tm_rope, tm_q, prm);
      launch_pdl(sm100::merge_kernel<true>, dim3(std::min(rows, sm100::kMergeTokenBlocks), kH / sm100::kMergeHeads),
                 dim3(32 * sm100::kMergeHeads), 0, st, prm.counts, prm.rows, 1, prm.k, P, (const float*)prm.part_o,
                 (const float*)prm.part_lse, prm.o_lat, lse);
      if (known && !forced) coop_mode[dev] = 3;
      break;
    }
    prm.merge_in_kernel = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * P);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = mode == 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, decode8_kernel, tm_codes, tm_rope, tm_q, prm) == cudaSuccess) {
      g_launches.fetch_add(1, std::memory_order_relaxed);
      if (known) coop_mode[dev] = mode;
      break;
    }
    (void)cudaGetLastError();   // a configuration the runtime refused: nothing was launched
  }
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace sm100f8
}  // namespace mla
