// The 8-bit latent cache written straight from the projection, and read back into the storage type.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "simt.cuh"

namespace mla {
namespace cache8 {

// Two E4M3 codes (low byte first) as fp32 values. Exact: every E4M3 value is an fp16 value.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Codes of four values over a scale: E4M3(v / s), to nearest, ties to even, saturated at +-448; a zero
// magnitude is +0. `safe` is s, or 1 for a zero row.
__device__ __forceinline__ uint32_t e4m3x4_codes(const float* v, float safe) {
  uint32_t out = 0;
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const float a = __fdiv_rn(v[k], safe), b = __fdiv_rn(v[k + 1], safe);
    uint16_t pr;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pr) : "f"(b), "f"(a));   // a -> low byte
    uint32_t lo = pr & 0xffu, hi = pr >> 8;
    if ((lo & 0x7fu) == 0u) lo = 0u;
    if ((hi & 0x7fu) == 0u) hi = 0u;
    out |= (lo | (hi << 8)) << (8 * k);
  }
  return out;
}

// =============================================================================================
// Append into the 8-bit cache, second half: as append_finish_kernel sums the K slices, normalises and
// rotates, but the latent row leaves as codes and one scale. The row is quantised from its fp32 values
// (no rounding to 16 bits in between), so the stored row is the nearest one to c itself. One block per
// new token; d_c % 16 == 0. 64 tokens: 5.9 us, a chain of latencies (28 slices, the norm, the largest value).
// =============================================================================================
template <typename T>
__global__ void append_fp8_finish_kernel(const float* part, int ksplit, int n_tok, int s_q, int d_c, int d_r,
                                         const T* gamma, float eps, float rope_base,
                                         const int32_t* seqlens, const int32_t* block_table,
                                         int max_pages, uint8_t* codes, int64_t code_stride, float* scales, T* rope,
                                         int64_t rope_stride, int num_pages, int groups) {
  extern __shared__ float z[];
  __shared__ float red[32];
  __shared__ long long s_row;   // the token's cache row; -1: none (reported)
  __shared__ int s_pos;
  grid_dependency_wait();   // launched with programmatic dependent launch after the projection
  allow_dependents();
  const int N = d_c + d_r;
  const float* cs_sn = simt::finish_gather(part, ksplit, n_tok, s_q, N, d_r, rope_base, seqlens, block_table, max_pages,
                                           num_pages, groups, z, &s_row, &s_pos);
  float ss = 0.f;
  for (int i = threadIdx.x; i < d_c; i += blockDim.x) ss = fmaf(z[i], z[i], ss);
  ss = block_sum(ss, red);
  const float inv = 1.0f / sqrtf(ss / (float)d_c + eps);
  const int64_t row = s_row;
  if (row < 0) return;
  float amax = 0.f;
  for (int i = threadIdx.x; i < d_c; i += blockDim.x) {
    const float v = z[i] * inv * (gamma ? ld(gamma + i) : 1.f);
    z[i] = v;
    amax = fmaxf(amax, fabsf(v));
  }
  amax = warp_max(amax);
  __syncthreads();   // red is reused; z is complete
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) amax = fmaxf(amax, red[w]);
  const float s = __fdiv_rn(amax, 448.f);
  const float safe = s > 0.f ? s : 1.f;
  uint8_t* dst = codes + row * code_stride;
  for (int i = threadIdx.x * 4; i < d_c; i += blockDim.x * 4)
    *reinterpret_cast<uint32_t*>(dst + i) = e4m3x4_codes(z + i, safe);
  if (threadIdx.x == 0) scales[row] = s;
  simt::finish_rope(z + d_c, d_r / 2, groups > 0 ? cs_sn : nullptr, s_pos, d_r, rope_base, rope + row * rope_stride);
}

// The same for many tokens (few K slices each): a warp per token, the whole row in registers, so that
// no block waits between the sums, the norm, the scale and the stores; the rotation's frequencies are made
// once per block. d_c % 16 == 0, (d_c + d_r) % 4 == 0, d_c <= 128 * kRowChunks, d_r <= 64 * kRowPairs, 16-byte
// aligned slices. 4096 tokens of 512 + 64 values: 104 us with a block a token (one slice), 9.0 us so (three
// slices, 28 MB of partial sums out of L2: 3.1 TB/s).
constexpr int kRowChunks = 8;     // most float4 pieces of the latent row a lane holds
constexpr int kRowPairs = 4;      // most rotated pairs a lane holds
constexpr int kRowWarps = 8;

// kChunks, kPairs: float4 pieces and rotated pairs a lane holds (4 and 1: rows of up to 512 + 64 values, in few
// enough registers for four blocks an SM, which then hide each other's loads).
template <typename T, int kChunks, int kPairs>
__global__ void __launch_bounds__(32 * kRowWarps, kChunks == 4 ? 4 : 2)
append_fp8_rows_kernel(const float* part, int ksplit, int n_tok, int s_q, int d_c, int d_r,
                       const T* gamma, float eps, float rope_base, const int32_t* seqlens,
                       const int32_t* block_table, int max_pages, uint8_t* codes, int64_t code_stride,
                       float* scales, T* rope, int64_t rope_stride, int num_pages) {
  __shared__ double inv_freq[32 * kRowPairs];
  for (int i = threadIdx.x; i < d_r / 2; i += blockDim.x) inv_freq[i] = rope_inv_freq(i, d_r, rope_base);
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  const int lane = threadIdx.x & 31;
  const int N = d_c + d_r, chunks = d_c / 4;
  const int64_t step = (int64_t)n_tok * N;   // one slice
  for (int tok = blockIdx.x * kRowWarps + (threadIdx.x >> 5); tok < n_tok; tok += gridDim.x * kRowWarps) {
    const int b = tok / s_q, pos = seqlens[b] - s_q + tok % s_q;
    int64_t row = -1;
    if (pos < 0 || (pos >> 6) >= max_pages) {
      if (lane == 0) report(MLA_ERR_DEVICE_CHECK);
    } else {
      const int page = block_table[(int64_t)b * max_pages + (pos >> 6)];
      if (page >= 0 && page < num_pages) row = (int64_t)page * 64 + (pos & 63);
      else if (lane == 0) report(MLA_ERR_DEVICE_CHECK);
    }
    if (row < 0) continue;
    const float* src = part + (int64_t)tok * N;
    float4 z[kChunks];
    float2 zr[kPairs];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) z[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) zr[j] = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int s = 0; s < ksplit; ++s) {   // a slice's loads all in flight
      const float* sl = src + s * step;
      float4 v[kChunks];
      float2 r[kPairs];
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
        v[j] = lane + 32 * j < chunks ? __ldcg(reinterpret_cast<const float4*>(sl) + lane + 32 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kPairs; ++j)
        r[j] = lane + 32 * j < d_r / 2 ? __ldcg(reinterpret_cast<const float2*>(sl + d_c) + lane + 32 * j) : make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) { z[j].x += v[j].x; z[j].y += v[j].y; z[j].z += v[j].z; z[j].w += v[j].w; }
#pragma unroll
      for (int j = 0; j < kPairs; ++j) { zr[j].x += r[j].x; zr[j].y += r[j].y; }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
      ss += fmaf(z[j].x, z[j].x, z[j].y * z[j].y) + fmaf(z[j].z, z[j].z, z[j].w * z[j].w);
    ss = warp_sum(ss);
    const float inv = 1.0f / sqrtf(ss / (float)d_c + eps);
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = lane + 32 * j;
      if (c < chunks) {
        z[j].x *= inv; z[j].y *= inv; z[j].z *= inv; z[j].w *= inv;
        if (gamma) {
          z[j].x *= ld(gamma + 4 * c); z[j].y *= ld(gamma + 4 * c + 1);
          z[j].z *= ld(gamma + 4 * c + 2); z[j].w *= ld(gamma + 4 * c + 3);
        }
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(z[j].x), fabsf(z[j].y)), fmaxf(fabsf(z[j].z), fabsf(z[j].w))));
      }
    }
    amax = warp_max(amax);
    const float s = __fdiv_rn(amax, 448.f);
    const float safe = s > 0.f ? s : 1.f;
    uint8_t* dst = codes + row * code_stride;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = lane + 32 * j;
      if (c < chunks) {
        const float v[4] = {z[j].x, z[j].y, z[j].z, z[j].w};
        *reinterpret_cast<uint32_t*>(dst + 4 * c) = e4m3x4_codes(v, safe);
      }
    }
    if (lane == 0) scales[row] = s;
    T* krow = rope + row * rope_stride;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int i = lane + 32 * j;
      if (i < d_r / 2) {
        float cs, sn;
        rope_cos_sin_at(pos, inv_freq[i], &cs, &sn);
        st(krow + 2 * i, zr[j].x * cs - zr[j].y * sn);
        st(krow + 2 * i + 1, zr[j].x * sn + zr[j].y * cs);
      }
    }
  }
}

// =============================================================================================
// Read back: out row r (row_offsets[b] <= r < row_offsets[b + 1]) = [s · value(code) ; k_r] of position
// first[b] + r - row_offsets[b] of sequence b. Bound by its bytes: d_c + 4 + d_r·e in, (d_c + d_r)·e out
// per row. A block takes up to kReadRows consecutive rows: one warp finds the sequence of the first by a
// 32-way search of row_offsets, a thread per row goes on from there and looks its cache row up, and
// then all threads move 16 codes each at a time. 262,144 rows of 512 + 64 bf16: 83.5 us, 5.6 TB/s (86 % of a
// plain copy's rate; blocks of 16, 64 and 128 rows took 90, 88 and 93 us); a few hundred rows: 4 us in blocks
// of 8 rows (11 us in blocks of 64).
// =============================================================================================
constexpr int kReadRows = 32;
constexpr int kReadThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kReadThreads)
read_fp8_kernel(const uint8_t* codes, int64_t code_stride, const float* scales,
                const T* rope, int64_t rope_stride, int num_pages, const int32_t* block_table,
                int max_pages, const int32_t* first, const int32_t* row_offsets, int B,
                int64_t n_rows, int rows_per_block, int d_c, int d_r, T* out, int64_t out_stride) {
  __shared__ int64_t src_row[kReadRows];   // -1: nothing to write there
  __shared__ float src_scale[kReadRows];
  __shared__ int s_b;
  grid_dependency_wait();
  allow_dependents();
  const int64_t r0 = (int64_t)blockIdx.x * rows_per_block;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    // the last b in [0, B] with row_offsets[b] <= r0: each step keeps the one of 32 pieces that holds it
    int lo = 0, hi = B;
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + (lane + 1) * step;
      const bool le = at <= hi && (int64_t)row_offsets[at] <= r0;
      const int n = __popc(__ballot_sync(0xffffffffu, le));   // offsets do not fall: the first n hold
      lo += n * step;
      hi = min(hi, lo + step - 1);
    }
    if (lane == 0) s_b = lo;
  }
  __syncthreads();
  if ((int)threadIdx.x < rows_per_block) {
    const int64_t r = r0 + threadIdx.x;
    int64_t row = -1;
    // the last b >= s_b with row_offsets[b] <= r: steps that double, then halve (short sequences may put
    // every row of the block in another one)
    int b = s_b, stride = 1;
    while (b + stride <= B && (int64_t)row_offsets[b + stride] <= r) { b += stride; stride *= 2; }
    for (; stride > 0; stride >>= 1)
      if (b + stride <= B && (int64_t)row_offsets[b + stride] <= r) b += stride;
    if (r < n_rows && b < B) {
      const int64_t p = (int64_t)(first ? first[b] : 0) + (r - row_offsets[b]);
      int page = -1;
      if (r >= row_offsets[b] && p >= 0 && (p >> 6) < max_pages) page = block_table[(int64_t)b * max_pages + (p >> 6)];
      if (page >= 0 && page < num_pages) row = (int64_t)page * 64 + (p & 63);
      else report(MLA_ERR_DEVICE_CHECK);
    }
    src_row[threadIdx.x] = row;
    src_scale[threadIdx.x] = row >= 0 ? scales[row] : 0.f;
  }
  __syncthreads();
  const int pieces = d_c / 16;
  for (int i = threadIdx.x; i < rows_per_block * pieces; i += kReadThreads) {
    const int r = i / pieces, c = i % pieces;
    const int64_t row = src_row[r];
    if (row < 0) continue;
    const uint4 v = *(reinterpret_cast<const uint4*>(codes + row * code_stride) + c);
    const float sc = src_scale[r];
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
    float f[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 x = e4m3x2_values(q[k >> 1] >> (16 * (k & 1)) & 0xffffu);
      f[2 * k] = x.x * sc;
      f[2 * k + 1] = x.y * sc;
    }
    T* dst = out + (r0 + r) * out_stride + 16 * c;
    constexpr int V = simt::Vec16<T>::n;
#pragma unroll
    for (int k = 0; k < 16; k += V) simt::Vec16<T>::store(dst + k, f + k);
  }
  // the RoPE keys are copied as stored
  constexpr int E = 16 / (int)sizeof(T);
  if (d_r % E == 0) {
    const int rp = d_r / E;
    for (int i = threadIdx.x; i < rows_per_block * rp; i += kReadThreads) {
      const int r = i / rp, c = i % rp;
      const int64_t row = src_row[r];
      if (row >= 0)
        reinterpret_cast<uint4*>(out + (r0 + r) * out_stride + d_c)[c] =
            __ldcs(reinterpret_cast<const uint4*>(rope + row * rope_stride) + c);
    }
  } else {
    for (int i = threadIdx.x; i < rows_per_block * d_r; i += kReadThreads) {
      const int r = i / d_r, c = i % d_r;
      const int64_t row = src_row[r];
      if (row >= 0) out[(r0 + r) * out_stride + d_c + c] = rope[row * rope_stride + c];
    }
  }
}

}  // namespace cache8
}  // namespace mla
