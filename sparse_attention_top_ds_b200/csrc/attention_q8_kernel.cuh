// attention_q8_kernel.cuh -- decode attention over the selected rows of a cache
// held in 8 bits (a float32 scale for each block of rows and KV head) plus a
// bfloat16 window, and the account of the weight every selected row received.
//
// For batch row b, KV head g and the query heads h of g's group, over the
// attended rows (the selected cache rows, then the window rows)
//     z[h, r] = scale * (q_h . row_r),   L[h] = sum_r e^z[h, r] + e^sink[h],
//     out[h]  = sum_r e^z[h, r] row_r / L[h],   lse[h] = log L[h],
// where row_r is key and value and a cache row is s[r / block, g] * code[r].
// The account adds  sum_h e^(z[h, r] - lse[h])  to mass[b, r].
#pragma once

#include <cuda_runtime.h>

#include "cache_format.cuh"
#include "ptx.cuh"

namespace dstopk {

struct AqParams {
  const uint16_t* q;       // bf16 [B, H, D]
  const uint8_t* cache;    // codes, or bf16 rows: [T, Hkv, D] per batch row
  const float* scales;     // [ceil(T / block), Hkv] per batch row; null for bf16
  const uint16_t* win;     // bf16 [B, W, Hkv, D] or null
  const int32_t* idx;      // [B, k] or null
  const int32_t* win_len;  // [B] or null
  const float* sink;       // [H] or null
  uint16_t* out;           // bf16 [B, H, D]
  float* lse;              // [B, H] or null; read by the account
  float* mass;             // the account: [T] per batch row
  int* status;
  uint64_t wait_ns;
  long long cache_bstride;   // elements from one batch row's cache to the next
  long long scales_bstride;  // scales from one batch row's to the next
  long long mass_bstride;
  int T, k, W, B, H, Hkv, D, log_block;
  float scale_log2;        // scale * log2(e)
};

// The cache row of slot j of batch row b, or -1 if the slot is skipped.
__device__ __forceinline__ int aq_slot(const AqParams& p, int b, int j) {
  const int r = p.idx[(size_t)b * p.k + j];
  debug_range(r >= -1 && r < p.T, p.status);
  return r >= 0 && r < p.T ? r : -1;
}

__device__ __forceinline__ int aq_window(const AqParams& p, int b) {
  int wl = p.win_len ? p.win_len[b] : p.W;
  debug_range(wl >= 0 && wl <= p.W, p.status);
  return min(max(wl, 0), p.W);
}

__device__ __forceinline__ float aq_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Element c of a row, without its scale.
template <int FMT>
__device__ __forceinline__ float aq_value(const uint8_t* row, int c) {
  if constexpr (FMT == kFmtBf16) return aq_bf16(reinterpret_cast<const uint16_t*>(row)[c]);
  uint32_t lo, hi;
  decode8x4<FMT>(row[c], lo, hi);
  return __uint_as_float(lo << 16);
}

template <int FMT>
__device__ __forceinline__ const uint8_t* aq_row(const AqParams& p, int b, int r, int g) {
  constexpr int kSize = FMT == kFmtBf16 ? 2 : 1;
  return p.cache + (b * p.cache_bstride + ((long long)r * p.Hkv + g) * p.D) * kSize;
}

template <int FMT>
__device__ __forceinline__ float aq_scale(const AqParams& p, int b, int r, int g) {
  if constexpr (FMT == kFmtBf16) return 1.0f;
  return p.scales[b * p.scales_bstride + (long long)(r >> p.log_block) * p.Hkv + g];
}

__device__ __forceinline__ float aq_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float aq_warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// One CTA per batch row and query head: the scores of every slot in shared
// memory (k + W floats), then the weighted sum column by column.
template <int FMT>
__global__ void __launch_bounds__(256) attn_q8_kernel(const AqParams p) {
  extern __shared__ float z_s[];
  __shared__ float red[9];
  pdl_wait();
  const int h = blockIdx.x % p.H, b = blockIdx.x / p.H, g = h / (p.H / p.Hkv);
  const int n = p.k + aq_window(p, b), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint16_t* q = p.q + ((size_t)b * p.H + h) * p.D;
  float m = -INFINITY;
  for (int j = warp; j < n; j += 8) {
    const int r = j < p.k ? aq_slot(p, b, j) : j - p.k;
    float z = -INFINITY;
    if (r >= 0) {
      float dot = 0.0f;
      if (j < p.k) {
        const uint8_t* row = aq_row<FMT>(p, b, r, g);
        for (int c = lane; c < p.D; c += 32) dot = fmaf(aq_bf16(q[c]), aq_value<FMT>(row, c), dot);
        dot *= aq_scale<FMT>(p, b, r, g);
      } else {
        const uint16_t* row = p.win + (((long long)b * p.W + r) * p.Hkv + g) * p.D;
        for (int c = lane; c < p.D; c += 32) dot = fmaf(aq_bf16(q[c]), aq_bf16(row[c]), dot);
      }
      z = aq_warp_sum(dot) * p.scale_log2;
    }
    if (lane == 0) z_s[j] = z;
    m = fmaxf(m, z);
  }
  const float sink = p.sink ? p.sink[h] * 1.4426950408889634f : -INFINITY;
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = sink;
  for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
  const float mu = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  for (int j = threadIdx.x; j < n; j += 256) {
    const float e = exp2f(z_s[j] - mu);
    z_s[j] = e;
    l += e;
  }
  l = aq_warp_sum(l);
  __syncthreads();
  if (lane == 0) red[warp] = l;
  __syncthreads();
  l = exp2f(sink - mu);
  for (int w = 0; w < 8; ++w) l += red[w];
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a NaN stays one
  for (int c = threadIdx.x; c < p.D; c += 256) {
    float acc = 0.0f;
    for (int j = 0; j < n; ++j) {
      const int r = j < p.k ? aq_slot(p, b, j) : j - p.k;
      if (r < 0) continue;
      const float v = j < p.k ? aq_value<FMT>(aq_row<FMT>(p, b, r, g), c) * aq_scale<FMT>(p, b, r, g)
                              : aq_bf16(p.win[(((long long)b * p.W + r) * p.Hkv + g) * p.D + c]);
      acc = fmaf(z_s[j], v, acc);
    }
    uint32_t u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(0.0f), "f"(acc * inv));
    p.out[((size_t)b * p.H + h) * p.D + c] = (uint16_t)u;
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[(size_t)b * p.H + h] = l == 0.0f ? -INFINITY : (mu + log2f(l)) * 0.6931471805599453f;
  pdl_launch_dependents();
}

// One warp per batch row and slot: the row's weight, summed over the heads.
template <int FMT>
__global__ void __launch_bounds__(256) attn_mass_kernel(const AqParams p) {
  pdl_wait();
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i < (long long)p.B * p.k) {
    const int b = (int)(i / p.k), r = aq_slot(p, b, (int)(i % p.k)), G = p.H / p.Hkv;
    if (r >= 0) {
      float w = 0.0f;
      for (int h = 0; h < p.H; ++h) {
        const uint16_t* q = p.q + ((size_t)b * p.H + h) * p.D;
        const uint8_t* row = aq_row<FMT>(p, b, r, h / G);
        float dot = 0.0f;
        for (int c = lane; c < p.D; c += 32) dot = fmaf(aq_bf16(q[c]), aq_value<FMT>(row, c), dot);
        dot = aq_warp_sum(dot) * aq_scale<FMT>(p, b, r, h / G);
        const float lse = p.lse[(size_t)b * p.H + h];
        if (lse != -INFINITY) w += exp2f(fmaf(dot, p.scale_log2, lse * -1.4426950408889634f));
      }
      if (lane == 0) atomicAdd(p.mass + b * p.mass_bstride + r, w);
    }
  }
  pdl_launch_dependents();
}

}  // namespace dstopk
