// cache_quant_kernel.cuh -- writing bfloat16 rows into a cache held in 8 bits
// with one float32 scale for each block of rows and KV head.
//
// For the rows r of the call that fall into one block, and one KV head:
//     a = max |x[r, c]|, at least 2^-100
//     s = a / M,  code[r, c] = rn8(x[r, c] * (M / a))
// with M = 448 (e4m3) or 127 (int8) and the quotients and the product in
// float32, so a code is a function of (x, a) alone and any IEEE evaluation
// gives the same one.  The floor on a keeps M / a finite (448 * 2^100 < 2^109)
// and the scale normal; a block of zeros has codes 0.  If a value of the block
// is not finite the scale is NaN and the codes are 0: the block reads as NaN.
#pragma once

#include <cuda_runtime.h>

#include "cache_format.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace dstopk {

struct CqParams {
  const uint16_t* rows;    // bf16: row r of batch row b at rows + b * rows_bstride + r * rows_rstride
  uint8_t* codes;          // batch row b's cache at codes + b * codes_bstride
  float* scales;           // batch row b's scales at scales + b * scales_bstride
  const int32_t* pos;      // [B] or null (= 0)
  const int32_t* len;      // [B] or null (= n)
  int* status;
  long long rows_bstride, rows_rstride, codes_bstride, scales_bstride;  // elements
  int B, n, Hkv, D, T;
  int log_block;
  int nblocks;             // blocks of n rows
};

// Rows of batch row b that are written, and the block its first row starts.
__device__ __forceinline__ int cq_live(const CqParams& p, int b, int* first_block) {
  const int pos = p.pos ? p.pos[b] : 0;
  const int block = 1 << p.log_block;
  const bool ok = pos >= 0 && pos <= p.T && (pos & (block - 1)) == 0;
  debug_range(ok, p.status);
  if (!ok) return 0;
  int live = p.len ? p.len[b] : p.n;
  debug_range(live >= 0 && live <= p.n && live <= p.T - pos, p.status);
  live = min(min(max(live, 0), p.n), p.T - pos);
  *first_block = pos >> p.log_block;
  return live;
}

template <int FMT>
__device__ __forceinline__ uint2 cq_encode8(const uint4& x, float inv) {
  if (inv == 0.0f) return make_uint2(0u, 0u);  // a block that is not finite
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = encode8x2<FMT>(__fmul_rn(__uint_as_float(w[i] << 16), inv), __fmul_rn(__uint_as_float(w[i] & 0xffff0000u), inv));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// NT threads to a block of rows and KV head (kCqGroup / NT of these to a CTA): each
// holds up to 8 pieces of 8 values in registers, so that a row is read once, and
// the block's largest magnitude is one integer maximum over the group (the bits of
// a magnitude order like its value).  NT is the smallest that holds the block.
// Bytes bound it, 2 read and 1 written for each value, but only just: a value costs
// about 5 instructions, so addresses are advanced, not worked out, per piece (8 x 16384
// rows of 512 in blocks of 64: 37.8 us in graph replays, 38.7 call by call, 5.2 to 5.3
// TB/s, 79 to 81% of the copy rate; worked out, 52).
constexpr int kCqPieces = 8;

template <int FMT, int NT>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT, NT <= 256 ? 4 : 1024 / NT) cache_quantize_kernel(const CqParams p) {
  constexpr int kGroups = NT < 256 ? 256 / NT : 1;
  __shared__ uint32_t warp_max[NT < 256 ? 8 : NT / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int group = threadIdx.x / NT, t = threadIdx.x % NT;
  const long long unit = (long long)blockIdx.x * kGroups + group;
  const int n = (int)(unit % p.nblocks), g = (int)(unit / p.nblocks % p.Hkv);
  const long long b = unit / p.nblocks / p.Hkv;
  int blk0 = 0;
  const int live = b < p.B ? cq_live(p, (int)b, &blk0) : 0;
  const int r0 = n << p.log_block, nr = min(1 << p.log_block, live - r0);
  const int per = p.D >> 3;                                // pieces of a row
  const int pieces = nr * per;
  // from one piece of this thread to its next, NT pieces on: `hop` on, and `wrap` more past a row's end
  const int step_row = NT / per, step_col = NT - step_row * per, row = t / per, col0 = t - row * per;
  const uint16_t* src = p.rows + b * p.rows_bstride + (r0 + row) * p.rows_rstride + (long long)g * p.D + col0 * 8;
  const long long hop = step_row * p.rows_rstride + step_col * 8, wrap = p.rows_rstride - p.D;
  uint4 v[kCqPieces];
  uint32_t a = 0;
  int col = col0;
#pragma unroll
  for (int i = 0; i < kCqPieces; ++i) {
    v[i] = t + i * NT < pieces ? __ldcs(reinterpret_cast<const uint4*>(src)) : make_uint4(0u, 0u, 0u, 0u);
    src += hop, col += step_col;
    if (col >= per) col -= per, src += wrap;
  }
#pragma unroll
  for (int i = 0; i < kCqPieces; ++i) a = max(a, max_abs_bf16x8(v[i]));
  a = __reduce_max_sync(0xffffffffu, a);
  if constexpr (NT > 32) {
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = a;
    if constexpr (NT >= 256)
      __syncthreads();
    else
      named_bar_sync(1 + group, NT);
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) a = max(a, warp_max[group * (NT / 32) + w]);
  }
  const BlockScale s = block_scale<FMT>(a);
  const long long first = ((long long)blk0 << p.log_block) + r0;
  const int width = p.Hkv * p.D;
  uint8_t* dst = p.codes + b * p.codes_bstride + (first + row) * width + (long long)g * p.D + col0 * 8;
  const int dhop = step_row * width + step_col * 8, dwrap = width - p.D;
  col = col0;
#pragma unroll
  for (int i = 0; i < kCqPieces; ++i) {
    if (t + i * NT < pieces) *reinterpret_cast<uint2*>(dst) = cq_encode8<FMT>(v[i], s.inv);
    dst += dhop, col += step_col;
    if (col >= per) col -= per, dst += dwrap;
  }
  if (t == 0 && nr > 0) p.scales[b * p.scales_bstride + (long long)(blk0 + n) * p.Hkv + g] = s.scale;
}

}  // namespace dstopk
