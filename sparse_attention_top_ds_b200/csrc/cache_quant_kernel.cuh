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

namespace dstopk {

struct CqParams {
  const uint16_t* rows;    // bf16: row r of batch row b at rows + b * rows_bstride + r * rows_rstride
  uint8_t* codes;          // batch row b's cache at codes + b * codes_bstride
  float* scales;           // batch row b's scales at scales + b * scales_bstride
  const int32_t* pos;      // [B] or null (= 0)
  const int32_t* len;      // [B] or null (= n)
  int* status;
  long long rows_bstride, rows_rstride, codes_bstride, scales_bstride;  // elements
  int n, Hkv, D, T;
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

// One CTA per block of rows and KV head, two passes over its rows.
template <int FMT>
__global__ void __launch_bounds__(256) cache_quantize_kernel(const CqParams p) {
  pdl_wait();
  const int n = blockIdx.x % p.nblocks, g = (blockIdx.x / p.nblocks) % p.Hkv, b = blockIdx.x / p.nblocks / p.Hkv;
  int blk0 = 0;
  const int live = cq_live(p, b, &blk0);
  const int r0 = n << p.log_block, nr = min(1 << p.log_block, live - r0);
  if (nr > 0) {
    const uint16_t* src = p.rows + b * p.rows_bstride + r0 * p.rows_rstride + (long long)g * p.D;
    const int per = p.D >> 3, pieces = nr * per;
    uint32_t a = 0;
    for (int i = threadIdx.x; i < pieces; i += 256) {
      const uint4 v = *(reinterpret_cast<const uint4*>(src + (i / per) * p.rows_rstride) + i % per);
      a = max(a, max_abs_bf16x8(v));
    }
    __shared__ uint32_t sa;
    if (threadIdx.x == 0) sa = 0;
    __syncthreads();
    atomicMax(&sa, a);
    __syncthreads();
    const BlockScale s = block_scale<FMT>(sa);
    const long long row = ((long long)blk0 << p.log_block) + r0;
    uint8_t* dst = p.codes + b * p.codes_bstride + (row * p.Hkv + g) * p.D;
    for (int i = threadIdx.x; i < pieces; i += 256) {
      const uint4 v = *(reinterpret_cast<const uint4*>(src + (i / per) * p.rows_rstride) + i % per);
      *(reinterpret_cast<uint2*>(dst + (long long)(i / per) * p.Hkv * p.D) + i % per) = cq_encode8<FMT>(v, s.inv);
    }
    if (threadIdx.x == 0) p.scales[b * p.scales_bstride + (long long)(blk0 + n) * p.Hkv + g] = s.scale;
  }
  pdl_launch_dependents();
}

}  // namespace dstopk
