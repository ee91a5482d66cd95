// cache_evict_kernel.cuh -- which blocks of a cache stay, by the attention
// weight their rows accumulated, and moving what stays to the front of another
// buffer.
//
// For batch row b with L rows in ceil(L / block) blocks, the key of a block is
// the sum of its valid rows' accounts.  The sum is taken in float64 and rounded
// once to float32, so that blocks next to the border do not change sides with
// the order of a sum.  What stays: the first keep_first and the last keep_last
// blocks, then the blocks with the largest keys, up to `budget` in all; equal
// keys go to the lower index, -0.0 equals +0.0, and a NaN ranks above +inf.
#pragma once

#include <cuda_runtime.h>

#include "ptx.cuh"

namespace dstopk {

struct CeParams {
  const float* mass;
  const int32_t* len;      // [B] or null (= T)
  int32_t* kept;           // [B, budget]
  int32_t* new_len;        // [B]
  int* status;
  long long mass_bstride;
  int T, block, budget, first, last;
};

__device__ __forceinline__ int ce_len(const int32_t* len, int T, int b, int* status) {
  const int L = len ? len[b] : T;
  debug_range(L >= 0 && L <= T, status);
  return min(max(L, 0), T);
}

// Order-preserving 32-bit key, larger first; protected blocks rank above all.
// 0 is below every key.
__device__ __forceinline__ uint32_t ce_key(const CeParams& p, const float* mass, int n, int nb, int L) {
  if (n < p.first || n >= nb - p.last) return 0xffffffffu;
  const int r0 = n * p.block, r1 = min(L, r0 + p.block);
  double sum = 0.0;
  for (int r = r0; r < r1; ++r) sum += (double)mass[r];
  const float v = (float)sum;
  if (v != v) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of one value per thread over a CTA of 1024, and of the threads before this one.
__device__ __forceinline__ int ce_scan(int v, int* warp_s, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_s[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < 32; ++w) {
    const int t = warp_s[w];
    if (w < warp) before += t;
    all += t;
  }
  *total = all;
  return before + x - v;
}

// One CTA per batch row: four 8-bit radix passes for the key of the last block
// that stays, then the list in ascending order.
__global__ void __launch_bounds__(1024) cache_evict_kernel(const CeParams p) {
  __shared__ int hist[256];
  __shared__ int warp_s[32];
  __shared__ uint32_t prefix_s;
  __shared__ int need_s;
  pdl_wait();
  const int b = blockIdx.x;
  const int L = ce_len(p.len, p.T, b, p.status), nb = (L + p.block - 1) / p.block;
  const float* mass = p.mass + b * p.mass_bstride;
  int32_t* kept = p.kept + (size_t)b * p.budget;
  uint32_t prefix = 0;
  int need = p.budget;  // blocks to take among those that match the prefix
  if (nb > p.budget) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (threadIdx.x < 256) hist[threadIdx.x] = 0;
      __syncthreads();
      for (int n = threadIdx.x; n < nb; n += 1024) {
        const uint32_t key = ce_key(p, mass, n, nb, L);
        if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        int d = 255;
        for (; d > 0 && hist[d] < need; --d) need -= hist[d];
        prefix_s = prefix | ((uint32_t)d << shift);
        need_s = need;
      }
      __syncthreads();
      prefix = prefix_s;
      need = need_s;
      __syncthreads();
    }
  }
  // blocks above the key stay, and the first `need` of those equal to it
  int out = 0, equal = 0;
  for (int n0 = 0; n0 < nb; n0 += 1024) {
    const int n = n0 + threadIdx.x;
    const uint32_t key = n < nb && nb > p.budget ? ce_key(p, mass, n, nb, L) : 0;
    int total = 0;
    const int eq = n < nb && nb > p.budget && key == prefix;
    const int rank = equal + ce_scan(eq, warp_s, &total);
    equal += total;
    const int stays = n < nb && (nb <= p.budget || key > prefix || (eq && rank < need));
    const int at = out + ce_scan(stays, warp_s, &total);
    out += total;
    if (stays) kept[at] = n;
    __syncthreads();
  }
  const int kept_n = min(nb, p.budget);
  for (int j = kept_n + threadIdx.x; j < p.budget; j += 1024) kept[j] = -1;
  __syncthreads();
  if (threadIdx.x == 0) {
    // the last block may be short: it stays exactly if it is the last of the list
    const int tail = nb > 0 && kept[kept_n - 1] == nb - 1 ? nb * p.block - L : 0;
    p.new_len[b] = kept_n * p.block - tail;
  }
  pdl_launch_dependents();
}

constexpr int kCcMaxArrays = 8;

struct CcArray {
  const uint8_t* src;
  uint8_t* dst;
  long long src_bstride, dst_bstride;  // bytes
  long long item;                      // bytes of a row, or of a block's entry
  int per_block;
  int vec;                             // bytes of one access: 16, 4 or 1
};

struct CcParams {
  CcArray a[kCcMaxArrays];
  const int32_t* kept;  // [B, budget]
  const int32_t* len;   // [B] or null (= T)
  int* status;
  int T, block, budget, n;
};

template <class V>
__device__ __forceinline__ void cc_move(uint8_t* dst, const uint8_t* src, long long bytes) {
  const long long words = bytes / (long long)sizeof(V);
  for (long long i = threadIdx.x; i < words; i += blockDim.x)
    reinterpret_cast<V*>(dst)[i] = reinterpret_cast<const V*>(src)[i];
}

// One CTA per kept entry: every array's bytes of one block.
__global__ void __launch_bounds__(256) cache_compact_kernel(const CcParams p) {
  pdl_wait();
  const int j = blockIdx.x % p.budget, b = blockIdx.x / p.budget;
  const int L = ce_len(p.len, p.T, b, p.status), nb = (L + p.block - 1) / p.block;
  const int n = p.kept[(size_t)b * p.budget + j];
  debug_range(n >= -1 && n < nb, p.status);
  if (n >= 0 && n < nb) {
    // as far as the block's rows are valid, and within the min(T, budget * block) rows of dst
    const int rows = min(min(p.block, L - n * p.block), p.T - j * p.block);
    for (int i = 0; i < p.n; ++i) {
      const CcArray& a = p.a[i];
      const long long unit = a.per_block ? a.item : a.item * p.block;
      const uint8_t* src = a.src + b * a.src_bstride + n * unit;
      uint8_t* dst = a.dst + b * a.dst_bstride + j * unit;
      const long long bytes = a.per_block ? a.item : a.item * rows;
      if (a.vec == 16)
        cc_move<uint4>(dst, src, bytes);
      else if (a.vec == 4)
        cc_move<uint32_t>(dst, src, bytes);
      else
        cc_move<uint8_t>(dst, src, bytes);
    }
  }
  pdl_launch_dependents();
}

}  // namespace dstopk
