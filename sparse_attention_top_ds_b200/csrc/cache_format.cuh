// cache_format.cuh -- the formats of a cached row: bfloat16 values, or 8-bit
// codes (e4m3 or int8) whose value is the code times the float32 scale of the
// row's block and KV head.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace dstopk {

constexpr int kFmtBf16 = 1, kFmtE4m3 = 2, kFmtI8 = 3;  // DS_BF16, DS_E4M3, DS_I8

// Two values to two 8-bit codes, nearest even (`lo` in the low byte); the
// values are at most the format's largest up to the rounding of one product.
template <int FMT>
__device__ __forceinline__ uint32_t encode8x2(float lo, float hi) {
  if constexpr (FMT == kFmtE4m3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    return ((uint32_t)__float2int_rn(lo) & 0xffu) | (((uint32_t)__float2int_rn(hi) & 0xffu) << 8);
  }
}

// Largest magnitude of 8 bfloat16 values, as the bits of its absolute value
// (a NaN's are the largest of all).
__device__ __forceinline__ uint32_t max_abs_bf16x8(const uint4& v) {
  const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
  const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  return max(m & 0xffffu, m >> 16);
}

struct BlockScale {
  float scale, inv;
};

// The scale of a block whose largest magnitude has the bfloat16 bits `amax`.
template <int FMT>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax) {
  constexpr float kTop = FMT == kFmtE4m3 ? 448.0f : 127.0f;
  if (amax >= 0x7f80u) return {__uint_as_float(0x7fc00000u), 0.0f};  // an infinity or a NaN in the block
  const float a = fmaxf(__uint_as_float(amax << 16), 0x1p-100f);
  return {__fdiv_rn(a, kTop), __fdiv_rn(kTop, a)};
}

// Four codes (a 32-bit word) to four bfloat16 values: codes 0 and 2 in `even`, 1
// and 3 in `odd`.  Exact: a code has at most 8 significant bits.  Pairs that lie
// 16 bits apart in the word need no byte permutation, which leaves 5 instructions
// to the integer pipe for a word instead of 8; what is stored this way has
// channels 1 and 2 of every 4 exchanged (swap_middle does it to other operands).
//  * e4m3: the 4 exponent and 3 mantissa bits are moved into a bfloat16's
//    fields, which gives the value times 2^-120 (the exponent biases are 7 and
//    127; subnormal codes become subnormal values), and multiplied by 2^120.  That
//    reads NaN as 480: `top` collects the largest such fields for e4m3_nan.
//  * int8: with s the sign bit and l the low 7 bits the value is
//    (128 + l) - (128 + 128 s), and both terms are 0x4300 with bits or-ed in.
template <int FMT>
__device__ __forceinline__ void decode8x4(uint32_t w, uint32_t& even, uint32_t& odd, uint32_t& top) {
  if constexpr (FMT == kFmtE4m3) {
    const uint32_t k = 0x7b807b80u;  // 2^120 twice
    even = (w << 4) & 0x07f007f0u, odd = (w >> 4) & 0x07f007f0u;
    top = __vmaxu2(__vmaxu2(top, even), odd);  // (cheaper than a look at the codes' bytes)
    even |= (w << 8) & 0x80008000u, odd |= w & 0x80008000u;
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(even) : "r"(k));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(odd) : "r"(k));
  } else {
    const uint32_t k = 0x43004300u, v = w >> 8;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(even) : "r"((w & 0x007f007fu) | k), "r"((w & 0x00800080u) | k));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(odd) : "r"((v & 0x007f007fu) | k), "r"((v & 0x00800080u) | k));
  }
}

// Was there a NaN among the codes of these largest fields?
__device__ __forceinline__ bool e4m3_nan(uint32_t top) { return ((top + 0x00100010u) & 0x08000800u) != 0; }

// 8 values of 16 bits with the middle two of every 4 exchanged.
__device__ __forceinline__ uint4 swap_middle(const uint4& x) {
  return make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x5410),
                    __byte_perm(x.z, x.w, 0x7632));
}

}  // namespace dstopk
