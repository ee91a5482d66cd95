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

#include <cuda.h>
#include <cuda_runtime.h>

#include "cache_format.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

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
  int HT, R, C;            // head tiles of a KV head, rows of a chunk, CTAs of a cluster
  float scale_log2;        // scale * log2(e)
  int fault;               // testing the failure detection: 1 = in CTA 0 the rows' barriers await an arrival more than come
};

__device__ __forceinline__ int aq_window(const AqParams& p, int b) {
  int wl = p.win_len ? p.win_len[b] : p.W;
  debug_range(wl >= 0 && wl <= p.W, p.status);
  return min(max(wl, 0), p.W);
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

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The wait for an mbarrier that is not there yet.  One that runs out records the timeout and
// sets the word at gave_up in shared memory, after which the CTA's other waits no longer
// last: its warps pass all their barriers and the CTA ends within about one limit.  (The
// attention's outputs then mean nothing.)  What is then still in flight, aq_drain waits
// for.
__device__ __forceinline__ void aq_poll(uint32_t bar, uint32_t parity, int* status, uint64_t limit, uint32_t gave_up) {
  if (limit == 0) limit = kWaitLimitNs;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) break;
    if ((it & 255u) == 0 && (globaltimer_ns() - t0 > limit || lds32(gave_up) != 0u)) {
      record_status(status, kErrTimeout);
      asm volatile("st.shared.u32 [%0], 1;" ::"r"(gave_up) : "memory");
      break;
    }
  }
}
static __device__ __noinline__ void aq_poll_far(uint32_t bar, uint32_t parity, int* status, uint64_t limit, uint32_t gave_up) {
  aq_poll(bar, parity, status, limit, gave_up);
}

// A warp's wait.  All lanes poll: a chunk's turn is a chain of a dozen such waits,
// and a wait by one lane with the others behind it woke up later each time (the
// decode call took 20.5 us instead of 19.0).  FAR: the polling is a call, which keeps
// the code short (8 decode rows 18.8 us, 19.5 polling in place), where what is live fits
// the registers that a call leaves alone (the workers' of 64 heads do not: 512 tokens over
// 2048 rows 601 us, 596 in place; nor does it help the account: 879 and 837 on the same).
template <bool FAR>
__device__ __forceinline__ void aq_wait(uint32_t bar, uint32_t parity, const AqParams& p, uint32_t gave_up) {
  if (!mbar_try_wait(bar, parity)) {
    if constexpr (FAR)
      aq_poll_far(bar, parity, p.status, p.wait_ns, gave_up);
    else
      aq_poll(bar, parity, p.status, p.wait_ns, gave_up);
  }
  __syncwarp();
}

// The end of a CTA that gave up, by the warp that issues: its MMAs and its last copy of
// queries (announced on bar_q in phase `parity`) are waited for once more, within the
// limit, before tensor and shared memory are given back.  `bar` has had no use before.
__device__ __forceinline__ void aq_drain(uint32_t bar, uint32_t bar_q, uint32_t parity, const AqParams& p) {
  if (elect_lane()) mma_commit(bar);
  __syncwarp();
  mbar_wait_bounded(bar, 0, p.status, p.wait_ns);
  mbar_wait_bounded(bar_q, parity, p.status, p.wait_ns);
  __syncwarp();
}

// ------------------------------------------------------------------ the rows of a chunk in shared memory

constexpr int kAqRows = 128;                 // rows of a chunk: M of S^T = rows . Q^T
constexpr int kAqBlock = kAqRows * 128;      // bytes of a chunk's rows in one 64-column block
constexpr int kAqMaxCluster = 16;

// A chunk: n rows, either slots j0.. of batch row b, or its window rows j0...
struct AqChunk {
  int j0, n;
  bool win;
};

// The row that place i of a chunk reads (a cache row or a window row), or -1: as
// it is read, so that its latency passes unseen until aq_checked looks at it.
__device__ __forceinline__ int aq_chunk_slot(const AqParams& p, const AqChunk& c, int b, int i) {
  int r = -1;
  if (i < c.n) {
    r = c.j0 + i;
    // (volatile: a plain read would be moved down to where it is used)
    if (!c.win) asm volatile("ld.global.b32 %0, [%1];" : "=r"(r) : "l"(p.idx + (size_t)b * p.k + c.j0 + i) : "memory");
  }
  return r;
}

// The row, or -1 if the slot is skipped.
__device__ __forceinline__ int aq_checked(const AqParams& p, bool win, int r) {
  if (win) return r;
  debug_range(r >= -1 && r < p.T, p.status);
  return r < p.T ? max(r, -1) : -1;
}

// A chunk's rows are widened to bfloat16 (exactly, without their scale) and
// stored as 64-column blocks of 128 rows x 128 bytes, 128-byte swizzle; skipped
// rows are zeros.  Read K-major the blocks are the rows operand of the scores,
// read MN-major that of the weighted sum.  Warp w takes rows 8 w .. + 7 of every
// block (with K = 2, for 8 warps, 64 + 8 w .. too), 4 lanes to a row and 16
// columns to a lane, so that a row's 64 (128) bytes are one request and the two
// 16-byte stores of 8 consecutive lanes meet 8 different bank groups.  A lane
// loads ahead (channels 1 and 2 of every 4 are stored exchanged, see decode8x4): a
// batch is 4 pieces of 16 bytes of each of its K rows, of codes
// those of 4 blocks, of bfloat16 rows those of 2 blocks.
template <int FMT, int K>
__device__ __forceinline__ void aq_load(uint4 (&v)[4 * K], const uint8_t* const (&src)[K], int batch, int DB) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int db = FMT == kFmtBf16 ? batch * 2 + (i >> 1) : batch * 4 + i;
      const uint8_t* at = FMT == kFmtBf16 ? src[k] + db * 128 + (i & 1) * 16 : src[k] + db * 64;
      v[k * 4 + i] = src[k] != nullptr && db < DB ? __ldcg(reinterpret_cast<const uint4*>(at)) : make_uint4(0u, 0u, 0u, 0u);
    }
}

// Store the pair of blocks 2 m, 2 m + 1 from its batch.
template <int FMT, int K>
__device__ __forceinline__ void aq_store(const uint4 (&v)[4 * K], int m, int n, int DB, uint32_t rows_s) {
  const int lane = threadIdx.x & 31, sub = (threadIdx.x >> 5) * 8 + (lane >> 2);
  const uint32_t at0 = rows_s + (uint32_t)(m * 2 * kAqBlock + sub * 128) + (((uint32_t)(lane & 3) * 32u) ^ ((uint32_t)(sub & 7) << 4));
#pragma unroll
  for (int k = 0; k < K; ++k) {
    // rows from the next multiple of 16 on meet weights that no MMA reads
    if ((int)(threadIdx.x >> 5) * 8 + k * 64 >= ((n + 15) & ~15)) break;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (2 * m + e >= DB) break;
      uint4 lo, hi;
      if constexpr (FMT == kFmtBf16) {
        lo = swap_middle(v[k * 4 + e * 2]), hi = swap_middle(v[k * 4 + e * 2 + 1]);
      } else {
        const uint4 x = v[k * 4 + (m & 1) * 2 + e];
        uint32_t top = 0;
        decode8x4<FMT>(x.x, lo.x, lo.y, top);
        decode8x4<FMT>(x.y, lo.z, lo.w, top);
        decode8x4<FMT>(x.z, hi.x, hi.y, top);
        decode8x4<FMT>(x.w, hi.z, hi.w, top);
        // one NaN makes the row's scores NaN, wherever it is.  (The check took 512 tokens
        // over 2048 rows from 560 us to 587, and the decode call from 19.1 to 19.5.)
        if (FMT == kFmtE4m3 && e4m3_nan(top)) lo.x = 0x7fc07fc0u;
      }
      const uint32_t at = at0 + (uint32_t)(e * kAqBlock + k * 64 * 128);
      sts128(at, lo);
      sts128(at ^ 16u, hi);
    }
  }
}

// The queries in the rows' order of channels: `bytes` of them in shared memory at
// q, by `threads` threads.
__device__ __forceinline__ void aq_swap_queries(uint32_t q, int bytes, int thread, int threads) {
  for (int i = thread * 16; i < bytes; i += threads * 16) sts128(q + (uint32_t)i, swap_middle(lds128(q + (uint32_t)i)));
  fence_proxy_async_smem();
}

// ------------------------------------------------------------------ attention
//
// A CTA owns a batch row, a KV head and N of its query heads, and every C-th
// chunk of up to 128 attended rows; the C CTAs of a cluster share one such
// tile.  Both products have the rows or the channels as M, so that a row's
// scale is one factor of a thread and the queries are the narrow operand:
//     S^T [rows, heads]    = rows . Q^T    (K = channels)
//     O^T [channels, heads] += rows^T . P^T  (K = rows), P = 2^(z - m) * scale,
// with S^T (N columns) and O^T (N columns for each 128 channels, or 2 N) in tensor
// memory: at most 320 of its 512 columns.  The widened rows serve both products
// (128 KiB at 512 channels), the queries stay (64 KiB), P^T takes 16 KiB.
//
// A weight times its row's scale is the sum of two bfloat16 numbers, the rounded value
// and the rounded rest (together off by at most 2^-16 of it), as long as N <= 32: they
// are 2 N columns of one P^T, an MMA of which takes as long as one of N, and O^T is
// their two halves' sum.  Rounded once, a weight is off by up to half a bfloat16 step
// (2^-8 of it); with few attended rows nothing averages that out, and the outputs were
// up to 1.7 times as far from the exact ones as their own rounding puts them.  With 64
// heads the second half would not fit tensor memory (576 columns).  A call of at most 64
// rows leaves half of P^T's 128 rows free: they take the rests, with MMAs of their own.
// More rows average the roundings out (512 tokens over 2048 rows: 1.3 times the distance),
// and such MMAs would add a fifth to a chunk's time: their weights are rounded once.
//
// A chunk passes through in turn: the widened rows serve both products, so
// nothing of the next chunk can be stored before the weighted sum has freed its
// pair of blocks, and widening and softmax never run at the same time.  All 8
// worker warps therefore do both: widen chunk i, block pair by block pair as it
// is freed (the scores' MMAs follow pair by pair), issue the loads of chunk
// i + 1, then take the softmax of chunk i, 32 rows and N/2 heads to a warp.  Warp
// 8 issues the MMAs.  (16 workers have 96 registers to a thread, which spills;
// with 8 the work of a thread is wide enough to cover its latencies.)
// A head's maximum runs over lanes: a butterfly that halves the heads at each
// step, then one exchange among the four warps of a part.  The running maximum is
// raised, and O^T rescaled, only when a chunk exceeds it by 2^8 (P stays below
// 2^8, and bfloat16 and float32 keep their relative precision).  A head's
// normaliser is summed from the unrounded weights in float32, one partial sum
// per row and thread, and reduced once at the end.
//
// The cluster's partial results meet in shared memory: every CTA sends each 32
// channels x 4 heads of its O^T to the CTA that owns them, and each owner adds
// the C contributions in rank order, scaled to the common maximum.
//
// 128 heads of 512 channels: 8 batch rows over 1024 + 128 rows take 19.2 us, 512 over
// 2048 rows of one cache 594 us (28% of the measured tensor rate).  What bounds it is
// the chain within a chunk, and shared memory: the MMAs and the widened rows want half
// of a chunk's time of its bandwidth.
constexpr int kAqWorkers = 8;
constexpr int kAqThreads = (kAqWorkers + 1) * 32;

template <int N>
struct AqSmem {
  __host__ __device__ static constexpr int q_off(int D) { return (D + 127) / 128 * 2 * kAqBlock; }
  __host__ __device__ static constexpr int p_off(int D) { return q_off(D) + D / 64 * N * 128; }
  __host__ __device__ static constexpr int st_off(int D) { return p_off(D) + kAqRows * 128; }  // float2 [16][N]
  __host__ __device__ static constexpr int ft_off(int D) { return st_off(D) + kAqMaxCluster * N * 8; }  // float [16][N]
  __host__ __device__ static constexpr int mx_off(int D) { return ft_off(D) + kAqMaxCluster * N * 4; }  // float [2][8][32]
  __host__ __device__ static constexpr int bc_off(int D) { return mx_off(D) + 2048; }   // float [8][2][32]
  __host__ __device__ static constexpr int bar_off(int D) { return bc_off(D) + 2048; }
  __host__ __device__ static constexpr int slot_off(int D) { return bar_off(D) + 16 * 8; }
  __host__ __device__ static constexpr int bytes(int D) { return slot_off(D) + 16 + 1024; }  // + alignment slack
};

// Reduce NH values, times the lane's f, over the warp's lanes; the lane's result
// is that of value lane % NH.
template <int NH, class Op>
__device__ __forceinline__ float aq_reduce_heads(const float (&v)[NH], float f, Op op) {
  const int lane = threadIdx.x & 31;
  float t[NH / 2];
#pragma unroll
  for (int i = 0; i < NH / 2; ++i) {
    const bool up = lane & (NH / 2);
    const float send = up ? v[i] : v[i + NH / 2], keep = up ? v[i + NH / 2] : v[i];
    t[i] = op(keep * f, __shfl_xor_sync(0xffffffffu, send * f, NH / 2));
  }
#pragma unroll
  for (int s = NH / 4; s > 0; s >>= 1) {
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const bool up = lane & s;
      const float send = up ? t[i] : t[i + s], keep = up ? t[i + s] : t[i];
      t[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, s));
    }
  }
  float r = t[0];
#pragma unroll
  for (int s = NH; s < 32; s <<= 1) r = op(r, __shfl_xor_sync(0xffffffffu, r, s));
  return r;
}

// NH consecutive TMEM columns of this thread's lane.
template <int NH>
__device__ __forceinline__ void aq_tmem_ld(uint32_t taddr, float (&z)[NH]) {
  if constexpr (NH == 4) {
    uint32_t r[4];
    tmem_ld4(taddr, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = __uint_as_float(r[e]);
  } else {
#pragma unroll
    for (int i = 0; i < NH; i += 8) {
      uint32_t r[8];
      tmem_ld8(taddr + (uint32_t)i, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i + e] = __uint_as_float(r[e]);
    }
  }
}

// 2^x, results below 2^-126 as 0.
__device__ __forceinline__ float aq_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t aq_pack(float lo, float hi) {
  uint32_t u;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
  return u;
}

// Two weights as bfloat16 numbers, and what they lose as two more.
__device__ __forceinline__ uint32_t aq_rest(float lo, float hi, uint32_t packed) {
  return aq_pack(lo - __uint_as_float(packed << 16), hi - __uint_as_float(packed & 0xffff0000u));
}

__device__ __forceinline__ void dsmem_st_f32x2(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

__device__ __forceinline__ void dsmem_st_f32x4(uint32_t addr, const float* v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3])
               : "memory");
}

// FEW (N = 64 only): chunks of at most 64 rows, whose weights' rests are rows 64 and up of P^T.
template <int FMT, int N, bool FEW>
__global__ void __launch_bounds__(kAqThreads, 1)
    attn_q8_kernel(const __grid_constant__ CUtensorMap tm_q, const AqParams p) {
  using L_ = AqSmem<N>;
  constexpr int NH = N / 2;  // heads of a softmax thread
  constexpr int kTerms = N <= 32 ? 2 : 1, NO = kTerms * N;  // columns of O^T for 128 channels
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int D = p.D, DB = D >> 6, MT = (D + 127) >> 7;
  const uint32_t rows_s = sbase, q_s = sbase + L_::q_off(D), p_s = sbase + L_::p_off(D);
  float2* st = reinterpret_cast<float2*>(smem + L_::st_off(D));
  float* ft = reinterpret_cast<float*>(smem + L_::ft_off(D));
  const uint32_t full0 = sbase + L_::bar_off(D), empty0 = full0 + 32u;  // pairs of blocks: stored [4], summed [4]
  const uint32_t bar_q = empty0 + 32u, bar_s = bar_q + 8u, bar_p = bar_s + 8u, bar_x = bar_p + 8u, bar_d = bar_x + 8u;
  const uint32_t gave_up = full0 + 16u * 8u + 4u;  // behind the address of tensor memory
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L_::slot_off(D));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = p.C, rank = blockIdx.x % C;
  const int G = p.H / p.Hkv, tile = blockIdx.x / C;
  const int ht = tile % p.HT, g = tile / p.HT % p.Hkv, b = tile / p.HT / p.Hkv;
  constexpr uint32_t kCols = N == 16 ? 256 : 512;  // >= 4 NO + N

  if (tid == 0) {
    for (int i = 0; i < MT; ++i) {
      mbar_init(full0 + 8u * i, kAqWorkers + (p.fault != 0 && blockIdx.x == 0 ? 1u : 0u));
      mbar_init(empty0 + 8u * i, 1);
    }
    mbar_init(bar_q, 1);
    mbar_init(bar_s, 1);
    mbar_init(bar_p, kAqWorkers);
    mbar_init(bar_x, kAqWorkers);  // queries reordered
    mbar_init(bar_d, 1);           // the end of a CTA that gave up
    tmem_slot[1] = 0u;             // gave_up
    fence_mbar_init();
  }
  if (warp == kAqWorkers) {
    tmem_alloc(smem_u32(tmem_slot), kCols);
    tmem_relinquish();
  }
  // shows the cluster that this CTA runs, so that its shared memory may be written
  if (C > 1) cluster_arrive_relaxed();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, tmem_st = tmem + (uint32_t)(MT * NO);
  pdl_wait();
  pdl_launch_dependents();

  const int wl = aq_window(p, b);
  const int nk = (p.k + p.R - 1) / p.R, nc = nk + (wl + p.R - 1) / p.R;  // chunks of slots, and all
  const int mine = nc > rank ? (nc - rank + C - 1) / C : 0;
  auto chunk = [&](int i) {
    const int c = rank + i * C;
    AqChunk a;
    a.win = c >= nk;
    a.j0 = (a.win ? c - nk : c) * p.R;
    a.n = min(p.R, (a.win ? wl : p.k) - a.j0);
    return a;
  };

  if (warp < kAqWorkers) {
    // Every address of chunk i + 1 is known while chunk i is worked on: its slots
    // are read before chunk i is widened, its rows and scales after that.
    const int sub = warp * 8 + (lane >> 2);  // this lane gathers rows sub and sub + 64 of a chunk
    int r2[2] = {-1, -1};
    const uint8_t* src[2] = {nullptr, nullptr};
    auto slots = [&](int i) {
      r2[0] = aq_chunk_slot(p, chunk(i), b, sub);
      r2[1] = aq_chunk_slot(p, chunk(i), b, sub + 64);
    };
    auto place = [&](bool w) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = aq_checked(p, w, r2[k]);
        src[k] = r < 0 ? nullptr
                 : w ? reinterpret_cast<const uint8_t*>(p.win + (((long long)b * p.W + r) * p.Hkv + g) * D) + (lane & 3) * 32
                     : aq_row<FMT>(p, b, r, g) + (lane & 3) * 16;
      }
    };
    uint4 v[8];  // batch 0 of a chunk, loaded before the softmax of the chunk before
    auto fetch = [&](uint4 (&x)[8], bool w, int batch) {
      if (w)
        aq_load<kFmtBf16, 2>(x, src, batch, DB);
      else
        aq_load<FMT, 2>(x, src, batch, DB);
    };
    // softmax: this thread's row and heads
    const int part = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    float* mx = reinterpret_cast<float*>(smem + L_::mx_off(D)) + part * 4 * 32;  // maxima of the part's warps
    float* lx = mx + 8 * 32;                                                     // and their sums
    float* bc = reinterpret_cast<float*>(smem + L_::bc_off(D)) + warp * 64;      // this warp's broadcasts
    float m_run = -INFINITY;  // head lane % NH of the part
    float l[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) l[h] = 0.0f;
    // (a skipped row's scale is read from block 0 and not used: nothing waits for the load here)
    auto row_scale = [&](int r, bool w) { return FMT == kFmtBf16 || w ? 1.0f : aq_scale<FMT>(p, b, max(r, 0), g); };
    int r = -1, r_next = -1;  // this thread's row, and its slot of the next chunk
    float scale_next = 1.0f;
    if (mine > 0) {
      const bool w0 = chunk(0).win;
      slots(0);
      r_next = aq_chunk_slot(p, chunk(0), b, row);
      place(w0);
      fetch(v, w0, 0);
      r_next = aq_checked(p, w0, r_next);
      scale_next = row_scale(r_next, w0);
    }
    for (int i = 0; i < mine; ++i) {
      const AqChunk c = chunk(i);
      r = r_next;
      const float rs = r >= 0 ? scale_next : 0.0f;
      if (i + 1 < mine) {
        slots(i + 1);
        r_next = aq_chunk_slot(p, chunk(i + 1), b, row);
      }
      // ---- widen chunk i
      uint4 w[8];
      fetch(w, c.win, 1);
      if (i == 0) {  // while the first rows are on their way
        aq_wait<(N < 64)>(bar_q, 0, p, gave_up);
        aq_swap_queries(q_s, DB * N * 128, tid, kAqWorkers * 32);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_x);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m >= MT) break;
        if (i > 0) aq_wait<(N < 64)>(empty0 + 8u * (uint32_t)m, (uint32_t)((i - 1) & 1), p, gave_up);
        if (c.win) {
          aq_store<kFmtBf16, 2>((m & 1) ? w : v, m, c.n, DB, rows_s);
          if (m < 2) aq_load<kFmtBf16, 2>((m & 1) ? w : v, src, m + 2, DB);
        } else {
          aq_store<FMT, 2>(m < 2 ? v : w, m, c.n, DB, rows_s);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full0 + 8u * (uint32_t)m);
      }
      // ---- the loads of chunk i + 1
      if (i + 1 < mine) {
        const bool w1 = chunk(i + 1).win;
        place(w1);
        fetch(v, w1, 0);
        r_next = aq_checked(p, w1, r_next);
        scale_next = row_scale(r_next, w1);
      }
      // ---- softmax of chunk i
      const float fac = r >= 0 ? rs * p.scale_log2 : 1.0f;
      aq_wait<(N < 64)>(bar_s, (uint32_t)(i & 1), p, gave_up);
      tc_fence_after();
      float z[NH];
      aq_tmem_ld<NH>(tmem_st + lane_base + (uint32_t)(part * NH), z);
      tmem_wait_ld();
      if (!__all_sync(0xffffffffu, r >= 0)) {
#pragma unroll
        for (int h = 0; h < NH; ++h) z[h] = r >= 0 ? z[h] : -INFINITY;
      }
      float cm = aq_reduce_heads<NH>(z, fac, [](float x, float y) { return fmaxf(x, y); });
      if (lane < NH) mx[(warp & 3) * 32 + lane] = cm;
      named_bar_sync(1 + part, 128);
      const int mh = lane & (NH - 1);
      cm = fmaxf(fmaxf(mx[mh], mx[32 + mh]), fmaxf(mx[64 + mh], mx[96 + mh]));
      // the same data and so the same decision in the part's four warps
      if (__any_sync(0xffffffffu, i == 0 || cm > m_run + 8.0f)) {
        const float m_new = fmaxf(m_run, cm);
        if (i > 0) {
          const float f = m_new == -INFINITY ? 1.0f : exp2f(m_run - m_new);
          __syncwarp();
          if (lane < NH) bc[32 + lane] = f;
          __syncwarp();
#pragma unroll
          for (int h = 0; h < NH; ++h) l[h] *= bc[32 + h];
          for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int j = 0; j < NH * kTerms; j += 8) {
              const int h = j % NH;  // (the first terms of this thread's heads, then the second)
              uint32_t o[8];
              const uint32_t at = tmem + lane_base + (uint32_t)(m * NO + j / NH * N + part * NH + h);
              tmem_ld8(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * bc[32 + h + e]);
              tmem_st8(at, o);
            }
          }
          tmem_wait_st();
        }
        m_run = m_new;
        __syncwarp();
        if (lane < NH) bc[lane] = m_new == -INFINITY ? 0.0f : m_new;
        __syncwarp();
      }
      const uint32_t prow = p_s + (uint32_t)row * 128u, sw7 = (uint32_t)(row & 7);
#pragma unroll
      for (int h = 0; h < NH; h += 8) {
        uint32_t u[4], u2[4];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 mu = *reinterpret_cast<const float4*>(bc + h + e);
          const float e0 = aq_ex2(fmaf(z[h + e], fac, -mu.x)), e1 = aq_ex2(fmaf(z[h + e + 1], fac, -mu.y));
          const float e2 = aq_ex2(fmaf(z[h + e + 2], fac, -mu.z)), e3 = aq_ex2(fmaf(z[h + e + 3], fac, -mu.w));
          l[h + e] += e0, l[h + e + 1] += e1, l[h + e + 2] += e2, l[h + e + 3] += e3;
          // the weighted sum's operand: the weight times the row's scale
          u[e / 2] = aq_pack(e0 * rs, e1 * rs);
          u[e / 2 + 1] = aq_pack(e2 * rs, e3 * rs);
          if constexpr (kTerms == 2 || FEW) {
            u2[e / 2] = aq_rest(e0 * rs, e1 * rs, u[e / 2]);
            u2[e / 2 + 1] = aq_rest(e2 * rs, e3 * rs, u[e / 2 + 1]);
          }
        }
        const uint32_t at = prow + (((uint32_t)((part * NH + h) >> 3) ^ sw7) << 4);
        if constexpr (kTerms == 2) {
          sts128(at, make_uint4(u[0], u[1], u[2], u[3]));
          sts128(prow + (((uint32_t)((N + part * NH + h) >> 3) ^ sw7) << 4), make_uint4(u2[0], u2[1], u2[2], u2[3]));
        } else if (!FEW || row < 64) {
          sts128(at, make_uint4(u[0], u[1], u[2], u[3]));
          if constexpr (FEW) sts128(at + 64u * 128u, make_uint4(u2[0], u2[1], u2[2], u2[3]));
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p);
    }
    // the heads' normalisers over this CTA's rows, to every CTA of the cluster
    if (C > 1) cluster_wait();
    const float ls = aq_reduce_heads<NH>(l, 1.0f, [](float x, float y) { return x + y; });
    if (lane < NH) lx[(warp & 3) * 32 + lane] = ls;
    named_bar_sync(1 + part, 128);
    if ((warp & 3) == 0 && lane < NH) {
      const float total = (lx[lane] + lx[32 + lane]) + (lx[64 + lane] + lx[96 + lane]);
      const uint32_t at = smem_u32(st + rank * N + part * NH + lane);
      if (C == 1)
        st[part * NH + lane] = make_float2(m_run, total);
      else
        for (int c = 0; c < C; ++c) dsmem_st_f32x2(dsmem_map(at, (uint32_t)c), m_run, total);
    }
    __syncwarp();
    if (mine > 0) {
      aq_wait<(N < 64)>(empty0 + 8u * (uint32_t)(MT - 1), (uint32_t)((mine - 1) & 1), p, gave_up);
      tc_fence_after();
    }
  } else {
    // ---------------- queries and MMAs: the warp runs as a whole, one elected lane
    // issues, and the steps are unrolled, so that an MMA's operands are a few
    // uniform additions (one lane on its own issues an MMA in about 120 cycles, the
    // tensor cores take one in 52)
    if (elect_lane()) {
      mbar_arrive_expect_tx(bar_q, (uint32_t)(DB * N * 128));
      tma_load_3d(q_s, &tm_q, 0, b * p.H + g * G + ht * N, 0, bar_q);
    }
    aq_wait<true>(mine > 0 ? bar_x : bar_q, 0, p, gave_up);  // (no copy may be in flight at the end)
    constexpr uint32_t id1 = idesc_bf16_f32(kAqRows, N);
    constexpr uint32_t id2 = idesc_bf16_f32(128, NO) | (1u << 15) | (1u << 16);
    const uint64_t ka = sw128_kmajor_desc(rows_s), kb = sw128_kmajor_desc(q_s);
    const uint64_t ma = sw128_mnmajor_desc(rows_s, kAqBlock, 1024u), mb = sw128_mnmajor_desc(p_s, kAqBlock, 1024u);
    for (int i = 0; i < mine; ++i) {
      const int steps = (chunk(i).n + 15) >> 4;
      for (int m = 0; m < MT; ++m) {
        aq_wait<true>(full0 + 8u * (uint32_t)m, (uint32_t)(i & 1), p, gave_up);
        tc_fence_after();
        if (elect_lane()) {
          const uint64_t a0 = desc_at(ka, (uint32_t)m * 2 * kAqBlock), b0 = desc_at(kb, (uint32_t)m * 2 * N * 128);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (kk < 4 || 2 * m + 1 < DB)
              mma_bf16_ss(tmem_st, desc_at(a0, (uint32_t)((kk >> 2) * kAqBlock + (kk & 3) * 32)),
                          desc_at(b0, (uint32_t)((kk >> 2) * N * 128 + (kk & 3) * 32)), id1, (m | kk) != 0 ? 1u : 0u);
          if (m == MT - 1) mma_commit(bar_s);
        }
        __syncwarp();
      }
      aq_wait<true>(bar_p, (uint32_t)(i & 1), p, gave_up);
      tc_fence_after();
      if (elect_lane()) {
        for (int m = 0; m < MT; ++m) {
          const uint64_t a0 = desc_at(ma, (uint32_t)m * 2 * kAqBlock);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (kk < steps)
              mma_bf16_ss(tmem + (uint32_t)(m * NO), desc_at(a0, (uint32_t)(kk * 2048)), desc_at(mb, (uint32_t)(kk * 2048)), id2,
                          (i | kk) != 0 ? 1u : 0u);
          if constexpr (FEW) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (kk < steps)
                mma_bf16_ss(tmem + (uint32_t)(m * NO), desc_at(a0, (uint32_t)(kk * 2048)),
                            desc_at(mb, (uint32_t)((kk + 4) * 2048)), id2, 1u);
          }
          mma_commit(empty0 + 8u * (uint32_t)m);
        }
      }
      __syncwarp();
    }
  }
  __syncwarp();

  // ---- the cluster's results.  The workers have waited for the last MMA:
  // past the barrier the rows' memory is free in every CTA, and the statistics
  // have arrived.
  if (C > 1 && warp == kAqWorkers) cluster_wait();
  tc_fence_before();
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const int q4 = warp & 3;
  uint16_t* out = p.out + ((size_t)b * p.H + (size_t)g * G) * D;
  const int U = (D >> 5) * (N / 4), per = (U + C - 1) / C;  // pieces of 32 channels x 4 heads; per owner
  // 16 heads of 32 channels of this CTA's O^T
  auto sums = [&](int m, int c16, float (&v)[16]) {
    const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16) + (uint32_t)(m * NO + c16 * 16);
    aq_tmem_ld<16>(at, v);
    if constexpr (kTerms == 2) {
      float w[16];
      aq_tmem_ld<16>(at + (uint32_t)N, w);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] += w[e];
    } else {
      tmem_wait_ld();
    }
  };
  const uint32_t inv_C = (65536u + (uint32_t)C - 1u) / (uint32_t)C;  // u / C = u * inv_C >> 16 for u <= 256
  if (warp == kAqWorkers) {
    for (int h = lane; h < N; h += 32) {
      const int hh = ht * N + h;
      const float sink = p.sink && hh < G ? p.sink[g * G + hh] * 1.4426950408889634f : -INFINITY;
      float M = sink, L = 0.0f;
      for (int c = 0; c < C; ++c)
        if (st[c * N + h].y != 0.0f) M = fmaxf(M, st[c * N + h].x);
      if (sink != -INFINITY) L = exp2f(sink - M);
      for (int c = 0; c < C; ++c) {
        const float2 s = st[c * N + h];
        const float f = s.y != 0.0f ? exp2f(s.x - M) : 0.0f;
        if (s.y != 0.0f) L = fmaf(s.y, f, L);
        ft[c * N + h] = f;
      }
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;  // a NaN stays one
      for (int c = 0; c < C; ++c) ft[c * N + h] *= inv;
      if (rank == 0 && p.lse && hh < G)
        p.lse[(size_t)b * p.H + g * G + hh] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
  } else if (C > 1) {
    // (each CTA begins elsewhere, so that they do not all send to one owner at once)
    const int items = MT * (N / 16), turned = items * rank / C;
    for (int j = warp >> 2; j < items; j += kAqWorkers / 4) {
      const int it = j + turned < items ? j + turned : j + turned - items;
      const int m = it / (N / 16), c16 = it % (N / 16);
      if (m * 128 + q4 * 32 >= D) continue;
      float v[16];
      if (mine > 0) {
        sums(m, c16, v);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.0f;
      }
      const int u = (m * 4 + q4) * (N / 4) + c16 * 4;
      int slot = (int)((uint32_t)u * inv_C >> 16), owner = u - slot * C;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t at = rows_s + (uint32_t)((rank * per + slot) * 512 + lane * 16);
        if (owner == rank)
          sts128(at, make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]), __float_as_uint(v[4 * e + 2]),
                                __float_as_uint(v[4 * e + 3])));
        else
          dsmem_st_f32x4(dsmem_map(at, (uint32_t)owner), v + 4 * e);
        if (++owner == C) owner = 0, ++slot;
      }
    }
  }
  __syncwarp();
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
  auto emit = [&](int u, const float* v) {
    // lane i of a piece holds the channel stored in place i of its 32
    const int hg = u % (N / 4), d = u / (N / 4) * 32 + (lane & 28) + ((lane & 1) << 1) + ((lane >> 1) & 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int hh = ht * N + hg * 4 + e;
      if (hh < G) out[(size_t)hh * D + d] = (uint16_t)aq_pack(v[e], 0.0f);
    }
  };
  if (C > 1 && warp < kAqWorkers) {
    for (int s = warp; s < per; s += kAqWorkers) {
      const int u = s * C + rank;
      if (u >= U) break;
      const int h = u % (N / 4) * 4;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
      for (int c = 0; c < C; ++c) {
        const float4 f = *reinterpret_cast<const float4*>(ft + c * N + h);
        const uint4 x = lds128(rows_s + (uint32_t)((c * per + s) * 512 + lane * 16));
        v[0] = fmaf(__uint_as_float(x.x), f.x, v[0]);
        v[1] = fmaf(__uint_as_float(x.y), f.y, v[1]);
        v[2] = fmaf(__uint_as_float(x.z), f.z, v[2]);
        v[3] = fmaf(__uint_as_float(x.w), f.w, v[3]);
      }
      emit(u, v);
    }
  } else if (warp < kAqWorkers) {
    for (int it = warp >> 2; it < MT * (N / 16); it += kAqWorkers / 4) {
      const int m = it / (N / 16), c16 = it % (N / 16);
      if (m * 128 + q4 * 32 >= D) continue;
      float v[16];
      if (mine > 0) {
        sums(m, c16, v);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 f = *reinterpret_cast<const float4*>(ft + c16 * 16 + 4 * e);
        v[4 * e] *= f.x, v[4 * e + 1] *= f.y, v[4 * e + 2] *= f.z, v[4 * e + 3] *= f.w;
        emit((m * 4 + q4) * (N / 4) + c16 * 4 + e, v + 4 * e);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kAqWorkers) {
    if (lds32(gave_up) != 0u) aq_drain(bar_d, bar_q, 0, p);
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// ------------------------------------------------------------------ the account
//
// A cluster owns a batch row and a chunk of up to 128 slots, its CTAs each a tile
// of up to 64 query heads of one KV head (and every C-th tile after that).  The
// scores are recomputed as above, S^T [rows, heads] = rows . Q^T: the account
// needs the weights in float32, which the attention rounds, and reading 2 bytes
// of a score for every head and row would cost more than the row's own bytes.
// With a row to a thread the sum over heads never leaves the thread: four
// threads share a row, their sums and then the CTAs' are added in a fixed order,
// and each slot's total is added to its account once.  8 batch rows of 128 heads of 512
// channels over 1024 rows take 7.4 us, a floor of 0.8: the chain slots, rows, scores.
// 512 of them over 2048 rows of one cache take 836 us, a floor of 83: a CTA takes one
// chunk, and nothing of the next is on its way meanwhile.
constexpr int kAmWorkers = 16;
constexpr int kAmThreads = (kAmWorkers + 1) * 32;
constexpr int kAmMaxCluster = 8;

template <int N>
struct AmSmem {
  __host__ __device__ static constexpr int q_off(int D) { return D / 64 * kAqBlock; }
  __host__ __device__ static constexpr int lse_off(int D) { return q_off(D) + D / 64 * N * 128; }  // float [N]
  __host__ __device__ static constexpr int part_off(int D) { return lse_off(D) + N * 4; }          // float [4][128]
  __host__ __device__ static constexpr int sum_off(int D) { return part_off(D) + 2048; }           // float [8][128]
  __host__ __device__ static constexpr int bar_off(int D) { return sum_off(D) + kAmMaxCluster * 512; }
  __host__ __device__ static constexpr int slot_off(int D) { return bar_off(D) + 8 * 8; }
  __host__ __device__ static constexpr int bytes(int D) { return slot_off(D) + 16 + 1024; }  // + alignment slack
};

template <int FMT, int N>
__global__ void __launch_bounds__(kAmThreads, 1)
    attn_mass_kernel(const __grid_constant__ CUtensorMap tm_q, const AqParams p) {
  using L_ = AmSmem<N>;
  constexpr int NH = N / 4;  // heads of an epilogue thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int D = p.D, DB = D >> 6, MT = (D + 127) >> 7;
  const uint32_t rows_s = sbase, q_s = sbase + L_::q_off(D);
  float* lse_s = reinterpret_cast<float*>(smem + L_::lse_off(D));
  float* part_s = reinterpret_cast<float*>(smem + L_::part_off(D));
  float* sum_s = reinterpret_cast<float*>(smem + L_::sum_off(D));
  const uint32_t full0 = sbase + L_::bar_off(D), bar_q = full0 + 32u, bar_s = bar_q + 8u, bar_x = bar_s + 8u, bar_d = bar_x + 8u;
  const uint32_t gave_up = full0 + 8u * 8u + 4u;  // behind the address of tensor memory
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L_::slot_off(D));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = p.C, rank = blockIdx.x % C;
  const int G = p.H / p.Hkv, tiles = p.Hkv * p.HT;
  const int nk = (p.k + p.R - 1) / p.R, b = (int)blockIdx.x / C / nk;
  const int j0 = (int)blockIdx.x / C % nk * p.R;
  const AqChunk chunk = {j0, min(p.R, p.k - j0), false};
  constexpr uint32_t kCols = N < 32 ? 32 : N;

  if (tid == 0) {
    for (int i = 0; i < MT; ++i) mbar_init(full0 + 8u * i, kAmWorkers + (p.fault != 0 && blockIdx.x == 0 ? 1u : 0u));
    mbar_init(bar_q, 1);
    mbar_init(bar_s, 1);
    mbar_init(bar_x, kAmWorkers);  // queries reordered
    mbar_init(bar_d, 1);           // the end of a CTA that gave up
    tmem_slot[1] = 0u;             // gave_up
    fence_mbar_init();
  }
  if (warp == kAmWorkers) {
    tmem_alloc(smem_u32(tmem_slot), kCols);
    tmem_relinquish();
  }
  if (C > 1) cluster_arrive_relaxed();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  const int sub = warp * 8 + (lane >> 2);                     // workers: the row this lane gathers,
  const int row = (warp & 3) * 32 + lane, part = warp >> 2;   // and the row and quarter of the heads it sums
  int r_load = warp < kAmWorkers ? aq_chunk_slot(p, chunk, b, sub) : -1;
  int r = warp < kAmWorkers ? aq_chunk_slot(p, chunk, b, row) : -1;
  r_load = aq_checked(p, false, r_load);
  r = aq_checked(p, false, r);
  float total = 0.0f;
  int turn = 0, loads = 0;  // tiles, and the copies of queries that were issued for them
  for (int t = rank, g_held = -1; t < tiles; t += C, ++turn) {
    const int g = t / p.HT, ht = t % p.HT, heads = min(N, G - ht * N);
    if (warp < kAmWorkers) {
      float fac = r >= 0 ? p.scale_log2 : 0.0f;  // (the scale's load is on its way while the rows are)
      if (FMT != kFmtBf16 && r >= 0) fac *= aq_scale<FMT>(p, b, r, g);
      auto swap_queries = [&]() {
        aq_wait<false>(bar_q, (uint32_t)(turn & 1), p, gave_up);
        aq_swap_queries(q_s, DB * N * 128, tid, kAmWorkers * 32);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_x);
      };
      if (g != g_held) {
        const uint8_t* src[1] = {r_load < 0 ? nullptr : aq_row<FMT>(p, b, r_load, g) + (lane & 3) * (FMT == kFmtBf16 ? 32 : 16)};
        uint4 v[4], w[4];
        aq_load<FMT, 1>(v, src, 0, DB);
        aq_load<FMT, 1>(w, src, 1, DB);
        swap_queries();
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= MT) break;
          if constexpr (FMT == kFmtBf16) {
            aq_store<FMT, 1>((m & 1) ? w : v, m, chunk.n, DB, rows_s);
            if (m < 2) aq_load<FMT, 1>((m & 1) ? w : v, src, m + 2, DB);
          } else {
            aq_store<FMT, 1>(m < 2 ? v : w, m, chunk.n, DB, rows_s);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full0 + 8u * (uint32_t)m);
        }
      } else {
        swap_queries();
        if (lane == 0)
          for (int m = 0; m < MT; ++m) mbar_arrive(full0 + 8u * (uint32_t)m);  // the rows are still there
      }
      // log2 units; infinite where a head adds nothing
      if (tid < N) {
        const float l = tid < heads ? p.lse[(size_t)b * p.H + g * G + ht * N + tid] : INFINITY;
        lse_s[tid] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
      }
      named_bar_sync(1, kAmWorkers * 32);
      aq_wait<false>(bar_s, (uint32_t)(turn & 1), p, gave_up);
      tc_fence_after();
      float z[NH];
      aq_tmem_ld<NH>(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(part * NH), z);
      tmem_wait_ld();
      float sum = 0.0f;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float ls = lse_s[part * NH + h];
        const float e = aq_ex2(fmaf(z[h], fac, -ls));
        sum += ls == INFINITY ? 0.0f : e;
      }
      total += sum;
      tc_fence_before();
      named_bar_sync(1, kAmWorkers * 32);  // lse_s and the scores have been read
    } else {
      // (the scores of the tile before have been read: the workers' barrier above precedes
      // their arrivals.  After a wait that ran out the copy before may not have landed, and
      // bar_q would get a second arrival in its phase)
      if (turn == 0 || __all_sync(0xffffffffu, lds32(gave_up) == 0u)) {
        if (elect_lane()) {
          mbar_arrive_expect_tx(bar_q, (uint32_t)(DB * N * 128));
          tma_load_3d(q_s, &tm_q, 0, b * p.H + g * G + ht * N, 0, bar_q);
        }
        ++loads;
      }
      aq_wait<false>(bar_x, (uint32_t)(turn & 1), p, gave_up);
      constexpr uint32_t id = idesc_bf16_f32(kAqRows, N);
      const uint64_t ka = sw128_kmajor_desc(rows_s), kb = sw128_kmajor_desc(q_s);
      for (int m = 0; m < MT; ++m) {
        aq_wait<false>(full0 + 8u * (uint32_t)m, (uint32_t)(turn & 1), p, gave_up);
        tc_fence_after();
        if (elect_lane()) {
          const uint64_t a0 = desc_at(ka, (uint32_t)m * 2 * kAqBlock), b0 = desc_at(kb, (uint32_t)m * 2 * N * 128);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (kk < 4 || 2 * m + 1 < DB)
              mma_bf16_ss(tmem, desc_at(a0, (uint32_t)((kk >> 2) * kAqBlock + (kk & 3) * 32)),
                          desc_at(b0, (uint32_t)((kk >> 2) * N * 128 + (kk & 3) * 32)), id, (m | kk) != 0 ? 1u : 0u);
          if (m == MT - 1) mma_commit(bar_s);
        }
        __syncwarp();
      }
      aq_wait<false>(bar_s, (uint32_t)(turn & 1), p, gave_up);  // the queries' memory is free
    }
    g_held = g;
  }

  // ---- the row's four sums, then the CTAs', in order
  if (warp < kAmWorkers) {
    part_s[part * kAqRows + row] = total;
    named_bar_sync(1, kAmWorkers * 32);
  }
  __syncwarp();
  if (C > 1) cluster_wait();
  if (tid < kAqRows) {
    float s = (part_s[tid] + part_s[kAqRows + tid]) + (part_s[2 * kAqRows + tid] + part_s[3 * kAqRows + tid]);
    if (lds32(gave_up) != 0u) s = 0.0f;  // not counted, rather than counted wrong
    if (C == 1)
      sum_s[tid] = s;
    else
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dsmem_map(smem_u32(sum_s + rank * kAqRows + tid), 0u)), "f"(s) : "memory");
  }
  __syncwarp();
  if (C > 1)
    cluster_sync();
  if (rank == 0 && tid < kAqRows && r >= 0) {
    float s = sum_s[tid];
    for (int i = 1; i < C; ++i) s += sum_s[i * kAqRows + tid];
    atomicAdd(p.mass + b * p.mass_bstride + r, s);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kAmWorkers) {
    if (lds32(gave_up) != 0u) aq_drain(bar_d, bar_q, (uint32_t)((loads - 1) & 1), p);
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

}  // namespace dstopk
