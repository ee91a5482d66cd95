// cache_ops.cuh -- the C ABI of the 8-bit cache: argument checks, launch-shape
// choice and launches of ds_cache_quantize, ds_sparse_attention_q8,
// ds_attention_mass, ds_cache_evict and ds_cache_compact.  Included by lib.cu
// after its helpers (device_state, set_pdl, wait_limit).  None of these
// allocates or keeps anything: calls on different streams may overlap.
#pragma once

namespace dstopk {

static bool cache_misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// log2 of a block size (1, 2, 4 .. DS_CACHE_MAX_BLOCK), or -1.
static int cache_log_block(int block) {
  for (int l = 0; (1 << l) <= DS_CACHE_MAX_BLOCK; ++l)
    if (block == 1 << l) return l;
  return -1;
}

static bool cache_is8(int dtype) { return dtype == DS_E4M3 || dtype == DS_I8; }

// One launch, chained to the kernel before it by programmatic dependent launch.
template <class P>
static int cache_launch(void (*kern)(P), const P& p, dim3 grid, int threads, size_t smem, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  set_pdl(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = pdl_on() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

// Queries [rows][D] bf16 in boxes of (64 channels, n heads, D/64 blocks), 128-byte swizzle.
static bool cache_encode_q(const void* q, long long rows, int D, int n, CUtensorMap* tq) {
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(D / 64)};
  cuuint64_t str[2] = {(cuuint64_t)D * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)n, (cuuint32_t)(D / 64)};
  cuuint32_t one[3] = {1, 1, 1};
  return g_encode(tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, str, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The attention's kernel for n = 16, 32 or 64 heads to a CTA; few: for calls of at most 64 rows.
typedef void (*AqKernel)(const CUtensorMap, const AqParams);
template <int FMT>
static AqKernel aq_kernel_of(int n, bool few) {
  if (n == 64) return few ? attn_q8_kernel<FMT, 64, true> : attn_q8_kernel<FMT, 64, false>;
  return n == 16 ? attn_q8_kernel<FMT, 16, false> : attn_q8_kernel<FMT, 32, false>;
}
static AqKernel aq_kernel(int dtype, int n, bool few) {
  return dtype == DS_E4M3 ? aq_kernel_of<kFmtE4m3>(n, few) : aq_kernel_of<kFmtI8>(n, few);
}
// Shared memory that a CTA of the attention or the account asks for at least.  Its
// cluster waits for all its CTAs, and a CTA waits for its tensor memory: two clusters
// that met on two SMs, each with the tensor memory that the other waits for, would
// wait for good.  With this much, no two CTAs of kernels that have both (these two,
// and the two below) fit one SM.  (Registers part them too, as compiled today.)
constexpr int kCacheAlone = 176 * 1024;
constexpr int kSmSmem = 228 * 1024, kCtaSmem = 1024;  // of an SM, and what a CTA takes besides its own
static_assert(2 * (kCacheAlone + kCtaSmem) > kSmSmem, "two CTAs of the 8-bit cache on an SM");
static_assert(kCacheAlone + PvSmem<1, 2>::bytes(1) + 2 * kCtaSmem > kSmSmem, "one beside the 16-bit attention's");
static_assert(kCacheAlone + QtSmem::kBytes + 2 * kCtaSmem > kSmSmem, "one beside the query projection's");
static int aq_smem(int n, int D) {
  return std::max(kCacheAlone, n == 16 ? AqSmem<16>::bytes(D) : n == 32 ? AqSmem<32>::bytes(D) : AqSmem<64>::bytes(D));
}

// The account's.
static AqKernel am_kernel(int dtype, int n) {
  if (dtype == DS_BF16)
    return n == 16 ? attn_mass_kernel<kFmtBf16, 16> : n == 32 ? attn_mass_kernel<kFmtBf16, 32> : attn_mass_kernel<kFmtBf16, 64>;
  if (dtype == DS_E4M3)
    return n == 16 ? attn_mass_kernel<kFmtE4m3, 16> : n == 32 ? attn_mass_kernel<kFmtE4m3, 32> : attn_mass_kernel<kFmtE4m3, 64>;
  return n == 16 ? attn_mass_kernel<kFmtI8, 16> : n == 32 ? attn_mass_kernel<kFmtI8, 32> : attn_mass_kernel<kFmtI8, 64>;
}
static int am_smem(int n, int D) {
  return std::max(kCacheAlone, n == 16 ? AmSmem<16>::bytes(D) : n == 32 ? AmSmem<32>::bytes(D) : AmSmem<64>::bytes(D));
}

static void cache_cluster(cudaLaunchAttribute& a, int C) {
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = (unsigned)C;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
}

static void aq_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int n, int D, unsigned ctas, int C) {
  cfg->gridDim = dim3(ctas, 1, 1);
  cfg->blockDim = dim3(kAqThreads, 1, 1);
  cfg->dynamicSmemBytes = (size_t)aq_smem(n, D);
  cache_cluster(attr[0], C);
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

// Once per device, from device_state: shared-memory limits, and how many
// clusters of each size of the attention run at once (0: none).
static cudaError_t cache_setup(DeviceState* s) {
  for (int dtype : {DS_E4M3, DS_I8})
    for (int n : {16, 32, 64})
      for (bool few : {false, true}) {
        const AqKernel kern = aq_kernel(dtype, n, few);
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, aq_smem(n, DS_ATTN_MAX_DIM));
        if (e != cudaSuccess) return e;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
          cudaGetLastError();
      }
  for (int dtype : {DS_BF16, DS_E4M3, DS_I8})
    for (int n : {16, 32, 64}) {
      const cudaError_t e = cudaFuncSetAttribute(am_kernel(dtype, n), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 am_smem(n, DS_ATTN_MAX_DIM));
      if (e != cudaSuccess) return e;
    }
  cudaError_t e = cudaFuncSetAttribute(cache_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCeKeys * 4);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(cache_compact_bulk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCcSmem);
  if (e != cudaSuccess) return e;
  for (int c = 1; c <= kAqMaxCluster; ++c) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    aq_config(&cfg, attr, 64, DS_ATTN_MAX_DIM, (unsigned)c, c);
    if (cudaOccupancyMaxActiveClusters(&s->aq_clusters[c], aq_kernel(DS_E4M3, 64, false), &cfg) != cudaSuccess) {
      cudaGetLastError();
      s->aq_clusters[c] = 0;
    }
  }
  return cudaSuccess;
}

// The arguments that the attention and the account share.
static int cache_attn_check(const void* q, const void* cache, int64_t cache_batch_stride, const float* scales,
                            int64_t scales_batch_stride, int dtype, int block, int T, const int32_t* idx, int k,
                            int batch, int heads, int kv_heads, int d, float scale) {
  if (!q || !cache || batch < 1 || batch > 65535 || T < 1 || k < 0 || k > DS_MAX_K || (k > 0 && !idx)) return DS_ERR_ARG;
  if (heads < 1 || heads > DS_ATTN_MAX_HEADS || kv_heads < 1 || heads % kv_heads != 0) return DS_ERR_ARG;
  if (d < 64 || d > DS_ATTN_MAX_DIM || d % 64 != 0 || !std::isfinite(scale)) return DS_ERR_ARG;
  if (cache_batch_stride < 0 || cache_misaligned(q, 16) || cache_misaligned(cache, 16) || cache_misaligned(idx, 4))
    return DS_ERR_ARG;
  if (cache_is8(dtype)) {
    if (!scales || cache_misaligned(scales, 4) || scales_batch_stride < 0 || cache_log_block(block) < 0) return DS_ERR_ARG;
  } else if (dtype != DS_BF16 || scales) {
    return DS_ERR_ARG;
  }
  return DS_OK;
}

}  // namespace dstopk

namespace dstopk {

// The bytes that an array has in each batch row: [at + b * step, at + b * step + bytes),
// step >= bytes where there is more than one.
struct CacheSpan {
  uintptr_t at;
  int64_t step, bytes;
};

// Does one array have a byte of the other?  Batch row by batch row, since one may lie
// in the other's gaps (two halves of one buffer [batch, 2, ...]).
static bool cache_overlap(const CacheSpan& x, const CacheSpan& y, int batch) {
  const auto end = [&](const CacheSpan& s) { return s.at + (uintptr_t)((batch - 1) * s.step + s.bytes); };
  if (end(x) <= y.at || end(y) <= x.at) return false;
  for (int i = 0, j = 0; i < batch && j < batch;) {
    const uintptr_t a = x.at + (uintptr_t)(i * x.step), b = y.at + (uintptr_t)(j * y.step);
    if (a + (uintptr_t)x.bytes <= b)
      ++i;
    else if (b + (uintptr_t)y.bytes <= a)
      ++j;
    else
      return true;
  }
  return false;
}

}  // namespace dstopk

extern "C" int ds_cache_quantize(const void* rows, int64_t rows_batch_stride, int64_t row_stride, int batch, int n,
                                 int kv_heads, int d, int dtype, int block, const int32_t* pos, const int32_t* len,
                                 void* codes, int64_t codes_batch_stride, float* scales, int64_t scales_batch_stride,
                                 int T, void* stream) {
  const int lb = cache_log_block(block);
  if (!rows || !codes || !scales || batch < 1 || batch > 65535 || n < 1 || T < 1 || lb < 0 || !cache_is8(dtype))
    return DS_ERR_ARG;
  if (kv_heads < 1 || kv_heads > DS_ATTN_MAX_HEADS || d < 64 || d > DS_ATTN_MAX_DIM || d % 64 != 0) return DS_ERR_ARG;
  const int64_t width = (int64_t)kv_heads * d;
  if (row_stride < width || row_stride % 8 != 0 || rows_batch_stride < 0 || rows_batch_stride % 8 != 0) return DS_ERR_ARG;
  const int64_t nb = ((int64_t)T + block - 1) / block;
  if (batch > 1 && (codes_batch_stride < T || scales_batch_stride < nb)) return DS_ERR_ARG;
  if (cache_misaligned(rows, 16) || cache_misaligned(codes, 16) || cache_misaligned(scales, 4) ||
      cache_misaligned(pos, 4) || cache_misaligned(len, 4))
    return DS_ERR_ARG;
  CqParams p = {};
  p.nblocks = (int)(((int64_t)n + block - 1) / block);
  const int64_t units = (int64_t)p.nblocks * kv_heads * batch;
  if (units > INT32_MAX) return DS_ERR_ARG;
  DeviceState* s = nullptr;
  const int rc = device_state(&s);
  if (rc != DS_OK) return rc;
  p.rows = static_cast<const uint16_t*>(rows);
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = scales;
  p.pos = pos;
  p.len = len;
  p.status = s->status;
  p.rows_bstride = rows_batch_stride;
  p.rows_rstride = row_stride;
  p.codes_bstride = codes_batch_stride * width;
  p.scales_bstride = scales_batch_stride * kv_heads;
  p.n = n;
  p.Hkv = kv_heads;
  p.D = d;
  p.T = T;
  p.log_block = lb;
  p.B = batch;
  const int pieces = (block * d) / 8;  // of 16 bytes, in a block of one KV head
  int nt = 32;
  while (nt * kCqPieces < pieces) nt *= 2;
  const int groups = nt < 256 ? 256 / nt : 1;
  const dim3 grid((unsigned)((units + groups - 1) / groups));
#define DS_CQ(NT)                                                                                                    \
  case NT:                                                                                                           \
    return cache_launch(dtype == DS_E4M3 ? cache_quantize_kernel<kFmtE4m3, NT> : cache_quantize_kernel<kFmtI8, NT>, p, \
                        grid, NT < 256 ? 256 : NT, 0, stream);
  switch (nt) {
    DS_CQ(32)
    DS_CQ(64)
    DS_CQ(128)
    DS_CQ(256)
    DS_CQ(512)
    DS_CQ(1024)
  }
#undef DS_CQ
  return DS_ERR_ARG;
}

extern "C" int ds_sparse_attention_q8(const void* q, const void* codes, int64_t codes_batch_stride, const float* scales,
                                      int64_t scales_batch_stride, int dtype, int block, int T, const int32_t* idx,
                                      int k, const void* win, int W, const int32_t* win_len, const float* sink,
                                      int batch, int heads, int kv_heads, int d, float scale, void* out, float* lse,
                                      void* stream) {
  int rc = cache_attn_check(q, codes, codes_batch_stride, scales, scales_batch_stride, dtype, block, T, idx, k, batch,
                            heads, kv_heads, d, scale);
  if (rc != DS_OK) return rc;
  if (!cache_is8(dtype) || !out || W < 0 || W > DS_ATTN_MAX_WINDOW || (W > 0 && !win)) return DS_ERR_ARG;
  if (cache_misaligned(out, 16) || cache_misaligned(win, 16) || cache_misaligned(win_len, 4) ||
      cache_misaligned(sink, 4) || cache_misaligned(lse, 4))
    return DS_ERR_ARG;
  DeviceState* s = nullptr;
  rc = device_state(&s);
  if (rc != DS_OK) return rc;
  AqParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.cache = static_cast<const uint8_t*>(codes);
  p.scales = scales;
  p.win = static_cast<const uint16_t*>(win);
  p.idx = idx;
  p.win_len = win_len;
  p.sink = sink;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.status = s->status;
  p.wait_ns = wait_limit();
  p.fault = take_planted_fault();
  p.cache_bstride = codes_batch_stride * kv_heads * d;
  p.scales_bstride = scales_batch_stride * kv_heads;
  p.T = T;
  p.k = k;
  p.W = W;
  p.B = batch;
  p.H = heads;
  p.Hkv = kv_heads;
  p.D = d;
  p.log_block = cache_log_block(block);
  p.scale_log2 = scale * 1.4426950408889634f;
  // Heads of a CTA, CTAs of a tile (while all tiles' clusters run at once) and rows
  // of a chunk.  Measured at 512 channels, a CTA's turn of a chunk takes 3.2, 3.5 and
  // 4.4 us with 16, 32 and 64 heads (the MMAs cost the same up to 64), the parts of a
  // call beside its turns 5.5, 5.5 and 8.5 us, and 7.1, 8.1 and 12.9 where a cluster
  // exchanges partial results; what has the least of both, over all waves of CTAs, is
  // taken.  128 heads over 1024 + 128 rows: one batch row 16 heads, 9 CTAs 9.7 us,
  // eight 32, 3 18.9 us, sixty-four 64, 1 63 us.  The figures are those of 512 channels
  // before e4m3 codes were checked for NaN (2 to 5% more), but what they choose is right
  // elsewhere too: of all heads and CTAs, each forced, on 40 shapes (64, 128, 192, 256 and
  // 512 channels; 1 to 300 batch rows; 8 to 128 heads to a KV head) none was more than 1%
  // faster, but for 16 batch rows of 128 heads, where 64, 3 takes 7 to 9% less than
  // the 32, 2 chosen at 64 to 256 channels, and 2% less at 512.
  const int G = heads / kv_heads;
  auto turns = [&](int r, int c) { return ((k + r - 1) / r + (W + r - 1) / r + c - 1) / c; };
  int n = 0;
  double best = 0.0;
  int64_t tiles = 0;
  static const struct {
    int n;
    double turn, alone, cluster;
  } kCost[] = {{16, 3.2, 5.5, 7.1}, {32, 3.5, 5.5, 8.1}, {64, 4.4, 8.5, 12.9}};
  for (const auto& w : kCost) {
    const int64_t t = (int64_t)batch * kv_heads * ((G + w.n - 1) / w.n);
    for (int c = 1; c <= kAqMaxCluster; ++c) {
      if (c > 1 && (t > s->aq_clusters[c] || turns(kAqRows, c) == turns(kAqRows, c - 1))) continue;
      const double waves = (double)((t * c + s->num_sms - 1) / s->num_sms);
      const double us = waves * turns(kAqRows, c) * w.turn + (c > 1 ? w.cluster : w.alone);
      if (n == 0 || us < best) n = w.n, best = us, tiles = t, p.C = c;
    }
    if (w.n >= G) break;
  }
  p.HT = (G + n - 1) / n;
  const int C = p.C;
  if (tiles * C > INT32_MAX) return DS_ERR_ARG;
  // the fewest rows that keep the number of turns
  for (p.R = kAqRows; p.R > 16 && turns(p.R - 16, C) == turns(kAqRows, C);) p.R -= 16;
  const bool few = k + W <= 64;  // (then R <= 64: slots and window rows are chunks of their own)
  CUtensorMap tq;
  if (!cache_encode_q(q, (long long)batch * heads, d, n, &tq)) return DS_ERR_ARG;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  aq_config(&cfg, attr, n, d, (unsigned)(tiles * C), C);
  cfg.stream = static_cast<cudaStream_t>(stream);
  set_pdl(attr[1]);
  cfg.numAttrs = pdl_on() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, aq_kernel(dtype, n, few), tq, p) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

extern "C" int ds_attention_mass(const void* q, const void* cache, int64_t cache_batch_stride, const float* scales,
                                 int64_t scales_batch_stride, int dtype, int block, int T, const int32_t* idx, int k,
                                 const float* lse, int batch, int heads, int kv_heads, int d, float scale, float* mass,
                                 int64_t mass_batch_stride, void* stream) {
  int rc = cache_attn_check(q, cache, cache_batch_stride, scales, scales_batch_stride, dtype, block, T, idx, k, batch,
                            heads, kv_heads, d, scale);
  if (rc != DS_OK) return rc;
  if (!lse || !mass || (batch > 1 && mass_batch_stride < T) || cache_misaligned(lse, 4) || cache_misaligned(mass, 4))
    return DS_ERR_ARG;
  DeviceState* s = nullptr;
  rc = device_state(&s);
  if (rc != DS_OK || k == 0) return rc;
  AqParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.scales = scales;
  p.idx = idx;
  p.lse = const_cast<float*>(lse);
  p.mass = mass;
  p.status = s->status;
  p.wait_ns = wait_limit();
  p.fault = take_planted_fault();
  p.cache_bstride = cache_batch_stride * kv_heads * d;
  p.scales_bstride = scales_batch_stride * kv_heads;
  p.mass_bstride = mass_batch_stride;
  p.T = T;
  p.k = k;
  p.B = batch;
  p.H = heads;
  p.Hkv = kv_heads;
  p.D = d;
  p.log_block = cache_is8(dtype) ? cache_log_block(block) : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  const int G = heads / kv_heads, n = G <= 16 ? 16 : G <= 32 ? 32 : 64;
  p.HT = (G + n - 1) / n;
  // a CTA to each head tile of a chunk, up to 8
  p.C = std::min(kAmMaxCluster, kv_heads * p.HT);
  // rows of a chunk: 128, or fewer while the chunks leave half of the SMs idle (the work of a CTA is mostly latency)
  p.R = kAqRows;
  while (p.R > 32 && (int64_t)batch * ((k + p.R / 2 - 1) / (p.R / 2)) * p.C <= s->num_sms) p.R /= 2;
  const int64_t ctas = (int64_t)batch * ((k + p.R - 1) / p.R) * p.C;
  CUtensorMap tq;
  if (!cache_encode_q(q, (long long)batch * heads, d, n, &tq)) return DS_ERR_ARG;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kAmThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)am_smem(n, d);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cache_cluster(attr[0], p.C);
  set_pdl(attr[1]);
  cfg.attrs = attr;
  cfg.numAttrs = pdl_on() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, am_kernel(dtype, n), tq, p) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

extern "C" int ds_cache_evict(const float* mass, int64_t mass_batch_stride, int batch, int T, const int32_t* len,
                              int block, int budget, int keep_first, int keep_last, int32_t* kept, int32_t* new_len,
                              void* stream) {
  if (!mass || !kept || !new_len || batch < 1 || batch > 65535 || T < 1 || T > kMaxRowElems || mass_batch_stride < 0)
    return DS_ERR_ARG;
  if (cache_log_block(block) < 0 || budget < 1 || budget > (T + block - 1) / block || keep_first < 0 || keep_last < 0 ||
      keep_first > budget || keep_last > budget - keep_first)
    return DS_ERR_ARG;
  if (cache_misaligned(mass, 4) || cache_misaligned(len, 4) || cache_misaligned(kept, 4) || cache_misaligned(new_len, 4))
    return DS_ERR_ARG;
  DeviceState* s = nullptr;
  const int rc = device_state(&s);
  if (rc != DS_OK) return rc;
  CeParams p = {};
  p.mass = mass;
  p.len = len;
  p.kept = kept;
  p.new_len = new_len;
  p.status = s->status;
  p.mass_bstride = mass_batch_stride;
  p.T = T;
  p.block = block;
  p.budget = budget;
  p.first = keep_first;
  p.last = keep_last;
  // CTAs of a batch row: a share of some 8192 rows to each.  8 rows of 32768 in blocks
  // of 64 take 9.3 us with 4 CTAs each, 9.9 with 2 and 12.1 with 8 (every CTA reads the
  // others' counts); in blocks of 1 15.3, 24.9 and 15.2.  4096 rows take 8.4 us with 1, 8.7
  // with 2.
  int C = 1;
  while (C < kCeMaxCluster && T / C > 8192) C *= 2;
  const int nb = (T + block - 1) / block;
  p.held = std::min((nb + C - 1) / C, kCeKeys);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3((unsigned)(batch * C), 1, 1);
  cfg.blockDim = dim3(kCeThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)p.held * 4;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cache_cluster(attr[0], C);
  set_pdl(attr[1]);
  cfg.attrs = attr;
  cfg.numAttrs = pdl_on() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, cache_evict_kernel, p) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

extern "C" int ds_cache_compact(const ds_cache_array* arrays, int n_arrays, const int32_t* kept, int budget,
                                const int32_t* len, int batch, int T, int block, void* stream) {
  if (!arrays || !kept || n_arrays < 1 || n_arrays > DS_CACHE_MAX_ARRAYS || batch < 1 || batch > 65535 || T < 1 ||
      T > kMaxRowElems || cache_log_block(block) < 0)
    return DS_ERR_ARG;
  const int64_t nb = ((int64_t)T + block - 1) / block;
  if (budget < 1 || budget > nb || cache_misaligned(kept, 4) || cache_misaligned(len, 4)) return DS_ERR_ARG;
  if ((int64_t)batch * budget > INT32_MAX) return DS_ERR_ARG;
  CcParams p = {};
  CacheSpan src[DS_CACHE_MAX_ARRAYS], dst[DS_CACHE_MAX_ARRAYS];
  for (int i = 0; i < n_arrays; ++i) {
    const ds_cache_array& a = arrays[i];
    if (!a.src || !a.dst || a.item_bytes < 1 || a.item_bytes > (int64_t(1) << 24) || (a.per_block != 0 && a.per_block != 1))
      return DS_ERR_ARG;
    const int64_t src_bytes = a.item_bytes * (a.per_block ? nb : T);
    const int64_t dst_bytes = a.item_bytes * (a.per_block ? budget : std::min<int64_t>(T, (int64_t)budget * block));
    if (batch > 1 && (a.src_batch_stride < src_bytes || a.dst_batch_stride < dst_bytes)) return DS_ERR_ARG;
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(a.src), d0 = reinterpret_cast<uintptr_t>(a.dst);
    src[i] = {s0, a.src_batch_stride, src_bytes};
    dst[i] = {d0, a.dst_batch_stride, dst_bytes};
    const uint64_t bits = (uint64_t)s0 | d0 | (uint64_t)a.item_bytes |
                          (batch > 1 ? (uint64_t)a.src_batch_stride | (uint64_t)a.dst_batch_stride : 0);
    CcArray& c = p.a[i];
    c.src = static_cast<const uint8_t*>(a.src);
    c.dst = static_cast<uint8_t*>(a.dst);
    c.src_bstride = a.src_batch_stride;
    c.dst_bstride = a.dst_batch_stride;
    c.item = a.item_bytes;
    c.per_block = a.per_block;
    c.vec = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
    c.row_per = (uint32_t)(c.item / c.vec);
    c.per = (uint32_t)(a.per_block ? 1 : block) * c.row_per;
  }
  // the moves are not ordered among themselves, so no array may be written where one is
  // read, or where another is written
  for (int i = 0; i < n_arrays; ++i)
    for (int j = 0; j < n_arrays; ++j)
      if (cache_overlap(src[i], dst[j], batch) || (i < j && cache_overlap(dst[i], dst[j], batch))) return DS_ERR_ARG;
  DeviceState* s = nullptr;
  const int rc = device_state(&s);
  if (rc != DS_OK) return rc;
  p.kept = kept;
  p.len = len;
  p.status = s->status;
  p.T = T;
  p.block = block;
  p.budget = budget;
  p.n = n_arrays;
  p.B = batch;
  p.wait_ns = wait_limit();
  // Arrays with blocks of 16 KiB and more, in multiples of 16 bytes, go by bulk copies,
  // ahead of the others: 67 MB of 32 KiB blocks, each read and written, moved in 20.7 us,
  // against 29.5 by the threads, of 16 KiB blocks in 21.0 against 27.3.  Of 8 KiB blocks
  // both take 27.5, of 4 KiB blocks the bulk copies 44.7 (a copy has a fixed cost) and
  // the threads 24.9.
  std::stable_partition(p.a, p.a + p.n, [&](CcArray& c) {
    const int64_t unit = c.item * (c.per_block ? 1 : block);
    c.parts = c.vec == 16 && unit >= 16384 ? (int)((unit + kCcPiece - 1) / kCcPiece) : 0;
    p.n_bulk += c.parts > 0;
    return c.parts > 0;
  });
  int64_t turn = 0, pieces = 0;
  for (int i = 0; i < p.n; ++i) {
    if (i < p.n_bulk)
      pieces += (int64_t)batch * budget * p.a[i].parts;
    else
      turn += p.a[i].per;
  }
  // Entries of a turn: two shares to a warp, or fewer while SMs are idle.  134 MB of rows
  // of 512 bytes with their accounts and scales, 8 x 16384 of 32768 kept: 25.5 us (5.3
  // TB/s) with 14 shares to a turn, 32.1 with 8 and 27.8 with 28.
  p.group = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(kCcMaxGroup, budget), 14 * kCcShare / std::max<int64_t>(turn, 1)));
  while (p.group > 1 && (int64_t)batch * ((budget + p.group - 1) / p.group) * 2 <= s->num_sms) p.group = (p.group + 1) / 2;
  const int64_t groups = (int64_t)batch * ((budget + p.group - 1) / p.group);
  if (p.n_bulk > 0) {
    p.fault = take_planted_fault();
    return cache_launch(cache_compact_bulk_kernel, p, dim3((unsigned)std::min<int64_t>(pieces, s->num_sms)), kCcBulkThreads,
                        kCcSmem, stream);
  }
  return cache_launch(cache_compact_kernel, p, dim3((unsigned)std::min<int64_t>(groups, 1 << 20)), 256, 0, stream);
}
