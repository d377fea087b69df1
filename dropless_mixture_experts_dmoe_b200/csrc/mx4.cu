// mx4.cu -- conversions to and from the microscaled 4-bit format (dmoe_mx4 of dmoe.h): blocks of
// 32 along a row, one power-of-two scale s each, elements q_i = e2m1(x_i / s) with
// s = 2^(floor(log2 max|x|) - 2).
#include "common.cuh"
#include "kernels.h"
#include "mx4.cuh"

namespace dmoe {

constexpr int kMx4Threads = 256;
constexpr int kMx4Warps = kMx4Threads / 32;

// One lane's 8 columns of a row: the elements, and (in every lane of the block's four) the
// block's scale byte.  All lanes of the warp take part.
__device__ __forceinline__ uint32_t quantize8(uint4 q, uint32_t &scale) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&q);
  uint32_t m = 0u;  // the largest |x| as fp32 bits (integers order like magnitudes)
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max((w[i] << 16) & 0x7FFF0000u, w[i] & 0x7FFF0000u));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  scale = mx4_scale_byte(m);
  if (scale == 255u) return 0u;
  const float inv = mx4_inverse(scale);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]) * inv;
    v[2 * i + 1] = bf16_hi(w[i]) * inv;
  }
  return mx4_pack8(v);
}

// The scale bytes of a lane group's 16 lanes (128 columns: four blocks) as one word, in the
// group's first lane.
__device__ __forceinline__ uint32_t scale_word16(uint32_t scale, int lane) {
  uint32_t w = scale << (8 * ((lane >> 2) & 3));
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 8);
  return w;
}

// src [rows, cols] bf16 -> codes [rows, cols / 2], scales in tiles.  A warp takes 256 columns of
// a row (two column tiles; the last one may be half).  Rows past `rows` of the last row tile
// get scale bytes 0.
__global__ void __launch_bounds__(kMx4Threads)
    k_mx4_quantize(long long rows, long long cols, const uint4 *__restrict__ src,
                   uint32_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long vpr = cols >> 3;  // 16-byte vectors (8 columns) per row
  const int ct = (int)(cols >> 7);
  const long long S = (vpr + 31) / 32;
  const long long rpad = (rows + 127) / 128 * 128;
  const long long nw = (long long)gridDim.x * kMx4Warps;
  for (long long it = (long long)blockIdx.x * kMx4Warps + (threadIdx.x >> 5); it < rpad * S;
       it += nw) {
    const long long r = it / S;
    const long long v = (it - r * S) * 32 + lane;
    const bool live = v < vpr;
    uint32_t c = 0u, sc = 0u;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (live && r < rows) q = __ldg(src + r * vpr + v);
    c = quantize8(q, sc);
    const uint32_t w = scale_word16(sc, lane);
    if (live && r < rows) codes[r * vpr + v] = c;
    if (live && (lane & 15) == 0)
      *reinterpret_cast<uint32_t *>(scales + mx4_scale_word(r, (int)(v >> 4), ct)) =
          r < rows ? w : 0u;
  }
}

// codes, scales -> dst [rows, cols] bf16 (exact: one bit of mantissa).
__global__ void __launch_bounds__(kMx4Threads)
    k_mx4_dequantize(long long rows, long long cols, const uint32_t *__restrict__ codes,
                     const uint8_t *__restrict__ scales, uint4 *__restrict__ dst) {
  pdl_wait();
  pdl_trigger();
  const long long vpr = cols >> 3;
  const int ct = (int)(cols >> 7);
  const long long n = rows * vpr;
  for (long long i = (long long)blockIdx.x * kMx4Threads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kMx4Threads) {
    const long long r = i / vpr;
    const int v = (int)(i - r * vpr);
    uint32_t o[4];
    mx4_unpack8(__ldg(codes + i), o);
    const float s = mx4_scale_value(scales[mx4_scale_word(r, v >> 4, ct) + ((v >> 2) & 3)]);
    uint4 d;
    uint32_t *dw = reinterpret_cast<uint32_t *>(&d);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[j] = pack_bf16x2(f16_lo(o[j]) * s, f16_hi(o[j]) * s);
    dst[i] = d;
  }
}

// The padded gather with the conversion in it: a warp converts 256 columns of a token row once
// and writes them to the token's padded rows; padding rows get elements and scales of zero.
__global__ void __launch_bounds__(kMx4Threads)
    k_mx4_gather(int T, int h, int k, int E, const uint4 *__restrict__ x,
                 const int32_t *__restrict__ dest_row, const int32_t *__restrict__ counts,
                 const int32_t *__restrict__ padded_bins, uint32_t *__restrict__ codes,
                 uint8_t *__restrict__ scales, const int32_t *__restrict__ offsets) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int vpr = h >> 3, ct = h >> 7;
  const int S = (vpr + 31) / 32;
  const long long ntok = (long long)T * S;
  const long long items = ntok + (long long)kBlock * E;
  const long long nw = (long long)gridDim.x * kMx4Warps;
  for (long long it = (long long)blockIdx.x * kMx4Warps + (threadIdx.x >> 5); it < items;
       it += nw) {
    if (it < ntok) {
      const int t = (int)(it / S);
      const int v = (int)(it - (long long)t * S) * 32 + lane;
      const bool live = v < vpr;
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (live) q = __ldg(x + (size_t)t * vpr + v);
      const long long base = offsets ? offsets[t] : (long long)t * k;
      const int cnt = offsets ? offsets[t + 1] - (int)base : k;
      uint32_t sc;
      const uint32_t c = quantize8(q, sc);
      const uint32_t w = scale_word16(sc, lane);
      for (int s = 0; s < cnt; ++s) {
        const int r = __ldg(dest_row + base + s);
        if (r < 0 || !live) continue;
        codes[(size_t)r * vpr + v] = c;
        if ((lane & 15) == 0)
          *reinterpret_cast<uint32_t *>(scales + mx4_scale_word(r, v >> 4, ct)) = w;
      }
    } else {
      const long long p = it - ntok;
      const int e = (int)(p / kBlock), r = (int)(p % kBlock);
      const int row = ((e > 0) ? padded_bins[e - 1] : 0) + counts[e] + r;
      if (row >= padded_bins[e]) continue;
      for (int v = lane; v < vpr; v += 32) {
        codes[(size_t)row * vpr + v] = 0u;
        if ((v & 15) == 0)
          *reinterpret_cast<uint32_t *>(scales + mx4_scale_word(row, v >> 4, ct)) = 0u;
      }
    }
  }
}

static int mx4_grid(long long items, long long per_cta) {
  long long g = (items + per_cta - 1) / per_cta;
  const long long cap = (long long)device_sm_count() * 8;
  if (g > cap) g = cap;
  return (int)(g < 1 ? 1 : g);
}

cudaError_t launch_mx4_quantize(long long rows, long long cols, const void *src, void *codes,
                                void *scales, cudaStream_t st) {
  const long long items = (rows + 127) / 128 * 128 * ((cols / 8 + 31) / 32);
  return launch_pdl(k_mx4_quantize, mx4_grid(items, kMx4Warps), kMx4Threads, 0, st, rows, cols,
                    static_cast<const uint4 *>(src), static_cast<uint32_t *>(codes),
                    static_cast<uint8_t *>(scales));
}

cudaError_t launch_mx4_dequantize(long long rows, long long cols, const void *codes,
                                  const void *scales, void *dst, cudaStream_t st) {
  return launch_pdl(k_mx4_dequantize, mx4_grid(rows * (cols / 8), kMx4Threads), kMx4Threads, 0, st,
                    rows, cols, static_cast<const uint32_t *>(codes),
                    static_cast<const uint8_t *>(scales), static_cast<uint4 *>(dst));
}

cudaError_t launch_mx4_gather(int T, int h, int k, int E, const void *x, const int32_t *dest_row,
                              const int32_t *counts, const int32_t *padded_bins, void *codes,
                              void *scales, cudaStream_t st, const int32_t *offsets) {
  const long long items = (long long)T * ((h / 8 + 31) / 32) + (long long)kBlock * E;
  return launch_pdl(k_mx4_gather, mx4_grid(items, kMx4Warps), kMx4Threads, 0, st, T, h, k, E,
                    static_cast<const uint4 *>(x), dest_row, counts, padded_bins,
                    static_cast<uint32_t *>(codes), static_cast<uint8_t *>(scales), offsets);
}

}  // namespace dmoe
