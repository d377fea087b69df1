// mx4.cu -- conversions to and from the microscaled 4-bit format (dmoe_mx4 of dmoe.h): blocks of
// 32 along a row, one power-of-two scale s each, elements q_i = e2m1(x_i / s) with
// s = 2^(floor(log2 max|x|) - 2).
#include "common.cuh"
#include "kernels.h"
#include "mx4.cuh"

namespace dmoe {

constexpr int kMx4Threads = 256;
constexpr int kMx4Warps = kMx4Threads / 32;

// A 16-byte load of data that is read once.
__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Per half: the larger of two unsigned 16-bit values.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The two bf16 values of w times a power of two (bf16), in fp32: exact.
__device__ __forceinline__ void scale_bf16x2(uint32_t w, uint16_t f, float &lo, float &hi) {
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "fma.rn.f32.bf16 %0, l, %3, %4;\n\tfma.rn.f32.bf16 %1, h, %3, %4;}"
      : "=f"(lo), "=f"(hi)
      : "r"(w), "h"(f), "f"(-0.0f));  // -0 keeps the sign of a zero
}

// One lane's 8 columns of a row: the elements, and (in every lane of the block's four) the
// block's scale byte.  All lanes of the warp take part.  Magnitudes of bf16 values order like
// their bits, two at a time.
__device__ __forceinline__ uint32_t quantize8(uint4 q, uint32_t &scale) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&q);
  uint32_t m = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                         max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
  m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  scale = mx4_scale_byte(max(m << 16, m & 0xFFFF0000u));
  // the inverse scale 2^(127 - s) as bf16 (s <= 252)
  const uint16_t inv = (uint16_t)((254u - min(scale, 253u)) << 7);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) scale_bf16x2(w[i], inv, v[2 * i], v[2 * i + 1]);
  const uint32_t c = mx4_pack8(v);
  return scale == 255u ? 0u : c;
}

// The scale bytes of a lane group's 16 lanes (128 columns: four blocks) as one word, in the
// group's first lane.
__device__ __forceinline__ uint32_t scale_word16(uint32_t scale, int lane) {
  uint32_t w = scale << (8 * ((lane >> 2) & 3));
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 8);
  return w;
}

// Rows l, l + 32, l + 64, l + 96 of a row tile go together: their scale words of a column tile
// are 16 consecutive bytes.
//
// src [rows, cols] bf16 -> codes [rows, cols / 2], scales in tiles.  A warp takes 256 columns (two
// column tiles; the last pair of a row may be half) of the four rows, all four 16-byte loads of
// a lane in flight at once (one row at a time: 202 us there and back for 65536 x 2048, bound by
// load latency; this form 131 us, 80 % of the copy rate, with the ALU the busiest pipe).
// Rows past `rows` of the last row tile get scale bytes 0.
__global__ void __launch_bounds__(kMx4Threads)
    k_mx4_quantize(long long rows, int vpr, const uint4 *__restrict__ src,
                   uint32_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int ct = vpr >> 4;  // column tiles; vpr = 16-byte vectors (8 columns) per row
  const long long groups = (rows + 127) / 128 * 32;  // of four rows
  const int v = blockIdx.y * 32 + lane;              // 256 columns per blockIdx.y
  for (long long lr = (long long)blockIdx.x * kMx4Warps + (threadIdx.x >> 5); lr < groups;
       lr += (long long)gridDim.x * kMx4Warps) {
    const long long r0 = (lr >> 5) * 128 + (lr & 31);
    const uint4 *sp = src + r0 * vpr + v;
    uint32_t *cp = codes + r0 * vpr + v;
    uint4 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = r0 + 32 * i;
      q[i] = (v < vpr && r < rows) ? ld_stream(sp + (size_t)(32 * i) * vpr)
                                   : make_uint4(0u, 0u, 0u, 0u);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = r0 + 32 * i;
      uint32_t sc;
      const uint32_t c = quantize8(q[i], sc);
      w[i] = (r < rows) ? scale_word16(sc, lane) : 0u;  // r is the same in the whole warp
      if (v < vpr && r < rows) cp[(size_t)(32 * i) * vpr] = c;
    }
    if (v < vpr && (lane & 15) == 0)
      *reinterpret_cast<uint4 *>(scales + mx4_scale_word(r0, v >> 4, ct)) =
          make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// codes, scales -> dst [rows, cols] bf16 (exact: one bit of mantissa), the same items.
__global__ void __launch_bounds__(kMx4Threads)
    k_mx4_dequantize(long long rows, int vpr, const uint32_t *__restrict__ codes,
                     const uint8_t *__restrict__ scales, uint4 *__restrict__ dst) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int ct = vpr >> 4;
  const long long groups = (rows + 127) / 128 * 32;
  const int v = blockIdx.y * 32 + lane;
  if (v >= vpr) return;
  for (long long lr = (long long)blockIdx.x * kMx4Warps + (threadIdx.x >> 5); lr < groups;
       lr += (long long)gridDim.x * kMx4Warps) {
    const long long r0 = (lr >> 5) * 128 + (lr & 31);
    const uint32_t *cp = codes + r0 * vpr + v;
    uint4 *dp = dst + r0 * vpr + v;
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = r0 + 32 * i;
      c[i] = (r < rows) ? __ldg(cp + (size_t)(32 * i) * vpr) : 0u;
    }
    const uint4 sw = __ldg(reinterpret_cast<const uint4 *>(scales + mx4_scale_word(r0, v >> 4, ct)));
    const uint32_t w[4] = {sw.x, sw.y, sw.z, sw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = r0 + 32 * i;
      if (r >= rows) break;
      uint32_t o[4];
      mx4_unpack8(c[i], o);
      const float s = mx4_scale_value((w[i] >> (8 * ((v >> 2) & 3))) & 0xFFu);
      uint4 d;
      uint32_t *dw = reinterpret_cast<uint32_t *>(&d);
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[j] = pack_bf16x2(f16_lo(o[j]) * s, f16_hi(o[j]) * s);
      dp[(size_t)(32 * i) * vpr] = d;
    }
  }
}

// The padded gather with the conversion in it: a warp converts up to 1024 columns of a token row
// once, all its loads in flight, and writes them to the token's padded rows, with each row's
// routing weight beside; padding rows get elements, scales and a weight of zero.
__global__ void __launch_bounds__(kMx4Threads)
    k_mx4_gather(int T, int h, int k, int E, const uint4 *__restrict__ x,
                 const int32_t *__restrict__ dest_row, const int32_t *__restrict__ counts,
                 const int32_t *__restrict__ padded_bins, uint32_t *__restrict__ codes,
                 uint8_t *__restrict__ scales, const int32_t *__restrict__ offsets,
                 const float *__restrict__ weights, float *__restrict__ row_weight) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int vpr = h >> 3, ct = h >> 7;
  constexpr int VPL = 4;
  const int S = (vpr + 32 * VPL - 1) / (32 * VPL);
  const long long ntok = (long long)T * S;
  const long long items = ntok + (long long)kBlock * E;
  const long long nw = (long long)gridDim.x * kMx4Warps;
  for (long long it = (long long)blockIdx.x * kMx4Warps + (threadIdx.x >> 5); it < items;
       it += nw) {
    if (it < ntok) {
      const int t = (int)(it / S);
      const int v0 = (int)(it - (long long)t * S) * 32 * VPL + lane;
      const long long base = offsets ? offsets[t] : (long long)t * k;
      const int cnt = offsets ? offsets[t + 1] - (int)base : k;
      uint4 q[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        q[i] = (v0 + 32 * i < vpr) ? __ldg(x + (size_t)t * vpr + v0 + 32 * i)
                                   : make_uint4(0u, 0u, 0u, 0u);
      uint32_t c[VPL], w[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        uint32_t sc;
        c[i] = quantize8(q[i], sc);
        w[i] = scale_word16(sc, lane);
      }
      for (int c0 = 0; c0 < cnt; c0 += 32) {
        const int nc = min(32, cnt - c0);
        const int d = (lane < nc) ? __ldg(dest_row + base + c0 + lane) : -1;
        if (v0 < 32 && d >= 0) row_weight[d] = __ldg(weights + base + c0 + lane);  // first slice
        for (int s = 0; s < nc; ++s) {
          const int r = __shfl_sync(0xFFFFFFFFu, d, s);
          if (r < 0) continue;
          uint32_t *dst = codes + (size_t)r * vpr + v0;
          uint8_t *sd = scales + mx4_scale_word(r, v0 >> 4, ct);
#pragma unroll
          for (int i = 0; i < VPL; ++i) {
            if (v0 + 32 * i >= vpr) break;
            dst[32 * i] = c[i];
            if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(sd + i * 2 * kMx4TileBytes) = w[i];
          }
        }
      }
    } else {
      const long long p = it - ntok;
      const int e = (int)(p / kBlock), r = (int)(p % kBlock);
      const int row = ((e > 0) ? padded_bins[e - 1] : 0) + counts[e] + r;
      if (row >= padded_bins[e]) continue;
      if (lane == 0) row_weight[row] = 0.0f;
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

// blockIdx.y: 256 columns; blockIdx.x strides over groups of four rows, eight per CTA.  (A grid's y
// extent ends at 65535; the entry points' 2^23 columns need 32768.)
static dim3 mx4_grid2(long long rows, long long cols) {
  const long long y = (cols / 8 + 31) / 32;
  long long x = (rows + 127) / 128 * 32 / kMx4Warps;
  const long long cap = ((long long)device_sm_count() * 8 + y - 1) / y;
  return dim3((unsigned)(x < cap ? x : cap), (unsigned)y);
}

cudaError_t launch_mx4_quantize(long long rows, long long cols, const void *src, void *codes,
                                void *scales, cudaStream_t st) {
  return launch_pdl(k_mx4_quantize, mx4_grid2(rows, cols), kMx4Threads, 0, st, rows,
                    (int)(cols / 8), static_cast<const uint4 *>(src),
                    static_cast<uint32_t *>(codes), static_cast<uint8_t *>(scales));
}

cudaError_t launch_mx4_dequantize(long long rows, long long cols, const void *codes,
                                  const void *scales, void *dst, cudaStream_t st) {
  return launch_pdl(k_mx4_dequantize, mx4_grid2(rows, cols), kMx4Threads, 0, st, rows,
                    (int)(cols / 8), static_cast<const uint32_t *>(codes),
                    static_cast<const uint8_t *>(scales), static_cast<uint4 *>(dst));
}

cudaError_t launch_mx4_gather(int T, int h, int k, int E, const void *x, const int32_t *dest_row,
                              const int32_t *counts, const int32_t *padded_bins, void *codes,
                              void *scales, cudaStream_t st, const int32_t *offsets,
                              const float *weights, float *row_weight) {
  const long long items = (long long)T * ((h / 8 + 127) / 128) + (long long)kBlock * E;
  return launch_pdl(k_mx4_gather, mx4_grid(items, kMx4Warps), kMx4Threads, 0, st, T, h, k, E,
                    static_cast<const uint4 *>(x), dest_row, counts, padded_bins,
                    static_cast<uint32_t *>(codes), static_cast<uint8_t *>(scales), offsets, weights,
                    row_weight);
}

}  // namespace dmoe
