// mx4_gemm.cu -- the expert FFN over many tokens with both operands in the microscaled 4-bit
// format (dmoe_mx4): grouped products over the non-empty 128-row blocks of the padded layout.
//   GLU   H = silu(X W1_e^T) * (X W3_e^T), H in fp32 converted to the format (blocks of 32 columns)
//   DOWN  Y_pad = w * (H W2_e^T), block floating point rows as dmoe_expert_down writes them
#include "common.cuh"
#include "kernels.h"
#include "mx4.cuh"

namespace dmoe {

constexpr int kMgThreads = 256;

// 32 elements (one block) of row r into fp32.
__device__ __forceinline__ void mg_load_block(const uint8_t *codes, const uint8_t *scales,
                                              long long r, int blk, int cols, float *o) {
  const uint4 q = __ldg(reinterpret_cast<const uint4 *>(codes + r * (cols >> 1)) + blk);
  const float s =
      mx4_scale_value(scales[mx4_scale_word(r, blk >> 2, cols >> 7) + (blk & 3)]);
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&q);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p[4];
    mx4_unpack8(w[i], p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[8 * i + 2 * j] = f16_lo(p[j]) * s;
      o[8 * i + 2 * j + 1] = f16_hi(p[j]) * s;
    }
  }
}

__global__ void __launch_bounds__(kMgThreads) k_mx4_glu(const Mx4GemmParams p) {
  __shared__ float sa[128][33], s1[32][33], s3[32][33];
  pdl_wait();
  pdl_trigger();
  const int nt = p.f / 32, nb = *p.num_blocks;
  const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
  for (long long tile = blockIdx.x; tile < (long long)nb * nt; tile += gridDim.x) {
    const int b = (int)(tile / nt), n = (int)(tile - (long long)b * nt);
    const long long e = p.block_expert[b];
    float a[16], u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i] = u[i] = 0.0f;
    for (int kb = 0; kb < p.h / 32; ++kb) {
      __syncthreads();
      const int q = threadIdx.x;
      if (q < 128)
        mg_load_block(p.a, p.as, (long long)b * 128 + q, kb, p.h, sa[q]);
      else if (q < 160)
        mg_load_block(p.w1, p.w1s, e * p.f + n * 32 + q - 128, kb, p.h, s1[q - 128]);
      else if (q < 192)
        mg_load_block(p.w3, p.w3s, e * p.f + n * 32 + q - 160, kb, p.h, s3[q - 160]);
      __syncthreads();
      for (int kk = 0; kk < 32; ++kk) {
        const float x = sa[row][kk];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          a[i] = fmaf(x, s1[half * 16 + i][kk], a[i]);
          u[i] = fmaf(x, s3[half * 16 + i][kk], u[i]);
        }
      }
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      a[i] = silu_f(a[i]) * u[i];
      m = max(m, __float_as_uint(a[i]) & 0x7FFFFFFFu);
    }
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    const uint32_t sc = mx4_scale_byte(m);
    const long long r = (long long)b * 128 + row;
    const float inv = sc == 255u ? 0.0f : mx4_inverse(sc);
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + r * (p.f >> 1)) + n * 4 + half * 2;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a[8 * g + i] * inv;
      dst[g] = sc == 255u ? 0u : mx4_pack8(v);
    }
    if (half == 0)
      p.outs[mx4_scale_word(r, n >> 2, p.f >> 7) + (n & 3)] = (uint8_t)sc;
  }
}

__global__ void __launch_bounds__(kMgThreads) k_mx4_down(const Mx4GemmParams p) {
  extern __shared__ float sm[];
  float(*sa)[33] = reinterpret_cast<float(*)[33]>(sm);
  float(*sb)[33] = sa + 128;
  pdl_wait();
  pdl_trigger();
  const int nt = p.h / 128, nb = *p.num_blocks;
  const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
  for (long long tile = blockIdx.x; tile < (long long)nb * nt; tile += gridDim.x) {
    const int b = (int)(tile / nt), n = (int)(tile - (long long)b * nt);
    const int e = p.block_expert[b];
    float a[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) a[i] = 0.0f;
    for (int kb = 0; kb < p.f / 32; ++kb) {
      __syncthreads();
      const int q = threadIdx.x;
      if (q < 128)
        mg_load_block(p.a, p.as, (long long)b * 128 + q, kb, p.f, sa[q]);
      else
        mg_load_block(p.w1, p.w1s, (long long)e * p.h + n * 128 + q - 128, kb, p.f, sb[q - 128]);
      __syncthreads();
      for (int kk = 0; kk < 32; ++kk) {
        const float x = sa[row][kk];
#pragma unroll
        for (int i = 0; i < 64; ++i) a[i] = fmaf(x, sb[half * 64 + i][kk], a[i]);
      }
    }
    const int r = b * 128 + row;
    const float w = bfp_row_weight(p.padded_bins, p.bins, p.indices, p.weights, e, r);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 64; ++i) m = fmaxf(m, fabsf(a[i]));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    float stored;
    const float k = bfp_scale(m * fabsf(w), stored) * w;
    if (half == 0) p.yscale[(size_t)r * dmoe_scale_stride(p.h) + n] = stored;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out) + ((size_t)r * p.h + n * 128 + half * 64) / 2;
#pragma unroll
    for (int i = 0; i < 32; ++i) dst[i] = pack_f16x2(a[2 * i] * k, a[2 * i + 1] * k);
  }
}

cudaError_t launch_mx4_glu(const Mx4GemmParams &p, long long max_blocks, cudaStream_t st) {
  const long long tiles = max_blocks * (p.f / 32);
  const long long cap = (long long)device_sm_count() * 4;
  return launch_pdl(k_mx4_glu, (int)(tiles < cap ? tiles : cap), kMgThreads, 0, st, p);
}

cudaError_t launch_mx4_down(const Mx4GemmParams &p, long long max_blocks, cudaStream_t st) {
  const long long tiles = max_blocks * (p.h / 128);
  const long long cap = (long long)device_sm_count() * 4;
  return launch_pdl(k_mx4_down, (int)(tiles < cap ? tiles : cap), kMgThreads,
                    256 * 33 * sizeof(float), st, p);
}

}  // namespace dmoe
