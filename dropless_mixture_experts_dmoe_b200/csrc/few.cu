// few.cu -- the whole layer for a few tokens (T <= DMOE_FEW_MAX_TOKENS): the decode step of a
// model whose prompts run through dmoe_forward.  With so few tokens the layer is bound by
// reading the weights of the experts in use, so nothing is padded or copied:
//   k_few_route  one warp per token: top-k of the logits and the softmax weights
//   k_few_glu    H_j = silu(W1_e x_t) * (W3_e x_t) per entry j = t*k + s, fp32
//   k_few_down   y_t = sum_s w_ts W2_e H_j
// Expert weights are bf16, or in the microscaled 4-bit format (dmoe_mx4).
#include "common.cuh"
#include "kernels.h"
#include "mx4.cuh"
#include "route_key.cuh"

namespace dmoe {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// One warp per token.  The k rounds of a warp-wide integer max over unique keys (the logit's
// order-preserving image, then the lower expert) pick the top-k in rank order, as the map's
// routing does; lane l holds experts l, l + 32, ...  The softmax terms use expf.
__global__ void __launch_bounds__(kFewThreads)
    k_few_route(const uint16_t *__restrict__ logits, int T, int E, int k, int renorm,
                int32_t *__restrict__ top, float *__restrict__ weights, int32_t *status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kFewWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  const uint16_t *row = logits + (size_t)t * E;
  bool bad = false;
  for (int e = lane; e < E; e += 32) bad |= (row[e] & 0x7F80u) == 0x7F80u;
  uint32_t last = 0xFFFFFFFFu, mine = 0u;
  for (int s = 0; s < k; ++s) {  // the largest key below the last pick
    uint32_t best = 0u;
    for (int e = lane; e < E; e += 32) {
      const uint32_t key = route_key_nan((uint32_t)row[e] << 16, 0xFFFFu - (uint32_t)e);
      if (key < last) best = max(best, key);
    }
    last = __reduce_max_sync(0xFFFFFFFFu, best);
    if (lane == s) mine = last;
  }
  const int e = 0xFFFF - (int)(mine & 0xFFFFu);
  const float v = (lane < k) ? __uint_as_float((uint32_t)row[e] << 16) : 0.0f;
  const float m = __shfl_sync(0xFFFFFFFFu, v, 0);
  float sum = 0.0f;
  if (renorm) {
    if (lane < k) sum = expf(v - m);
  } else {
    for (int i = lane; i < E; i += 32) sum += expf(__uint_as_float((uint32_t)row[i] << 16) - m);
  }
  sum = warp_sum(sum);
  if (lane < k) {
    top[(size_t)t * k + lane] = e;
    weights[(size_t)t * k + lane] = expf(v - m) / sum;
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) set_status(status, DMOE_STATUS_NONFINITE_LOGITS);
}

// Given experts: report ids outside [0, E) (their entries add nothing) and repeats.
__global__ void __launch_bounds__(kFewThreads)
    k_few_check(const int32_t *__restrict__ top, int T, int E, int k, int32_t *status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kFewWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  int e = -1 - lane, flags = 0;
  if (lane < k) {
    e = top[(size_t)t * k + lane];
    if (e < 0 || e >= E) {
      flags = DMOE_STATUS_EXPERT_OUT_OF_RANGE;
      e = -1 - lane;
    }
  }
  const unsigned peers = __match_any_sync(0xFFFFFFFFu, e);
  if (e >= 0 && __popc(peers) > 1) flags |= DMOE_STATUS_DUPLICATE_EXPERT;
  flags = __reduce_or_sync(0xFFFFFFFFu, flags);
  if (flags && lane == 0) set_status(status, flags);
}

// Eight consecutive weights (columns 8v .. 8v+7 of row r) in fp32.
__device__ __forceinline__ void weights8(const FewWeights &w, long long r, int v, int cols,
                                         float (&o)[8]) {
  if (w.scales) {
    uint32_t p[4];
    mx4_unpack8(__ldg(static_cast<const uint32_t *>(w.data) + r * (cols >> 3) + v), p);
    const float s = mx4_scale_value(static_cast<const uint8_t *>(
        w.scales)[mx4_scale_word(r, v >> 4, cols >> 7) + ((v >> 2) & 3)]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = f16_lo(p[i]) * s;
      o[2 * i + 1] = f16_hi(p[i]) * s;
    }
  } else {
    const uint4 q = __ldg(static_cast<const uint4 *>(w.data) + r * (cols >> 3) + v);
    const uint32_t *p = reinterpret_cast<const uint32_t *>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = bf16_lo(p[i]);
      o[2 * i + 1] = bf16_hi(p[i]);
    }
  }
}

__global__ void __launch_bounds__(kFewThreads) k_few_glu(const FewParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long items = (long long)p.T * p.k * p.f;
  const long long nw = (long long)gridDim.x * kFewWarps;
  for (long long it = (long long)blockIdx.x * kFewWarps + (threadIdx.x >> 5); it < items;
       it += nw) {
    const long long j = it / p.f;
    const int c = (int)(it - j * p.f), t = (int)(j / p.k);
    const int e = p.top[j];
    if (e < 0 || e >= p.E) continue;
    const long long r = (long long)e * p.f + c;
    float a = 0.0f, b = 0.0f;
    for (int v = lane; v < (p.h >> 3); v += 32) {
      const uint4 q = __ldg(static_cast<const uint4 *>(p.x) + (size_t)t * (p.h >> 3) + v);
      const uint32_t *xw = reinterpret_cast<const uint32_t *>(&q);
      float w1[8], w3[8];
      weights8(p.w1, r, v, p.h, w1);
      weights8(p.w3, r, v, p.h, w3);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xv = (i & 1) ? bf16_hi(xw[i >> 1]) : bf16_lo(xw[i >> 1]);
        a = fmaf(xv, w1[i], a);
        b = fmaf(xv, w3[i], b);
      }
    }
    a = warp_sum(a);
    b = warp_sum(b);
    if (lane == 0) p.hbuf[it] = silu_f(a) * b;
  }
}

__global__ void __launch_bounds__(kFewThreads) k_few_down(const FewParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long items = (long long)p.T * p.h;
  const long long nw = (long long)gridDim.x * kFewWarps;
  for (long long it = (long long)blockIdx.x * kFewWarps + (threadIdx.x >> 5); it < items;
       it += nw) {
    const int t = (int)(it / p.h), c = (int)(it - (long long)t * p.h);
    float y = 0.0f;
    for (int s = 0; s < p.k; ++s) {
      const long long j = (long long)t * p.k + s;
      const int e = p.top[j];
      if (e < 0 || e >= p.E) continue;
      float a = 0.0f;
      for (int v = lane; v < (p.f >> 3); v += 32) {
        float w[8];
        weights8(p.w2, (long long)e * p.h + c, v, p.f, w);
        const float4 *hv = reinterpret_cast<const float4 *>(p.hbuf + j * p.f) + 2 * v;
        const float4 h0 = hv[0], h1 = hv[1];
        a = fmaf(w[0], h0.x, a);
        a = fmaf(w[1], h0.y, a);
        a = fmaf(w[2], h0.z, a);
        a = fmaf(w[3], h0.w, a);
        a = fmaf(w[4], h1.x, a);
        a = fmaf(w[5], h1.y, a);
        a = fmaf(w[6], h1.z, a);
        a = fmaf(w[7], h1.w, a);
      }
      y = fmaf(p.weights[j], warp_sum(a), y);
    }
    if (lane == 0) p.y[it] = __float2bfloat16(y);
  }
}

static int few_grid(long long warps) {
  long long g = (warps + kFewWarps - 1) / kFewWarps;
  const long long cap = (long long)device_sm_count() * 8;
  return (int)(g < cap ? g : cap);
}

cudaError_t launch_few(const FewParams &p, const uint16_t *logits, bool renorm, int32_t *top,
                       float *weights, int32_t *status, cudaStream_t st) {
  const int rg = (p.T + kFewWarps - 1) / kFewWarps;
  cudaError_t e;
  if (logits)
    e = launch_pdl(k_few_route, rg, kFewThreads, 0, st, logits, p.T, p.E, p.k, renorm ? 1 : 0, top,
                   weights, status);
  else
    e = launch_pdl(k_few_check, rg, kFewThreads, 0, st, (const int32_t *)top, p.T, p.E, p.k,
                   status);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_few_glu, few_grid((long long)p.T * p.k * p.f), kFewThreads, 0, st, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_few_down, few_grid((long long)p.T * p.h), kFewThreads, 0, st, p);
}

}  // namespace dmoe
