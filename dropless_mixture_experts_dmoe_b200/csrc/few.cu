// few.cu -- the whole layer for a few tokens (T <= DMOE_FEW_MAX_TOKENS): the decode step of a
// model whose prompts run through dmoe_forward or dmoe_mx4_forward.
//   k_few_route  top-k of the logits and the softmax weights (and x in fp16, for 4-bit weights)
//   k_few_glu    H_j = silu(W1_e x_t) * (W3_e x_t) per entry j = t*k + s
//   k_few_down   y_t = sum_s w_ts W2_e H_j
// With so few tokens the layer is bound by reading the weights of the experts in use once:
// nothing is padded, x and H are read from L2, and every kernel is a stream of weight tiles.
//
// A CTA multiplies tiles of 16 R weight rows (8 R gate and 8 R up rows in k_few_glu) by the
// columns of up to 8 NT of the expert's tokens.  Its warps are R row tiles x S slices of K, and
// one more that fills a ring of stages: TMA boxes of the weight rows (swizzled), bulk copies of
// the tokens' rows and of the scales.  The products run on mma.sync m16n8k16 with the weights
// as the 16-row operand: a tile of 16 rows costs one instruction per 16 K and 8 tokens, far
// below the tensor rate at these sizes; what counts is that 80 KB and more per SM are in flight
// at all times, so the ring runs on from one tile into the next, across experts, and that the
// multiplying warps spend few instructions on anything but the products.  tcgen05 would need
// 128-row tiles and a full shared-memory operand for 1 to 8 columns, and the 4-bit weights
// converted into it.
//   bf16 weights: x as bf16; H as the sum of two bf16 (16 bits), multiplied in turn.
//   4-bit weights: e2m1 -> fp16 is exact, so x and H go in fp16 under a power-of-two scale, x per
//     row (exact down to 2^-29 of the row's largest), H per 32 columns (11 bits); the 32
//     products of a weight block are summed first, then scaled by the block's scale.
// The few partial sums over S and over the experts of a token are added in a fixed order.
//
// Measured: one token, E = 8, top-2, hidden 4096, ffn 14336 (0.70 GB of bf16 weights) 111 us, 97 % of
// the copy rate; in counters the first product keeps DRAM 76 % busy and issues on 26 % of the cycles,
// the second 64 % (its 45 us hold the launch, the routing and the joining of sums).  With 4-bit
// weights (187 MB) 53 us: the first product is bound by its instructions (34 per 16 x 32 block of
// weights: unpacking to fp16 and the scales; 51 % of issue slots, 25 of its 32 us for the loads alone).
#include "common.cuh"
#include "kernels.h"
#include "mx4.cuh"
#include "route_key.cuh"

namespace dmoe {

namespace {

constexpr int kRouteWarps = 8;
constexpr int kRouteRegs = 8;  // experts per lane of a routing warp in registers
constexpr float kMaxBf16 = 0x1.FEp127f;
constexpr int kFewSmem = 226 * 1024;  // dynamic shared memory of a CTA at most

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// Exponent of the factor that takes a block of largest finite magnitude amax (fp32 bits) into
// fp16: amax lands in [2^14, 2^15); the factor stops at 2^126 (blocks below 2^-112).
__device__ __forceinline__ int f16_block_exp(uint32_t amax_bits) {
  const int ef = (int)(amax_bits >> 23);
  return (amax_bits == 0u) ? 0 : min(141 - ef, 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// |v| as fp32 bits if finite, else 0 (infinities and NaN pass through the conversion).
__device__ __forceinline__ uint32_t finite_abs(uint32_t b) {
  b &= 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// One token's routing by one warp.  The k rounds of a warp-wide integer max over unique keys
// (the logit's order-preserving image, then the lower expert) pick the top-k in rank order, as
// the map's routing does; lane l holds experts l, l + 32, ..., up to 256 experts in registers.
// The softmax terms use expf.  Lane s < k returns pick s and its weight; `bad`: a logit is not
// finite.
__device__ __forceinline__ void route_token(const uint16_t *__restrict__ row, int E, int k,
                                            bool renorm, int lane, int &expert, float &weight,
                                            bool &bad) {
  auto image = [&](int e) -> uint32_t { return (uint32_t)__ldcg(row + e) << 16; };
  auto key_of = [&](uint32_t im, int e) { return route_key_nan(im, 0xFFFFu - (uint32_t)e); };
  constexpr int R = kRouteRegs;
  uint32_t im[R], key[R];
  bad = false;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = lane + 32 * i;
    im[i] = (e < E) ? image(e) : 0u;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = lane + 32 * i;
    key[i] = (e < E) ? key_of(im[i], e) : 0u;
    bad |= (im[i] & 0x7F800000u) == 0x7F800000u;
  }
  for (int e = lane + 32 * R; e < E; e += 32) bad |= (image(e) & 0x7F800000u) == 0x7F800000u;
  uint32_t last = 0xFFFFFFFFu, mine = 0u;
  for (int s = 0; s < k; ++s) {  // the largest key below the last pick
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < R; ++i) best = max(best, key[i] < last ? key[i] : 0u);
    for (int e = lane + 32 * R; e < E; e += 32) {
      const uint32_t ke = key_of(image(e), e);
      if (ke < last) best = max(best, ke);
    }
    last = __reduce_max_sync(0xFFFFFFFFu, best);
    if (lane == s) mine = last;
  }
  expert = (lane < k) ? 0xFFFF - (int)(mine & 0xFFFFu) : 0;
  const float v = (lane < k) ? __uint_as_float(image(expert)) : 0.0f;
  const float m = __shfl_sync(0xFFFFFFFFu, v, 0);
  float sum = 0.0f;
  if (renorm) {
    if (lane < k) sum = expf(v - m);
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (lane + 32 * i < E) sum += expf(__uint_as_float(im[i]) - m);
    for (int e = lane + 32 * R; e < E; e += 32) sum += expf(__uint_as_float(image(e)) - m);
  }
  sum = warp_sum(sum);
  weight = expf(v - m) / sum;
  bad = __any_sync(0xFFFFFFFFu, bad);
}

// ... with its results stored; `status` may be NULL.
__device__ __forceinline__ void route_store(const uint16_t *__restrict__ row, int E, int k,
                                            bool renorm, int32_t *top, float *weights,
                                            int32_t *status, int lane) {
  int e;
  float w;
  bool bad;
  route_token(row, E, k, renorm, lane, e, w, bad);
  if (lane < k) {
    top[lane] = e;
    weights[lane] = w;
  }
  if (bad && lane == 0 && status) set_status(status, DMOE_STATUS_NONFINITE_LOGITS);
}

// Given experts: report ids outside [0, E) (their entries add nothing) and repeats.
__device__ __forceinline__ void check_token(const int32_t *__restrict__ top, int E, int k,
                                            int32_t *status, int lane) {
  int e = -1 - lane, flags = 0;
  if (lane < k) {
    e = top[lane];
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

// One CTA per token: warp 0 routes (or checks) it; when the weights have four bits the other
// warps convert its row of x to fp16 under one power-of-two scale.
__global__ void __launch_bounds__(32 * kRouteWarps)
    k_few_route(const uint16_t *__restrict__ logits, int E, int k, int renorm, int h,
                int32_t *__restrict__ top, float *__restrict__ weights, int32_t *status,
                const uint4 *__restrict__ x, uint4 *__restrict__ x16, float *__restrict__ xs) {
  __shared__ uint32_t s_max;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t t = blockIdx.x;
  const int vpr = h >> 3;
  if (x16) {
    if (threadIdx.x == 0) s_max = 0u;
    __syncthreads();
    if (warp > 0) {
      uint32_t m = 0u;
      for (int v = threadIdx.x - 32; v < vpr; v += 32 * (kRouteWarps - 1)) {
        const uint4 q = __ldg(x + t * vpr + v);
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&q);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m = max(m, max(finite_abs(w[i] << 16), finite_abs(w[i] & 0xFFFF0000u)));
      }
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      if (lane == 0) atomicMax(&s_max, m);
    }
    __syncthreads();
  }
  if (warp == 0) {
    if (logits)
      route_store(logits + t * E, E, k, renorm != 0, top + t * k, weights + t * k, status, lane);
    else
      check_token(top + t * k, E, k, status, lane);
  } else if (x16) {
    const int es = f16_block_exp(s_max);
    const float f = pow2(es);
    if (threadIdx.x == 32) xs[t] = pow2(-es);
    for (int v = threadIdx.x - 32; v < vpr; v += 32 * (kRouteWarps - 1)) {
      const uint4 q = __ldg(x + t * vpr + v);
      const uint32_t *w = reinterpret_cast<const uint32_t *>(&q);
      uint4 o;
      uint32_t *ow = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
      for (int i = 0; i < 4; ++i) ow[i] = pack_f16x2(bf16_lo(w[i]) * f, bf16_hi(w[i]) * f);
      x16[t * vpr + v] = o;
    }
  }
}

// ---- the product kernels -----------------------------------------------------------------------

// Copy `bytes` (a multiple of 16, both addresses too) to this CTA's shared memory, counted on bar.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// 16 bytes, past L1.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on bar when all of this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(
                   smem_u32(bar))
               : "memory");
}
// Shared-memory reads of the products: volatile, so that they stay behind the barrier waits, but
// without claiming other memory, so that the compiler moves them among the products.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void lds128(uint32_t (&v)[4], uint32_t a) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b + c
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
        "f"(c[3]));
}

// Shape of a variant: MX4 weights in four bits; DOWN the second product; NT tiles of 8 tokens;
// R x S multiplying warps of KU columns; P stages.  BR: copies of the token rows (two: H's
// upper and lower bf16).  SB: the token operand has a scale per 32 columns (H in fp16).
template <bool MX4_, bool DOWN_, int NT_, int R_, int S_, int KU_, int P_, int CTAS_,
          bool WIDE_ = false>
struct FewCfg {
  static constexpr bool MX4 = MX4_, DOWN = DOWN_, SB = MX4 && DOWN, WIDE = WIDE_;
  static constexpr int NT = NT_, R = R_, S = S_, KU = KU_, P = P_;
  static constexpr int min_ctas = CTAS_;  // CTAs per SM
  static constexpr int CH = S * KU;  // columns per stage
  static constexpr bool xbulk = CH * 2 >= 512 && NT <= 2;  // see load_x()
  static constexpr int warps = R * S, loaders = xbulk ? 1 : 4, threads = 32 * (warps + loaders);
  static constexpr int BR = (DOWN && !MX4) ? 2 : 1;
  // weights: [W1, W3 | W2][slices of SC columns][rows][row_b bytes], as TMA boxes land
  static constexpr int SC = MX4 ? (WIDE ? 256 : 128) : 64, slices = CH / SC;
  static constexpr int row_b = MX4 && !WIDE ? 64 : 128;
  static constexpr int mats = DOWN ? 1 : 2, rows_m = DOWN ? 16 * R : 8 * R;
  static constexpr int w_mat = slices * rows_m * row_b, w_bytes = mats * w_mat;
  static constexpr int sc_mat = MX4 ? CH / 128 * kMx4TileBytes : 0;  // whole scale tiles
  // token rows: a stride that is 16 (ldmatrix) or 64 (16-byte loads of 4 lanes a row) bytes off
  // a multiple of 128 keeps the reads free of bank conflicts
  static constexpr int x_row = CH * 2 + (MX4 ? 64 : 16);
  static constexpr int x_bytes = BR * 8 * NT * x_row;
  static constexpr int sb_row = CH / 8 + 16;  // a token's block scales
  static constexpr int sb_bytes = SB ? 8 * NT * sb_row : 0;
  static constexpr int o_sc = w_bytes, o_x = o_sc + mats * sc_mat, o_sb = o_x + x_bytes;
  static constexpr int stage = (o_sb + sb_bytes + 1023) / 1024 * 1024;
  static constexpr int outs = DOWN ? 16 * R : 8 * R;  // output columns per tile
  // partial sums of the slices of K past the first, and for GLU MX4 a tile's H in fp32
  static constexpr int red = (S - 1) * R * NT * 512;
  static constexpr int hrow = outs + 4;
  static constexpr int hbuf = (MX4 && !DOWN) ? 8 * NT * hrow * 4 : 0;
  // y sums: rows of `outs` plus 8 floats (four tokens x eight rows meet no bank twice)
  enum { yrow = DOWN ? outs + 8 : 0 };
  static constexpr int o_red = P * stage, o_hbuf = o_red + red, o_bars = o_hbuf + hbuf,
                       o_lists = o_bars + 128;
  static constexpr int fixed = 1024 + o_lists;  // the ring starts on a 1024-byte boundary
  static_assert(w_mat % 1024 == 0 && (!MX4 || DOWN || outs % 32 == 0), "boxes, whole blocks of H");
  static_assert(2 * P * 8 <= 112, "barriers");
  static_assert(P * stage >= 16 * DMOE_MAX_EXPERTS, "masks");
};

// Bytes of the expert lists: entries [n] (j | token << 16), a factor of each [n] (DOWN: its
// weight; GLU with 4-bit weights: the scale of its token's x), a word per expert, groups of
// up to 8 NT entries of one expert (at most one per expert in use and one per 8 entries, and where
// the last one ends); and with the
// routing done in the kernel the experts and weights [n].
__host__ __device__ inline size_t few_list_bytes(const FewParams &p) {
  const int n = p.T * p.k;
  const size_t a = (size_t)n * (p.logits ? 16 : 8) + (size_t)p.E * 4 +
                   (size_t)((p.E < n ? p.E : n) + n / 8 + 1) * 4;
  return (a + 15) / 16 * 16;
}

struct FewLists {
  uint32_t *ent;
  float *fac;
  int32_t *top;    // the routing, if this kernel does it
  float *weights;
  int *start;
  uint32_t *act;  // expert | first entry << 16
  __device__ __forceinline__ FewLists(uint8_t *base, const FewParams &p) {
    const int n = p.T * p.k, routed = p.logits ? n : 0;
    ent = reinterpret_cast<uint32_t *>(base);
    fac = reinterpret_cast<float *>(ent + n);
    top = reinterpret_cast<int32_t *>(fac + n);
    weights = reinterpret_cast<float *>(top + routed);
    start = reinterpret_cast<int *>(weights + routed);
    act = reinterpret_cast<uint32_t *>(start + p.E);
  }
};

// Expert of entry j, or -1 for one that is not listed: an id outside [0, E), or an expert that an
// earlier slot of the token names too (its weights are added up, see few_weight).  Read through
// L2: k_few_down comes here before it waits for the kernel in front of it.
__device__ __forceinline__ int few_entry(const FewParams &p, const FewLists &l, int j) {
  if (p.logits) return l.top[j];  // routed here
  const int e = __ldcg(p.top + j);
  if (e < 0 || e >= p.E) return -1;
  if (p.given)  // computed experts are distinct
    for (int i = j - j % p.k; i < j; ++i)
      if (__ldcg(p.top + i) == e) return -1;
  return e;
}

// Weight of expert e for the token of its listed entry j.
__device__ __forceinline__ float few_weight(const FewParams &p, const FewLists &l, int j, int e) {
  if (p.logits) return l.weights[j];
  float w = __ldcg(p.weights + j);
  if (p.given)
    for (int i = j + 1; i < j - j % p.k + p.k; ++i)
      if (__ldcg(p.top + i) == e) w += __ldcg(p.weights + i);
  return w;
}

// Entry j of expert e takes place `at` of the lists.
template <class C>
__device__ __forceinline__ void few_put(const FewParams &p, const FewLists &l, int j, int e,
                                        int at) {
  const int t = j / p.k;
  l.ent[at] = (uint32_t)j | ((uint32_t)t << 16);
  // 4-bit products come out halved (see blocks())
  if (C::DOWN)
    l.fac[at] = few_weight(p, l, j, e) * (C::MX4 ? 0.5f : 1.0f);
  else if (C::MX4)
    l.fac[at] = 0.5f * __ldcg(p.xscale + t);
}

// The lists of up to 32 entries, by one warp: places by counting smaller keys (expert, entry).
// One token, E = 128, top-8: 13.7 us, 16.4 with the lists for any number.
template <class C>
__device__ __forceinline__ int few_lists32(const FewParams &p, const FewLists &l, int lane) {
  const int n = p.T * p.k;
  const int e = lane < n ? few_entry(p, l, lane) : -1;
  const uint32_t key = e < 0 ? 0xFFFFFFFFu : (uint32_t)(e << 5 | lane);
  int at = 0, first = 0;
  for (int i = 0; i < n; ++i) {
    const uint32_t o = __shfl_sync(0xFFFFFFFFu, key, i);
    at += o < key;
    first += (o >> 5) < (key >> 5);
  }
  const bool head = e >= 0 && (at - first) % (8 * C::NT) == 0;  // of a group
  const uint32_t head_key = head ? key : 0xFFFFFFFFu;
  int group = 0;
  for (int i = 0; i < n; ++i) group += __shfl_sync(0xFFFFFFFFu, head_key, i) < key;
  if (e >= 0) few_put<C>(p, l, lane, e, at);
  if (head) l.act[group] = (uint32_t)e | ((uint32_t)at << 16);
  const int groups = __popc(__ballot_sync(0xFFFFFFFFu, head));
  const int total = __popc(__ballot_sync(0xFFFFFFFFu, e >= 0));
  if (lane == 0) l.act[groups] = (uint32_t)total << 16;
  return groups;
}

// The experts in use, in increasing order, in groups of up to 8 NT entries, and their entries,
// one group's behind another's.  Returns the number of groups.  Where an expert may have more
// than one group, its entries go by token, so that every CTA makes the same groups: by the tokens
// of each expert as four words of bits (`mask`, in place of the stages, which are not in use yet).
// Where it has one, an entry's place decides only which column of the product it is, and the
// order that atomics give, which is quicker, does not show in any result.
template <class C>
__device__ __forceinline__ int few_lists(const FewParams &p, const FewLists &l, int *s_act,
                                         uint32_t *mask) {
  constexpr int THREADS = C::threads;
  const int n = p.T * p.k, lane = threadIdx.x & 31;
  int *start = l.start;
  if (p.logits) {  // a few tokens: every CTA routes them, a warp each, the first one writes it down
    for (int t = threadIdx.x >> 5; t < p.T; t += THREADS / 32) {
      int e;
      float w;
      bool bad;
      route_token(p.logits + (size_t)t * p.E, p.E, p.k, p.renorm, lane, e, w, bad);
      if (lane < p.k) {
        l.top[t * p.k + lane] = e;
        l.weights[t * p.k + lane] = w;
        if (!C::DOWN && blockIdx.x == 0) {
          p.top_out[t * p.k + lane] = e;
          p.weights_out[t * p.k + lane] = w;
        }
      }
      if (!C::DOWN && blockIdx.x == 0 && bad && lane == 0)
        set_status(p.status, DMOE_STATUS_NONFINITE_LOGITS);
    }
  }
  if (n <= 32) {
    __syncthreads();
    if (threadIdx.x < 32) {
      const int groups = few_lists32<C>(p, l, lane);
      if (lane == 0) *s_act = groups;
    }
    __syncthreads();
    return *s_act;
  }
  const bool by_token = p.T > 8 * C::NT;
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
    if (by_token)
      *reinterpret_cast<uint4 *>(mask + 4 * e) = make_uint4(0u, 0u, 0u, 0u);
    else
      start[e] = 0;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += THREADS) {
    const int e = few_entry(p, l, j);
    if (e < 0) continue;
    if (by_token)
      atomicOr(&mask[4 * e + (j / p.k >> 5)], 1u << (j / p.k & 31));
    else
      atomicAdd(&start[e], 1);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0, na = 0;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      int c = 0;
      if (e < p.E) {
        if (by_token) {
          const uint4 m = *reinterpret_cast<const uint4 *>(mask + 4 * e);
          c = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
        } else {
          c = start[e];
        }
      }
      const int groups = (c + 8 * C::NT - 1) / (8 * C::NT);
      int v = c | (groups << 16);  // both sums at once (at most 4096 each)
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, off);
        if (lane >= off) v += u;
      }
      const int end = carry + (v & 0xFFFF), g1 = na + (v >> 16);
      for (int g = 0; g < groups; ++g)
        l.act[g1 - groups + g] = (uint32_t)e | ((uint32_t)(end - c + 8 * C::NT * g) << 16);
      if (e < p.E) start[e] = by_token ? end - c : end;  // else filled in from the back
      v = __shfl_sync(0xFFFFFFFFu, v, 31);
      carry += v & 0xFFFF;
      na += v >> 16;
    }
    if (lane == 0) {
      l.act[na] = (uint32_t)carry << 16;
      *s_act = na;
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += THREADS) {
    const int e = few_entry(p, l, j);
    if (e < 0) continue;
    int at;
    if (by_token) {
      const int t = j / p.k;
      at = start[e];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t m = mask[4 * e + w], below = (1u << (t & 31)) - 1u;
        at += __popc(w < (t >> 5) ? m : w == (t >> 5) ? m & below : 0u);
      }
    } else {
      at = atomicSub(&start[e], 1) - 1;
    }
    few_put<C>(p, l, j, e, at);
  }
  if (by_token) fence_async_smem();  // the stages are the copies' again
  __syncthreads();
  return *s_act;
}

// A place in a CTA's stream of stages: item (GLU: group, row tile; DOWN: group, part of K), chunk
// of K.  Groups of one expert are items of their own, which different CTAs take: with a CTA
// that went through all groups of its expert, 96 tokens on a skewed router took 105 us, now 92.
struct FewPos {
  int a, b;             // group; tile or part
  int e, n0, cnt;       // expert, first entry, entries (8 NT at most, which its users say again:
                        // the bound keeps loops over them out of the loading warp)
  int chunk, c0, c1;    // chunks [c0, c1) of K
  bool on;
};

template <class C>
struct FewKernel {
  const FewParams &p;
  const FewLists &l;
  uint32_t ring;
  uint64_t *full, *empty;
  volatile int *abort_flag;
  int K, chunks, na;
  int per, step;         // items per group; items from one of this CTA's to its next
  int tile, part;        // DOWN: the CTA's row tile, chunks per part of K

  __device__ __forceinline__ void open(FewPos &q) const {
    if (q.b >= per) {
      const int d = q.b / per;
      q.a += d;
      q.b -= d * per;
    }
    q.on = q.a < na;
    if (!q.on) return;
    const uint32_t g = l.act[q.a];
    q.e = (int)(g & 0xFFFFu);
    q.n0 = (int)(g >> 16);
    q.cnt = (int)(l.act[q.a + 1] >> 16) - q.n0;
    q.c0 = C::DOWN ? q.b * part : 0;
    q.c1 = C::DOWN ? min(chunks, q.c0 + part) : chunks;
    q.chunk = q.c0;
  }
  __device__ __forceinline__ FewPos first(int item) const {
    FewPos q;
    q.a = 0;
    q.b = item;
    open(q);
    return q;
  }
  __device__ __forceinline__ void next(FewPos &q) const {
    if (++q.chunk < q.c1) return;
    q.b += step;
    open(q);
  }
  __device__ __forceinline__ int tile_of(const FewPos &q) const { return C::DOWN ? tile : q.b; }

  // ---- the loading warps (the first one brings the weights) ----

  // Columns of K in the stage, and the bytes that its copies bring.
  __device__ __forceinline__ int width(const FewPos &q) const {
    return min(C::CH, K - q.chunk * C::CH);
  }
  __device__ __forceinline__ uint32_t bytes(const FewPos &q) const {  // that bulk copies bring
    const uint32_t w = width(q), nr = min(q.cnt, 8 * C::NT);
    return p.withheld + C::w_bytes + (C::MX4 ? C::mats * (w >> 7) * kMx4TileBytes : 0) +
           (C::xbulk ? nr * (C::BR * w * 2 + (C::SB ? w >> 3 : 0)) : 0);
  }
  // Weights and their scales (one lane).
  __device__ __forceinline__ void load_w(const FewPos &q, int st) const {
    const uint32_t dst = ring + st * C::stage, bar = smem_u32(&full[st]);
    const int row = C::DOWN ? q.e * p.h + tile * C::outs : q.e * p.f + q.b * C::outs;
    tma_load_3d(dst, &p.tw[0], bar, 0, row, q.chunk * C::slices);
    if (!C::DOWN) tma_load_3d(dst + C::w_mat, &p.tw[1], bar, 0, row, q.chunk * C::slices);
    if (C::MX4) {
      const uint32_t n = (width(q) >> 7) * kMx4TileBytes;
      const size_t at = ((size_t)(row >> 7) * (K >> 7) + q.chunk * (C::CH / 128)) * kMx4TileBytes;
      bulk_load(dst + C::o_sc, p.ws[0] + at, n, bar);
      if (!C::DOWN) bulk_load(dst + C::o_sc + C::sc_mat, p.ws[1] + at, n, bar);
    }
  }
  // Token rows, and their block scales.  A bulk copy is issued lane by lane, so few long rows (512
  // bytes and more of a stage) go as one copy each, more or shorter ones as 16 bytes per lane of four
  // loading warps (the layer of 32 tokens, E = 64, 4-bit weights: 77 us, 93 with one warp's bulk
  // copies).  Columns past K are not loaded and not used.
  __device__ __forceinline__ void load_x(const FewPos &q, int st, int loader, int lane) const {
    const uint32_t dst = ring + st * C::stage;
    const int nr = min(q.cnt, 8 * C::NT), w = width(q);
    const size_t k0 = (size_t)q.chunk * C::CH;
    if constexpr (C::xbulk) {
      const uint32_t bar = smem_u32(&full[st]);
      for (int n = lane; n < nr; n += 32) {
        const uint32_t v = l.ent[q.n0 + n], d = dst + C::o_x + n * C::x_row;
        const size_t at = (size_t)(C::DOWN ? v & 0xFFFFu : v >> 16) * K + k0;
        bulk_load(d, p.xin + at, w * 2, bar);
        if (C::BR == 2) bulk_load(d + 8 * C::NT * C::x_row, p.xlo + at, w * 2, bar);
        if (C::SB) bulk_load(dst + C::o_sb + n * C::sb_row, p.xscale + (at >> 5), w >> 3, bar);
      }
    } else {
      constexpr int segs = C::CH / 8;
#pragma unroll 4
      for (int i = 32 * loader + lane; i < nr * segs; i += 32 * C::loaders) {
        const int n = i / segs, seg = i % segs;
        if (seg * 8 >= w) continue;
        const uint32_t v = l.ent[q.n0 + n];
        const size_t at = (size_t)(C::DOWN ? v & 0xFFFFu : v >> 16) * K + k0 + seg * 8;
        const uint32_t d = dst + C::o_x + n * C::x_row + seg * 16;
        cp16(d, p.xin + at);
        if (C::BR == 2) cp16(d + 8 * C::NT * C::x_row, p.xlo + at);
      }
      if constexpr (C::SB) {
        constexpr int sbs = C::CH / 128;  // four blocks each
        for (int i = 32 * loader + lane; i < nr * sbs; i += 32 * C::loaders) {
          const int n = i / sbs, seg = i % sbs;
          if (seg * 128 >= w) continue;
          const size_t row = l.ent[q.n0 + n] & 0xFFFFu;
          cp16(dst + C::o_sb + n * C::sb_row + seg * 16,
               p.xscale + row * (K >> 5) + (k0 >> 5) + seg * 4);
        }
      }
      cp_arrive(&full[st]);
    }
  }

  // pre: the weights of the first stages are loaded before the wait for the earlier kernels.
  __device__ __forceinline__ void produce(int item0, bool pre, int loader, int lane) const {
    FewPos q = first(item0), w = q;
    if (pre) {
      for (int st = 0; st < C::P && w.on; ++st) {
        if (loader == 0 && lane == 0) {
          mbar_arrive_expect_tx(&full[st], bytes(w));
          load_w(w, st);
        }
        next(w);
      }
      pdl_wait();
    }
    int st = 0;
    uint32_t phase = 0;
    long long issued = 0;
    while (q.on) {
      if (issued >= C::P) {
        int good = 1;
        if (lane == 0)
          good = mbar_wait(&empty[st], phase ^ 1u, p.status, abort_flag, p.wait_cycles) ? 1 : 0;
        if (!__shfl_sync(0xFFFFFFFFu, good, 0)) break;
      }
      if (loader == 0 && lane == 0 && !(pre && issued < C::P)) {
        mbar_arrive_expect_tx(&full[st], bytes(q));
        load_w(q, st);
      }
      if (C::xbulk) __syncwarp();  // the expected bytes are set before any of them can arrive
      load_x(q, st, loader, lane);
      ++issued;
      next(q);
      if (++st == C::P) {
        st = 0;
        phase ^= 1u;
      }
    }
    if (lane == 0)  // every copy has landed before the CTA's memory is given up
      for (long long i = (issued > C::P ? issued - C::P : 0); i < issued; ++i)
        mbar_wait_plain(&full[i % C::P], (uint32_t)((i / C::P) & 1), p.wait_cycles);
  }

  // ---- the multiplying warps ----

  // Four blocks (128 columns, a slice) of a warp's 16 rows times the token tiles, added to acc
  // times two (the entries' factors halve them): 2^(s - 126) has the exponent field s + 1, which is
  // right for every s up to 253, 0 included.  LARGE: for scale bytes above 127 in the stage (254
  // and 255, NaN, among them), the factor 2^(s - 127) made case by case.  wl: this lane's word of
  // row lane / 4 in the slice; xb, sb: its token row and the token scales.
  template <bool LARGE>
  __device__ __forceinline__ void blocks(uint32_t wl, uint32_t xb, uint32_t sb, uint32_t sca,
                                         uint32_t scb, int ntl, const float (&zero)[4],
                                         float (&acc)[C::NT][4]) const {
    constexpr int up = C::DOWN ? 8 * C::row_b : C::w_mat;  // from row i to row i + 8
    constexpr bool ahead = C::SB && C::NT <= 2;  // a slice's token scales fit in registers
    uint32_t s0[C::NT][4], s1[C::NT][4];
    if constexpr (ahead) {
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) {
        if (nt > 0 && nt >= ntl) break;
        lds128(s0[nt], sb + nt * 8 * C::sb_row);
        lds128(s1[nt], sb + (nt * 8 + 1) * C::sb_row);
      }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t wa = wl ^ (b << 4);
      uint32_t lo[4], hi[4];
      mx4_unpack8(lds32(wa), lo);
      mx4_unpack8(lds32(wa + up), hi);
      float fa, fb;
      if (LARGE) {
        fa = mx4_scale_value((sca >> (8 * b)) & 0xFFu);
        fb = mx4_scale_value((scb >> (8 * b)) & 0xFFu);
      } else {  // sca, scb: the bytes plus one
        fa = __uint_as_float((b < 3 ? sca << (23 - 8 * b) : sca >> 1) & 0x7F800000u);
        fb = __uint_as_float((b < 3 ? scb << (23 - 8 * b) : scb >> 1) & 0x7F800000u);
      }
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) {
        if (nt > 0 && nt >= ntl) break;
        uint32_t x[4];
        lds128(x, xb + nt * 8 * C::x_row + b * 64);
        float h[4], c[4];
        mma_f16(h, lo[0], hi[0], lo[1], hi[1], x[0], x[1], zero);
        mma_f16(c, lo[2], hi[2], lo[3], hi[3], x[2], x[3], h);
        if constexpr (C::SB) {
          if constexpr (!ahead) {
            s0[nt][b] = lds32(sb + nt * 8 * C::sb_row + 4 * b);
            s1[nt][b] = lds32(sb + (nt * 8 + 1) * C::sb_row + 4 * b);
          }
          const float u = __uint_as_float(s0[nt][b]), v = __uint_as_float(s1[nt][b]);
          c[0] *= u;
          c[1] *= v;
          c[2] *= u;
          c[3] *= v;
        }
        if (LARGE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i] += c[i];
        }
        acc[nt][0] = fmaf(c[0], fa, acc[nt][0]);
        acc[nt][1] = fmaf(c[1], fa, acc[nt][1]);
        acc[nt][2] = fmaf(c[2], fb, acc[nt][2]);
        acc[nt][3] = fmaf(c[3], fb, acc[nt][3]);
      }
    }
  }

  // tile0: the item's first row within its 128-row scale tile.
  __device__ __forceinline__ void multiply(const FewPos &q, int tile0, int st, int r, int s,
                                           int lane, const float (&zero)[4],
                                           float (&acc)[C::NT][4]) const {
    const int left = K - q.chunk * C::CH - s * C::KU;
    if (left <= 0) return;
    const uint32_t base = ring + st * C::stage;
    const int ntl = (min(q.cnt, 8 * C::NT) + 7) >> 3;
    if constexpr (C::MX4) {
      const int g = lane >> 2, t = lane & 3;
      const int row = r * (C::DOWN ? 16 : 8) + g;  // of the box
      constexpr int js = C::KU / 128;
      // this lane's word of block 0 (an exclusive or with 16 b gives block b's: the boxes are
      // swizzled by row, 64-byte rows every second one)
      const uint32_t w = base + s * (C::KU / C::SC) * C::rows_m * C::row_b + row * C::row_b +
                         ((C::WIDE ? row & 7 : (row >> 1) & 3) << 4) + 4 * t;
      auto wj = [&](int j) {  // 128 columns on
        return C::WIDE ? (w + (j >> 1) * C::rows_m * 128) ^ ((j & 1) << 6) : w + j * C::rows_m * 64;
      };
      // the tile's rows start at a multiple of 8: rows 0..7 and 8..15 stay in one 32-row group
      const int r128 = tile0 + row;
      const uint32_t sw =
          base + C::o_sc + s * js * kMx4TileBytes + (r128 & 31) * 16 + (r128 >> 5) * 4;
      constexpr int sup = C::DOWN ? 128 : C::sc_mat;
      const uint32_t xb = base + C::o_x + g * C::x_row + (s * C::KU + 8 * t) * 2;
      const uint32_t sb = base + C::o_sb + 2 * t * C::sb_row + s * (C::KU / 8);
      uint32_t sca[js], scb[js], any = 0u;
#pragma unroll
      for (int j = 0; j < js; ++j) {  // (the slice past an odd end holds an earlier stage's)
        sca[j] = lds32(sw + j * kMx4TileBytes);
        scb[j] = lds32(sw + j * kMx4TileBytes + sup);
        any |= sca[j] | scb[j];
      }
      if (__any_sync(0xFFFFFFFFu, any & 0x80808080u)) {
#pragma unroll
        for (int j = 0; j < js; ++j)
          if (j * 128 < left)
            blocks<true>(wj(j), xb + j * 256, sb + j * 16, sca[j], scb[j], ntl, zero, acc);
      } else {
#pragma unroll
        for (int j = 0; j < js; ++j)
          if (j * 128 < left)
            blocks<false>(wj(j), xb + j * 256, sb + j * 16, sca[j] + 0x01010101u,
                          scb[j] + 0x01010101u, ntl, zero, acc);
      }
    } else {
      const int ar = lane & 15;
      const uint32_t wr = base + s * C::rows_m * 128 +
                          (C::DOWN ? (r * 16 + ar) * 128
                                   : (ar >> 3) * C::w_mat + (r * 8 + (ar & 7)) * 128);
      const uint32_t xb = base + C::o_x + (lane & 7) * C::x_row + (s * C::KU + (lane >> 3) * 8) * 2;
#pragma unroll
      for (int kk = 0; kk < 4; kk += 2) {
        uint32_t a0[4], a1[4];
        ldsm4(a0, wr + (((2 * kk + (lane >> 4)) ^ (ar & 7)) << 4));
        ldsm4(a1, wr + (((2 * kk + 2 + (lane >> 4)) ^ (ar & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          if (nt > 0 && nt >= ntl) break;
#pragma unroll
          for (int br = 0; br < C::BR; ++br) {
            uint32_t x[4];
            ldsm4(x, xb + (br * 8 * C::NT + nt * 8) * C::x_row + kk * 32);
            mma_bf16(acc[nt], a0, x[0], x[1]);
            mma_bf16(acc[nt], a1, x[2], x[3]);
          }
        }
      }
    }
  }

  // Among the multiplying warps.
  __device__ __forceinline__ static void sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * C::warps) : "memory");
  }

  // done(pos, nt, sums): called by the first slice's warps with the sums of token tile nt over
  // the item's K: words 2 i + c are row lane / 4 + 8 i of the warp's 16 and token
  // 8 nt + 2 (lane % 4) + c; end(pos): by all multiplying threads after them.
  template <class Done, class End>
  __device__ __forceinline__ void consume(int item0, float *red, int warp, int lane, Done done,
                                          End end) const {
    const int r = warp / C::S, s = warp % C::S;
    float acc[C::NT][4];
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
    // four zero registers, kept: the accumulator that each block's first product starts from
    float zero[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("mov.f32 %0, 0f00000000;" : "=f"(zero[i]));
    int st = 0;
    uint32_t phase = 0;
    bool good = true;  // until a wait expires
    int tile0 = 0;
    for (FewPos q = first(item0); q.on; next(q)) {
      if (C::MX4 && q.chunk == q.c0) tile0 = (tile_of(q) * C::outs) & 127;
      if (!mbar_wait(&full[st], phase, p.status, abort_flag, p.wait_cycles)) {
        *abort_flag = 1;
        good = false;
      }
      multiply(q, tile0, st, r, s, lane, zero, acc);
      __syncwarp();
      // a stage that was not waited for to the end, and those behind it, are not given back: their
      // copies may be under way, and the loading warps then stop at the abort flag
      if (lane == 0 && good) mbar_arrive(&empty[st]);
      if (++st == C::P) {
        st = 0;
        phase ^= 1u;
      }
      if (q.chunk < q.c1 - 1) continue;
      const int ntl = (min(q.cnt, 8 * C::NT) + 7) >> 3;
      // slices past the first hand over their sums
      float4 *part4 = reinterpret_cast<float4 *>(red) + r * C::NT * 32 + lane;
      if (C::S > 1) {
        if (s > 0) {
#pragma unroll
          for (int nt = 0; nt < C::NT; ++nt)
            if (nt < ntl)
              part4[((s - 1) * C::R * C::NT + nt) * 32] =
                  make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
        }
        sync();
      }
      if (s == 0) {
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          if (nt < ntl) {
#pragma unroll
            for (int o = 0; o < C::S - 1; ++o) {
              const float4 v = part4[(o * C::R * C::NT + nt) * 32];
              acc[nt][0] += v.x;
              acc[nt][1] += v.y;
              acc[nt][2] += v.z;
              acc[nt][3] += v.w;
            }
            done(q, nt, r, acc[nt]);
          }
        }
      }
      end(q);
      if (C::S > 1) sync();  // the partial sums are read before they are written again
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
    }
  }
};

// The CTA's dynamic shared memory from the first 1024-byte boundary on; barriers set up (the
// caller synchronises the CTA before they are used).
template <class C>
__device__ __forceinline__ uint8_t *few_setup(uint8_t *raw, uint64_t *&full, uint64_t *&empty,
                                              volatile int *&abort_flag) {
  uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  full = reinterpret_cast<uint64_t *>(smem + C::o_bars);
  empty = full + C::P;
  abort_flag = reinterpret_cast<volatile int *>(smem + C::o_bars + 120);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::P; ++i) {
      mbar_init(&full[i], C::xbulk ? 1 : 1 + 32 * C::loaders);  // bulk bytes, and the lanes' own copies
      mbar_init(&empty[i], C::warps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  return smem;
}

template <class C>
__global__ void __launch_bounds__(C::threads, C::min_ctas)
    k_few_glu(const __grid_constant__ FewParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ int s_act;
  uint64_t *full, *empty;
  volatile int *abort_flag;
  uint8_t *smem = few_setup<C>(raw, full, empty, abort_flag);
  const FewLists l(smem + C::o_lists, p);
  pdl_wait();
  pdl_trigger();
  const int na = few_lists<C>(p, l, &s_act, reinterpret_cast<uint32_t *>(smem));
  const FewKernel<C> k{p, l, smem_u32(smem), full, empty, abort_flag, p.h,
                       (p.h + C::CH - 1) / C::CH, na, p.f / C::outs, (int)gridDim.x, 0, 0};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp >= C::warps) {
    k.produce(blockIdx.x, false, warp - C::warps, lane);
    return;
  }
  float *hb = reinterpret_cast<float *>(smem + C::o_hbuf);
  const int g = lane >> 2, t2 = 2 * (lane & 3);
  k.consume(
      blockIdx.x, reinterpret_cast<float *>(smem + C::o_red), warp, lane,
      [&](const FewPos &q, int nt, int r, const float (&v)[4]) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // gate v[c], up v[2 + c] of one column and token n
          const int n = 8 * nt + t2 + c, col = r * 8 + g;
          if (n >= q.cnt) continue;
          const uint32_t en = l.ent[q.n0 + n];
          if constexpr (C::MX4) {
            const float xs = l.fac[q.n0 + n];
            hb[n * C::hrow + col] = silu_f(v[c] * xs) * (v[2 + c] * xs);
          } else {
            const float hv = silu_f(v[c]) * v[2 + c];
            const size_t at = (size_t)(en & 0xFFFFu) * p.f + q.b * C::outs + col;
            // the upper part stops at bf16's largest value: up to fp32's the lower part holds the
            // rest, and of an inf or NaN the lower part is one
            const __nv_bfloat16 hi = __float2bfloat16(fminf(fmaxf(hv, -kMaxBf16), kMaxBf16));
            p.hout[at] = __bfloat16_as_ushort(hi);
            p.hlo[at] = __bfloat16_as_ushort(__float2bfloat16(hv - __bfloat162float(hi)));
          }
        }
      },
      [&](const FewPos &q) {
        if constexpr (C::MX4) {  // blocks of 32 columns to fp16, a warp each
          k.sync();
          const int nr = min(q.cnt, 8 * C::NT);
          for (int i = warp; i < nr * (C::outs / 32); i += C::warps) {
            const int n = i / (C::outs / 32), b = i % (C::outs / 32);
            const float hv = hb[n * C::hrow + b * 32 + lane];
            const int es =
                f16_block_exp(__reduce_max_sync(0xFFFFFFFFu, finite_abs(__float_as_uint(hv))));
            const size_t at =
                (size_t)(l.ent[q.n0 + n] & 0xFFFFu) * p.f + q.b * C::outs + b * 32 + lane;
            p.hout[at] = __half_as_ushort(__float2half_rn(hv * pow2(es)));
            if (lane == 0) p.hscale[at >> 5] = pow2(-es);
          }
          if (C::S == 1) k.sync();  // hb is read before the next tile writes it
        }
      });
}

// A cluster of G CTAs shares a row tile, each with every G-th of the groups or parts of K; their
// sums are added in rank order through distributed shared memory.
template <class C>
__global__ void __launch_bounds__(C::threads, C::min_ctas)
    k_few_down(const __grid_constant__ FewParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ int s_act;
  uint64_t *full, *empty;
  volatile int *abort_flag;
  uint8_t *smem = few_setup<C>(raw, full, empty, abort_flag);
  const FewLists l(smem + C::o_lists, p);
  float *ysum = reinterpret_cast<float *>(smem + C::o_lists + few_list_bytes(p));
  // Before the wait for k_few_glu: only what was complete when that kernel passed its own
  // wait (it lets this one start after that): the routing, and the caller's W2.
  const int na = few_lists<C>(p, l, &s_act, reinterpret_cast<uint32_t *>(smem));
  const int G = p.groups, rank = (int)cluster_ctarank();
  const int chunks = (p.f + C::CH - 1) / C::CH;
  const FewKernel<C> k{p, l, smem_u32(smem), full, empty, abort_flag, p.f, chunks, na,
                       p.kparts, G, (int)blockIdx.x / G, (chunks + p.kparts - 1) / p.kparts};
  for (int i = threadIdx.x; i < p.T * C::yrow; i += C::threads) ysum[i] = 0.0f;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp >= C::warps) {
    k.produce(rank, true, warp - C::warps, lane);
  } else {
    pdl_wait();
    pdl_trigger();
    const int g = lane >> 2, t2 = 2 * (lane & 3);
    k.consume(
        rank, reinterpret_cast<float *>(smem + C::o_red), warp, lane,
        [&](const FewPos &q, int nt, int r, const float (&v)[4]) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int n = 8 * nt + t2 + c;
            if (n >= q.cnt) continue;
            const uint32_t en = l.ent[q.n0 + n];  // an expert's entries: distinct tokens
            const float w = l.fac[q.n0 + n];
            float *y = ysum + (en >> 16) * C::yrow + r * 16 + g;
            y[0] = fmaf(w, v[c], y[0]);
            y[8] = fmaf(w, v[2 + c], y[8]);
          }
          __syncwarp();  // another lane may add to these sums for the next expert
        },
        [](const FewPos &) {});
  }
  __syncwarp();
  cluster_sync_all();
  const int h0 = k.tile * C::outs;
  const uint32_t mine = smem_u32(ysum);
  for (int i = rank * C::threads + threadIdx.x; i < p.T * (C::outs / 2); i += G * C::threads) {
    const int t = i / (C::outs / 2), c = 2 * (i % (C::outs / 2));
    float a = 0.0f, b = 0.0f;
    for (int o = 0; o < G; ++o) {
      float u, v;
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                   : "=f"(u), "=f"(v)
                   : "r"(mapa_shared(mine, o) + (uint32_t)((t * C::yrow + c) * 4))
                   : "memory");
      a += u;
      b += v;
    }
    *reinterpret_cast<uint32_t *>(p.y + (size_t)t * p.h + h0 + c) = pack_bf16x2(a, b);
  }
  cluster_sync_all();  // no CTA leaves while another reads its sums
}

// ---- host side ---------------------------------------------------------------------------------

// Weights [rows, K] as slices of SC columns: {SC, rows, K / SC}; a box is a tile's rows of all the
// slices of a stage (slices past K read zeros).
template <class C>
bool few_map(CUtensorMap *m, const void *ptr, long long rows, int K) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t pitch = (cuuint64_t)K * (C::MX4 ? 1 : 4) / 2;
  const cuuint32_t dim0 = C::MX4 ? C::row_b : 64;  // bytes, or bf16
  cuuint64_t dims[3] = {dim0, (cuuint64_t)rows, (cuuint64_t)(K / C::SC)};
  cuuint64_t strides[2] = {pitch, (cuuint64_t)C::row_b};
  cuuint32_t box[3] = {dim0, (cuuint32_t)C::rows_m, (cuuint32_t)C::slices}, estr[3] = {1, 1, 1};
  return enc(m, C::MX4 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             C::row_b == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of `smem` bytes that the device holds at once (1 KB of each is the system's).
template <class C>
int few_places(size_t smem) {
  const int n = (int)(228 * 1024 / (smem + 1024 + 64));
  return device_sm_count() * (n < 1 ? 1 : n < C::min_ctas ? n : C::min_ctas);
}

// Limit of the kernel's waits, and what its stages wait for in vain.
void few_limits(FewParams &p) {
  const int inject = take_inject_stall();
  p.withheld = inject ? 16u : 0u;
  p.wait_cycles = inject ? kInjectedWaitCycles : kWaitCycles;
}

template <class C>
cudaError_t launch_few_glu(FewParams p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_few_glu<C>, done, kFewSmem);
  if (e != cudaSuccess) return e;
  const long long ef = (long long)p.E * p.f;
  if (!few_map<C>(&p.tw[0], p.w1.data, ef, p.h) || !few_map<C>(&p.tw[1], p.w3.data, ef, p.h))
    return cudaErrorInvalidValue;
  few_limits(p);
  p.ws[0] = static_cast<const uint8_t *>(p.w1.scales);
  p.ws[1] = static_cast<const uint8_t *>(p.w3.scales);
  const size_t smem = C::fixed + few_list_bytes(p);
  const long long n = (long long)p.T * p.k;
  const long long items = ((n < p.E ? n : p.E) + n / (8 * C::NT)) * (p.f / C::outs);
  const long long ctas = few_places<C>(smem);
  return launch_pdl(k_few_glu<C>, (int)(items < ctas ? items : ctas), C::threads, smem, st, p);
}

template <class C>
cudaError_t launch_few_down(FewParams p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_few_down<C>, done, kFewSmem);
  if (e != cudaSuccess) return e;
  if (!few_map<C>(&p.tw[0], p.w2.data, (long long)p.E * p.h, p.f)) return cudaErrorInvalidValue;
  few_limits(p);
  p.tw[1] = p.tw[0];
  p.ws[0] = p.ws[1] = static_cast<const uint8_t *>(p.w2.scales);
  const size_t smem = C::fixed + few_list_bytes(p) +
                      (size_t)p.T * C::yrow * sizeof(float);
  const long long n = (long long)p.T * p.k;
  const int experts = (int)(n < p.E ? n : p.E);
  const int tiles = p.h / C::outs;
  // the experts are spread over up to eight CTAs per row tile until there is one CTA for each
  // place on the SMs; with fewer experts than that, K is cut into parts as well (whole chunks)
  const int places = few_places<C>(smem);
  int G = 1;
  while (G < 8 && tiles * G * 2 <= places) G *= 2;
  const int chunks = (p.f + C::CH - 1) / C::CH;
  int parts = 1;
  while (parts * 2 <= chunks &&
         (experts * parts < G || (experts * parts < 4 * G && chunks >= 16 * parts)))
    parts *= 2;  // a long K in parts of eight chunks and more evens out the CTAs of a tile, too
  const int part = (chunks + parts - 1) / parts;
  p.kparts = (chunks + part - 1) / part;  // no empty part
  while (G > 1 && experts * p.kparts < G) G /= 2;
  p.groups = G;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * G);
  cfg.blockDim = dim3(C::threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = DMOE_PDL;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = G;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_few_down<C>, p);
}

template <class G, class D>
cudaError_t launch_few_pair(const FewParams &p, const FewParams &d, cudaStream_t st) {
  const cudaError_t e = launch_few_glu<G>(p, st);
  return e == cudaSuccess ? launch_few_down<D>(d, st) : e;
}

// Shape of a product: R row tiles x S slices of KU columns, P stages, CTAs per SM.
template <int R_, int S_, int KU_, int P_, int CTAS_>
struct FewShape {
  static constexpr int R = R_, S = S_, KU = KU_, P = P_, CTAS = CTAS_;
};

// 4-bit weights whose rows are whole 128-byte pieces (K a multiple of 256) are fetched in boxes of
// 128-byte rows, others in boxes of 64-byte rows.
template <bool MX4, int NT, class G, class D>
cudaError_t launch_few_shapes(const FewParams &p, const FewParams &d, cudaStream_t st) {
  using G0 = FewCfg<MX4, false, NT, G::R, G::S, G::KU, G::P, G::CTAS>;
  using D0 = FewCfg<MX4, true, NT, D::R, D::S, D::KU, D::P, D::CTAS>;
  if constexpr (MX4) {
    constexpr bool gw = G::KU % 256 == 0 || G::S % 2 == 0, dw = D::KU % 256 == 0 || D::S % 2 == 0;
    using G1 = FewCfg<MX4, false, NT, G::R, G::S, G::KU, G::P, G::CTAS, true>;
    using D1 = FewCfg<MX4, true, NT, D::R, D::S, D::KU, D::P, D::CTAS, true>;
    static_assert(gw && dw && G::KU == 256 && D::KU == 256, "slices of 256 columns");
    if (p.h % 256 == 0)
      return p.f % 256 == 0 ? launch_few_pair<G1, D1>(p, d, st) : launch_few_pair<G1, D0>(p, d, st);
    return p.f % 256 == 0 ? launch_few_pair<G0, D1>(p, d, st) : launch_few_pair<G0, D0>(p, d, st);
  } else {
    return launch_few_pair<G0, D0>(p, d, st);
  }
}

}  // namespace

// The shapes of the first (G) and second (D) product, by weights (M: 4 bits, B: bf16) and token
// tiles of 8.
using MG1 = FewShape<4, 2, 256, 3, 2>;
using MD1 = FewShape<4, 2, 256, 3, 2>;
using MG2 = FewShape<4, 2, 256, 2, 2>;
using MD2 = FewShape<4, 2, 256, 2, 2>;
using MG4 = FewShape<8, 1, 256, 2, 2>;
using MD4 = FewShape<4, 2, 256, 2, 1>;
using BG1 = FewShape<1, 8, 64, 4, 2>;
using BD1 = FewShape<2, 4, 64, 4, 2>;
using BG2 = FewShape<2, 4, 64, 4, 2>;
using BD2 = FewShape<2, 4, 64, 3, 2>;
using BG4 = FewShape<4, 2, 64, 3, 2>;
using BD4 = FewShape<4, 2, 64, 3, 2>;
using BG8 = FewShape<8, 2, 64, 3, 1>;
using BD8 = FewShape<8, 1, 64, 3, 1>;

// Token tiles that a call's experts are given at a time.  An expert with more tokens reads its
// weights again (from L2); one with fewer still has the larger tile's stages, fewer CTAs per SM
// and rows to load.  The host knows T and the mean number of tokens per expert, mean = T k / E, not
// the routing.
//   4 bits: one tile up to 16 tokens (16 tokens, E = 64, top-8: 61 us, 68 with two), two up to a
//     mean of 16 (32 tokens, E = 64: 77 us, 92 with one and 93 with four), then four (128 tokens,
//     E = 8, top-2, hidden 4096, ffn 14336: 728 us, 785 with two)
//   bf16: up to 32 tokens one (32, E = 64, top-8: 136 us, 174 with two), from a mean of 4 on two
//     (24, E = 16, top-4: 79 us, 86 with one); beyond that four, which a skewed router needs (96
//     tokens, skewed: 92 us, 196 with two; 128 over E = 256: 311 us, 436 with two); from a mean of
//     16 on eight (128 over E = 8: 737 us, 984 with four)
static int few_token_tiles(bool mx4, int T, int k, int E) {
  const long long n = (long long)T * k;
  if (T <= 8) return 1;
  if (mx4) return T <= 16 ? 1 : n < 16LL * E ? 2 : 4;
  if (n >= 16LL * E) return 8;
  return T > 32 ? 4 : n <= 4LL * E ? 1 : 2;
}

cudaError_t launch_few(const FewParams &p_in, const uint16_t *logits, bool renorm, int32_t *top,
                       float *weights, int32_t *status, cudaStream_t st) {
  FewParams p = p_in;
  p.status = status;
  p.renorm = renorm;
  const bool mx4 = p.w1.scales != nullptr;
  cudaError_t e = cudaSuccess;
  // Up to 8 tokens (one per warp) and bf16 weights the two product kernels route the tokens
  // themselves, in every CTA, instead of waiting for a kernel that does: one launch less (7.9 us of
  // host time a call, 10.1 with it; one token, E = 128, top-8 takes 13.7 us in all).  With more
  // experts than a warp keeps in registers each CTA would read the logits again for every pick
  // (hidden 1536, ffn 256, top-8: one token at E = 1024 42.8 us, 27.2 with the kernel; at E = 512
  // 24.5 and 18.0; with top-2 12.0 and 14.2).
  if (logits && !mx4 && p.T <= 8 && p.E <= kRouteRegs * 32) {
    p.logits = logits;
    p.top_out = top;
    p.weights_out = weights;
  } else {
    e = launch_pdl(k_few_route, p.T, mx4 ? 32 * kRouteWarps : 32, 0, st, logits, p.E, p.k,
                   renorm ? 1 : 0, p.h, top, weights, status, static_cast<const uint4 *>(p.x),
                   reinterpret_cast<uint4 *>(p.x16), p.x16scale);
  }
  if (e != cudaSuccess) return e;
  FewParams d = p;
  p.xin = mx4 ? p.x16 : static_cast<const uint16_t *>(p.x);
  p.xscale = p.x16scale;
  d.xin = p.hout;
  d.xlo = p.hlo;
  d.xscale = p.hscale;
  const int nt = few_token_tiles(mx4, p.T, p.k, p.E);
  if (mx4) {
    if (nt == 1) return launch_few_shapes<true, 1, MG1, MD1>(p, d, st);
    if (nt == 2) return launch_few_shapes<true, 2, MG2, MD2>(p, d, st);
    return launch_few_shapes<true, 4, MG4, MD4>(p, d, st);
  }
  if (nt == 1) return launch_few_shapes<false, 1, BG1, BD1>(p, d, st);
  if (nt == 2) return launch_few_shapes<false, 2, BG2, BD2>(p, d, st);
  if (nt == 4) return launch_few_shapes<false, 4, BG4, BD4>(p, d, st);
  return launch_few_shapes<false, 8, BG8, BD8>(p, d, st);
}

}  // namespace dmoe
