// few.cu -- the whole layer for a few tokens (T <= DMOE_FEW_MAX_TOKENS): the decode step of a
// model whose prompts run through dmoe_forward or dmoe_mx4_forward.
//   k_few_route  top-k of the logits and the softmax weights (and x in fp16, for 4-bit weights)
//   k_few_glu    H_j = silu(W1_e x_t) * (W3_e x_t) per entry j = t*k + s
//   k_few_down   y_t = sum_s w_ts W2_e H_j
// With so few tokens the layer is bound by reading the weights of the experts in use once:
// nothing is padded, x and H are read from L2, and every kernel is a stream of weight tiles.
//
// A CTA multiplies tiles of 16 R weight rows (8 R gate and 8 R up rows in k_few_glu) by the
// columns of up to 8 NT of the expert's tokens.  Its warps are R row tiles x S slices of K; a
// stage of the ring holds each warp's 16 rows x KU columns, fetched by the warp itself with
// 16-byte cp.async (a lane group per 128-byte line), and the tokens' S * KU columns.  The
// products run on mma.sync m16n8k16 with the weights as the 16-row operand: a tile of 16 rows
// costs one instruction per 16 K and 8 tokens, far below the tensor rate at these sizes; what
// counts is that 40 KB and more per SM are in flight at all times, so the ring runs on from one
// tile into the next, across experts.  tcgen05 would need 128-row tiles and a full shared-memory
// operand for 1 to 8 columns, and the 4-bit weights converted into it.
//   bf16 weights: x as bf16; H as the sum of two bf16 (16 bits), multiplied in turn.
//   4-bit weights: e2m1 -> fp16 is exact, so x and H go in fp16 under a power-of-two scale per
//     row and 32 columns (11 bits at the block's largest, exact for x down to 2^-29 of it);
//     the 32 products of a block are summed first, then scaled by the block's two scales.
// The few partial sums over S and over the experts of a token are added in a fixed order.
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "mx4.cuh"
#include "route_key.cuh"

namespace dmoe {

namespace {

constexpr int kRouteWarps = 8;
constexpr int kMaxSmem = 227 * 1024;

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
// the map's routing does; lane l holds experts l, l + 32, ...  The softmax terms use expf.
__device__ __forceinline__ void route_token(const uint16_t *__restrict__ row, int E, int k,
                                            bool renorm, int32_t *__restrict__ top,
                                            float *__restrict__ weights, int32_t *status,
                                            int lane) {
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
    top[lane] = e;
    weights[lane] = expf(v - m) / sum;
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) set_status(status, DMOE_STATUS_NONFINITE_LOGITS);
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

// One CTA per token: warp 0 routes (or checks) it, the others convert its row of x to fp16 when
// the weights have four bits.
__global__ void __launch_bounds__(32 * kRouteWarps)
    k_few_route(const uint16_t *__restrict__ logits, int E, int k, int renorm, int h,
                int32_t *__restrict__ top, float *__restrict__ weights, int32_t *status,
                const uint4 *__restrict__ x, uint4 *__restrict__ x16, float *__restrict__ xs) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t t = blockIdx.x;
  if (warp == 0) {
    if (logits)
      route_token(logits + t * E, E, k, renorm != 0, top + t * k, weights + t * k, status, lane);
    else
      check_token(top + t * k, E, k, status, lane);
  } else if (x16) {
    const int vpr = h >> 3;  // h is a multiple of 128: whole lane groups of four per block
    for (int v = threadIdx.x - 32; v < vpr; v += 32 * (kRouteWarps - 1)) {
      const uint4 q = __ldg(x + t * vpr + v);
      const uint32_t *w = reinterpret_cast<const uint32_t *>(&q);
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m = max(m, max(finite_abs(w[i] << 16), finite_abs(w[i] & 0xFFFF0000u)));
      const unsigned grp = 0xFu << (lane & 28);  // the block's four lanes
      m = max(m, __shfl_xor_sync(grp, m, 1));
      m = max(m, __shfl_xor_sync(grp, m, 2));
      const int es = f16_block_exp(m);
      const float f = pow2(es);
      uint4 o;
      uint32_t *ow = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
      for (int i = 0; i < 4; ++i) ow[i] = pack_f16x2(bf16_lo(w[i]) * f, bf16_hi(w[i]) * f);
      x16[t * vpr + v] = o;
      if ((lane & 3) == 0) xs[t * (h >> 5) + (v >> 2)] = pow2(-es);
    }
  }
}

// ---- the product kernels -----------------------------------------------------------------------

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shape of a variant: MX4 weights in four bits; NT tiles of 8 tokens; R x S warps; P stages;
// DOWN the second product.  BR: copies of the token rows (two: H's upper and lower bf16).
template <bool MX4_, bool DOWN_, int NT_, int R_, int S_, int P_>
struct FewCfg {
  static constexpr bool MX4 = MX4_, DOWN = DOWN_;
  static constexpr int NT = NT_, R = R_, S = S_, P = P_;
  static constexpr int warps = R * S, threads = 32 * warps;
  static constexpr int min_ctas = threads == 256 ? 2 : 1;
  static constexpr int KU = MX4 ? 128 : 64;  // columns per warp and stage
  static constexpr int CH = S * KU;          // columns per stage
  static constexpr int BR = (DOWN && !MX4) ? 2 : 1;
  static constexpr int w_warp = MX4 ? 1024 : 2048;  // weight bytes per warp and stage
  static constexpr int sc_warp = MX4 ? 256 : 0;     // weight scales: 16 bytes per row
  // token rows: a stride that is 16 (ldmatrix) or 64 (16-byte loads of 4 lanes a row) bytes off
  // a multiple of 128 keeps the reads free of bank conflicts
  static constexpr int x_row = CH * 2 + (MX4 ? 64 : 16);
  static constexpr int x_bytes = BR * 8 * NT * x_row;
  static constexpr int sb_bytes = MX4 ? (CH / 32) * 8 * NT * 4 : 0;  // token scales [block][token]
  static constexpr int o_sc = warps * w_warp, o_x = o_sc + warps * sc_warp, o_sb = o_x + x_bytes;
  static constexpr int stage = o_sb + sb_bytes;
  // partial sums of every warp; with two slices of K the first slice's warps add theirs to the
  // second's in place
  static constexpr int red_s = S == 2 ? 1 : S;
  static constexpr int red = R * red_s * NT * 512;
  static constexpr int rows = 16 * R;           // weight rows per tile
  static constexpr int outs = DOWN ? rows : rows / 2;  // output columns per tile
  static_assert(stage % 128 == 0 && o_x % 16 == 0 && x_row % 16 == 0, "alignment");
};

// Bytes of the expert lists: counts / starts [E + 1] int, active experts and entries (uint16).
__host__ __device__ inline size_t few_list_bytes(int E, int n) {
  const size_t a = (size_t)(E + 1) * 4 + (size_t)(E < n ? E : n) * 2 + (size_t)n * 2 + 8;
  return (a + 15) / 16 * 16;
}

// Expert of entry j, or -1 for one that is not listed: an id outside [0, E), or an expert that an
// earlier slot of the token names too (its weights are added up, see few_weight).  Read through
// L2: k_few_down comes here before it waits for the kernel in front of it.
__device__ __forceinline__ int few_entry(const FewParams &p, int j) {
  const int e = __ldcg(p.top + j);
  if (e < 0 || e >= p.E) return -1;
  if (p.given)  // computed experts are distinct
    for (int i = j - j % p.k; i < j; ++i)
      if (__ldcg(p.top + i) == e) return -1;
  return e;
}

// Weight of expert e for the token of its listed entry j.
__device__ __forceinline__ float few_weight(const FewParams &p, int j, int e) {
  float w = __ldg(p.weights + j);
  if (p.given)
    for (int i = j + 1; i < j - j % p.k + p.k; ++i)
      if (__ldg(p.top + i) == e) w += __ldg(p.weights + i);
  return w;
}

// The experts in use, in increasing order, and their entries.  start[e] .. start[e + 1] are e's entries in ent; returns the number of
// experts in use.  An entry's place in its expert's list decides only which column of the
// product it is, so the order the atomics give does not show in any result.
template <int THREADS>
__device__ __forceinline__ int few_lists(const FewParams &p, int *start, uint16_t *act,
                                         uint16_t *ent, int *s_act) {
  const int n = p.T * p.k, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e <= p.E; e += THREADS) start[e] = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += THREADS) {
    const int e = few_entry(p, j);
    if (e >= 0) atomicAdd(&start[e], 1);
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // ends of the lists (the entries are filled in from the back)
    int carry = 0, na = 0;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      const int c = (e < p.E) ? start[e] : 0;
      const unsigned on = __ballot_sync(0xFFFFFFFFu, c > 0);
      int v = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, off);
        if (lane >= off) v += u;
      }
      if (c > 0) act[na + __popc(on & ((1u << lane) - 1u))] = (uint16_t)e;
      if (e < p.E) start[e] = carry + v;
      na += __popc(on);
      carry += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (lane == 0) {
      start[p.E] = carry;
      *s_act = na;
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += THREADS) {
    const int e = few_entry(p, j);
    if (e >= 0) ent[atomicSub(&start[e], 1) - 1] = (uint16_t)j;
  }
  __syncthreads();  // start[e] is now the first entry of e
  return *s_act;
}

// A place in a CTA's stream of stages: item (expert, row tile), group of 8 NT entries, chunk of K.
struct FewPos {
  int item, e, tile, n0, cnt, chunk;  // cnt: entries of the expert from n0 on (may exceed 8 NT)
  bool on;
};

template <class C>
struct FewKernel {
  const FewParams &p;
  const int *start;
  const uint16_t *act, *ent;
  uint32_t ring;
  int warp, lane, r, s;
  int K, chunks, tiles;
  int item_end, item_step;  // GLU: items are (expert, tile) pairs; DOWN: experts of one tile
  int fixed_tile;

  __device__ __forceinline__ void open(FewPos &q) const {
    q.on = q.item < item_end;
    if (!q.on) return;
    const int a = C::DOWN ? q.item : q.item / tiles;
    q.tile = C::DOWN ? fixed_tile : q.item - a * tiles;
    q.e = act[a];
    q.n0 = start[q.e];
    q.cnt = start[q.e + 1] - q.n0;
    q.chunk = 0;
  }
  __device__ __forceinline__ void next(FewPos &q) const {
    if (++q.chunk < chunks) return;
    if (q.cnt > 8 * C::NT) {
      q.n0 += 8 * C::NT;
      q.cnt -= 8 * C::NT;
      q.chunk = 0;
      return;
    }
    q.item += item_step;
    open(q);
  }

  // This warp's 16 weight rows of the stage.
  __device__ __forceinline__ void load_w(const FewPos &q, int st) const {
    const int k0 = q.chunk * C::CH + s * C::KU;
    if (k0 >= K) return;
    const uint32_t dst = ring + st * C::stage + warp * C::w_warp;
    const FewWeights &wa = C::DOWN ? p.w2 : p.w1;
    const FewWeights &wb = C::DOWN ? p.w2 : p.w3;
    const long long row0 = C::DOWN ? (long long)q.e * p.h + q.tile * C::rows + r * 16
                                   : (long long)q.e * p.f + q.tile * (C::rows / 2) + r * 8;
    const long long rb0 = C::DOWN ? row0 + 8 : row0;  // rows 8..15
    if constexpr (C::MX4) {
      const int rr = lane >> 2, seg = lane & 3;
      const size_t col = (size_t)(k0 >> 1) + seg * 16;
      const uint32_t d = dst + rr * 64 + ((seg ^ ((rr >> 1) & 3)) << 4);
      cp16(d, static_cast<const uint8_t *>(wa.data) + (size_t)(row0 + rr) * (K >> 1) + col);
      cp16(d + 512, static_cast<const uint8_t *>(wb.data) + (size_t)(rb0 + rr) * (K >> 1) + col);
      if (lane < 16) {  // the 16-byte piece with the row's word in it (past L1, as the elements)
        const FewWeights &w = lane < 8 ? wa : wb;
        const long long row = (lane < 8 ? row0 : rb0) + (lane & 7);
        cp16(ring + st * C::stage + C::o_sc + warp * C::sc_warp + lane * 16,
             static_cast<const uint8_t *>(w.scales) +
                 (mx4_scale_word(row, k0 >> 7, K >> 7) & ~(size_t)15));
      }
    } else {
      const int rr = lane >> 3, seg = lane & 7;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + rr;
        const FewWeights &w = i < 2 ? wa : wb;
        const long long g = (i < 2 ? row0 : rb0) + (row & 7);
        cp16(dst + row * 128 + ((seg ^ (row & 7)) << 4),
             static_cast<const uint16_t *>(w.data) + (size_t)g * K + k0 + seg * 8);
      }
    }
  }

  // The token rows of the stage (columns past K are not loaded and not used).
  __device__ __forceinline__ void load_x(const FewPos &q, int st) const {
    constexpr int segs = C::CH / 8;  // 16-byte pieces per row
    const int nr = min(q.cnt, 8 * C::NT);
    const int c0 = q.chunk * C::CH;
    const uint32_t dst = ring + st * C::stage + C::o_x;
    for (int i = threadIdx.x; i < nr * segs; i += C::threads) {
      const int n = i / segs, seg = i % segs;
      if (c0 + seg * 8 >= K) continue;
      const int j = ent[q.n0 + n];
      const size_t row = C::DOWN ? (size_t)j : (size_t)(j / p.k);
#pragma unroll
      for (int b = 0; b < C::BR; ++b) {
        const uint16_t *src = b ? p.xlo : p.xin;
        cp16(dst + (b * 8 * C::NT + n) * C::x_row + seg * 16, src + row * K + c0 + seg * 8);
      }
    }
    if constexpr (C::MX4) {
      constexpr int nb = C::CH / 32;
      for (int i = threadIdx.x; i < nr * nb; i += C::threads) {
        const int n = i / nb, b = i % nb;
        if (c0 + b * 32 >= K) continue;
        const int j = ent[q.n0 + n];
        const size_t row = C::DOWN ? (size_t)j : (size_t)(j / p.k);
        cp4(ring + st * C::stage + C::o_sb + (b * 8 * C::NT + n) * 4,
            p.xscale + row * (K >> 5) + (c0 >> 5) + b);
      }
    }
  }

  __device__ __forceinline__ void multiply(const FewPos &q, int st, float (&acc)[C::NT][4]) const {
    if (q.chunk * C::CH + s * C::KU >= K) return;
    const uint32_t base = ring + st * C::stage;
    const uint32_t w = base + warp * C::w_warp;
    const int ntl = (min(q.cnt, 8 * C::NT) + 7) >> 3;
    if constexpr (C::MX4) {
      const int g = lane >> 2, t = lane & 3;
      // rows 0..7 and 8..15 of a tile start at multiples of 8: one 32-row group each
      const int ra = q.tile * C::outs + r * (C::DOWN ? 16 : 8);
      const uint32_t sw = base + C::o_sc + warp * C::sc_warp + g * 16 + ((ra >> 5) & 3) * 4;
      const uint32_t sca = lds32(sw), scb = lds32(sw + 128);
      const uint32_t xb = base + C::o_x + g * C::x_row + (s * C::KU + 8 * t) * 2;
      const uint32_t sb = base + C::o_sb + (s * (C::KU / 32) * 8 * C::NT + 2 * t) * 4;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t wa = w + g * 64 + ((b ^ ((g >> 1) & 3)) << 4) + 4 * t;
        uint32_t lo[4], hi[4];
        mx4_unpack8(lds32(wa), lo);
        mx4_unpack8(lds32(wa + 512), hi);
        const float fa = mx4_scale_value((sca >> (8 * b)) & 0xFFu);
        const float fb = mx4_scale_value((scb >> (8 * b)) & 0xFFu);
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          if (nt >= ntl) break;
          uint32_t x0, x1, x2, x3;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                       : "r"(xb + nt * 8 * C::x_row + b * 64)
                       : "memory");
          float s0, s1;
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                       : "=f"(s0), "=f"(s1)
                       : "r"(sb + (b * 8 * C::NT + nt * 8) * 4)
                       : "memory");
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_f16(c, lo[0], hi[0], lo[1], hi[1], x0, x1);
          mma_f16(c, lo[2], hi[2], lo[3], hi[3], x2, x3);
          acc[nt][0] = fmaf(c[0] * s0, fa, acc[nt][0]);
          acc[nt][1] = fmaf(c[1] * s1, fa, acc[nt][1]);
          acc[nt][2] = fmaf(c[2] * s0, fb, acc[nt][2]);
          acc[nt][3] = fmaf(c[3] * s1, fb, acc[nt][3]);
        }
      }
    } else {
      const int ar = lane & 15;
      const uint32_t xb = base + C::o_x + (lane & 7) * C::x_row + (s * C::KU + (lane >> 3) * 8) * 2;
#pragma unroll
      for (int kk = 0; kk < 4; kk += 2) {
        uint32_t a0[4], a1[4];
        ldsm4(a0, w + ar * 128 + (((2 * kk + (lane >> 4)) ^ (ar & 7)) << 4));
        ldsm4(a1, w + ar * 128 + (((2 * kk + 2 + (lane >> 4)) ^ (ar & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          if (nt >= ntl) break;
#pragma unroll
          for (int br = 0; br < C::BR; ++br) {
            uint32_t x[4];
            ldsm4(x, xb + (br * 8 * C::NT + nt * 8) * C::x_row + kk * 32);
            mma_bf16(acc[nt], a0[0], a0[1], a0[2], a0[3], x[0], x[1]);
            mma_bf16(acc[nt], a1[0], a1[1], a1[2], a1[3], x[2], x[3]);
          }
        }
      }
    }
  }
};

// Element (row i of the tile, token n) of warp (r, s)'s sums in red: the accumulator of lane
// 4 (i % 8) + n / 2, word 2 (i / 8) + n % 2.
template <class C>
__device__ __forceinline__ float red_sum(const float *red, int i16, int r, int n) {
  const float *v = red + (((size_t)r * C::red_s) * C::NT + (n >> 3)) * 128 +
                   (4 * (i16 & 7) + ((n & 7) >> 1)) * 4 + 2 * (i16 >> 3) + (n & 1);
  float a = v[0];
#pragma unroll
  for (int q = 1; q < C::red_s; ++q) a += v[(size_t)q * C::NT * 128];
  return a;
}

// The stream of stages that both products share.  PRE: issued before the wait for the earlier
// kernels are the weight rows only.  done(pos): called by all threads when the sums of a
// tile and entry group are in red.
template <class C, class Done>
__device__ __forceinline__ void few_stream(const FewKernel<C> &k, int item0, float *red,
                                           bool pre, Done done) {
  FewPos pq;  // what is loaded next
  pq.item = item0;
  k.open(pq);
  FewPos cq = pq;
  if (pre) {  // weights of the first stages now, their token rows once the earlier kernel is done
    FewPos w = pq;
#pragma unroll
    for (int i = 0; i < C::P - 1; ++i) {
      if (w.on) {
        k.load_w(w, i);
        k.next(w);
      }
      cp_commit();
    }
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < C::P - 1; ++i) {
      if (pq.on) {
        k.load_x(pq, i);
        k.next(pq);
      }
      cp_commit();
    }
  } else {
#pragma unroll
    for (int i = 0; i < C::P - 1; ++i) {
      if (pq.on) {
        k.load_w(pq, i);
        k.load_x(pq, i);
        k.next(pq);
      }
      cp_commit();
    }
  }
  float acc[C::NT][4];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
  int st = 0, ld = C::P - 1;
  while (cq.on) {
    cp_wait<C::P - 2>();
    __syncthreads();  // the stage has landed; every warp is done with the stage before it
    if (pq.on) {
      k.load_w(pq, ld);
      k.load_x(pq, ld);
      k.next(pq);
    }
    cp_commit();
    if (++ld == C::P) ld = 0;
    k.multiply(cq, st, acc);
    if (++st == C::P) st = 0;
    if (cq.chunk == k.chunks - 1) {
      const int ntl = (min(cq.cnt, 8 * C::NT) + 7) >> 3;
      float4 *mine = reinterpret_cast<float4 *>(red) + k.lane +
                     (size_t)(C::red_s == 1 ? k.r : k.warp) * C::NT * 32;
      auto put = [&](bool add) {
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          if (nt < ntl) {
            float4 v = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
            if (add) {
              const float4 o = mine[nt * 32];
              v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
            }
            mine[nt * 32] = v;
          }
        }
      };
      if (C::S != 2) {
        put(false);
      } else {
        if (k.s == 1) put(false);
        __syncthreads();
        if (k.s == 0) put(true);
      }
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
      __syncthreads();
      done(cq);  // red is next written after the stage barrier of a later iteration
    }
    k.next(cq);
  }
  cp_wait<0>();
}

template <class C>
__device__ __forceinline__ FewKernel<C> few_kernel(const FewParams &p, const int *start,
                                                   const uint16_t *act, const uint16_t *ent,
                                                   uint32_t ring) {
  const int warp = threadIdx.x >> 5;
  const int K = C::DOWN ? p.f : p.h;
  return FewKernel<C>{p,    start, act, ent, ring, warp, (int)(threadIdx.x & 31), warp / C::S,
                      warp % C::S, K, (K + C::CH - 1) / C::CH,
                      C::DOWN ? p.h / C::rows : p.f / (C::rows / 2), 0, 1, 0};
}

// Dynamic shared memory: ring | red | lists (| y sums).
template <class C>
struct FewSmem {
  static constexpr int ring = C::P * C::stage, red = ring + C::red;
};

template <class C>
__global__ void __launch_bounds__(C::threads, C::min_ctas) k_few_glu(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  float *red = reinterpret_cast<float *>(smem + FewSmem<C>::ring);
  int *start = reinterpret_cast<int *>(smem + FewSmem<C>::red);
  uint16_t *act = reinterpret_cast<uint16_t *>(start + p.E + 1);
  uint16_t *ent = act + min(p.E, p.T * p.k);
  __shared__ int s_act;
  pdl_wait();
  pdl_trigger();
  const int na = few_lists<C::threads>(p, start, act, ent, &s_act);
  FewKernel<C> k = few_kernel<C>(p, start, act, ent, smem_u32(smem));
  k.item_end = na * k.tiles;
  k.item_step = gridDim.x;
  few_stream(k, blockIdx.x, red, false, [&](const FewPos &q) {
    const int nr = min(q.cnt, 8 * C::NT);
    const int f0 = q.tile * C::outs;
    for (int i = threadIdx.x; i < nr * C::outs; i += C::threads) {
      const int n = i / C::outs, c = i % C::outs;
      const float a = red_sum<C>(red, c & 7, c >> 3, n);
      const float b = red_sum<C>(red, (c & 7) + 8, c >> 3, n);
      const float hv = silu_f(a) * b;
      const size_t at = (size_t)ent[q.n0 + n] * p.f + f0 + c;
      if constexpr (C::MX4) {  // 32 lanes hold one block of 32 columns
        static_assert(!C::MX4 || C::outs % 32 == 0, "whole blocks");
        const int es = f16_block_exp(__reduce_max_sync(0xFFFFFFFFu, finite_abs(__float_as_uint(hv))));
        p.hout[at] = __half_as_ushort(__float2half_rn(hv * pow2(es)));
        if ((threadIdx.x & 31) == 0) p.hscale[at >> 5] = pow2(-es);
      } else {
        const __nv_bfloat16 hi = __float2bfloat16(hv);
        const float rest = hv - __bfloat162float(hi);
        p.hout[at] = __bfloat16_as_ushort(hi);
        // inf - inf: the upper part already says it
        p.hlo[at] = __bfloat16_as_ushort(__float2bfloat16(rest == rest ? rest : 0.0f));
      }
    }
  });
}

// A cluster of G CTAs shares a row tile, each with a contiguous G-th of the experts in use;
// their sums are added in rank order through distributed shared memory.
template <class C>
__global__ void __launch_bounds__(C::threads, C::min_ctas) k_few_down(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  float *red = reinterpret_cast<float *>(smem + FewSmem<C>::ring);
  int *start = reinterpret_cast<int *>(smem + FewSmem<C>::red);
  uint16_t *act = reinterpret_cast<uint16_t *>(start + p.E + 1);
  uint16_t *ent = act + min(p.E, p.T * p.k);
  float *ysum = reinterpret_cast<float *>(smem + FewSmem<C>::red + few_list_bytes(p.E, p.T * p.k));
  __shared__ int s_act;
  // Before the wait for k_few_glu: only what was complete when that kernel passed its own
  // wait (it lets this one start after that): the routing, and the caller's W2.
  const int na = few_lists<C::threads>(p, start, act, ent, &s_act);
  const int G = p.groups, g = (int)cluster_ctarank();
  FewKernel<C> k = few_kernel<C>(p, start, act, ent, smem_u32(smem));
  k.fixed_tile = blockIdx.x / G;
  const int per = (na + G - 1) / G;
  k.item_end = min(na, (g + 1) * per);
  for (int i = threadIdx.x; i < p.T * C::outs; i += C::threads) ysum[i] = 0.0f;
  few_stream(k, g * per, red, true, [&](const FewPos &q) {
    const int nr = min(q.cnt, 8 * C::NT);
    for (int i = threadIdx.x; i < nr * C::outs; i += C::threads) {
      const int n = i / C::outs, c = i % C::outs;
      const int j = ent[q.n0 + n];  // an expert's entries belong to distinct tokens
      float &y = ysum[(j / p.k) * C::outs + c];
      y = fmaf(few_weight(p, j, q.e), red_sum<C>(red, c & 15, c >> 4, n), y);
    }
  });
  cluster_sync_all();
  const int h0 = k.fixed_tile * C::outs;
  const uint32_t mine = smem_u32(ysum);
  for (int i = g * C::threads + threadIdx.x; i < p.T * (C::outs / 2); i += G * C::threads) {
    const int t = i / (C::outs / 2), c = 2 * (i % (C::outs / 2));
    float a = 0.0f, b = 0.0f;
    for (int o = 0; o < G; ++o) {
      float u, v;
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                   : "=f"(u), "=f"(v)
                   : "r"(mapa_shared(mine, o) + (uint32_t)((t * C::outs + c) * 4))
                   : "memory");
      a += u;
      b += v;
    }
    *reinterpret_cast<uint32_t *>(p.y + (size_t)t * p.h + h0 + c) = pack_bf16x2(a, b);
  }
  cluster_sync_all();  // no CTA leaves while another reads its sums
}

// ---- host side ---------------------------------------------------------------------------------

// Opt the kernel in to large shared memory, once per device.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev < 64) ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - 1024);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <class C>
cudaError_t launch_few_glu(const FewParams &p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_few_glu<C>, done);
  if (e != cudaSuccess) return e;
  const size_t smem = FewSmem<C>::red + few_list_bytes(p.E, p.T * p.k);
  const long long n = (long long)p.T * p.k;
  const long long items = (n < p.E ? n : p.E) * (p.f / C::outs);
  long long ctas = device_sm_count();
  if (2 * (smem + 2048) <= 228 * 1024 && C::min_ctas > 1) ctas *= 2;
  return launch_pdl(k_few_glu<C>, (int)(items < ctas ? items : ctas), C::threads, smem, st, p);
}

template <class C>
cudaError_t launch_few_down(FewParams p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_few_down<C>, done);
  if (e != cudaSuccess) return e;
  const size_t smem = FewSmem<C>::red + few_list_bytes(p.E, p.T * p.k) +
                      (size_t)p.T * C::outs * sizeof(float);
  const long long n = (long long)p.T * p.k;
  const int experts = (int)(n < p.E ? n : p.E);
  const int tiles = p.h / C::outs;
  // experts split over up to eight CTAs per row tile until the SMs are covered
  int G = 1;
  while (G < 8 && 2 * G <= experts && tiles * G < device_sm_count()) G *= 2;
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

template <bool MX4, int NT, int R, int S, int PG, int PD>
cudaError_t launch_few_pair(const FewParams &p, const FewParams &d, cudaStream_t st) {
  cudaError_t e = launch_few_glu<FewCfg<MX4, false, NT, R, S, PG>>(p, st);
  if (e != cudaSuccess) return e;
  return launch_few_down<FewCfg<MX4, true, NT, R, S, PD>>(d, st);
}

}  // namespace

cudaError_t launch_few(const FewParams &p_in, const uint16_t *logits, bool renorm, int32_t *top,
                       float *weights, int32_t *status, cudaStream_t st) {
  FewParams p = p_in;
  const bool mx4 = p.w1.scales != nullptr;
  cudaError_t e = launch_pdl(k_few_route, p.T, mx4 ? 32 * kRouteWarps : 32, 0, st, logits, p.E, p.k,
                             renorm ? 1 : 0, p.h, top, weights, status,
                             static_cast<const uint4 *>(p.x), reinterpret_cast<uint4 *>(p.x16),
                             p.x16scale);
  if (e != cudaSuccess) return e;
  FewParams d = p;
  p.xin = mx4 ? p.x16 : static_cast<const uint16_t *>(p.x);
  p.xscale = p.x16scale;
  d.xin = p.hout;
  d.xlo = p.hlo;
  d.xscale = p.hscale;
  if (mx4) {
    if (p.T <= 8) return launch_few_pair<true, 1, 4, 2, 5, 5>(p, d, st);
    if (p.T <= 16) return launch_few_pair<true, 2, 4, 2, 4, 4>(p, d, st);
    if (p.T <= 32) return launch_few_pair<true, 4, 8, 2, 4, 4>(p, d, st);
    return launch_few_pair<true, 4, 8, 2, 4, 3>(p, d, st);
  }
  if (p.T <= 8) return launch_few_pair<false, 1, 1, 8, 4, 3>(p, d, st);
  if (p.T <= 16) return launch_few_pair<false, 2, 2, 4, 4, 3>(p, d, st);
  if (p.T <= 32) return launch_few_pair<false, 4, 4, 2, 3, 3>(p, d, st);
  return launch_few_pair<false, 8, 8, 1, 3, 3>(p, d, st);
}

}  // namespace dmoe
