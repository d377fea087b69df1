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
//   4-bit weights: e2m1 -> fp16 is exact, so x and H go in fp16 under a power-of-two scale, x per
//     row (exact down to 2^-29 of the row's largest), H per 32 columns (11 bits); the 32
//     products of a weight block are summed first, then scaled by the block's scale.
// The few partial sums over S and over the experts of a token are added in a fixed order.
#include <stdlib.h>

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
      route_token(logits + t * E, E, k, renorm != 0, top + t * k, weights + t * k, status, lane);
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
// The same with a zero accumulator going in.
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shape of a variant: MX4 weights in four bits; DOWN the second product; NT tiles of 8 tokens;
// R x S warps of KU columns; P stages.  BR: copies of the token rows (two: H's upper and lower
// bf16).  SB: the token operand has a scale per 32 columns (H in fp16).
template <bool MX4_, bool DOWN_, int NT_, int R_, int S_, int KU_, int P_>
struct FewCfg {
  static constexpr bool MX4 = MX4_, DOWN = DOWN_, SB = MX4 && DOWN;
  static constexpr int NT = NT_, R = R_, S = S_, KU = KU_, P = P_;
  static constexpr int warps = R * S, threads = 32 * warps;
  static constexpr int min_ctas = threads == 256 ? 2 : 1;
  static constexpr int CH = S * KU;  // columns per stage
  static constexpr int BR = (DOWN && !MX4) ? 2 : 1;
  static constexpr int wbits = MX4 ? 4 : 16;
  static constexpr int w_warp = 16 * KU * wbits / 8;       // weight bytes per warp and stage
  static constexpr int sc_warp = MX4 ? KU / 128 * 256 : 0;  // scales: 16 bytes per row and 128 K
  // token rows: a stride that is 16 (ldmatrix) or 64 (16-byte loads of 4 lanes a row) bytes off
  // a multiple of 128 keeps the reads free of bank conflicts
  static constexpr int x_row = CH * 2 + (MX4 ? 64 : 16);
  static constexpr int x_bytes = BR * 8 * NT * x_row;
  static constexpr int sb_bytes = SB ? (CH / 32) * 8 * NT * 4 : 0;  // token scales [block][token]
  static constexpr int o_sc = warps * w_warp, o_x = o_sc + warps * sc_warp, o_sb = o_x + x_bytes;
  static constexpr int stage = o_sb + sb_bytes;
  static constexpr int rows = 16 * R;                  // weight rows per tile
  static constexpr int outs = DOWN ? rows : rows / 2;  // output columns per tile
  // partial sums: of the slices of K past the first, and for GLU MX4 a tile's H in fp32
  static constexpr int red = (S - 1) * R * NT * 512;
  static constexpr int hrow = outs + 4;
  static constexpr int hbuf = (MX4 && !DOWN) ? 8 * NT * hrow * 4 : 0;
  // y sums: rows of `outs` plus 8 floats (four tokens x eight rows meet no bank twice)
  static constexpr int yrow = outs + 8;
  static constexpr int o_red = P * stage, o_hbuf = o_red + red, o_lists = o_hbuf + hbuf;
  static_assert(stage % 16 == 0 && o_x % 16 == 0 && x_row % 16 == 0, "alignment");
  static_assert(!MX4 || DOWN || outs % 32 == 0, "whole blocks of H");
};

// Bytes of the expert lists: entries [n] (j | token << 16), starts [E + 1], experts in use
// (uint16).
__host__ __device__ inline size_t few_list_bytes(int E, int n) {
  const size_t a = (size_t)n * 4 + (size_t)(E + 1) * 4 + (size_t)(E < n ? E : n) * 2;
  return (a + 15) / 16 * 16;
}

struct FewLists {
  uint32_t *ent;
  int *start;
  uint16_t *act;
  __device__ __forceinline__ FewLists(uint8_t *base, int E, int n)
      : ent(reinterpret_cast<uint32_t *>(base)), start(reinterpret_cast<int *>(ent + n)),
        act(reinterpret_cast<uint16_t *>(start + E + 1)) {}
};

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

// The experts in use, in increasing order, and their entries: start[e] .. start[e + 1] in ent.
// Returns the number of experts in use.  An entry's place in its expert's list decides only
// which column of the product it is, so the order the atomics give does not show in any result.
template <int THREADS>
__device__ __forceinline__ int few_lists(const FewParams &p, const FewLists &l, int *s_act) {
  const int n = p.T * p.k, lane = threadIdx.x & 31;
  int *start = l.start;
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
      if (c > 0) l.act[na + __popc(on & ((1u << lane) - 1u))] = (uint16_t)e;
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
    if (e >= 0) l.ent[atomicSub(&start[e], 1) - 1] = (uint32_t)j | ((uint32_t)(j / p.k) << 16);
  }
  __syncthreads();  // start[e] is now the first entry of e
  return *s_act;
}

// A place in a CTA's stream of stages: item (GLU: expert, row tile; DOWN: expert, part of K),
// group of 8 NT entries, chunk of K.
struct FewPos {
  int item, e, tile, n0, cnt;  // cnt: entries of the expert from n0 on (may exceed 8 NT)
  int chunk, c0, c1;           // chunks [c0, c1) of K
  bool on;
};

template <class C>
struct FewKernel {
  const FewParams &p;
  const FewLists &l;
  uint32_t ring;
  int warp, lane, r, s;
  int K, chunks, tiles;
  int item_end, item_step;
  int fixed_tile, part;  // DOWN: the CTA's row tile, chunks per part of K
  // this lane's rows of the tile being loaded (rows 0..7 in a, 8..15 in b), at its slice of K
  const uint8_t *wa, *wb, *ws;

  __device__ __forceinline__ FewKernel(const FewParams &p_, const FewLists &l_, uint32_t ring_)
      : p(p_), l(l_), ring(ring_), warp(threadIdx.x >> 5), lane(threadIdx.x & 31),
        r(warp / C::S), s(warp % C::S), K(C::DOWN ? p_.f : p_.h), chunks((K + C::CH - 1) / C::CH),
        tiles(C::DOWN ? p_.h / C::rows : p_.f / (C::rows / 2)), item_end(0), item_step(1),
        fixed_tile(0), part(C::DOWN ? (chunks + p_.kparts - 1) / p_.kparts : 0), wa(nullptr), wb(nullptr), ws(nullptr) {}

  __device__ __forceinline__ void open(FewPos &q) const {
    q.on = q.item < item_end;
    if (!q.on) return;
    const int per = C::DOWN ? p.kparts : tiles;
    const int a = q.item / per, b = q.item - a * per;
    q.tile = C::DOWN ? fixed_tile : b;
    q.e = l.act[a];
    q.n0 = l.start[q.e];
    q.cnt = l.start[q.e + 1] - q.n0;
    q.c0 = C::DOWN ? b * part : 0;
    q.c1 = C::DOWN ? min(chunks, q.c0 + part) : chunks;
    q.chunk = q.c0;
  }
  __device__ __forceinline__ void next(FewPos &q) const {
    if (++q.chunk < q.c1) return;
    if (q.cnt > 8 * C::NT) {
      q.n0 += 8 * C::NT;
      q.cnt -= 8 * C::NT;
      q.chunk = q.c0;
      return;
    }
    q.item += item_step;
    open(q);
  }

  // Row 0 (a) and row 8 (b) of this warp's 16 in the tile.
  __device__ __forceinline__ void rows_of(const FewPos &q, long long &a, long long &b) const {
    if (C::DOWN) {
      a = (long long)q.e * p.h + q.tile * C::rows + r * 16;
      b = a + 8;
    } else {
      a = b = (long long)q.e * p.f + q.tile * (C::rows / 2) + r * 8;
    }
  }

  // This warp's 16 weight rows of the stage.
  __device__ __forceinline__ void load_w(const FewPos &q, int st) {
    constexpr int seg_lanes = C::MX4 ? C::KU / 32 : 8;  // lanes (16 bytes each) per row
    constexpr int row_step = 32 / seg_lanes;
    const int rr = lane / seg_lanes, seg = lane % seg_lanes;
    const size_t pitch = (size_t)K * C::wbits / 8;
    if (q.chunk == q.c0) {
      const FewWeights &fa = C::DOWN ? p.w2 : p.w1;
      const FewWeights &fb = C::DOWN ? p.w2 : p.w3;
      long long a, b;
      rows_of(q, a, b);
      const size_t col = (size_t)(q.c0 * C::CH + s * C::KU) * C::wbits / 8 + seg * 16;
      wa = static_cast<const uint8_t *>(fa.data) + (size_t)(a + rr) * pitch + col;
      wb = static_cast<const uint8_t *>(fb.data) + (size_t)(b + rr) * pitch + col;
      if (C::MX4 && lane < 16)  // the 16-byte piece with the row's word in it (past L1)
        ws = static_cast<const uint8_t *>(lane < 8 ? fa.scales : fb.scales) +
             (mx4_scale_word((lane < 8 ? a : b) + (lane & 7), (q.c0 * C::CH + s * C::KU) >> 7, K >> 7) &
              ~(size_t)15);
    }
    const int left = K - q.chunk * C::CH - s * C::KU;  // a multiple of 64 (4 bits: of 128)
    if (left > 0) {
      const uint32_t dst = ring + st * C::stage + warp * C::w_warp;
      if (seg * (C::MX4 ? 32 : 8) < left) {
#pragma unroll
        for (int i = 0; i < 8; i += row_step) {
          const int row = i + rr;
          const uint32_t d = dst + row * (seg_lanes * 16) + (swz(row, seg) << 4);
          cp16(d, wa + i * pitch);
          cp16(d + 8 * seg_lanes * 16, wb + i * pitch);
        }
      }
      if (C::MX4 && lane < 16) {
        const uint32_t d = ring + st * C::stage + C::o_sc + warp * C::sc_warp + lane * 16;
#pragma unroll
        for (int j = 0; j < C::KU / 128; ++j)
          if (j * 128 < left) cp16(d + 256 * j, ws + kMx4TileBytes * j);
      }
    }
    wa += C::CH * C::wbits / 8;
    wb += C::CH * C::wbits / 8;
    ws += (C::CH / 128) * kMx4TileBytes;
  }

  // Place of 16-byte piece `seg` of a weight row in its row of the stage.  bf16: ldmatrix reads
  // one piece of eight rows.  4 bits: eight rows' four words of a piece (32 lanes) are read; rows
  // of 64 bytes share their banks with every second row, rows of 128 bytes with every row.
  __device__ __forceinline__ static int swz(int row, int seg) {
    if (!C::MX4) return seg ^ (row & 7);
    return C::KU == 128 ? seg ^ ((row >> 1) & 3) : seg ^ (row & 7);
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
      const uint32_t v = l.ent[q.n0 + n];
      const size_t at = (size_t)(C::DOWN ? v & 0xFFFFu : v >> 16) * K + c0 + seg * 8;
      cp16(dst + n * C::x_row + seg * 16, p.xin + at);
      if (C::BR == 2) cp16(dst + (8 * C::NT + n) * C::x_row + seg * 16, p.xlo + at);
    }
    if constexpr (C::SB) {
      constexpr int nb = C::CH / 32;
      for (int i = threadIdx.x; i < nr * nb; i += C::threads) {
        const int n = i / nb, b = i % nb;
        if (c0 + b * 32 >= K) continue;
        const size_t row = l.ent[q.n0 + n] & 0xFFFFu;
        cp4(ring + st * C::stage + C::o_sb + (b * 8 * C::NT + n) * 4,
            p.xscale + row * (K >> 5) + (c0 >> 5) + b);
      }
    }
  }

  // Whether a byte of w is 0 or 255 (exact for "any": a borrow needs a zero byte below it).
  __device__ __forceinline__ static bool odd_scales(uint32_t w) {
    return (((w - 0x01010101u) & ~w) | ((~w - 0x01010101u) & w)) & 0x80808080u;
  }

  // Four blocks (128 columns) of this warp's 16 rows times the token tiles.
  template <bool ODD>
  __device__ __forceinline__ void blocks(int j, uint32_t w, uint32_t xb, uint32_t sb, uint32_t sca,
                                         uint32_t scb, int ntl, float (&acc)[C::NT][4]) const {
    const int g = lane >> 2, t = lane & 3;
    constexpr int wrow = C::KU / 2;
#pragma unroll
    for (int b4 = 0; b4 < 4; ++b4) {
      const int b = 4 * j + b4;
      const uint32_t wl = w + g * wrow + (swz(g, b) << 4) + 4 * t;
      uint32_t lo[4], hi[4];
      mx4_unpack8(lds32(wl), lo);
      mx4_unpack8(lds32(wl + 8 * wrow), hi);
      float fa, fb;
      if (ODD) {
        fa = mx4_scale_value((sca >> (8 * b4)) & 0xFFu);
        fb = mx4_scale_value((scb >> (8 * b4)) & 0xFFu);
      } else {
        fa = __uint_as_float((b4 < 3 ? sca << (23 - 8 * b4) : sca >> 1) & 0x7F800000u);
        fb = __uint_as_float((b4 < 3 ? scb << (23 - 8 * b4) : scb >> 1) & 0x7F800000u);
      }
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) {
        if (nt >= ntl) break;
        uint32_t x0, x1, x2, x3;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                     : "r"(xb + nt * 8 * C::x_row + b * 64)
                     : "memory");
        float c[4];
        mma_f16_zero(c, lo[0], hi[0], lo[1], hi[1], x0, x1);
        mma_f16(c, lo[2], hi[2], lo[3], hi[3], x2, x3);
        if constexpr (C::SB) {
          float s0, s1;
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                       : "=f"(s0), "=f"(s1)
                       : "r"(sb + (b * 8 * C::NT + nt * 8) * 4)
                       : "memory");
          c[0] *= s0;
          c[1] *= s1;
          c[2] *= s0;
          c[3] *= s1;
        }
        acc[nt][0] = fmaf(c[0], fa, acc[nt][0]);
        acc[nt][1] = fmaf(c[1], fa, acc[nt][1]);
        acc[nt][2] = fmaf(c[2], fb, acc[nt][2]);
        acc[nt][3] = fmaf(c[3], fb, acc[nt][3]);
      }
    }
  }

  __device__ __forceinline__ void multiply(const FewPos &q, int st, float (&acc)[C::NT][4]) const {
    const int left = K - q.chunk * C::CH - s * C::KU;
    if (left <= 0) return;
    const uint32_t base = ring + st * C::stage;
    const uint32_t w = base + warp * C::w_warp;
    const int ntl = (min(q.cnt, 8 * C::NT) + 7) >> 3;
    if constexpr (C::MX4) {
      const int g = lane >> 2, t = lane & 3;
      // rows 0..7 and 8..15 of a tile start at multiples of 8: one 32-row group each
      const int ra = q.tile * C::outs + r * (C::DOWN ? 16 : 8);
      const uint32_t sw = base + C::o_sc + warp * C::sc_warp + g * 16 + ((ra >> 5) & 3) * 4;
      const uint32_t xb = base + C::o_x + g * C::x_row + (s * C::KU + 8 * t) * 2;
      const uint32_t sb = base + C::o_sb + (s * (C::KU / 32) * 8 * C::NT + 2 * t) * 4;
#pragma unroll
      for (int j = 0; j < C::KU / 128; ++j) {
        if (j * 128 >= left) break;
        const uint32_t sca = lds32(sw + 256 * j), scb = lds32(sw + 256 * j + 128);
        // scale bytes 1 .. 254 are exponent fields as they stand; 0 (2^-127) and 255 (NaN) are not
        if (__any_sync(0xFFFFFFFFu, odd_scales(sca) | odd_scales(scb)))
          blocks<true>(j, w, xb, sb, sca, scb, ntl, acc);
        else
          blocks<false>(j, w, xb, sb, sca, scb, ntl, acc);
      }
    } else {
      const int ar = lane & 15;
      const uint32_t xb = base + C::o_x + (lane & 7) * C::x_row + (s * C::KU + (lane >> 3) * 8) * 2;
#pragma unroll
      for (int kk = 0; kk < 4; kk += 2) {
        uint32_t a0[4], a1[4];
        ldsm4(a0, w + ar * 128 + (swz(ar, 2 * kk + (lane >> 4)) << 4));
        ldsm4(a1, w + ar * 128 + (swz(ar, 2 * kk + 2 + (lane >> 4)) << 4));
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

// The stream of stages that both products share.  pre: before the wait for the earlier kernels
// only weights are loaded.  done(pos, nt, sums): called by the first slice's warps with the
// sums of token tile nt over all of K: words 2 i + c are row lane / 4 + 8 i of the warp's 16 and
// token 8 nt + 2 (lane % 4) + c; end(pos): by all threads after them.
template <class C, class Done, class End>
__device__ __forceinline__ void few_stream(FewKernel<C> &k, int item0, float *red, bool pre,
                                           Done done, End end) {
  FewPos pq;  // what is loaded next
  pq.item = item0;
  k.open(pq);
  FewPos cq = pq;
  if (pre) {  // weights of the first stages now, their token rows once the earlier kernel is done
    FewPos xq = pq;
#pragma unroll
    for (int i = 0; i < C::P - 1; ++i) {
      if (pq.on) {
        k.load_w(pq, i);
        k.next(pq);
      }
      cp_commit();
    }
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < C::P - 1; ++i) {
      if (xq.on) {
        k.load_x(xq, i);
        k.next(xq);
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
    if (cq.chunk == cq.c1 - 1) {
      const int ntl = (min(cq.cnt, 8 * C::NT) + 7) >> 3;
      // slices past the first hand over their sums (red is next written after the stage
      // barrier of a later iteration)
      float4 *part = reinterpret_cast<float4 *>(red) + k.r * C::NT * 32 + k.lane;
      if (C::S > 1) {
        if (k.s > 0) {
#pragma unroll
          for (int nt = 0; nt < C::NT; ++nt)
            if (nt < ntl)
              part[((k.s - 1) * C::R * C::NT + nt) * 32] =
                  make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
        }
        __syncthreads();
      }
      if (k.s == 0) {
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          if (nt < ntl) {
#pragma unroll
            for (int q = 0; q < C::S - 1; ++q) {
              const float4 v = part[(q * C::R * C::NT + nt) * 32];
              acc[nt][0] += v.x;
              acc[nt][1] += v.y;
              acc[nt][2] += v.z;
              acc[nt][3] += v.w;
            }
            done(cq, nt, acc[nt]);
          }
        }
      }
      end(cq);
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
    }
    k.next(cq);
  }
  cp_wait<0>();
}

template <class C>
__global__ void __launch_bounds__(C::threads, C::min_ctas)
    k_few_glu(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const FewLists l(smem + C::o_lists, p.E, p.T * p.k);
  __shared__ int s_act;
  pdl_wait();
  pdl_trigger();
  const int na = few_lists<C::threads>(p, l, &s_act);
  FewKernel<C> k(p, l, smem_u32(smem));
  k.item_end = na * k.tiles;
  k.item_step = gridDim.x;
  float *hb = reinterpret_cast<float *>(smem + C::o_hbuf);
  const int g = k.lane >> 2, t2 = 2 * (k.lane & 3);
  few_stream(
      k, blockIdx.x, reinterpret_cast<float *>(smem + C::o_red), false,
      [&](const FewPos &q, int nt, const float (&v)[4]) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // gate v[c], up v[2 + c] of column f, token n
          const int n = 8 * nt + t2 + c, col = k.r * 8 + g;
          if (n >= q.cnt) continue;
          const uint32_t en = l.ent[q.n0 + n];
          if constexpr (C::MX4) {
            const float xs = __ldg(p.xscale + (en >> 16));
            hb[n * C::hrow + col] = silu_f(v[c] * xs) * (v[2 + c] * xs);
          } else {
            const float hv = silu_f(v[c]) * v[2 + c];
            const size_t at = (size_t)(en & 0xFFFFu) * p.f + q.tile * C::outs + col;
            const __nv_bfloat16 hi = __float2bfloat16(hv);
            const float rest = hv - __bfloat162float(hi);
            p.hout[at] = __bfloat16_as_ushort(hi);
            // inf - inf: the upper part already says it
            p.hlo[at] = __bfloat16_as_ushort(__float2bfloat16(rest == rest ? rest : 0.0f));
          }
        }
      },
      [&](const FewPos &q) {
        if constexpr (C::MX4) {  // blocks of 32 columns to fp16, a warp each
          __syncthreads();
          const int nr = min(q.cnt, 8 * C::NT);
          for (int i = k.warp; i < nr * (C::outs / 32); i += C::warps) {
            const int n = i / (C::outs / 32), b = i % (C::outs / 32);
            const float hv = hb[n * C::hrow + b * 32 + k.lane];
            const int es =
                f16_block_exp(__reduce_max_sync(0xFFFFFFFFu, finite_abs(__float_as_uint(hv))));
            const size_t at =
                (size_t)(l.ent[q.n0 + n] & 0xFFFFu) * p.f + q.tile * C::outs + b * 32 + k.lane;
            p.hout[at] = __half_as_ushort(__float2half_rn(hv * pow2(es)));
            if (k.lane == 0) p.hscale[at >> 5] = pow2(-es);
          }
        }
      });
}

// A cluster of G CTAs shares a row tile, each with every G-th of the experts in use (neighbouring
// experts of a skewed router hold similar numbers of tokens); their sums are added in rank
// order through distributed shared memory.
template <class C>
__global__ void __launch_bounds__(C::threads, C::min_ctas)
    k_few_down(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const FewLists l(smem + C::o_lists, p.E, p.T * p.k);
  float *ysum = reinterpret_cast<float *>(smem + C::o_lists + few_list_bytes(p.E, p.T * p.k));
  __shared__ int s_act;
  // Before the wait for k_few_glu: only what was complete when that kernel passed its own
  // wait (it lets this one start after that): the routing, and the caller's W2.
  const int na = few_lists<C::threads>(p, l, &s_act);
  const int G = p.groups, rank = (int)cluster_ctarank();
  FewKernel<C> k(p, l, smem_u32(smem));
  k.fixed_tile = blockIdx.x / G;
  k.item_end = na * p.kparts;
  k.item_step = G;
  for (int i = threadIdx.x; i < p.T * C::yrow; i += C::threads) ysum[i] = 0.0f;
  const int g = k.lane >> 2, t2 = 2 * (k.lane & 3);
  few_stream(
      k, rank, reinterpret_cast<float *>(smem + C::o_red), true,
      [&](const FewPos &q, int nt, const float (&v)[4]) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int n = 8 * nt + t2 + c;
          if (n >= q.cnt) continue;
          const uint32_t en = l.ent[q.n0 + n];  // an expert's entries belong to distinct tokens
          const float w = few_weight(p, en & 0xFFFFu, q.e);
          float *y = ysum + (en >> 16) * C::yrow + k.r * 16 + g;
          y[0] = fmaf(w, v[c], y[0]);
          y[8] = fmaf(w, v[2 + c], y[8]);
        }
      },
      [](const FewPos &) {});
  cluster_sync_all();
  const int h0 = k.fixed_tile * C::outs;
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
  const size_t smem = C::o_lists + few_list_bytes(p.E, p.T * p.k);
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
  const size_t smem = C::o_lists + few_list_bytes(p.E, p.T * p.k) +
                      (size_t)p.T * C::yrow * sizeof(float);
  const long long n = (long long)p.T * p.k;
  const int experts = (int)(n < p.E ? n : p.E);
  const int tiles = p.h / C::outs;
  // the experts are spread over up to eight CTAs per row tile until there is one CTA for each
  // place on the SMs; with fewer experts than that, K is cut into parts as well (whole chunks)
  int places = device_sm_count();
  if (2 * (smem + 2048) <= 228 * 1024 && C::min_ctas > 1) places *= 2;
  int G = 1;
  while (G < 8 && tiles * G * 2 <= places) G *= 2;
  const int chunks = (p.f + C::CH - 1) / C::CH;
  int parts = 1;
  while (experts * parts < G && parts * 2 <= chunks) parts *= 2;
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

template <bool MX4, int NT, int R, int S, int KU, int PG, int PD>
cudaError_t launch_few_pair(const FewParams &p, const FewParams &d, cudaStream_t st) {
  cudaError_t e = launch_few_glu<FewCfg<MX4, false, NT, R, S, KU, PG>>(p, st);
  if (e != cudaSuccess) return e;
  return launch_few_down<FewCfg<MX4, true, NT, R, S, KU, PD>>(d, st);
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
  const char *v = getenv("FEWV");
  const int var = v ? atoi(v) : 0;
  const double mean = (double)p.T * p.k / p.E;
  int nt = p.T <= 8 || mean <= 3 ? 1 : p.T <= 16 || mean <= 8 ? 2 : p.T <= 32 || mean <= 20 ? 4 : 8;
  if (var) nt = var;
  if (mx4) {
    if (nt == 1) return launch_few_pair<true, 1, 4, 2, 256, 3, 3>(p, d, st);
    if (nt == 2) return launch_few_pair<true, 2, 4, 2, 128, 4, 4>(p, d, st);
    if (p.T <= 32) return launch_few_pair<true, 4, 8, 2, 128, 4, 4>(p, d, st);
    return launch_few_pair<true, 4, 8, 2, 128, 4, 3>(p, d, st);
  }
  if (nt == 1) return launch_few_pair<false, 1, 1, 8, 64, 4, 3>(p, d, st);
  if (nt == 2) return launch_few_pair<false, 2, 2, 4, 64, 4, 3>(p, d, st);
  if (nt == 4) return launch_few_pair<false, 4, 4, 2, 64, 3, 3>(p, d, st);
  return launch_few_pair<false, 8, 8, 1, 64, 3, 3>(p, d, st);
}

}  // namespace dmoe
