// mx4_gemm.cu -- the expert FFN over many tokens with both operands of every product in the
// microscaled 4-bit format (dmoe_mx4 of dmoe.h), on the block-scaled tensor cores
// (tcgen05.mma kind::mxf4: e2m1 elements, one e8m0 scale per 32 along K, fp32 accumulation).
//
//   GLU   H = silu(X W1_e^T) * (X W3_e^T); H is converted to the format from fp32 in the epilogue
//         (a thread holds a row's 32-column block, so its maximum needs no exchange)
//   DOWN  Y_pad = w * (H W2_e^T) in block floating point, as the bf16 down GEMM writes it
//
// One SM pair per tile (cta_group::2, M = 256, N = 256): at four bits a 128 x 256 tile on one
// SM would need 100 bytes of operands per clock from L2; the pair needs 66.  The unit of work is
// a pair of consecutive row blocks of one expert times a column tile, enumerated from
// padded_bins on the device.  Persistent clusters of two CTAs, 320 threads each:
//   warp 0      TMA producer: per stage of 256 K this CTA's 128 rows of A (16 KB, 128-byte
//               swizzle), its half of B (16 KB), the scale tiles of its A rows (1 KB) and of
//               all 256 rows of B (2 KB; each SM of the pair multiplies by all of them)
//   warp 1      one thread of the leader: tcgen05.cp of the stage's scale tiles into tensor memory
//               (six 512-byte tiles, each 32 lanes x 4 columns repeated for the four lane
//               groups), then four MMAs of 64 K
//   warps 2..9  epilogue: a warp takes 32 rows and half of the columns
// Tensor memory: 256 accumulator columns, and 32 columns of scales per stage, which are
// rewritten only after the stage's MMAs are done.  Two accumulators and scales do not
// fit in 512 columns; instead the epilogue takes its 128 columns into registers at once and
// releases the accumulator before it converts and stores them.
//
// Every mbarrier wait is bounded; on expiry the kernel sets DMOE_STATUS_TIMEOUT, raises an
// abort flag for the other roles of its CTA, drains what it issued and returns.
#include <string.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "mx4.cuh"

namespace dmoe {

namespace {

constexpr int XM = 128;           // rows per CTA
constexpr int XN = 256;           // columns per tile
constexpr int XK = 256;           // K per stage: one 128-byte swizzle row of elements
constexpr int X_OP = XM * XK / 2;  // an operand's bytes per stage and CTA: 16 KB
constexpr int X_SFA = 2 * kMx4TileBytes;  // two column tiles of scales
constexpr int X_SFB = 4 * kMx4TileBytes;  // ... of both 128-row tiles of B
constexpr int X_STAGE = 2 * X_OP + X_SFA + X_SFB;  // 35 KB
constexpr int X_STAGES = 5;
constexpr int X_EPI = 8;
constexpr int X_THREADS = 64 + 32 * X_EPI;
constexpr int X_BOX = 32 * 128;  // a result box: 32 rows x 128 B
constexpr int X_TMEM = 512;
constexpr int X_SF_COL = 256;     // scales of stage s: columns 256 + 32 s ..
static_assert(X_SF_COL + 32 * X_STAGES <= X_TMEM, "tensor memory");
constexpr size_t X_SMEM = 1024 + (size_t)X_STAGES * X_STAGE + X_EPI * X_BOX + 256 +
                          sizeof(int) * (DMOE_MAX_EXPERTS + 1);
static_assert(X_SMEM <= 227 * 1024, "shared memory");

struct MxParams {
  CUtensorMap ta, tsa;            // A elements and scales
  CUtensorMap tb[2], tsb[2];      // B of the leader's / the peer's half: W1 / W3, or W2 twice
  CUtensorMap ty;                 // DOWN: Y_pad
  const int32_t *padded_bins, *bins, *indices;
  const float *weights;
  int E, h, f;
  int n_tiles, k_tiles;  // column tiles per unit; 128-wide K tiles
  int nblk_cap, group;
  int inject;
  long long wait_cycles;
  uint8_t *hq, *hs;  // GLU
  float *yscale;     // DOWN
  int32_t *status;
};

struct MxTile {
  int e, n, row0;
  bool dummy;
};

// Tile t -> expert, column tile, this CTA's rows; units of an expert in chunks of p.group, the
// unit varying fastest so that concurrent pairs share B.
__device__ __forceinline__ MxTile mx_decode(const MxParams &p, int t, const int *ustart,
                                            uint32_t rank) {
  const int vu = t / p.n_tiles;
  int lo = 0, hi = p.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ustart[mid] <= vu)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int units = ustart[lo + 1] - ustart[lo];
  const int c0 = ((vu - ustart[lo]) / p.group) * p.group;
  const int cs = min(p.group, units - c0);
  const int lt = t - (ustart[lo] + c0) * p.n_tiles;
  MxTile tl;
  tl.e = lo;
  tl.n = lt / cs;
  const int unit = c0 + (lt - tl.n * cs);
  const int first = ((lo > 0) ? p.padded_bins[lo - 1] : 0) / XM;
  const int b = first + 2 * unit + (int)rank;
  tl.dummy = b >= p.padded_bins[lo] / XM;
  tl.row0 = (tl.dummy ? p.nblk_cap : b) * XM;  // past the last row: loads read zeros
  return tl;
}

__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  // 32 rows of 16 bytes, eight rows (128 B) per core matrix, no swizzle
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// Instruction descriptor, kind::mxf4: A and B e2m1 (1), K-major; bit 23 e8m0 scales; bits 4-5
// and 29-30 which of the four bytes of a scale word the MMA starts at (B, A); N >> 3, M >> 4.
__host__ __device__ constexpr uint32_t idesc_mx4(int M, int N, int sf) {
  return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 4) << 24) | ((uint32_t)sf << 29);
}

__device__ __forceinline__ void tc_mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], "
      "p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ int mx_snake(int r, int cluster, int nclusters) {
  return r * nclusters + ((r & 1) ? nclusters - 1 - cluster : cluster);
}

// Two MX blocks (64 columns of H) of this thread's row from gate g and up u.
__device__ __forceinline__ void glu_store(const MxParams &p, const uint32_t (&g)[2][32],
                                          const uint32_t (&u)[2][32], int row, int n, int half) {
  uint32_t sc[2];
  uint4 *dst = reinterpret_cast<uint4 *>(p.hq + (size_t)row * (p.f >> 1) + n * 64 + half * 32);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float v[32];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v[i] = silu_f(__uint_as_float(g[j][i])) * __uint_as_float(u[j][i]);
      m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    sc[j] = mx4_scale_byte(m);
    const float inv = mx4_inverse(min(sc[j], 252u));
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = v[8 * q + i] * inv;
      w[q] = (sc[j] == 255u) ? 0u : mx4_pack8(o);
    }
    dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  *reinterpret_cast<uint16_t *>(p.hs + mx4_scale_word(row, n, p.f >> 7) + 2 * half) =
      (uint16_t)(sc[0] | (sc[1] << 8));
}

template <bool GLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(X_THREADS, 1)
    k_mx4_gemm(const __grid_constant__ MxParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_u32 = smem_u32(smem_raw);
  uint8_t *tiles = smem_raw + ((1024u - (base_u32 & 1023u)) & 1023u);
  // operands of all stages first (1024-byte aligned), then result boxes, scales, barriers
  uint8_t *outbuf = tiles + X_STAGES * 2 * X_OP;
  uint8_t *scales = outbuf + X_EPI * X_BOX;
  uint64_t *bars = reinterpret_cast<uint64_t *>(scales + X_STAGES * (X_SFA + X_SFB));
  uint64_t *full = bars, *empty = bars + X_STAGES;
  uint64_t *tfull = bars + 2 * X_STAGES, *tempty = tfull + 1, *drain = tfull + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tfull + 3);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *ustart = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(bars) + 256);  // [E + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < X_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * X_EPI);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.ta);
    prefetch_tmap(&p.tsa);
    prefetch_tmap(&p.tb[rank]);
    prefetch_tmap(&p.tsb[0]);
    prefetch_tmap(&p.tsb[1]);
  }
  pdl_wait();  // the next kernel is released as this grid's CTAs exit
  for (int e = threadIdx.x; e < p.E; e += X_THREADS) {
    const int blocks = (p.padded_bins[e] - ((e > 0) ? p.padded_bins[e - 1] : 0)) / XM;
    ustart[e + 1] = (blocks + 1) / 2;
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      int v = (e < p.E) ? ustart[e + 1] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int nv = __shfl_up_sync(0xFFFFFFFFu, v, off);
        if (lane >= off) v += nv;
      }
      if (e < p.E) ustart[e + 1] = carry + v;
      carry += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (lane == 0) ustart[0] = 0;
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, X_TMEM);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = ustart[p.E] * p.n_tiles;
  const int k_stages = (p.k_tiles + 1) / 2;
  const uint32_t leader_full0 = mapa_shared(smem_u32(&full[0]), 0);
  const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    for (int r = 0, t = mx_snake(0, cluster, nclusters); ok && t < total;
         t = mx_snake(++r, cluster, nclusters)) {
      const MxTile tl = mx_decode(p, t, ustart, rank);
      // B rows: this CTA's half; scale row tiles of both halves
      const int brow = GLU ? tl.e * p.f + tl.n * (XN / 2)
                           : tl.e * p.h + tl.n * XN + (int)rank * (XN / 2);
      const int s0 = (GLU ? brow : tl.e * p.h + tl.n * XN) / 128;
      const int s1 = GLU ? s0 : s0 + 1;
      for (int kb = 0; kb < k_stages; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, p.status, abort_flag, p.wait_cycles)) {
          ok = false;
          break;
        }
        const uint32_t bar = leader_full0 + (uint32_t)(stage * sizeof(uint64_t));
        if (p.inject && leader && issued == 0) {
          // test-only stall: this stage is never armed, so the MMA's wait on it expires
        } else {
          uint8_t *sa = tiles + stage * 2 * X_OP;
          uint8_t *sf = scales + stage * (X_SFA + X_SFB);
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * X_STAGE);
          tma_load_2d_pair(sa, &p.ta, bar, kb * (XK / 2), tl.row0);
          tma_load_2d_pair(sa + X_OP, &p.tb[rank], bar, kb * (XK / 2), brow);
          // scale tiles of K tiles 2 kb, 2 kb + 1 (one past an odd end is loaded, not used)
          tma_load_2d_pair(sf, &p.tsa, bar, 0, tl.row0 / 128 * p.k_tiles + 2 * kb);
          tma_load_2d_pair(sf + X_SFA, &p.tsb[0], bar, 0, s0 * p.k_tiles + 2 * kb);
          tma_load_2d_pair(sf + 2 * X_SFA, &p.tsb[1], bar, 0, s1 * p.k_tiles + 2 * kb);
        }
        ++issued;
        if (++stage == X_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (leader)  // every issued copy (of both CTAs) has landed before exit
      for (long long i = (issued > X_STAGES ? issued - X_STAGES : 0); i < issued; ++i)
        mbar_wait_plain(&full[i % X_STAGES], (uint32_t)((i / X_STAGES) & 1), p.wait_cycles);
  } else if (warp == 1 && lane == 0 && leader) {
    // ---------------- scales and MMAs (leader only) ----------------
    int stage = 0;
    uint32_t phase = 0, acc_phase = 0;
    for (int r = 0, t = mx_snake(0, cluster, nclusters); t < total;
         t = mx_snake(++r, cluster, nclusters)) {
      if (!mbar_wait(tempty, acc_phase ^ 1u, p.status, abort_flag, p.wait_cycles)) break;
      tc_fence_after();
      bool ok = true;
      for (int kb = 0; kb < k_stages; ++kb) {
        if (!mbar_wait(&full[stage], phase, p.status, abort_flag, p.wait_cycles)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(tiles + stage * 2 * X_OP), b = a + X_OP;
        const uint32_t sf = smem_u32(scales + stage * (X_SFA + X_SFB));
        const uint32_t ca = tmem_base + X_SF_COL + 32 * stage, cb = ca + 8;
        const int kt = min(2, p.k_tiles - 2 * kb);  // 128-wide K tiles in this stage
        for (int j = 0; j < kt; ++j) {
          tc_cp_scales(ca + 4 * j, sdesc_scales(sf + j * kMx4TileBytes));
          tc_cp_scales(cb + 8 * j, sdesc_scales(sf + X_SFA + j * kMx4TileBytes));
          tc_cp_scales(cb + 8 * j + 4, sdesc_scales(sf + 2 * X_SFA + j * kMx4TileBytes));
        }
        for (int j = 0; j < kt; ++j) {
#pragma unroll
          for (int i = 0; i < 2; ++i)  // 64 K (32 bytes, two scales) each
            tc_mma_mx4(tmem_base, sdesc_kmajor_sw128(a + (2 * j + i) * 32),
                       sdesc_kmajor_sw128(b + (2 * j + i) * 32), idesc_mx4(2 * XM, XN, 2 * i),
                       ca + 4 * j, cb + 8 * j, (kb | j | i) != 0 ? 1u : 0u);
        }
        tc_commit_pair_mc(&empty[stage]);
        if (++stage == X_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      tc_commit_pair_mc(tfull);
      acc_phase ^= 1u;
    }
    tc_commit_pair(drain);
    mbar_wait_plain(drain, 0, p.wait_cycles);
  } else if (warp >= 2) {
    // ---------------- epilogue (both CTAs) ----------------
    const int sub = warp & 3;          // tensor-memory lanes of this warp
    const int half = (warp - 2) >> 2;  // its half of the columns
    const uint32_t box = smem_u32(outbuf) + (uint32_t)((warp - 2) * X_BOX);
    uint32_t acc_phase = 0;
    for (int r = 0, t = mx_snake(0, cluster, nclusters); t < total;
         t = mx_snake(++r, cluster, nclusters)) {
      const MxTile tl = mx_decode(p, t, ustart, rank);
      const int row = tl.row0 + sub * 32 + lane;
      float wr = 0.0f;
      if (!GLU && !tl.dummy)
        wr = bfp_row_weight(p.padded_bins, p.bins, p.indices, p.weights, tl.e, row);
      int good = 1;
      if (lane == 0) good = mbar_wait(tfull, acc_phase, p.status, abort_flag, p.wait_cycles) ? 1 : 0;
      if (!__shfl_sync(0xFFFFFFFFu, good, 0)) break;
      acc_phase ^= 1u;
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(sub * 32) << 16);
      uint32_t v0[2][32], v1[2][32];
      // GLU: 64 gate columns and their 64 up columns; DOWN: 128 columns
      const int c0 = GLU ? 64 * half : 128 * half, c1 = GLU ? 128 + c0 : c0 + 64;
      tmem_ld32(tb + c0, v0[0]);
      tmem_ld32(tb + c0 + 32, v0[1]);
      tmem_ld32(tb + c1, v1[0]);
      tmem_ld32(tb + c1 + 32, v1[1]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty);  // accumulator free: values in registers
      if (tl.dummy) continue;
      if (GLU) {
        glu_store(p, v0, v1, row, tl.n, half);
      } else {
        const int n0 = tl.n * XN + half * 128;
        if (n0 >= p.h) continue;
        uint32_t mb = 0u;  // largest magnitude, as integers (NaN above inf)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          mb = max(max(mb, max(v0[0][i] & 0x7FFFFFFFu, v0[1][i] & 0x7FFFFFFFu)),
                   max(v1[0][i] & 0x7FFFFFFFu, v1[1][i] & 0x7FFFFFFFu));
        const float m = __uint_as_float(mb);
        float stored;
        const float k = bfp_scale(m * fabsf(wr), stored) * wr;
        p.yscale[(size_t)row * dmoe_scale_stride(p.h) + n0 / 128] = stored;
#pragma unroll
        for (int b = 0; b < 2; ++b) {  // 64 columns per box
          const uint32_t(&v)[2][32] = b ? v1 : v0;
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          const uint32_t dst = box + (uint32_t)(lane * 128);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[i] = pack_f16x2(__uint_as_float(v[c >> 2][8 * (c & 3) + 2 * i]) * k,
                                __uint_as_float(v[c >> 2][8 * (c & 3) + 2 * i + 1]) * k);
            st_shared_v4(dst + (uint32_t)((c ^ (lane & 7)) << 4), o[0], o[1], o[2], o[3]);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d_u32(&p.ty, box, n0 + 64 * b, tl.row0 + sub * 32);
            bulk_commit();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, X_TMEM);
  }
}

// Elements [rows, cols / 2] bytes: boxes of 128 rows x 128 bytes, 128-byte swizzle.
bool map_codes(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols / 2, rows}, strides[1] = {cols / 2};
  cuuint32_t box[2] = {XK / 2, XM}, estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles [rows/128 * cols/128] of 512 bytes (128 words): boxes of two consecutive tiles.
bool map_scales(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {kMx4TileBytes / 4, rows / 128 * (cols / 128)}, strides[1] = {kMx4TileBytes};
  cuuint32_t box[2] = {kMx4TileBytes / 4, 2}, estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Y_pad [rows, cols] fp16: boxes of 32 rows x 64 columns, 128-byte swizzle.
bool map_rows16(CUtensorMap *m, void *ptr, uint64_t rows, uint64_t cols) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * 2};
  cuuint32_t box[2] = {64, 32}, estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, ptr, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool GLU>
cudaError_t launch_mx(const GemmProblem &g, MxParams &p, cudaStream_t st) {
  p.padded_bins = g.padded_bins;
  p.bins = g.bins;
  p.indices = g.indices;
  p.weights = g.weights;
  p.E = g.E;
  p.h = g.h;
  p.f = g.f;
  p.nblk_cap = g.nblk_cap;
  p.status = g.status;
  p.inject = take_inject_stall();
  p.wait_cycles = p.inject ? kInjectedWaitCycles : kWaitCycles;
  // units whose A rows (2 x 128 x K / 2 bytes each) fill about 40 MB of L2 share B tiles
  const long long per_unit = 2LL * XM * p.k_tiles * 64;
  const long long group = (40LL << 20) / per_unit;
  p.group = (int)(group < 1 ? 1 : group > 64 ? 64 : group);
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  static int max_clusters = 0;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(k_mx4_gemm<GLU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)X_SMEM);
    if (attr_err != cudaSuccess) return;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (device_sm_count() / 2), 1, 1);
    cfg.blockDim = dim3(X_THREADS, 1, 1);
    cfg.dynamicSmemBytes = X_SMEM;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k_mx4_gemm<GLU>, &cfg) != cudaSuccess || n < 1)
      n = device_sm_count() / 2;
    max_clusters = n;
  });
  if (attr_err != cudaSuccess) return attr_err;
  const long long max_tiles = ((long long)g.nblk_cap / 2 + g.E) * p.n_tiles;
  const long long clusters = max_tiles < max_clusters ? max_tiles : max_clusters;
  return launch_pdl(k_mx4_gemm<GLU>, (int)(2 * clusters), X_THREADS, X_SMEM, st, p);
}

}  // namespace

cudaError_t launch_mx4_glu(const GemmProblem &g, const void *xq, const void *xs, const void *w1,
                           const void *s1, const void *w3, const void *s3, void *hq, void *hs,
                           cudaStream_t st) {
  MxParams p;
  memset(&p, 0, sizeof(p));
  const uint64_t P = (uint64_t)g.nblk_cap * XM, EF = (uint64_t)g.E * g.f;
  if (!map_codes(&p.ta, xq, P, g.h) || !map_scales(&p.tsa, xs, P, g.h) ||
      !map_codes(&p.tb[0], w1, EF, g.h) || !map_scales(&p.tsb[0], s1, EF, g.h) ||
      !map_codes(&p.tb[1], w3, EF, g.h) || !map_scales(&p.tsb[1], s3, EF, g.h))
    return cudaErrorInvalidValue;
  p.ty = p.ta;
  p.hq = static_cast<uint8_t *>(hq);
  p.hs = static_cast<uint8_t *>(hs);
  p.n_tiles = g.f / (XN / 2);
  p.k_tiles = g.h / 128;
  return launch_mx<true>(g, p, st);
}

cudaError_t launch_mx4_down(const GemmProblem &g, const void *hq, const void *hs, const void *w2,
                            const void *s2, void *y_pad, float *y_scale, cudaStream_t st) {
  MxParams p;
  memset(&p, 0, sizeof(p));
  const uint64_t P = (uint64_t)g.nblk_cap * XM, EH = (uint64_t)g.E * g.h;
  if (!map_codes(&p.ta, hq, P, g.f) || !map_scales(&p.tsa, hs, P, g.f) ||
      !map_codes(&p.tb[0], w2, EH, g.f) || !map_scales(&p.tsb[0], s2, EH, g.f) ||
      !map_rows16(&p.ty, y_pad, P, g.h))
    return cudaErrorInvalidValue;
  p.tb[1] = p.tb[0];
  p.tsb[1] = p.tsb[0];
  p.yscale = y_scale;
  p.n_tiles = (g.h + XN - 1) / XN;
  p.k_tiles = g.f / 128;
  return launch_mx<false>(g, p, st);
}

}  // namespace dmoe
