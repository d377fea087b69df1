// mx4_gemm.cu -- the expert FFN over many tokens with both operands of every product in the
// microscaled 4-bit format (dmoe_mx4 of dmoe.h), on the block-scaled tensor cores
// (tcgen05.mma kind::mxf4: e2m1 elements, one e8m0 scale per 32 along K, fp32 accumulation).
//
//   GLU   H = silu(X W1_e^T) * (X W3_e^T); H is converted to the format from fp32 in the epilogue
//         (a thread holds a row's 32-column block, so its maximum needs no exchange)
//   DOWN  Y_pad = w * (H W2_e^T) in block floating point, as the bf16 down GEMM writes it
//
// One SM pair per tile (cta_group::2, M = 256): at four bits a 128 x 256 tile on one SM would need
// 100 bytes of operands per clock from L2; a pair's 256 x 256 needs 66.  The unit of work is a
// pair of consecutive row blocks of one expert times a column tile, enumerated from padded_bins
// on the device.  GLU tiles are 256 columns wide (128 of gate, 128 of up).  DOWN tiles are 128
// wide with two accumulators: its K (ffn) is short, so that the hand-over of the accumulator,
// not the operands, bounds it.  Persistent clusters of two CTAs, 608 threads each:
//   warp 0      TMA producer: per stage of 256 K this CTA's half of B with 128-byte swizzle, and
//               the scale tiles of all rows of B (each SM of the pair multiplies by all of them);
//               and its 128 rows of A (16 KB) with their scales: GLU for every stage (a ring of six;
//               a stage's round trip is about 4000 clocks, its MMAs 512), DOWN (K up to 1024) once
//               per unit, which leaves room for a ring of nine stages of B.  A pair takes a unit's
//               columns in a row
//   warp 18     leader only: tcgen05.cp of a stage's scale tiles into tensor memory (512-byte
//               tiles, each 32 lanes x 4 columns repeated for the four lane groups)
//   warp 1      leader only: four MMAs of 64 K per stage.  One warp that did both took 1000
//               clocks a stage, where the MMAs take 512
//   warps 2..17 epilogue: a warp takes 32 rows and 64 accumulator columns
//               (eight warps with twice the columns measured level)
// Tensor memory: 256 accumulator columns, and 32 columns of scales per stage, which are
// rewritten only after the stage's MMAs are done.  Two GLU accumulators and scales do not fit in
// 512 columns; instead an epilogue warp takes its 64 columns into registers at once and releases
// the accumulator before it converts and stores them.
//
// Measured at T = 4096, hidden 2048, ffn 1024, E = 64, top-8 (412 GFLOP): GLU 70 us, DOWN 68 us;
// without the epilogue's work 67 and 61, without MMAs and scale copies as well 54 and 55.  Loads,
// MMAs and epilogue each come near the whole time, and overlap up to the ring's and the
// accumulators' hand-overs.  (A second pair of issuing warps for DOWN's second accumulator, each
// with a ring of its own: 66 us there, 110 instead of 105 at K = 256.  Weights fetched into L2 a
// tile or more ahead: slower.)
//
// Every mbarrier wait is bounded; on expiry the kernel sets DMOE_STATUS_TIMEOUT, raises an
// abort flag for the other roles of its CTA, drains what it issued and returns; DOWN's epilogue
// warps, which exchange maxima in pairs, leave in pairs.
#include <string.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "mx4.cuh"

namespace dmoe {

namespace {

constexpr int XM = 128;            // rows per CTA
constexpr int XK = 256;            // K per stage: one 128-byte swizzle row of elements
constexpr int X_A = XM * XK / 2;   // A's bytes per stage and CTA: 16 KB
constexpr int X_SF = 2 * kMx4TileBytes;  // scales of 128 rows: two column tiles
constexpr int X_EPI = 16;
constexpr int X_THREADS = 96 + 32 * X_EPI;
constexpr int X_BOX = 32 * 128;  // a result box: 32 rows x 128 B
constexpr int X_TMEM = 512;

// DOWN stages its results in one box per epilogue warp, GLU stores from registers.
template <bool GLU>
struct MxCfg {
  static constexpr int N = GLU ? 256 : 128;  // columns per tile (accumulator)
  static constexpr int nacc = GLU ? 1 : 2;
  static constexpr int sfb = N / 128;             // 128-row scale tiles of B
  static constexpr int b_bytes = N / 2 * XK / 2;  // this CTA's half of B
  static constexpr int b_stage = b_bytes + sfb * X_SF, a_stage = X_A + X_SF;
  static constexpr int stages = GLU ? 6 : 9;  // ring of B
  static constexpr int slots = GLU ? 6 : 4;   // stages of A
  static constexpr int out = GLU ? 0 : X_EPI * X_BOX;
  static constexpr int amax = GLU ? 0 : X_EPI * 32 * 4;
  static constexpr int tables = 2;  // per expert: units and row blocks before it
  // barriers: full, empty, sfull [stages], tfull, tempty, drain [2]; the tensor-memory address and
  // the abort flag behind them
  static constexpr int bar_bytes = ((3 * stages + 6) * 8 + 8 + 127) / 128 * 128;
  static constexpr size_t smem = 1024 + (size_t)stages * b_stage + (size_t)slots * a_stage + out +
                                 amax + bar_bytes + sizeof(int) * tables * (DMOE_MAX_EXPERTS + 1);
  // tensor memory: accumulators | scales of A's slots | scales of B's stages
  static constexpr int sfa_col = 256, sfb_col = sfa_col + 8 * slots;
  // arrivals that release an accumulator: the epilogue warps of both CTAs that read it
  static constexpr int epi_arrivals = 2 * X_EPI / nacc;
  static_assert(nacc * N <= sfa_col && sfb_col + 8 * sfb * stages <= X_TMEM, "tensor memory");
  static_assert(smem <= 227 * 1024, "shared memory");
};

struct MxParams {
  CUtensorMap ta, tsa;            // A elements and scales
  CUtensorMap tb[2], tsb[2];      // B of the leader's / the peer's half: W1 / W3, or W2 twice
  CUtensorMap ty;                 // DOWN: Y_pad
  const int32_t *padded_bins;
  const float *row_weight;  // DOWN: [P_max] routing weight of each padded row
  int E, h, f;
  int n_tiles, k_tiles;  // column tiles per unit; 128-wide K tiles
  int nblk_cap;
  int inject;
  long long wait_cycles;
  uint8_t *hq, *hs;  // GLU
  float *yscale;     // DOWN
  int32_t *status;
};

// A tile: column tile n of unit vu (of all experts' units in a row), this CTA's rows.
struct MxTile {
  int vu, n, e, row0;
  bool dummy;
  bool first;  // of its unit on this cluster
};

// A cluster's tiles, in order: as many whole units as every cluster can have, one from each round
// of `clusters` neighbouring units, so that clusters at work on the same expert share its
// weights in L2 (with contiguous shares of all tiles, units of an expert were far apart in time: the
// first product of the fine-grained layer took 78 us, now 70); then a contiguous share [r0, r0 + count - whole) of the remaining units' tiles.
struct MxShare {
  int cluster, clusters, n_tiles;
  int whole, count;  // tiles of whole units, of all
  int rest, r0;      // first of the remaining units; first tile from there on
  __device__ __forceinline__ MxShare(int c, int nc, int units, int nt)
      : cluster(c), clusters(nc), n_tiles(nt) {
    const int rounds = units / nc;
    rest = rounds * nc;
    whole = rounds * nt;
    const int tiles = (units - rest) * nt;  // nt times fewer than nc
    r0 = (int)((long long)c * tiles / nc);
    count = whole + (int)((long long)(c + 1) * tiles / nc) - r0;
  }
};

// The schedule's tables in shared memory, [E + 1] each: units and row blocks before expert e.
struct MxTables {
  const int *ustart, *bstart;
};

// The expert and rows of tl.vu.  The whole warp looks for the last expert with ustart[e] <= vu,
// first at every 32nd, then at the 32 from there on.
__device__ __forceinline__ void mx_unit(const MxParams &p, MxTile &tl, const MxTables &tb,
                                        uint32_t rank) {
  const int lane = threadIdx.x & 31;
  const int g = 32 * lane, e0 =
      32 * (__popc(__ballot_sync(0xFFFFFFFFu, g < p.E && tb.ustart[min(g, p.E)] <= tl.vu)) - 1);
  const int c = e0 + lane;
  tl.e = e0 + __popc(__ballot_sync(0xFFFFFFFFu, c < p.E && tb.ustart[min(c, p.E)] <= tl.vu)) - 1;
  const int b = tb.bstart[tl.e] + 2 * (tl.vu - tb.ustart[tl.e]) + (int)rank;
  tl.dummy = b >= tb.bstart[tl.e + 1];
  tl.row0 = (tl.dummy ? p.nblk_cap : b) * XM;  // past the last row: loads read zeros
}

// The cluster's i-th tile.
__device__ __forceinline__ MxTile mx_tile(const MxParams &p, const MxShare &sh, int i,
                                          const MxTables &tb, uint32_t rank) {
  MxTile tl;
  const bool whole = i < sh.whole;
  const int j = whole ? i : sh.r0 + i - sh.whole, u = j / sh.n_tiles;
  tl.n = j - u * sh.n_tiles;
  tl.vu = whole ? u * sh.clusters + sh.cluster : sh.rest + u;
  tl.first = tl.n == 0 || i == 0 || i == sh.whole;
  mx_unit(p, tl, tb, rank);
  return tl;
}

// ... from tl, the one `by` tiles before it.
__device__ __forceinline__ void mx_next(const MxParams &p, const MxShare &sh, MxTile &tl, int i,
                                        int by, const MxTables &tb, uint32_t rank) {
  if (tl.n + by < sh.n_tiles && (i < sh.whole || i - by >= sh.whole)) {  // of the same unit
    tl.n += by;
    tl.first = false;
  } else {
    tl = mx_tile(p, sh, i, tb, rank);
  }
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

// Arrival on a barrier of the pair's leader that hands over nothing but tensor memory already
// read (tcgen05.wait::ld and the fence come before it).  A cluster-scope release here would
// wait for this thread's earlier global stores: it took over 1000 clocks a tile.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// One lane of a converged warp.  The producer and MMA warps run their loops as whole warps and
// elect the lane only around the instructions: their operands then stay in uniform registers
// (as a loop of one lane the MMA warp took about 900 clocks a stage).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// silu(z) u with one reciprocal: e^-z overflowing to inf gives 1 / inf = 0, the limit.
__device__ __forceinline__ float silu_mul(float z, float u) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-z)));
  return z * r * u;
}

// One block (32 columns of H) of this thread's row from gate g and up u, block `blk` of the row.
__device__ __forceinline__ void glu_store(const MxParams &p, const uint32_t (&g)[32],
                                          const uint32_t (&u)[32], int row, int blk) {
  float v[32];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = silu_mul(__uint_as_float(g[i]), __uint_as_float(u[i]));
    m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  const uint32_t sc = mx4_scale_byte(m);
  const float inv = mx4_inverse(min(sc, 252u));
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[8 * q + i] * inv;
    w[q] = (sc == 255u) ? 0u : mx4_pack8(o);
  }
  *reinterpret_cast<uint4 *>(p.hq + (size_t)row * (p.f >> 1) + blk * 16) =
      make_uint4(w[0], w[1], w[2], w[3]);
  p.hs[mx4_scale_word(row, blk >> 2, p.f >> 7) + (blk & 3)] = (uint8_t)sc;
}

template <bool GLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(X_THREADS, 1)
    k_mx4_gemm(const __grid_constant__ MxParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_u32 = smem_u32(smem_raw);
  uint8_t *tiles = smem_raw + ((1024u - (base_u32 & 1023u)) & 1023u);
  using C = MxCfg<GLU>;
  constexpr int X_STAGES = C::stages;
  uint8_t *abuf = tiles, *bbuf = abuf + C::slots * X_A;  // elements: 1024-byte aligned
  uint8_t *outbuf = bbuf + X_STAGES * C::b_bytes;
  uint8_t *ascale = outbuf + C::out, *bscale = ascale + C::slots * X_SF;
  uint64_t *bars = reinterpret_cast<uint64_t *>(bscale + X_STAGES * C::sfb * X_SF);
  uint64_t *full = bars, *empty = bars + X_STAGES;
  uint64_t *sfull = bars + 2 * X_STAGES;  // leader: the stage's scales are in tensor memory
  uint64_t *tfull = bars + 3 * X_STAGES, *tempty = tfull + 2, *drain = tfull + 4;  // [2] each
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tfull + 6);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  float *amax = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(bars) + C::bar_bytes);
  int *ustart = reinterpret_cast<int *>(amax + MxCfg<GLU>::amax / 4);
  int *bstart = ustart + p.E + 1;  // [E + 1] each
  const MxTables tables{ustart, bstart};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < X_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], 1);
    }
    for (int a = 0; a < C::nacc; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], C::epi_arrivals);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.ta);
    prefetch_tmap(&p.tsa);
    prefetch_tmap(&p.tb[rank]);
    prefetch_tmap(&p.tsb[0]);
    prefetch_tmap(&p.tsb[1]);
  }
  // GLU: the gather lets this kernel start after its own wait, so the map is complete; only the
  // producer waits for the gather's rows.  (The next kernel is released as this grid's CTAs exit.)
  if (!GLU) pdl_wait();
  for (int e = threadIdx.x; e < p.E; e += X_THREADS) {
    const int end = __ldcg(p.padded_bins + e) / XM;
    const int first = (e > 0) ? __ldcg(p.padded_bins + e - 1) / XM : 0;
    ustart[e + 1] = (end - first + 1) / 2;
    bstart[e + 1] = end;
  }
  if (threadIdx.x == 0) bstart[0] = 0;
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
  const MxShare share(cluster, nclusters, ustart[p.E], p.n_tiles);
  const int count = share.count;
  const int k_stages = (p.k_tiles + 1) / 2;
  // DOWN: A stays in its slots while the unit's columns pass, in `groups` sets of slots by turns.
  // GLU, and a K too long for the slots: A passes through with B, stage by stage.  (For DOWN that
  // leaves four stages: hidden 4096, ffn 14336, E = 8, top-2 takes 399 us in all at 1024 tokens,
  // 3.5 times the floor of its weights' bytes.)
  const bool resident = !GLU && k_stages <= C::slots;
  const int groups = resident ? C::slots / k_stages : 1;
  const int ring = resident || GLU ? C::stages : C::slots;
  const uint32_t leader_full0 = mapa_shared(smem_u32(&full[0]), 0);
  const uint32_t leader_tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    int stage = 0, group = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    MxTile tl;
    if (count > 0) tl = mx_tile(p, share, 0, tables, rank);
    if (GLU) pdl_wait();
    for (int t = 0; ok && t < count; ++t) {
      const bool fresh = tl.first || !resident;  // A has to be loaded
      if (t > 0 && tl.first && ++group == groups) group = 0;
      // B rows: this CTA's half; scale row tiles of all of B
      const int brow =
          GLU ? tl.e * p.f + tl.n * 128 : tl.e * p.h + tl.n * 128 + (int)rank * 64;
      const int s0 = brow / 128 * p.k_tiles, sa0 = tl.row0 / 128 * p.k_tiles, row0 = tl.row0;
      for (int kb = 0; kb < k_stages; ++kb) {
        ok = mbar_wait(&empty[stage], phase ^ 1u, p.status, abort_flag, p.wait_cycles);
        if (resident && fresh) {  // the slot's last use, groups * k_stages stages ago at the latest
          const int last = (int)issued - groups * k_stages, turn = last / ring;
          if (ok && last >= 0)
            ok = mbar_wait(&empty[last - turn * ring], (uint32_t)turn & 1u, p.status, abort_flag,
                           p.wait_cycles);
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        const uint32_t bar = leader_full0 + (uint32_t)(stage * sizeof(uint64_t));
        // test-only stall (inject): the first stage is never armed, so the MMA's wait on it expires
        if (!(p.inject && leader && issued == 0) && elect_one()) {
          if (leader)
            mbar_arrive_expect_tx(&full[stage], 2 * (C::b_stage + (fresh ? C::a_stage : 0)));
          uint8_t *sf = bscale + stage * C::sfb * X_SF;
          // scale tiles of K tiles 2 kb, 2 kb + 1 (one past an odd end is loaded, not used)
          tma_load_2d_pair(bbuf + stage * C::b_bytes, &p.tb[rank], bar, kb * (XK / 2), brow);
          tma_load_2d_pair(sf, &p.tsb[0], bar, 0, s0 + 2 * kb);
          if (GLU) tma_load_2d_pair(sf + X_SF, &p.tsb[1], bar, 0, s0 + 2 * kb);
          if (fresh) {
            const int slot = resident ? group * k_stages + kb : stage;
            tma_load_2d_pair(abuf + slot * X_A, &p.ta, bar, kb * (XK / 2), row0);
            tma_load_2d_pair(ascale + slot * X_SF, &p.tsa, bar, 0, sa0 + 2 * kb);
          }
        }
        if (kb == 0 && t + 1 < count)  // the next tile, while this one loads
          mx_next(p, share, tl, t + 1, 1, tables, rank);
        ++issued;
        if (++stage == ring) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
    if (leader && lane == 0)  // every issued copy (of both CTAs) has landed before exit
      for (long long i = (issued > ring ? issued - ring : 0); i < issued; ++i)
        mbar_wait_plain(&full[i % ring], (uint32_t)((i / ring) & 1), p.wait_cycles);
  } else if ((warp == 1 || warp == X_EPI + 2) && leader) {
    // ---------------- MMAs (warp 1) and scale copies (the last warp), leader only ----------------
    const bool copier = warp != 1;
    const int n = count * k_stages;  // stages of this cluster, over all of its tiles
    // ring stage, K step, tile and its column, set of A's slots
    int stage = 0, kb = 0, t = 0, col = share.whole > 0 ? 0 : share.r0 % p.n_tiles, group = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    for (int i = 0; i < n; ++i) {
      bool ok = true;
      if (copier) {
        ok = mbar_wait(&full[stage], phase, p.status, abort_flag, p.wait_cycles);
      } else {
        if (kb == 0)
          ok = mbar_wait(&tempty[acc], acc_phase ^ 1u, p.status, abort_flag, p.wait_cycles);
        ok = ok && mbar_wait(&sfull[stage], phase, p.status, abort_flag, p.wait_cycles);
      }
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      const int slot = resident ? group * k_stages + kb : stage;
      const uint32_t ca = tmem_base + C::sfa_col + 8 * slot;
      const uint32_t cb = tmem_base + C::sfb_col + 8 * C::sfb * stage;
      const bool two = 2 * kb + 1 < p.k_tiles;  // 128-wide K tiles; the last stage may have one
      if (copier) {
        const bool fresh = t == 0 || col == 0 || t == share.whole || !resident;
        const uint64_t sa = sdesc_scales(smem_u32(ascale) + slot * X_SF);
        const uint64_t sb = sdesc_scales(smem_u32(bscale) + stage * C::sfb * X_SF);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (j == 1 && !two) break;
            if (fresh) tc_cp_scales(ca + 4 * j, sa + j * (kMx4TileBytes / 16));
#pragma unroll
            for (int q = 0; q < C::sfb; ++q)
              tc_cp_scales(cb + 4 * C::sfb * j + 4 * q, sb + (q * X_SF + j * kMx4TileBytes) / 16);
          }
          tc_commit_pair(&sfull[stage]);
        }
      } else {
        const uint64_t ad = sdesc_kmajor_sw128(smem_u32(abuf) + slot * X_A);
        const uint64_t bd = sdesc_kmajor_sw128(smem_u32(bbuf) + stage * C::b_bytes);
        const uint32_t d = tmem_base + (uint32_t)(acc * C::N);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (j == 1 && !two) break;
#pragma unroll
            for (int q = 0; q < 2; ++q)  // 64 K (32 bytes, two scales) each
              tc_mma_mx4(d, ad + 2 * (2 * j + q), bd + 2 * (2 * j + q),
                         idesc_mx4(2 * XM, C::N, 2 * q), ca + 4 * j, cb + 4 * C::sfb * j,
                         (kb | j | q) != 0 ? 1u : 0u);
          }
          tc_commit_pair_mc(&empty[stage]);
          if (kb == k_stages - 1) tc_commit_pair_mc(&tfull[acc]);
        }
      }
      __syncwarp();
      if (++stage == ring) {
        stage = 0;
        phase ^= 1u;
      }
      if (++kb == k_stages) {
        kb = 0;
        if (++acc == C::nacc) {
          acc = 0;
          acc_phase ^= 1u;
        }
        if (++col == p.n_tiles) {
          col = 0;
          if (++group == groups) group = 0;
        }
        if (++t == share.whole) col = share.r0 % p.n_tiles;
      }
    }
    if (elect_one()) tc_commit_pair(&drain[copier]);
    __syncwarp();
    mbar_wait_plain(&drain[copier], 0, p.wait_cycles);
  } else if (warp >= 2 && warp < X_EPI + 2) {
    // ---------------- epilogue (both CTAs) ----------------
    // GLU: 16 warps per tile, a quarter of the columns each.  DOWN: the two halves of the warps
    // take every second tile (accumulator), half of the columns each.
    const int sub = warp & 3;  // tensor-memory lanes of this warp
    const int quarter = (warp - 2) >> 2;
    const int part = GLU ? quarter : quarter & 1, mine_acc = GLU ? 0 : quarter >> 1;
    const uint32_t box = smem_u32(outbuf) + (uint32_t)((warp - 2) * X_BOX);
    // a tile's rows, and the routing weight of this thread's row, are looked up while the tile
    // before it is converted and stored
    auto weight_of = [&](const MxTile &tl) -> float {
      return (GLU || tl.dummy) ? 0.0f : __ldg(p.row_weight + tl.row0 + sub * 32 + lane);
    };
    uint32_t acc_phase = 0;
    int t = mine_acc;
    int good = 1;  // 0 once a wait of this warp expired
    MxTile nx;
    float wnx = 0.0f;
    if (t < count) {
      nx = mx_tile(p, share, t, tables, rank);
      wnx = weight_of(nx);
    }
    while (t < count) {
      const MxTile tl = nx;
      const float wr = wnx;
      const int row = tl.row0 + sub * 32 + lane;
      if (lane == 0 && good)
        good = mbar_wait(&tfull[mine_acc], acc_phase, p.status, abort_flag, p.wait_cycles) ? 1 : 0;
      good = __shfl_sync(0xFFFFFFFFu, good, 0);
      // DOWN: one warp of a pair may see the abort flag where the other's wait still passed, so a
      // warp goes on to the pair's next barrier, says so there, and both leave at the same tile
      if (GLU && !good) break;
      acc_phase ^= 1u;
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(sub * 32) << 16) + (uint32_t)(mine_acc * C::N);
      uint32_t v0[32], v1[32];
      // GLU: 32 gate columns and their 32 up columns; DOWN: 64 columns
      const int c0 = (GLU ? 32 : 64) * part, c1 = GLU ? 128 + c0 : c0 + 32;
      tmem_ld32(tb + c0, v0);
      tmem_ld32(tb + c1, v1);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && good)  // accumulator free: values in registers
        mbar_arrive_remote(leader_tempty0 + (uint32_t)(mine_acc * sizeof(uint64_t)));
      t += C::nacc;
      if (t < count) {
        const int vu = nx.vu;
        mx_next(p, share, nx, t, C::nacc, tables, rank);
        if (nx.vu != vu) wnx = weight_of(nx);
      }
      if (tl.dummy) continue;
      if (GLU) {
        glu_store(p, v0, v1, row, tl.n * 4 + part);
      } else {
        const int n0 = tl.n * 128 + part * 64;
        uint32_t mb = 0u;  // largest magnitude, as integers (NaN above inf)
#pragma unroll
        for (int i = 0; i < 32; ++i) mb = max(mb, max(v0[i] & 0x7FFFFFFFu, v1[i] & 0x7FFFFFFFu));
        constexpr uint32_t kExpired = 0xFFFFFFFFu;  // above every magnitude
        if (!good) mb = kExpired;
        // ... of the 128-column group: exchanged with the warp of its other 64 columns
        uint32_t *mine = reinterpret_cast<uint32_t *>(amax) + (warp - 2) * 32 + lane;
        uint32_t *other = mine + (part ? -128 : 128);  // four warps on
        const int bar = 1 + mine_acc * 4 + sub;
        *mine = mb;
        asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
        mb = max(mb, *other);
        asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");  // read before the next tile's
        if (mb == kExpired) break;  // in every lane of both warps
        float stored;
        const float k = bfp_scale(__uint_as_float(mb) * fabsf(wr), stored) * wr;
        if (part == 0) p.yscale[(size_t)row * dmoe_scale_stride(p.h) + n0 / 128] = stored;
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        const uint32_t dst = box + (uint32_t)(lane * 128);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t(&v)[32] = c < 4 ? v0 : v1;
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = pack_f16x2(__uint_as_float(v[8 * (c & 3) + 2 * i]) * k,
                              __uint_as_float(v[8 * (c & 3) + 2 * i + 1]) * k);
          st_shared_v4(dst + (uint32_t)((c ^ (lane & 7)) << 4), o[0], o[1], o[2], o[3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d_u32(&p.ty, box, n0, tl.row0 + sub * 32);
          bulk_commit();
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

// Elements [rows, cols / 2] bytes: boxes of box_rows x 128 bytes, 128-byte swizzle.
bool map_codes(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols / 2, rows}, strides[1] = {cols / 2};
  cuuint32_t box[2] = {XK / 2, box_rows}, estr[2] = {1, 1};
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
  p.E = g.E;
  p.h = g.h;
  p.f = g.f;
  p.nblk_cap = g.nblk_cap;
  p.status = g.status;
  p.inject = take_inject_stall();
  p.wait_cycles = p.inject ? kInjectedWaitCycles : kWaitCycles;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(k_mx4_gemm<GLU>, done, (int)MxCfg<GLU>::smem);
  if (e != cudaSuccess) return e;
  static std::once_flag once;
  static int max_clusters = 0;
  std::call_once(once, [] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (device_sm_count() / 2), 1, 1);
    cfg.blockDim = dim3(X_THREADS, 1, 1);
    cfg.dynamicSmemBytes = MxCfg<GLU>::smem;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k_mx4_gemm<GLU>, &cfg) != cudaSuccess || n < 1)
      n = device_sm_count() / 2;
    max_clusters = n;
  });
  const long long max_tiles = ((long long)g.nblk_cap / 2 + g.E) * p.n_tiles;
  const long long clusters = max_tiles < max_clusters ? max_tiles : max_clusters;
  return launch_pdl(k_mx4_gemm<GLU>, (int)(2 * clusters), X_THREADS, MxCfg<GLU>::smem, st, p);
}

}  // namespace

cudaError_t launch_mx4_glu(const GemmProblem &g, const void *xq, const void *xs, const void *w1,
                           const void *s1, const void *w3, const void *s3, void *hq, void *hs,
                           cudaStream_t st) {
  MxParams p;
  memset(&p, 0, sizeof(p));
  const uint64_t P = (uint64_t)g.nblk_cap * XM, EF = (uint64_t)g.E * g.f;
  if (!map_codes(&p.ta, xq, P, g.h, XM) || !map_scales(&p.tsa, xs, P, g.h) ||
      !map_codes(&p.tb[0], w1, EF, g.h, 128) || !map_scales(&p.tsb[0], s1, EF, g.h) ||
      !map_codes(&p.tb[1], w3, EF, g.h, 128) || !map_scales(&p.tsb[1], s3, EF, g.h))
    return cudaErrorInvalidValue;
  p.ty = p.ta;
  p.hq = static_cast<uint8_t *>(hq);
  p.hs = static_cast<uint8_t *>(hs);
  p.n_tiles = g.f / 128;
  p.k_tiles = g.h / 128;
  return launch_mx<true>(g, p, st);
}

cudaError_t launch_mx4_down(const GemmProblem &g, const void *hq, const void *hs, const void *w2,
                            const void *s2, const float *row_weight, void *y_pad, float *y_scale,
                            cudaStream_t st) {
  MxParams p;
  memset(&p, 0, sizeof(p));
  p.row_weight = row_weight;
  const uint64_t P = (uint64_t)g.nblk_cap * XM, EH = (uint64_t)g.E * g.h;
  if (!map_codes(&p.ta, hq, P, g.f, XM) || !map_scales(&p.tsa, hs, P, g.f) ||
      !map_codes(&p.tb[0], w2, EH, g.f, 64) || !map_scales(&p.tsb[0], s2, EH, g.f) ||
      !map_rows16(&p.ty, y_pad, P, g.h))
    return cudaErrorInvalidValue;
  p.tb[1] = p.tb[0];
  p.tsb[1] = p.tsb[0];
  p.yscale = y_scale;
  p.n_tiles = g.h / 128;
  p.k_tiles = g.f / 128;
  return launch_mx<false>(g, p, st);
}

}  // namespace dmoe
