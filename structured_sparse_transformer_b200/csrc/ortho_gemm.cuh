// The Newton-Schulz products of the orthogonalisation (sm_100a).
//
// Per round, on the short side m of a stack of matrices X [m x n]:
//   Gram    G = X X^T / s^2            (X = s times the iterate)
//   Poly    P = a I + b G + c G^2      (G symmetric, so G^2 = G G^T)
//   Apply   X <- P X
// The last round's product with X goes to its destination in a kernel of its own
// (orth_last_kernel): the 16-bit result, or the weight, W <- keep W - step (P X), W16 <- W.
//
// orth_products_kernel is one cooperative launch of CTA pairs (tcgen05 cta_group::2, 256 x 256
// tiles, fp16 operands, fp32 accumulation) that runs all other phases one after another.  A
// phase needs everything the one before wrote, so at its end every CTA counts up a counter of
// the phase once its epilogue warps' stores are complete, and every TMA producer waits for the
// count and tells its epilogue warps: tensor memory, barriers and descriptors stay set up.
// (As 15 launches, each phase paid for launch, set-up and drain: about 9 us each.)  At 1600 x 6400
// this kernel's 14 phases take 302 us, 240 us of them stages at 0.36-0.40 us; the rest is the
// exchange of split tiles and the hand-over between phases.
// Small matrices (CLUSTER) take a cluster of CTA pairs each instead: they need not wait for one
// another, no cooperative launch is needed, and the counts become arrivals on an mbarrier of
// every CTA of the cluster instead of counters in L2.
//
// Gram and Poly are symmetric: only tiles on and below the diagonal are computed, and a tile
// below it is stored a second time, transposed (stmatrix.trans on the same registers), so
// they cost half of the full product.  Where a phase has fewer tiles than pairs, or a last
// wave does, its tiles are split along K (PairSchedule).  Each part then finishes its share of
// the tile's 32-column chunks: it passes the others' chunks on as fp32 partial sums and adds
// what they passed for its own, in part order (every part writes and reads (s-1)/s of a tile,
// where one part adding all of them would wait for s-1 whole tiles).
//
// orth_last_kernel's tensor-memory lanes are the matrix's columns, so that a warp's 32 lanes
// touch 32 neighbouring entries of a row whatever its alignment: a tall matrix takes P X as
// it is (X holds its transpose), a wide one (P X)^T = X^T P with X as the MN-major A operand.
//
// Fewer bits: the iterate, G and P are held in fp16.  With X scaled by a power of two s near
// sqrt(n), its entries are of the order of one whatever the size of the matrix and at most 2 s,
// so fp16 neither overflows nor loses small entries, and its 11-bit significand leaves about
// 1e-3 of relative error after five rounds, where bf16 (8 bits) leaves about 9e-3.  Folding
// a I into P (instead of adding a X in the epilogue) spares the epilogue a read of X and
// leaves the same error.
//
// Warps: 0 = TMA producer, 1 = TMEM allocation and (leader) MMA issue, 2-9 = epilogue, two
// groups of four warps on one half of the columns each.  A phase's tail is its last tiles'
// epilogues, so a warp takes half of its 32 x 128 block through every step at once (tensor
// memory -> registers -> fp16 pairs -> stmatrix -> TMA store): chunk by chunk, each step's
// latency is paid four times (3.6 us a tile).  Every wait is bounded.
#pragma once
#include "gemm_sp.cuh"
#include "sp24_ops.cuh"

namespace sp24 {

enum : int { kOrthGram = 0, kOrthPoly = 1, kOrthApply = 2 };

constexpr int kOgTileBytes = 32 * 32 * 2;              // staging tile: 32 x 32 16-bit values, 64B-swizzled
constexpr int kOgBarBytes = 512;
constexpr int kOgEpiWarps = 8;
constexpr int kOgThreads = 64 + 32 * kOgEpiWarps;
constexpr int kOgStageBytes = 2 * 128 * 128;           // A 128 rows and B 128 rows (or two atoms) of 128 bytes
constexpr int kOgChunks = 4;                           // 32-column chunks of a warp: 128 of the tile's 256 columns
constexpr int kOgStagingBytes = kOgChunks * kOgTileBytes;   // per epilogue warp
constexpr int kOgStages = 5;
constexpr int kOgSmem = kOgStages * kOgStageBytes + kOgEpiWarps * kOgStagingBytes + kOgBarBytes + 1024;
constexpr int kOgMaxSplit = 4;                         // parts of a split tile (chunk kk of n belongs to part kk parts / n)
constexpr int kOgMaxPairs = 80;
constexpr int kOgMaxSteps = 16;
// Partial sums of one CTA of a split tile: per epilogue warp and chunk, the registers of its
// tensor-memory load as eight float4 per lane.
constexpr int64_t kOgPartFloats = (int64_t)kOgEpiWarps * kOgChunks * 8 * 32 * 4;
// Counters at the front of the workspace, zero at launch: per phase, the CTAs that have finished
// it; then per (CTA, epilogue warp), 1 + the last phase whose partial sums it has passed on.
constexpr int kOgPhaseCounters = 64;
constexpr int kOgCounters = kOgPhaseCounters + 2 * kOgMaxPairs * kOgEpiWarps;
static_assert(3 * kOgMaxSteps <= kOgPhaseCounters, "a counter per phase");
static_assert(kOgSmem <= 232448 && 8 * (2 * kOgStages + 7 + kOgEpiWarps) <= kOgBarBytes,
              "shared memory per CTA");

struct OrthMaps {
  // Boxes of 64 columns x 128 rows (rows) or 64 rows (half: a K-major operand of narrow tiles,
  // or X MN-major); st: 32 x 32 store tiles.
  CUtensorMap x_rows[2], x_half[2], x_st[2], g_rows, g_half, g_st, p_rows, p_st;
};

struct OrthProducts {
  int m, n;                  // short and long side
  int batch, phases;
  int bn[3];                 // by kind: columns of a tile (256 or 128),
  int tiles[3];              //   tiles per matrix,
  int split[3];              //   parts of a tail tile
  uint64_t wait_budget;
  float gram_alpha;          // 1 / s^2
  const float *gamma;        // [batch] round 0: s X0 = gamma X
  int cluster;               // CLUSTER: CTAs per matrix
  float a, b, c;
  float *part;
  unsigned *counters;
};

struct OrthPhase {
  int kind, in, num_kt, bn, tiles, split;
  __device__ OrthPhase(const OrthProducts &p, int ph) {
    kind = ph % 3;
    in = (ph / 3) & 1;
    num_kt = ((kind == kOrthGram ? p.n : p.m) + 63) >> 6;
    bn = p.bn[kind];
    tiles = p.batch * p.tiles[kind];
    split = p.split[kind];
  }
};

// Tiles of a symmetric product: rows in blocks of 256, columns in blocks of bn (R = 256/bn per
// row block); row block i has column blocks 0 .. R(i+1)-1, cut at the matrix's edge.
__host__ __device__ constexpr int64_t orth_sym_tiles(int64_t m, int bn) {
  const int64_t rb = (m + 255) / 256, r = 256 / bn, cb = (m + bn - 1) / bn;
  return r * rb * (rb - 1) / 2 + (cb < r * rb ? cb : r * rb);
}

// Matrix, first row and first column of a tile; `below`: strictly below the diagonal blocks.
__device__ __forceinline__ void orth_tile(const OrthProducts &p, const OrthPhase &f, int b0, int t, int &b, int &m0, int &n0,
                                          bool &below) {
  b = t / p.tiles[f.kind];
  t -= b * p.tiles[f.kind];
  b += b0;
  if (f.kind != kOrthApply) {
    const int R = 256 / f.bn;
    int i = (int)((sqrtf(1.0f + 8.0f * (float)t / (float)R) - 1.0f) * 0.5f);
    while (R * i * (i + 1) / 2 > t) --i;
    while (R * (i + 1) * (i + 2) / 2 <= t) ++i;
    m0 = i * 256;
    n0 = (t - R * i * (i + 1) / 2) * f.bn;
    below = n0 < m0;
  } else {
    const int num_mt = (p.m + 255) / 256;
    m0 = (t % num_mt) * 256;
    n0 = (t / num_mt) * f.bn;
    below = false;
  }
}

// Passes on a warp's chunks that other parts finish.  Not inlined: inlined, the compiler keeps
// its registers beside the epilogue's and spills.
__device__ __noinline__ void orth_pass_chunks(uint32_t taddr, int nch, int halves, int part, int parts, float4 *slot) {
#pragma unroll 1
  for (int kk = 0; kk < nch; ++kk) {
    if (((kk * parts) >> halves) == part) continue;
    uint32_t r[2][16];
    tmem_ld_16x256b_x4(taddr + (uint32_t)(32 * kk), r[0]);
    tmem_ld_16x256b_x4(taddr + (uint32_t)(32 * kk) + (16u << 16), r[1]);
    tmem_wait_ld();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      regs_fence(r[h]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        __stcg(slot + (kk * 8 + 4 * h + e) * 32,
               make_float4(__uint_as_float(r[h][4 * e]), __uint_as_float(r[h][4 * e + 1]),
                           __uint_as_float(r[h][4 * e + 2]), __uint_as_float(r[h][4 * e + 3])));
    }
  }
}

// Two 32-column chunks (the first n of them) as the fragments of 16x256b: [chunk][h].
__device__ __forceinline__ void orth_load_half(uint32_t taddr, int n, uint32_t (&r)[2][2][16]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < n) {
      tmem_ld_16x256b_x4(taddr + (uint32_t)(32 * k), r[k][0]);
      tmem_ld_16x256b_x4(taddr + (uint32_t)(32 * k) + (16u << 16), r[k][1]);
    }
  tmem_wait_ld();
#pragma unroll
  for (int k = 0; k < 4; ++k) regs_fence(r[k >> 1][k & 1]);
}

// Launched in clusters of 2 (a cooperative grid, all matrices in every phase), or with CLUSTER of
// p.cluster CTAs (cluster i has matrix i; no tile is split).
template <bool CLUSTER>
__global__ void __launch_bounds__(kOgThreads, 1)
    orth_products_kernel(const __grid_constant__ OrthMaps maps, const __grid_constant__ OrthProducts p) {
  constexpr int kStages = kOgStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *epi_smem = smem + kStages * kOgStageBytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + kOgEpiWarps * kOgStagingBytes);
  uint64_t *full = bars;                       // [stages] leader: TMA (both CTAs) -> MMA
  uint64_t *empty = bars + kStages;            // [stages] MMA -> this CTA's TMA
  uint64_t *acc_full = bars + 2 * kStages;     // [2] MMA -> this CTA's epilogue
  uint64_t *acc_empty = acc_full + 2;          // [2] leader: both epilogues -> MMA
  uint64_t *drain = acc_empty + 2;
  uint64_t *ready = drain + 1;                 // producer -> epilogue: the phase's inputs are written
  uint64_t *g_bars = ready + 1;                // [epilogue warps] G's entries of a Poly tile
  uint64_t *phase_done = g_bars + kOgEpiWarps; // CLUSTER: the cluster's epilogue warps have finished the phase
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(phase_done + 1);
  volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const uint32_t rank = cta & 1;               // in the pair
  const bool is_leader = rank == 0;
  const uint16_t pair_mask = (uint16_t)(3u << (cta - rank));
  const int pair = (int)(CLUSTER ? cta : blockIdx.x) >> 1;
  const int npairs = (int)(CLUSTER ? (unsigned)p.cluster : gridDim.x) >> 1;
  const int b0 = CLUSTER ? (int)blockIdx.x / p.cluster : 0;   // the first matrix
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kOgEpiWarps);
    }
    mbar_init(drain, 1);
    mbar_init(ready, 1);
    mbar_init(phase_done, (uint32_t)((CLUSTER ? p.cluster : 1) * kOgEpiWarps));
    for (int w = 0; w < kOgEpiWarps; ++w) mbar_init(&g_bars[w], 1);
    *s_abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&maps.x_rows[0]);
    prefetch_tensormap(&maps.g_rows);
    prefetch_tensormap(&maps.g_st);
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the cluster's barriers exist before any cross-CTA arrive or byte count
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  if (CLUSTER) {
    pdl_launch_dependents();
    pdl_wait();
  }

  if (warp == 0) {
    // ------------------------------------------------------ producer (both CTAs)
    // What does not depend on the phase before is done ahead of the wait for it.
    uint32_t g = 0;
    bool ok = true;
    for (int ph = 0; ok && ph < p.phases; ++ph) {
      const OrthPhase f(p, ph);
      const bool b_mn = f.kind == kOrthApply;
      const CUtensorMap *ma = f.kind == kOrthGram ? &maps.x_rows[f.in] : (f.kind == kOrthPoly ? &maps.g_rows : &maps.p_rows);
      const CUtensorMap *mb = b_mn ? &maps.x_half[f.in]
                                   : (f.bn == 256 ? ma : (f.kind == kOrthGram ? &maps.x_half[f.in] : &maps.g_half));
      if (lane == 0) {
        prefetch_tensormap(ma);
        prefetch_tensormap(mb);
      }
      PairSchedule sched(f.split, pair, npairs, f.tiles, f.num_kt);
      int tile, kb, ke, b = 0, m0 = 0, n0 = 0;
      bool below, more = sched.next(tile, kb, ke);
      if (more) orth_tile(p, f, b0, tile, b, m0, n0, below);
      bool up = true;   // all of the phase before is written
      if (CLUSTER) {
        if (ph > 0) up = mbar_wait_cluster_bounded(phase_done, (uint32_t)(ph - 1) & 1u, p.wait_budget, s_abort);
      } else if (ph > 0 && lane == 0) {
        up = flag_spin_bounded(p.counters + ph - 1, gridDim.x, p.wait_budget, s_abort);
      }
      if (!__all_sync(0xFFFFFFFFu, up)) break;
      __syncwarp();
      fence_proxy_async_all();
      if (lane == 0) mbar_arrive(ready);
      while (ok && more) {
        const int a_row = m0 + (int)rank * 128, b_row = n0 + (int)rank * (f.bn / 2);
        for (int kt = kb; kt < ke; ++kt, ++g) {
          const int s = (int)(g % kStages);
          const bool got = mbar_wait_bounded(&empty[s], ((g / kStages) & 1u) ^ 1u, p.wait_budget, s_abort);
          if (!(ok = __all_sync(0xFFFFFFFFu, got))) break;
          if (elect_one()) {
            uint8_t *st = smem + s * kOgStageBytes;
            if (is_leader) mbar_arrive_expect_tx(&full[s], 2 * (16384 + 64 * f.bn));
            // K-major: rows of 64 entries along K; MN-major: 64-column atoms of 64 rows.
            tma_load_3d_pair(st, ma, &full[s], kt * 64, a_row, b);
            if (b_mn) {
              tma_load_3d_pair(st + 16384, mb, &full[s], b_row, kt * 64, b);
              if (f.bn == 256) tma_load_3d_pair(st + 24576, mb, &full[s], b_row + 64, kt * 64, b);
            } else {
              tma_load_3d_pair(st + 16384, mb, &full[s], kt * 64, b_row, b);
            }
          }
          __syncwarp();
        }
        more = sched.next(tile, kb, ke);
        if (more) orth_tile(p, f, b0, tile, b, m0, n0, below);
      }
    }
    // The leader's `full` barriers count both CTAs' bytes: let every copy land.
    if (is_leader && lane == 0) {
      for (uint32_t i = g > kStages ? g - kStages : 0; i < g; ++i) {
        volatile int no_abort = 0;
        mbar_wait_bounded(&full[i % kStages], (i / kStages) & 1u, kDrainBudget, &no_abort);
      }
    }
  } else if (warp == 1 && is_leader) {
    // ----------------------------------------------------- MMA issuer (leader)
    uint32_t g = 0;
    bool ok = true;
    int j = 0;
    for (int ph = 0; ok && ph < p.phases; ++ph) {
      const OrthPhase f(p, ph);
      const bool b_mn = f.kind == kOrthApply;
      const uint32_t idesc = make_idesc_dense(false, 256, f.bn) | (b_mn ? 1u << 16 : 0u);
      const uint64_t a_desc0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      const uint64_t b_desc0 = smem_desc(smem_u32(smem + 16384), b_mn ? 8192 : 16, 1024, kSwizzle128B);
      // A K step of 16 moves 32 bytes along the rows, or 16 rows of 128 bytes.
      const uint64_t b_step = b_mn ? 2048 >> 4 : 2;
      PairSchedule sched(f.split, pair, npairs, f.tiles, f.num_kt);
      int tile, kb, ke;
      for (; ok && sched.next(tile, kb, ke); ++j) {
        const int buf = j & 1;
        const bool freed = mbar_wait_bounded(&acc_empty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u, p.wait_budget, s_abort);
        if (!(ok = __all_sync(0xFFFFFFFFu, freed))) break;
        tc_fence_after();
        const uint32_t acc = tmem_base + (uint32_t)(buf * 256);
        for (int kt = kb; kt < ke; ++kt, ++g) {
          const int s = (int)(g % kStages);
          const bool got = mbar_wait_bounded(&full[s], (g / kStages) & 1u, p.wait_budget, s_abort);
          if (!(ok = __all_sync(0xFFFFFFFFu, got))) break;
          tc_fence_after();
          const uint64_t so = (uint64_t)((s * kOgStageBytes) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_f16_pair(acc, a_desc0 + so + 2 * kk, b_desc0 + so + kk * b_step, idesc,
                              (kt != kb || kk != 0) ? 1u : 0u);
            tc_commit_pair(&empty[s], pair_mask);
            if (kt == ke - 1) tc_commit_pair(&acc_full[buf], pair_mask);
          }
          __syncwarp();
        }
      }
    }
    // The last MMAs are over before tensor and shared memory go, even if an epilogue gave up waiting for them.
    if (elect_one()) tc_commit_pair(drain, (uint16_t)(1u << cta));
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait_bounded(drain, 0, kDrainBudget, &no_abort);
  } else if (warp >= 2) {
    // ---------------------------------------------------- epilogue (both CTAs)
    // Warp w drains lanes 32q..32q+31 (q = w%4) at its half (grp) of the columns, four or two chunks
    // of 32, two at a time: register 4i + 2 sub + e of [chunk][h], lane l, is row 16h + 8 sub +
    // l/4, column 8i + 2(l%4) + e of the chunk.
    const int ew = warp - 2, grp = ew >> 2, q = warp & 3;
    uint8_t *stg = epi_smem + ew * kOgStagingBytes;
    const uint32_t stg_u32 = smem_u32(stg);
    uint64_t *g_bar = &g_bars[ew];
    uint32_t g_issued = 0, g_used = 0;   // Poly tiles' loads of G
    const int lr = lane >> 2, lc = 2 * (lane & 3);
    // stmatrix and ldmatrix of a 16 x 16 block: lane l names row l%8 of matrix l/8; matrix
    // 2i + sub holds rows 8 sub.., columns 8i...
    const int d_row = 8 * ((lane >> 3) & 1) + (lane & 7), d_unit = lane >> 4;
    const int t_row = 8 * (lane >> 4) + (lane & 7), t_unit = (lane >> 3) & 1;
    // Split tiles: this warp's slot and counter; those of the part d pairs on are 2 d CTAs further.
    float4 *part_own = reinterpret_cast<float4 *>(p.part + (int64_t)blockIdx.x * kOgPartFloats) +
                       (int64_t)ew * kOgChunks * 8 * 32 + lane;
    unsigned *flag_own = p.counters + kOgPhaseCounters + (int64_t)blockIdx.x * kOgEpiWarps + ew;
    bool alive = true;
    int j = 0;
    for (int ph = 0; ph < p.phases; ++ph) {   // (to the end, with or without work: its barrier counts all warps)
      const OrthPhase f(p, ph);
      const CUtensorMap *mo = f.kind == kOrthGram ? &maps.g_st : (f.kind == kOrthPoly ? &maps.p_st : &maps.x_st[1 - f.in]);
      const int N = f.kind == kOrthApply ? p.n : p.m;
      if (lane == 0) prefetch_tensormap(mo);
      PairSchedule sched(f.split, pair, npairs, f.tiles, f.num_kt);
      int tile, kb, ke;
      for (; alive && sched.next(tile, kb, ke); ++j) {
        int b, m0, n0;
        bool below;
        orth_tile(p, f, b0, tile, b, m0, n0, below);
        m0 += (int)rank * 128 + 32 * q;
        n0 += f.bn / 2 * grp;
        const int halves = f.bn / 128;                        // pairs of chunks of this warp
        const bool split = !CLUSTER && ke - kb < f.num_kt;
        const int part = split ? pair % f.split : 0, parts = split ? f.split : 1;
        const int nch = min(2 * halves, (N - n0 + 31) >> 5);  // chunks inside the matrix (none: <= 0)
        const int buf = j & 1;
        auto mine = [&](int kk) { return kk < nch && ((kk * parts) >> halves) == part; };   // chunks that this part finishes
        // The other parts have passed on this warp's chunks: one lane waits for each.
        auto others_ready = [&]() {
          bool ready_flag = true;
          if (lane < parts && lane != part)
            ready_flag = flag_spin_bounded(flag_own + 2 * (lane - part) * kOgEpiWarps, (unsigned)ph + 1, p.wait_budget, s_abort);
          const bool all = __all_sync(0xFFFFFFFFu, ready_flag);
          __syncwarp();
          return all;
        };
        auto flag_passed = [&]() {
          __syncwarp();
          if (lane == 0) flag_store_release(flag_own, (unsigned)ph + 1);
        };
        auto release_acc = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_leader(&acc_empty[buf]);
        };
        const uint32_t t_base = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * 256 + f.bn / 2 * grp);

        // Poly: G's entries of the warp's chunks, by TMA into its staging tiles, once the phase
        // before is written (the producer acquired it for the CTA).
        int n_mine = 0;
#pragma unroll
        for (int kk = 0; kk < kOgChunks; ++kk) n_mine += mine(kk) ? 1 : 0;
        const bool any = n_mine > 0 && m0 < p.m;
        if (f.kind == kOrthPoly && any) {
          const bool up = mbar_wait_bounded(ready, (uint32_t)ph & 1u, p.wait_budget, s_abort);
          if (!__all_sync(0xFFFFFFFFu, up)) {
            alive = false;
            break;
          }
          ++g_issued;
          if (lane == 0) {
            bulk_wait_group_read<0>();   // the last tile's stores have read the staging tiles
            fence_proxy_async_all();
            mbar_arrive_expect_tx(g_bar, (uint32_t)(n_mine * kOgTileBytes));
            for (int kk = 0; kk < kOgChunks; ++kk)
              if (mine(kk)) tma_load_3d(stg + kk * kOgTileBytes, &maps.g_st, g_bar, n0 + 32 * kk, m0, b);
          }
          __syncwarp();
        }
        const bool got = mbar_wait_bounded(&acc_full[buf], (uint32_t)(j >> 1) & 1u, p.wait_budget, s_abort);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          alive = false;
          break;
        }
        tc_fence_after();
        if (split) {
          orth_pass_chunks(t_base, nch, halves, part, parts, part_own);
          flag_passed();
          if (!others_ready()) {
            alive = false;
            break;
          }
        }
        if (!any) {
          release_acc();
          continue;
        }
        if (f.kind == kOrthPoly) {
          const bool here = mbar_wait_bounded(g_bar, g_used & 1u, p.wait_budget, s_abort);
          if (!__all_sync(0xFFFFFFFFu, here)) {
            alive = false;
            break;
          }
          ++g_used;
        } else {
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
        }
        const float gamma = ph < 3 ? __ldg(p.gamma + b) : 1.0f;
        const float alpha = f.kind == kOrthGram ? p.gram_alpha * gamma * gamma : gamma;
#pragma unroll 1
        for (int half = 0; half < halves; ++half) {
          uint32_t r[2][2][16];
          orth_load_half(t_base + (uint32_t)(64 * half), nch - 2 * half, r);
          if (half == halves - 1) release_acc();
          if (!mine(2 * half) && !mine(2 * half + 1)) continue;
          if (split) {   // add the other parts' sums to its own, in part order
#pragma unroll 1
            for (int d = 0; d < parts; ++d) {
              if (d == part) continue;
              const float4 *src = part_own + (int64_t)(2 * (d - part)) * (kOgPartFloats / 4) + 2 * half * 8 * 32;
              float4 pv[2][2][4];
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  pv[k][e >> 2][e & 3] = mine(2 * half + k) ? __ldcg(src + (8 * k + e) * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 v = pv[k][e >> 2][e & 3];
                  uint32_t *a = &r[k][e >> 2][4 * (e & 3)];
                  a[0] = __float_as_uint(__fadd_rn(__uint_as_float(a[0]), v.x));
                  a[1] = __float_as_uint(__fadd_rn(__uint_as_float(a[1]), v.y));
                  a[2] = __float_as_uint(__fadd_rn(__uint_as_float(a[2]), v.z));
                  a[3] = __float_as_uint(__fadd_rn(__uint_as_float(a[3]), v.w));
                }
            }
          }
          // fp16 pairs in place (register 4g + e of [k][h], e = 2 (i % 2) + sub, i = 2g + e / 2),
          // and to the staging tiles.  A chunk that is not this part's is packed too, its
          // tile is not stored.
          const uint32_t d_at = stg_u32 + (uint32_t)(2 * half * kOgTileBytes);
          if (f.kind == kOrthPoly) {
            const int diag = m0 + lr - (n0 + 64 * half + lc);   // row - column of the first entry
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                  uint32_t gv[4];
                  ldmatrix_x4(d_at + (uint32_t)(k * kOgTileBytes) + swz64(16 * h + d_row, 2 * g + d_unit), gv);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const int d = diag + 16 * h + 8 * (e & 1) - 32 * k - 16 * g - 8 * (e >> 1);
                    float gx, gy;
                    unpack2<false>(gv[e], gx, gy);
                    const float x = fmaf(p.c, __uint_as_float(r[k][h][8 * g + 2 * e]), p.b * gx) + (d == 0 ? p.a : 0.0f);
                    const float y = fmaf(p.c, __uint_as_float(r[k][h][8 * g + 2 * e + 1]), p.b * gy) + (d == 1 ? p.a : 0.0f);
                    r[k][h][4 * g + e] = pack2<false>(x, y);
                  }
                }
            __syncwarp();   // every lane has its entries of G: P takes their places
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  r[k][h][e] = pack2<false>(alpha * __uint_as_float(r[k][h][2 * e]), alpha * __uint_as_float(r[k][h][2 * e + 1]));
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const uint32_t pk[4] = {r[k][h][4 * g], r[k][h][4 * g + 1], r[k][h][4 * g + 2], r[k][h][4 * g + 3]};
                stmatrix_x4(d_at + (uint32_t)(k * kOgTileBytes) + swz64(16 * h + d_row, 2 * g + d_unit), pk);
              }
          auto store = [&](bool transposed) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {   // the TMA unit clips rows and columns past the matrix
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int kk = 2 * half + k;
                if (!mine(kk)) continue;
                if (transposed) tma_store_3d(mo, stg + kk * kOgTileBytes, m0, n0 + 32 * kk, b);
                else tma_store_3d(mo, stg + kk * kOgTileBytes, n0 + 32 * kk, m0, b);
              }
              bulk_commit_group();
            }
          };
          store(false);
          if (below) {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                  const uint32_t pk[4] = {r[k][h][4 * g], r[k][h][4 * g + 1], r[k][h][4 * g + 2], r[k][h][4 * g + 3]};
                  stmatrix_x4_trans(d_at + (uint32_t)(k * kOgTileBytes) + swz64(16 * g + t_row, 2 * h + t_unit), pk);
                }
            store(true);
          }
        }
      }
      __syncwarp();
      if (lane == 0) bulk_wait_group<0>();   // this warp's stores of the phase are complete
      // No warp leaves a phase before its inputs were written (the producer acquired that for the CTA).
      // One without a tile would run ahead otherwise: `ready` and `phase_done` tell two phases apart, not
      // three, so its next wait for G would pass on the phase before last, and its arrival would
      // count for a phase that is still open.
      if (alive) {
        const bool up = mbar_wait_bounded(ready, (uint32_t)ph & 1u, p.wait_budget, s_abort);
        alive = __all_sync(0xFFFFFFFFu, up);
        __syncwarp();
      }
      if (!CLUSTER) {
        named_barrier_sync(1, 32 * kOgEpiWarps);
        if (ew == 0 && lane == 0 && alive) flag_add_release(p.counters + ph, 1u);
      } else if (alive && lane < p.cluster) {
        mbar_arrive_cluster(phase_done, (uint32_t)lane);
      }
    }
    if (lane == 0) {
      bulk_wait_group<0>();
      if (g_used < g_issued) {   // after an abort, let the load of G in flight land
        volatile int no_abort = 0;
        mbar_wait_bounded(g_bar, g_used & 1u, kDrainBudget, &no_abort);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  pair_abort_pause(s_abort);
  cluster_sync();  // the peer's MMAs, copies and arrivals into this CTA are over
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ------------------------------------------------------------------ short sides up to 256
// G and P are one 256 x 256 tile then, so every CTA pair of a matrix's cluster computes them for
// itself and keeps them in its shared memory: S holds 128 rows of G, then of P, per CTA in the
// K-major operand layout, four blocks of 64 columns, which serves as both operands of G G^T
// and as A of P X.  Gram takes X's rows as both operands too, so a stage is one 16 KB load.
// Only P X is shared out (tiles of bn columns), and only X' passes through global memory:
// one hand-over a round instead of three (orthogonalising 256 x 512 took 77 us with a cluster's
// phases, 64 this way; 64 x 64 50 and 39).
// With the last round's P stored by the first pair, orth_last_kernel follows as always.
constexpr int kOsStages = 8;
constexpr int kOsStageBytes = 128 * 128;
constexpr int kOsSBytes = 4 * 128 * 128;
constexpr int kOsStagingBytes = 2 * kOgTileBytes;      // per epilogue warp
constexpr int kOsSmem = kOsStages * kOsStageBytes + kOsSBytes + kOgEpiWarps * kOsStagingBytes + kOgBarBytes + 1024;
static_assert(kOsSmem <= 232448 && 8 * (2 * kOsStages + 8) <= kOgBarBytes, "shared memory per CTA");

__global__ void __launch_bounds__(kOgThreads, 1)
    orth_small_kernel(const __grid_constant__ OrthMaps maps, const __grid_constant__ CUtensorMap p_st128,
                      const __grid_constant__ OrthProducts p) {
  constexpr int kStages = kOsStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *s_mat = smem + kStages * kOsStageBytes;
  uint8_t *epi_smem = s_mat + kOsSBytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + kOgEpiWarps * kOsStagingBytes);
  uint64_t *full = bars;                       // [stages] leader: TMA (both CTAs) -> MMA
  uint64_t *empty = bars + kStages;            // [stages] MMA -> this CTA's TMA
  uint64_t *acc_full = bars + 2 * kStages;     // [2] MMA -> this CTA's epilogue
  uint64_t *acc_empty = acc_full + 2;          // [2] leader: both epilogues -> MMA
  uint64_t *drain = acc_empty + 2;
  uint64_t *s_ready = drain + 1;               // leader: both epilogues have written S
  uint64_t *round_done = s_ready + 1;          // the cluster's epilogue warps have finished the round
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(round_done + 1);
  volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const uint32_t rank = cta & 1;               // in the pair
  const bool is_leader = rank == 0;
  const uint16_t pair_mask = (uint16_t)(3u << (cta - rank));
  const int pair = (int)cta >> 1, npairs = p.cluster >> 1;
  const int b = (int)blockIdx.x / p.cluster;   // the matrix
  const int rounds = (p.phases + 1) / 3;
  const int kt_n = (p.n + 63) >> 6, kt_m = (p.m + 63) >> 6;
  const int bn = p.bn[kOrthApply], tiles = p.tiles[kOrthApply];

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kOgEpiWarps);
    }
    mbar_init(drain, 1);
    mbar_init(s_ready, 2 * kOgEpiWarps);
    mbar_init(round_done, (uint32_t)(p.cluster * kOgEpiWarps));
    *s_abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&maps.x_rows[0]);
    prefetch_tensormap(&maps.x_half[0]);
    prefetch_tensormap(&maps.x_st[1]);
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the cluster's barriers exist before any cross-CTA arrive or byte count
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------------ producer (both CTAs)
    uint32_t g = 0;
    bool ok = true;
    auto stage = [&](uint8_t *&st, uint64_t *&bar) {   // the next stage, once it is free
      const int s = (int)(g % kStages);
      const bool got = mbar_wait_bounded(&empty[s], ((g / kStages) & 1u) ^ 1u, p.wait_budget, s_abort);
      ok = __all_sync(0xFFFFFFFFu, got);
      st = smem + s * kOsStageBytes;
      bar = &full[s];
      if (ok) ++g;
      return ok;
    };
    uint8_t *st;
    uint64_t *bar;
    for (int r = 0; ok && r < rounds; ++r) {
      const int in = r & 1;
      if (r > 0) {   // X of this round is written
        const bool over = mbar_wait_cluster_bounded(round_done, (uint32_t)(r - 1) & 1u, p.wait_budget, s_abort);
        if (!(ok = __all_sync(0xFFFFFFFFu, over))) break;
        fence_proxy_async_all();
      }
      for (int kt = 0; kt < kt_n && stage(st, bar); ++kt) {
        if (elect_one()) {
          if (is_leader) mbar_arrive_expect_tx(bar, 2 * 64 * 256);
          tma_load_3d_pair(st, &maps.x_rows[in], bar, kt * 64, (int)rank * 128, b);
        }
        __syncwarp();
      }
      if (r + 1 == rounds) break;
      for (int t = pair; ok && t < tiles; t += npairs) {
        const int col = t * bn + (int)rank * (bn / 2);   // 64-column atoms of 64 rows; narrow tiles leave half a stage
        for (int kt = 0; kt < kt_m && stage(st, bar); ++kt) {
          if (elect_one()) {
            if (is_leader) mbar_arrive_expect_tx(bar, 2 * 64 * 256);
            tma_load_3d_pair(st, &maps.x_half[in], bar, col, kt * 64, b);
            tma_load_3d_pair(st + 8192, &maps.x_half[in], bar, bn == 256 ? col + 64 : col, kt * 64, b);
          }
          __syncwarp();
        }
      }
    }
    // The leader's `full` barriers count both CTAs' bytes: let every copy land.
    if (is_leader && lane == 0) {
      for (uint32_t i = g > kStages ? g - kStages : 0; i < g; ++i) {
        volatile int no_abort = 0;
        mbar_wait_bounded(&full[i % kStages], (i / kStages) & 1u, kDrainBudget, &no_abort);
      }
    }
  } else if (warp == 1 && is_leader) {
    // ----------------------------------------------------- MMA issuer (leader)
    constexpr uint32_t idesc_sym = make_idesc_dense(false, 256, 256);
    const uint32_t idesc_apply = make_idesc_dense(false, 256, bn) | (1u << 16);
    const uint64_t st_desc = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
    const uint64_t st_desc_mn = smem_desc(smem_u32(smem), 8192, 1024, kSwizzle128B);
    const uint64_t s_desc = smem_desc(smem_u32(s_mat), 16, 1024, kSwizzle128B);
    uint32_t g = 0, n_ready = 0;
    int j = 0;
    bool ok = true;
    auto acc_free = [&]() {
      const bool got = mbar_wait_bounded(&acc_empty[j & 1], ((uint32_t)(j >> 1) & 1u) ^ 1u, p.wait_budget, s_abort);
      ok = __all_sync(0xFFFFFFFFu, got);
      tc_fence_after();
      return ok;
    };
    auto loaded = [&](uint64_t &so) {
      const int s = (int)(g % kStages);
      const bool got = mbar_wait_bounded(&full[s], (g / kStages) & 1u, p.wait_budget, s_abort);
      ok = __all_sync(0xFFFFFFFFu, got);
      tc_fence_after();
      so = (uint64_t)((s * kOsStageBytes) >> 4);
      return ok;
    };
    auto s_written = [&]() {
      const bool got = mbar_wait_cluster_bounded(s_ready, n_ready & 1u, p.wait_budget, s_abort);
      ok = __all_sync(0xFFFFFFFFu, got);
      ++n_ready;
      tc_fence_after();
      return ok;
    };
    uint64_t so;
    for (int r = 0; ok && r < rounds; ++r) {
      if (!acc_free()) break;   // Gram: a stage is both operands
      for (int kt = 0; kt < kt_n && loaded(so); ++kt, ++g) {
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f16_pair(tmem_base + (uint32_t)((j & 1) * 256), st_desc + so + 2 * kk, st_desc + so + 2 * kk, idesc_sym,
                            (kt != 0 || kk != 0) ? 1u : 0u);
          tc_commit_pair(&empty[g % kStages], pair_mask);
          if (kt == kt_n - 1) tc_commit_pair(&acc_full[j & 1], pair_mask);
        }
        __syncwarp();
      }
      if (!ok) break;
      ++j;
      if (!s_written() || !acc_free()) break;   // Poly: S is both operands
      if (elect_one()) {
        for (int kt = 0; kt < kt_m; ++kt)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t at = s_desc + (uint64_t)(kt * (16384 >> 4) + 2 * kk);
            tc_mma_f16_pair(tmem_base + (uint32_t)((j & 1) * 256), at, at, idesc_sym, (kt != 0 || kk != 0) ? 1u : 0u);
          }
        tc_commit_pair(&acc_full[j & 1], pair_mask);
      }
      __syncwarp();
      ++j;
      if (r + 1 == rounds) break;
      if (!s_written()) break;
      for (int t = pair; ok && t < tiles; t += npairs) {   // P X: A is S, B a stage of X, MN-major
        if (!acc_free()) break;
        for (int kt = 0; kt < kt_m && loaded(so); ++kt, ++g) {
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_f16_pair(tmem_base + (uint32_t)((j & 1) * 256), s_desc + (uint64_t)(kt * (16384 >> 4) + 2 * kk),
                              st_desc_mn + so + (uint64_t)(kk * (2048 >> 4)), idesc_apply, (kt != 0 || kk != 0) ? 1u : 0u);
            tc_commit_pair(&empty[g % kStages], pair_mask);
            if (kt == kt_m - 1) tc_commit_pair(&acc_full[j & 1], pair_mask);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++j;
      }
    }
    // The last MMAs are over before tensor and shared memory go, even if an epilogue gave up waiting for them.
    if (elect_one()) tc_commit_pair(drain, (uint16_t)(1u << cta));
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait_bounded(drain, 0, kDrainBudget, &no_abort);
  } else if (warp >= 2) {
    // ---------------------------------------------------- epilogue (both CTAs)
    // Warps, chunks and registers as in orth_products_kernel.
    const int ew = warp - 2, grp = ew >> 2, q = warp & 3;
    uint8_t *stg = epi_smem + ew * kOsStagingBytes;
    const uint32_t stg_u32 = smem_u32(stg);
    const int lr = lane >> 2, lc = 2 * (lane & 3);
    const int d_row = 8 * ((lane >> 3) & 1) + (lane & 7), d_unit = lane >> 4;
    const int row0 = (int)rank * 128 + 32 * q;   // of the matrix
    const float gamma = __ldg(p.gamma + b);
    // This lane's address of the 16 x 16 block (h, g) of chunk kk in S.
    auto s_at = [&](int kk, int h, int g) {
      return smem_u32(s_mat) + (uint32_t)((2 * grp + (kk >> 1)) * 16384) +
             swz128(32 * q + 16 * h + d_row, 4 * (kk & 1) + 2 * g + d_unit);
    };
    bool alive = true;
    int j = 0;
    auto acc_here = [&]() {
      const bool got = mbar_wait_bounded(&acc_full[j & 1], (uint32_t)(j >> 1) & 1u, p.wait_budget, s_abort);
      alive = __all_sync(0xFFFFFFFFu, got);
      tc_fence_after();
      return alive;
    };
    auto release_acc = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(&acc_empty[j & 1]);
    };
    for (int r = 0; alive && r < rounds; ++r) {
      // G, then P, to S (entries past the matrix are zeros, but for a on P's diagonal, whose
      // rows are clipped and whose columns meet X's zero rows).
#pragma unroll 1
      for (int poly = 0; poly < 2 && acc_here(); ++poly, ++j) {
        const float alpha = r == 0 ? p.gram_alpha * gamma * gamma : p.gram_alpha;
        const uint32_t t_base = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)((j & 1) * 256 + 128 * grp);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t v[2][2][16];
          orth_load_half(t_base + (uint32_t)(64 * half), 2, v);
          if (half == 1) release_acc();
          if (poly) {
            const int diag = row0 + lr - (128 * grp + 64 * half + lc);   // row - column of the first entry
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                  uint32_t gv[4];
                  ldmatrix_x4(s_at(2 * half + k, h, g), gv);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const int dd = diag + 16 * h + 8 * (e & 1) - 32 * k - 16 * g - 8 * (e >> 1);
                    float gx, gy;
                    unpack2<false>(gv[e], gx, gy);
                    const float x = fmaf(p.c, __uint_as_float(v[k][h][8 * g + 2 * e]), p.b * gx) + (dd == 0 ? p.a : 0.0f);
                    const float y = fmaf(p.c, __uint_as_float(v[k][h][8 * g + 2 * e + 1]), p.b * gy) + (dd == 1 ? p.a : 0.0f);
                    v[k][h][4 * g + e] = pack2<false>(x, y);
                  }
                }
            __syncwarp();   // every lane has its entries of G: P takes their places
          } else {
#pragma unroll
            for (int kh = 0; kh < 4; ++kh)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[kh >> 1][kh & 1][e] = pack2<false>(alpha * __uint_as_float(v[kh >> 1][kh & 1][2 * e]),
                                                     alpha * __uint_as_float(v[kh >> 1][kh & 1][2 * e + 1]));
          }
#pragma unroll
          for (int kh = 0; kh < 4; ++kh)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const uint32_t *a = &v[kh >> 1][kh & 1][4 * g];
              const uint32_t pk[4] = {a[0], a[1], a[2], a[3]};
              stmatrix_x4(s_at(2 * half + (kh >> 1), kh & 1, g), pk);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (poly && r + 1 == rounds) {   // the last P goes to orth_last_kernel
          if (lane == 0 && pair == 0 && row0 < p.m) {
            for (int k = 0; k < 2; ++k)
              if (128 * grp + 64 * k < p.m)
                tma_store_3d(&p_st128, s_mat + (2 * grp + k) * 16384 + 32 * q * 128, 128 * grp + 64 * k, row0, b);
            bulk_commit_group();
          }
        } else if (lane == 0) {
          mbar_arrive_cluster(s_ready, cta - rank);
        }
      }
      if (!alive || r + 1 == rounds) break;
      for (int t = pair; t < tiles && acc_here(); t += npairs, ++j) {
        const int n0 = t * bn + bn / 2 * grp, halves = bn / 128;
        const int nch = min(2 * halves, (p.n - n0 + 31) >> 5);   // chunks inside the matrix (none: <= 0)
        const float alpha = r == 0 ? gamma : 1.0f;
        const uint32_t t_base = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)((j & 1) * 256 + bn / 2 * grp);
#pragma unroll 1
        for (int half = 0; half < halves; ++half) {
          uint32_t v[2][2][16];
          orth_load_half(t_base + (uint32_t)(64 * half), 2, v);
          if (half == halves - 1) release_acc();
          if (2 * half >= nch || row0 >= p.m) continue;
#pragma unroll
          for (int kh = 0; kh < 4; ++kh)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              v[kh >> 1][kh & 1][e] = pack2<false>(alpha * __uint_as_float(v[kh >> 1][kh & 1][2 * e]),
                                                   alpha * __uint_as_float(v[kh >> 1][kh & 1][2 * e + 1]));
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
#pragma unroll
          for (int kh = 0; kh < 4; ++kh)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const uint32_t *a = &v[kh >> 1][kh & 1][4 * g];
              const uint32_t pk[4] = {a[0], a[1], a[2], a[3]};
              stmatrix_x4(stg_u32 + (uint32_t)((kh >> 1) * kOgTileBytes) + swz64(16 * (kh & 1) + d_row, 2 * g + d_unit), pk);
            }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {   // the TMA unit clips rows and columns past the matrix
            tma_store_3d(&maps.x_st[1 - (r & 1)], stg, n0 + 64 * half, row0, b);
            if (2 * half + 1 < nch)
              tma_store_3d(&maps.x_st[1 - (r & 1)], stg + kOgTileBytes, n0 + 64 * half + 32, row0, b);
            bulk_commit_group();
          }
        }
      }
      if (!alive) break;
      if (lane == 0) bulk_wait_group<0>();   // this warp's part of X' is written
      __syncwarp();
      if (lane < p.cluster) mbar_arrive_cluster(round_done, (uint32_t)lane);
    }
    if (lane == 0) bulk_wait_group<0>();
  }

  tc_fence_before();
  __syncthreads();
  pair_abort_pause(s_abort);
  cluster_sync();  // the cluster's MMAs, copies and arrivals into this CTA are over
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ------------------------------------------------------------------ the last product
struct OrthLast {
  int rows, cols;            // the matrices; tall: X holds their transposes
  int num_kt;
  int batch, tiles;          // tiles per matrix
  uint64_t wait_budget;
  float alpha;               // 1/s, or step/s
  const float *gamma;        // [batch], with one round: s X0 = gamma X; else null
  float keep;
  float *w;                  // [batch][rows][cols]
  uint16_t *out16;           // [batch][rows][cols]; UPDATE: may be null
};

constexpr int kOlEpiWarps = 16;
constexpr int kOlThreads = 64 + 32 * kOlEpiWarps;
constexpr int kOlStages = 6;
constexpr int kOlSmem = kOlStages * kOgStageBytes + kOgBarBytes + 1024;   // (stages sized for BN = 256)

// 32 rows of a column with pitch ld, `left` of them inside the matrix (the last one repeats).
__device__ __forceinline__ void orth_load_rows(const float *src, int ld, int left, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i, src += i < left ? ld : 0) v[i] = __ldcs(src);
}

// Lane = column of the matrix, accumulator column = row.  Persistent over tiles of 256 columns x
// BN rows, two accumulators; BN = 128 where there would be few tiles.  16 epilogue warps take 32
// columns x BN/4 rows of the tile each, in chunks of 32 rows; the first chunk's W is loaded before
// the accumulator is ready, the second's before the first is stored, so 64 KB of W per SM are in
// flight behind the main loop.  Bound, with UPDATE, by memory: 10 bytes per entry.
template <bool BF16, bool UPDATE, bool TALL, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kOlThreads, 1)
    orth_last_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const OrthLast p) {
  constexpr int kStages = kOlStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * kOgStageBytes);
  uint64_t *full = bars;                       // [stages] leader: TMA (both CTAs) -> MMA
  uint64_t *empty = bars + kStages;            // [stages] MMA -> this CTA's TMA
  uint64_t *acc_full = bars + 2 * kStages;     // [2] MMA -> this CTA's epilogue
  uint64_t *acc_empty = acc_full + 2;          // [2] leader: both epilogues -> MMA
  uint64_t *drain = acc_empty + 2;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool is_leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int num_tiles = p.batch * p.tiles;
  const int num_mt = (p.cols + 255) / 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kOlEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrive or byte count
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  pdl_launch_dependents();
  pdl_wait();

  auto tile_at = [&](int tile, int &b, int &m0, int &n0) {
    b = tile / p.tiles;
    const int t = tile - b * p.tiles;
    m0 = (t % num_mt) * 256;
    n0 = (t / num_mt) * BN;
  };
  if (warp == 0) {
    // ------------------------------------------------------ producer (both CTAs)
    uint32_t g = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < num_tiles; tile += npairs) {
      int b, m0, n0;
      tile_at(tile, b, m0, n0);
      const int a_row = m0 + (int)rank * 128, b_row = n0 + (int)rank * (BN / 2);
      for (int kt = 0; kt < p.num_kt; ++kt, ++g) {
        const int s = (int)(g % kStages);
        const bool got = mbar_wait_bounded(&empty[s], ((g / kStages) & 1u) ^ 1u, p.wait_budget, s_abort);
        if (!(ok = __all_sync(0xFFFFFFFFu, got))) break;
        if (elect_one()) {
          uint8_t *st = smem + s * kOgStageBytes;
          if (is_leader) mbar_arrive_expect_tx(&full[s], 2 * (16384 + 64 * BN));
          // P K-major, X in two 64-column atoms of 64 rows.
          if (TALL) {
            tma_load_3d_pair(st, &tm_a, &full[s], kt * 64, a_row, b);
            tma_load_3d_pair(st + 16384, &tm_b, &full[s], b_row, kt * 64, b);
            if (BN == 256) tma_load_3d_pair(st + 24576, &tm_b, &full[s], b_row + 64, kt * 64, b);
          } else {
            tma_load_3d_pair(st, &tm_a, &full[s], a_row, kt * 64, b);
            tma_load_3d_pair(st + 8192, &tm_a, &full[s], a_row + 64, kt * 64, b);
            tma_load_3d_pair(st + 16384, &tm_b, &full[s], kt * 64, b_row, b);
          }
        }
        __syncwarp();
      }
    }
    // The leader's `full` barriers count both CTAs' bytes: let every copy land.
    if (is_leader) {
      for (uint32_t i = g > kStages ? g - kStages : 0; i < g; ++i) {
        volatile int no_abort = 0;
        mbar_wait_bounded(&full[i % kStages], (i / kStages) & 1u, kDrainBudget, &no_abort);
      }
    }
  } else if (warp == 1 && is_leader) {
    // ----------------------------------------------------- MMA issuer (leader)
    constexpr uint32_t idesc = make_idesc_dense(false, 256, BN) | (TALL ? 1u << 16 : 1u << 15);
    const uint64_t a_desc0 = smem_desc(smem_u32(smem), TALL ? 16 : 8192, 1024, kSwizzle128B);
    const uint64_t b_desc0 = smem_desc(smem_u32(smem + 16384), TALL ? 8192 : 16, 1024, kSwizzle128B);
    uint32_t g = 0;
    bool ok = true;
    int j = 0;
    for (int tile = pair; ok && tile < num_tiles; tile += npairs, ++j) {
      const int buf = j & 1;
      const bool freed = mbar_wait_bounded(&acc_empty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u, p.wait_budget, s_abort);
      if (!(ok = __all_sync(0xFFFFFFFFu, freed))) break;
      tc_fence_after();
      const uint32_t acc = tmem_base + (uint32_t)(buf * 256);
      for (int kt = 0; kt < p.num_kt; ++kt, ++g) {
        const int s = (int)(g % kStages);
        const bool got = mbar_wait_bounded(&full[s], (g / kStages) & 1u, p.wait_budget, s_abort);
        if (!(ok = __all_sync(0xFFFFFFFFu, got))) break;
        tc_fence_after();
        const uint64_t so = (uint64_t)((s * kOgStageBytes) >> 4);
        // A K step of 16 moves 32 bytes along the rows, or, MN-major, 16 rows of 128 bytes.
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f16_pair(acc, a_desc0 + so + kk * (TALL ? 2 : 2048 >> 4), b_desc0 + so + kk * (TALL ? 2048 >> 4 : 2),
                            idesc, (kt != 0 || kk != 0) ? 1u : 0u);
          tc_commit_pair(&empty[s], 0x3);
          if (kt == p.num_kt - 1) tc_commit_pair(&acc_full[buf], 0x3);
        }
        __syncwarp();
      }
    }
    // The last MMAs are over before tensor and shared memory go, even if an epilogue gave up waiting for them.
    if (elect_one()) tc_commit_pair(drain, 0x1);
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait_bounded(drain, 0, kDrainBudget, &no_abort);
  } else if (warp >= 2) {
    // ---------------------------------------------------- epilogue (both CTAs)
    const int ew = warp - 2, grp = ew >> 2, q = warp & 3;
    bool alive = true;
    int j = 0;
    for (int tile = pair; alive && tile < num_tiles; tile += npairs, ++j) {
      int b, m0, n0;
      tile_at(tile, b, m0, n0);
      const int col = m0 + (int)rank * 128 + 32 * q + lane;
      const int row0 = n0 + BN / 4 * grp;
      const int left = p.rows - row0;   // rows of the matrix from this warp's first on
      const int64_t at = ((int64_t)b * p.rows + row0) * p.cols;
      const float alpha = p.gamma ? p.alpha * __ldg(p.gamma + b) : p.alpha;
      const float *w_src = p.w + at + min(col, p.cols - 1);   // loads past the last column repeat it
      float pre[32];
      if (UPDATE && left > 0) orth_load_rows(w_src, p.cols, left, pre);
      const int buf = j & 1;
      const bool got = mbar_wait_bounded(&acc_full[buf], (uint32_t)(j >> 1) & 1u, p.wait_budget, s_abort);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        alive = false;
        break;
      }
      tc_fence_after();
      const uint32_t t_base = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * 256 + BN / 4 * grp);
#pragma unroll
      for (int k = 0; k < BN / 128; ++k) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_base + (uint32_t)(32 * k), r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));   // uses stay below the wait
        if (k == BN / 128 - 1) {   // the accumulator goes back to the MMA
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_leader(&acc_empty[buf]);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float acc = __uint_as_float(r[i]);
          r[i] = __float_as_uint(UPDATE ? fmaf(-alpha, acc, p.keep * pre[i]) : alpha * acc);
        }
        if (UPDATE && BN == 256 && k == 0 && left > 32) orth_load_rows(w_src + (int64_t)32 * p.cols, p.cols, left - 32, pre);
        const int n_rows = col < p.cols ? left - 32 * k : 0;
        float *w_at = p.w + at + (int64_t)(32 * k) * p.cols + col;
        uint16_t *o_at = p.out16 + at + (int64_t)(32 * k) * p.cols + col;
        const bool out = !UPDATE || p.out16 != nullptr;
#pragma unroll
        for (int i = 0; i < 32; ++i, w_at += p.cols, o_at += p.cols) {
          if (i < n_rows) {
            if (UPDATE) __stcs(w_at, __uint_as_float(r[i]));
            if (out) *o_at = (uint16_t)f32_to_bits<BF16>(__uint_as_float(r[i]));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  pair_abort_pause(s_abort);
  cluster_sync();  // the peer's MMAs, copies and arrivals into this CTA are over
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

}  // namespace sp24
