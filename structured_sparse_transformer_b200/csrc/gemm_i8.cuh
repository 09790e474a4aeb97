// 8-bit forward product on CTA pairs (tcgen05 kind::i8, cta_group::2, sm_100a):
//   Y[T x N] = (Xq Wq^T) sw sx, optionally gelu of it.
//
// A = Wq (feature = tensor-memory lane), B = Xq (token = accumulator column), both K-major in
// rows of 128 bytes; exact 32-bit integer accumulation, then (float(acc) * sw[n]) * sx[t] in
// fp32 and one rounding to the dtype.  A pair computes 256 features x 256 tokens; each CTA
// holds 128 rows of Wq and 128 rows of Xq per 128-deep stage, the pair's even CTA issues the
// MMAs (K = 32 each).  Persistent over tiles, features fastest (the pairs running at once
// share token tiles through L2), two accumulators, so a tile's epilogue overlaps the next
// tile's main loop.
//
// Warps: 0 = TMA producer, 1 = TMEM allocation and (leader) MMA issue, 2-17 = epilogue, four
// groups of four warps on alternate 32-token chunks: registers -> 16-bit pairs ->
// stmatrix.trans into a staging tile [32 tokens x 32 features] -> one TMA store.  Every wait
// is bounded.
//
// Bound by the tensor cores: 32768 x 6400 x 1600 in 227-277 us (2.4-3.0 POP/s, by the box's power),
// 2047 x 1024 x 4096 with GELU in 14.2 us (its epilogue's 4 us a tile against 3 us of stages).  At
// 8192 tokens the tensor pipe is busy 68% of 63 us; DRAM reads are the operands once.
#pragma once
#include "gemm_sp.cuh"
#include "sp24_ops.cuh"

namespace sp24 {

constexpr int kI8EpiWarps = 16;
constexpr int kI8Threads = 64 + 32 * kI8EpiWarps;
constexpr int kI8BarBytes = 512;
constexpr int kI8TileBytes = 32 * 32 * 2;              // staging tile, 64B-swizzled

// gelu2 with the factor of t clamped as t's polynomial is (half_r2: at 4 sqrt 2).  A product past fp32's range
// then goes to its limit, infinity or 0, where |x| t would be infinity times 0; and beyond the clamp, where |x| R(|x|/sqrt 2)
// is nearly constant (1 - 1/x^2 + ... of sqrt(2/pi)), the tail is off by 3% at most, where |x| R(4) grows away from it.
__device__ __forceinline__ float2 gelu2_to_limits(float2 x) {
  const float2 ax = make_float2(fabsf(x.x), fabsf(x.y));
  const float2 t = __fmul2_rn(half_r2(ax), gauss_e2(x));
  const float2 c = make_float2(fminf(ax.x, 5.65685424949238f), fminf(ax.y, 5.65685424949238f));
  return __ffma2_rn(make_float2(-c.x, -c.y), t, make_float2(fmaxf(x.x, 0.0f), fmaxf(x.y, 0.0f)));
}

struct I8Geom {
  static constexpr int BN = 256;
  static constexpr int kSmemA = 128 * 128;
  static constexpr int kSmemB = (BN / 2) * 128;
  static constexpr int kStageBytes = kSmemA + kSmemB;
  static constexpr int kFixed = 1024 + kI8BarBytes + kI8EpiWarps * kI8TileBytes;
  static constexpr int kStages = (232448 - kFixed) / kStageBytes < 8 ? (232448 - kFixed) / kStageBytes : 8;
  static constexpr int kSmem = kStages * kStageBytes + kFixed;
  static constexpr int kChunks = BN / 32;
  static_assert(kStages >= 4 && 8 * (2 * kStages + 6) <= kI8BarBytes, "shared memory per CTA");
  static_assert(kStageBytes % 1024 == 0, "128B-swizzled tiles need 1 KB aligned starts");
};

template <bool BF16, bool GELU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                   const __grid_constant__ CUtensorMap tm_y, int N, int T, int num_kt, uint64_t wait_budget,
                   const float *__restrict__ sw, const float *__restrict__ sx) {
  using G = I8Geom;
  constexpr int BN = G::BN;
  constexpr int kStages = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *epi_smem = smem + kStages * G::kStageBytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + kI8EpiWarps * kI8TileBytes);
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
  const int num_mt = (N + 255) / 256;
  const int num_tiles = num_mt * ((T + BN - 1) / BN);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kI8EpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_x);
    prefetch_tensormap(&tm_y);
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

  if (warp == 0) {
    // ------------------------------------------------------ producer (both CTAs)
    uint32_t g = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < num_tiles; tile += npairs) {
      const int w_row = (tile % num_mt) * 256 + (int)rank * 128, x_row = (tile / num_mt) * BN + (int)rank * (BN / 2);
      for (int kt = 0; kt < num_kt; ++kt, ++g) {
        const int s = (int)(g % kStages);
        const bool got = mbar_wait_bounded(&empty[s], ((g / kStages) & 1u) ^ 1u, wait_budget, s_abort);
        if (!(ok = __all_sync(0xFFFFFFFFu, got))) break;
        if (elect_one()) {
          uint8_t *st = smem + s * G::kStageBytes;
          if (is_leader) mbar_arrive_expect_tx(&full[s], 2 * G::kStageBytes);
          tma_load_2d_pair(st, &tm_w, &full[s], kt * 128, w_row);
          tma_load_2d_pair(st + G::kSmemA, &tm_x, &full[s], kt * 128, x_row);
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
    constexpr uint32_t idesc = make_idesc_i8(256, BN);
    const uint64_t a_desc0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
    const uint64_t b_desc0 = smem_desc(smem_u32(smem + G::kSmemA), 16, 1024, kSwizzle128B);
    uint32_t g = 0;
    bool ok = true;
    int j = 0;
    for (int tile = pair; ok && tile < num_tiles; tile += npairs, ++j) {
      const int buf = j & 1;
      const bool freed = mbar_wait_bounded(&acc_empty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u, wait_budget, s_abort);
      if (!(ok = __all_sync(0xFFFFFFFFu, freed))) break;
      tc_fence_after();
      const uint32_t acc = tmem_base + (uint32_t)(buf * BN);
      for (int kt = 0; kt < num_kt; ++kt, ++g) {
        const int s = (int)(g % kStages);
        const bool got = mbar_wait_bounded(&full[s], (g / kStages) & 1u, wait_budget, s_abort);
        if (!(ok = __all_sync(0xFFFFFFFFu, got))) break;
        tc_fence_after();
        const uint64_t so = (uint64_t)((s * G::kStageBytes) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)   // 32 bytes along the 128-byte swizzled rows each
            tc_mma_i8_pair(acc, a_desc0 + so + 2 * kk, b_desc0 + so + 2 * kk, idesc, (kt != 0 || kk != 0) ? 1u : 0u);
          tc_commit_pair(&empty[s], 0x3);
          if (kt == num_kt - 1) tc_commit_pair(&acc_full[buf], 0x3);
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
    // Warp w drains lanes 32q..32q+31 (q = w%4) at the 32-token chunks grp, grp + 4.  Register
    // 4i + 2 sub + e of block [h][g], lane l: feature 16h + 8 sub + l/4, token 16g + 8i +
    // 2(l%4) + e of the chunk.
    const int ew = warp - 2, grp = ew >> 2, q = warp & 3;
    uint8_t *stg = epi_smem + ew * kI8TileBytes;
    const uint32_t stg_u32 = smem_u32(stg);
    const int lr = lane >> 2, lc = 2 * (lane & 3);
    bool alive = true;
    int j = 0;
    for (int tile = pair; alive && tile < num_tiles; tile += npairs, ++j) {
      const int m0 = (tile % num_mt) * 256 + (int)rank * 128 + 32 * q, n0 = (tile / num_mt) * BN;
      const int nch = min(G::kChunks, (T - n0 + 31) / 32);
      float fw[4];   // [2h + sub]
#pragma unroll
      for (int e = 0; e < 4; ++e) fw[e] = m0 + 8 * e + lr < N ? __ldg(sw + m0 + 8 * e + lr) : 0.0f;
      float2 fx[2][2];   // the first chunk's token scales, [g][i]
      auto load_sx = [&](int c0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = c0 + 8 * e + lc;
          fx[e >> 1][e & 1] = make_float2(t < T ? __ldg(sx + t) : 0.0f, t + 1 < T ? __ldg(sx + t + 1) : 0.0f);
        }
      };
      load_sx(n0 + 32 * grp);
      const int buf = j & 1;
      const bool got = mbar_wait_bounded(&acc_full[buf], (uint32_t)(j >> 1) & 1u, wait_budget, s_abort);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        alive = false;
        break;
      }
      tc_fence_after();
      const uint32_t t_base = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * BN);
      constexpr int kPerWarp = (G::kChunks + 3) / 4;
#pragma unroll
      for (int k = 0; k < kPerWarp; ++k) {
        const int ch = grp + 4 * k;
        uint32_t r[2][2][8];
        if (ch < nch) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < 2; ++g)
              tmem_ld_16x256b_x2(t_base + ((uint32_t)(16 * h) << 16) + (uint32_t)(32 * ch + 16 * g), r[h][g]);
          tmem_wait_ld();
#pragma unroll
          for (int hg = 0; hg < 4; ++hg) reg_fence(r[hg >> 1][hg & 1]);
        }
        if (k == kPerWarp - 1) {   // the accumulator goes back to the MMA
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_leader(&acc_empty[buf]);
        }
        if (ch >= nch) continue;
        const int c0 = n0 + 32 * ch;
        if (k > 0) load_sx(c0);
        uint32_t pk[2][2][4];   // [h][g][2i + sub]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float s = fw[2 * h + (e & 1)];
              const float2 x = fx[g][e >> 1];
              float2 v = make_float2((__int2float_rn((int)r[h][g][2 * e]) * s) * x.x,
                                     (__int2float_rn((int)r[h][g][2 * e + 1]) * s) * x.y);
              if (GELU) v = gelu2_to_limits(v);
              pk[h][g][e] = pack2<BF16>(v.x, v.y);
            }
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int g = 0; g < 2; ++g)
            stmatrix_x4_trans(stg_u32 + swz64(16 * g + 8 * (lane >> 4) + (lane & 7), 2 * h + ((lane >> 3) & 1)), pk[h][g]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && m0 < N) {   // the TMA unit clips features and tokens past the matrix
          tma_store_2d(&tm_y, stg, m0, c0);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
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

// ------------------------------------------------------------------ few tokens
// Where the 256-feature tiles above would leave most pairs idle and K is long: bound by reading Wq
// and by latency, so K is spread too.  A cluster of S CTAs (S = 1, 2, 4 or 8) computes 128
// features x TP tokens, each CTA an S-th of K: M = 128, N = TP MMAs (cta_group::1) on tiles that
// a warp (one elected lane issues) loads as fast as the ring of stages takes them.  The 32-bit
// integer partial sums meet through distributed shared memory: each CTA leaves its own in shared
// memory, and CTA r adds all of them for tokens r, r + S, ..., scales and stores (integer sums:
// the order does not matter).
// At T = 37, K = 5120, N = 1280: 6.7 us, where the pairs' five tiles would take 15.
constexpr int kI8sThreads = 64 + 256;                  // producer, MMA, eight epilogue warps
constexpr int kI8sMaxStages = 8;

template <int TP>
struct I8sGeom {
  static constexpr int kSmemW = 128 * 128;
  static constexpr int kStageBytes = kSmemW + TP * 128;
  static constexpr int kPartBytes = TP * 128 * 4;      // partial sums [token][feature], over the stages
  static constexpr int kBarBytes = 256;
  static constexpr int smem_for(int stages) {
    return (stages * kStageBytes > kPartBytes ? stages * kStageBytes : kPartBytes) + kBarBytes + 1024;
  }
  static constexpr int kMost = (232448 - kBarBytes - 1024) / kStageBytes;
  static constexpr int kStagesMost = kMost < kI8sMaxStages ? kMost : kI8sMaxStages;
  static_assert(TP == 16 || TP == 32 || TP == 64 || TP == 128, "token tiles");
  static_assert(smem_for(kStagesMost) <= 232448 && 8 * (2 * kI8sMaxStages + 2) + 16 <= kBarBytes, "shared memory per CTA");
};

template <int TP, bool BF16, bool GELU>
__global__ void __launch_bounds__(kI8sThreads)
    gemm_i8_few_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, int N, int T,
                       int num_kt, int split, int stages, uint64_t wait_budget, const float *__restrict__ sw,
                       const float *__restrict__ sx, uint16_t *__restrict__ Y) {
  using G = I8sGeom<TP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int body = max(stages * G::kStageBytes, G::kPartBytes);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + body);   // [stages] TMA -> MMA
  uint64_t *empty = full + kI8sMaxStages;                       // [stages] MMA -> TMA
  uint64_t *acc_full = empty + kI8sMaxStages;                   // MMA -> epilogue
  uint64_t *drain = acc_full + 1;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);
  int *part = reinterpret_cast<int *>(smem);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = blockIdx.x % split;
  const int f0 = (blockIdx.x / split) * 128, t0 = blockIdx.y * TP;
  T = min(T - t0, TP);   // tokens of this tile
  sx += t0;
  Y += (int64_t)t0 * N;
  const int kb = (int)((int64_t)rank * num_kt / split), ke = (int)((int64_t)(rank + 1) * num_kt / split);
  constexpr uint32_t kCols = TP < 32 ? 32 : TP;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  pdl_launch_dependents();
  pdl_wait();

  bool done = true;   // epilogue warps: the accumulator was there
  if (warp == 0) {
    int g = 0, s = 0;
    uint32_t turn = 0;   // of the ring (counted: a division by `stages` costs as much as the rest of the loop)
    for (int kt = kb; kt < ke; ++kt, ++g) {
      const bool got = mbar_wait_bounded(&empty[s], turn ^ 1u, wait_budget, s_abort);
      if (!__all_sync(0xFFFFFFFFu, got)) break;
      if (elect_one()) {
        uint8_t *st = smem + s * G::kStageBytes;
        mbar_arrive_expect_tx(&full[s], G::kStageBytes);
        tma_load_2d(st, &tm_w, &full[s], kt * 128, f0);
        tma_load_2d(st + G::kSmemW, &tm_x, &full[s], kt * 128, t0);
      }
      __syncwarp();
      if (++s == stages) {
        s = 0;
        turn ^= 1u;
      }
    }
    for (int i = g > stages ? g - stages : 0; i < g; ++i) {   // every copy lands before the block ends
      volatile int no_abort = 0;
      mbar_wait_bounded(&full[i % stages], (uint32_t)(i / stages) & 1u, kDrainBudget, &no_abort);
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = make_idesc_i8(128, TP);
    const uint64_t a_desc0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
    const uint64_t b_desc0 = smem_desc(smem_u32(smem + G::kSmemW), 16, 1024, kSwizzle128B);
    int s = 0;
    uint32_t turn = 0;
    bool ok = true;
    for (int kt = kb; kt < ke; ++kt) {
      const bool got = mbar_wait_bounded(&full[s], turn, wait_budget, s_abort);
      if (!(ok = __all_sync(0xFFFFFFFFu, got))) break;
      tc_fence_after();
      const uint64_t so = (uint64_t)((s * G::kStageBytes) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)   // 32 bytes along the 128-byte swizzled rows each
          tc_mma_i8(tmem_base, a_desc0 + so + 2 * kk, b_desc0 + so + 2 * kk, idesc, (kt != kb || kk != 0) ? 1u : 0u);
        tc_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == stages) {
        s = 0;
        turn ^= 1u;
      }
    }
    uint64_t *over = ok ? acc_full : drain;
    if (elect_one()) tc_commit(over);
    __syncwarp();
    // The last MMAs are over before tensor and shared memory go, even if an epilogue gave up waiting for them.
    volatile int no_abort = 0;
    mbar_wait_bounded(over, 0, kDrainBudget, &no_abort);
    // Tensor memory goes back before this CTA waits for its cluster: another of them may still be waiting for its
    // own, held by a kernel that in turn waits for what this one holds.
    if (split > 1) {
      named_barrier_sync(1, kI8sThreads - 32);   // the epilogue has read it
      cluster_arrive();
      tc_fence_after();
      tmem_dealloc(tmem_base, kCols);
      cluster_wait();
    }
  } else if (warp >= 2) {
    // This lane's feature of the tile; the two warps of a lane quadrant take tokens in turn.
    const int q = warp & 3, f = 32 * q + lane, turn = (warp - 2) >> 2;
    const float w = f0 + f < N ? __ldg(sw + f0 + f) : 0.0f;
    // kB sums of one feature, tokens t, t + step, ...: all scales are loaded before any is used.
    // (Two at a time where there are few tokens: a short kernel's time is also that of fetching its
    // code.)
    constexpr int kB = TP <= 32 ? 2 : 8;
    auto put = [&](int t, int step, const int (&acc)[kB]) {
      float x[kB];
#pragma unroll
      for (int i = 0; i < kB; ++i) x[i] = t + i * step < T ? __ldg(sx + t + i * step) : 0.0f;
#pragma unroll
      for (int i = 0; i < kB; i += 2) {
        float2 y = make_float2((__int2float_rn(acc[i]) * w) * x[i], (__int2float_rn(acc[i + 1]) * w) * x[i + 1]);
        if (GELU) y = gelu2_to_limits(y);
        const uint32_t v = pack2<BF16>(y.x, y.y);
        uint16_t *at = Y + (int64_t)(t + i * step) * N + f0 + f;
        if (t + i * step < T) at[0] = (uint16_t)(v & 0xFFFFu);
        if (t + (i + 1) * step < T) at[(int64_t)step * N] = (uint16_t)(v >> 16);
      }
    };
    const bool got = mbar_wait_bounded(acc_full, 0, wait_budget, s_abort);
    done = __all_sync(0xFFFFFFFFu, got);
    if (done) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 16 * turn; c < T; c += 32) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)c, r);
        tmem_wait_ld();
        regs_fence(r);
        if (split > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(c + i) * 128 + f] = (int)r[i];
        } else if (f0 + f < N) {
#pragma unroll
          for (int i = 0; i < 16; i += kB) {
            int v[kB];
#pragma unroll
            for (int e = 0; e < kB; ++e) v[e] = (int)r[i + e];
            if (c + i < T) put(c + i, 1, v);
          }
        }
      }
    }
    tc_fence_before();
    if (split > 1) {
      named_barrier_arrive(1, kI8sThreads - 32);
      cluster_sync();   // every CTA's sums are in its shared memory
      if (done && f0 + f < N) {
        // kB tokens at a time, four CTAs' words of them in flight together.
#pragma unroll 1
        for (int t = rank + kB * split * turn; t < T; t += 2 * kB * split) {
          int sum[kB] = {};
#pragma unroll 1
          for (int c0 = 0; c0 < split; c0 += 4) {
            int v[4][kB];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t remote = cluster_addr(smem_u32(part + f), (uint32_t)min(c0 + c, split - 1));
#pragma unroll
              for (int i = 0; i < kB; ++i)
                v[c][i] = c0 + c < split && t + i * split < T ? ld_cluster_s32(remote + 512u * (uint32_t)(t + i * split)) : 0;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < kB; ++i) sum[i] += v[c][i];
          }
          put(t, split, sum);
        }
      }
    }
  }
  if (split > 1) {
    __syncwarp();
    if (warp == 0) cluster_sync();
    __syncwarp();
    cluster_sync();   // no CTA leaves while its sums are read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1 && split == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kCols);
  }
}

// ------------------------------------------------------------------ one to eight tokens
// Bound by reading Wq once, and by latency: no tensor memory, no barriers, no tensor maps to
// encode on the host.  A block takes four features; a thread takes every 128th 16-byte unit of
// K for all four and TT tokens (dp4a, exact), so each unit of Xq serves four rows of Wq.
constexpr int kI8vThreads = 128;
constexpr int kI8vRows = 4;

template <int TT, int KB, bool BF16, bool GELU>
__global__ void __launch_bounds__(kI8vThreads)
    gemv_i8_kernel(const int8_t *__restrict__ Xq, const float *__restrict__ sx, int T, int K,
                   const int8_t *__restrict__ Wq, const float *__restrict__ sw, int N, uint16_t *__restrict__ Y) {
  __shared__ int s_sum[kI8vThreads / 32][kI8vRows * TT];
  pdl_launch_dependents();
  pdl_wait();
  const int n0 = blockIdx.x * kI8vRows;
  const int4 *w = reinterpret_cast<const int4 *>(Wq + (int64_t)n0 * K);
  const int4 *x = reinterpret_cast<const int4 *>(Xq);
  const int units = K >> 4;
  int acc[kI8vRows][TT] = {};
  // KB units of a thread in flight at once, the last of them guarded one by one (a remainder loop
  // would take K = 6400, 400 units, in turns of one load latency each: 12.4 us at N = 6400, T = 1,
  // against 10.0).  One where a thread has no more (K <= 2048): twice the blocks fit an SM
  // (1600 x 6400 at T = 2: 3.9 us against 5.0).
  for (int u0 = threadIdx.x; u0 < units; u0 += KB * kI8vThreads) {
    int4 wv[KB][kI8vRows], xv[KB][TT];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int u = u0 + i * kI8vThreads;
      const bool in = u < units;
#pragma unroll
      for (int r = 0; r < kI8vRows; ++r) wv[i][r] = in ? __ldcs(w + (int64_t)r * units + u) : make_int4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[i][t] = in ? __ldg(x + (int64_t)min(t, T - 1) * units + u) : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < KB; ++i)
#pragma unroll
      for (int r = 0; r < kI8vRows; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          acc[r][t] = __dp4a(wv[i][r].x, xv[i][t].x,
                             __dp4a(wv[i][r].y, xv[i][t].y, __dp4a(wv[i][r].z, xv[i][t].z, __dp4a(wv[i][r].w, xv[i][t].w, acc[r][t]))));
  }
#pragma unroll
  for (int r = 0; r < kI8vRows; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int v = __reduce_add_sync(0xFFFFFFFFu, acc[r][t]);
      if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5][kI8vRows * t + r] = v;
    }
  __syncthreads();
  const int t = threadIdx.x / kI8vRows, n = n0 + threadIdx.x % kI8vRows;
  if (t < T && t < TT) {
    int v = 0;
#pragma unroll
    for (int i = 0; i < kI8vThreads / 32; ++i) v += s_sum[i][threadIdx.x];
    const float y = (__int2float_rn(v) * __ldg(sw + n)) * __ldg(sx + t);
    Y[(int64_t)t * N + n] = (uint16_t)f32_to_bits<BF16>(GELU ? gelu2_to_limits(make_float2(y, y)).x : y);
  }
}

}  // namespace sp24
