// Tensor-core products of the optimiser's orthogonalisation (fp16 operands) and of the
// 8-bit forward (int8 operands), on CTA pairs (tcgen05 cta_group::2, sm_100a).
//
// One kernel, D[m0.., n0..] = A * B^T over a batch of matrices, with A read K-major in
// rows of 128 bytes (64 fp16 or 128 int8) and B either the same way or, for the product
// with X, MN-major.  A pair computes 256 x BN outputs; each CTA holds 128 rows of A and
// BN/2 rows (columns, MN-major) of B per stage, and the pair's even CTA issues the MMAs.
// Persistent: pair p takes tiles p, p + P, ...  Accumulators are double-buffered in tensor
// memory (2 x BN columns), so a tile's epilogue overlaps the next tile's main loop.
//
// Products (MODE):
//   kNtI8      Y[T x N] = (Xq Wq^T) sw sx [, GELU].  A = Wq (feature = tensor-memory lane),
//              B = Xq; exact 32-bit integer accumulation (kind::i8), then
//              (float(acc) * sw[n]) * sx[t] in fp32 and one rounding to the dtype.
//   kNtGram    G = alpha X X^T      (X = the iterate, fp16, scaled by s; alpha = 1/s^2)
//   kNtPoly    P = a I + b G + c G G^T   (G is symmetric, so G G^T = G^2)
//   kNtApply   X <- P X             (B = X read MN-major)
//   kNtOrth    the last product, stored as the 16-bit result (transposed for a tall matrix)
//   kNtMuon    the last product, applied to the weight: W <- keep W - step (P X), W16 <- W
// Gram and Poly are symmetric: only tiles on and below the diagonal are computed, and a
// tile strictly below it is stored a second time, transposed (stmatrix.trans on the same
// registers), so they cost half of the full product.
//
// Fewer bits: the iterate, G and P are held in fp16.  With X scaled by a power of two s
// near sqrt(longer side), its entries are of the order of one whatever the size of the
// matrix and at most 2 s, so fp16 neither overflows nor loses small entries, and its 11-bit
// significand leaves about 1e-3 of relative error after five rounds, where bf16 (8 bits)
// leaves about 9e-3; products accumulate in fp32.  Folding a I into P (instead of adding
// a X in the epilogue) spares the epilogue a read of X and measures the same error.
//
// Warps: 0 = TMA producer, 1 = TMEM allocation and (leader) MMA issue, 2-9 = epilogue,
// two groups of four warps on alternate 32-column chunks.  Every wait is bounded.
#pragma once
#include "gemm_sp.cuh"

namespace sp24 {

enum : int { kNtI8 = 0, kNtGram = 1, kNtPoly = 2, kNtApply = 3, kNtOrth = 4, kNtMuon = 5 };

constexpr int kNtEpiWarps = 8;
constexpr int kNtThreads = 64 + 32 * kNtEpiWarps;
constexpr int kNtBarBytes = 512;
constexpr int kNtTileBytes = 32 * 32 * 2;              // staging tile: 32 x 32 16-bit values, 64B-swizzled

template <int MODE, int BN>
struct NtGeom {
  static constexpr bool kSym = MODE == kNtGram || MODE == kNtPoly;
  static constexpr bool kBmn = MODE == kNtApply || MODE == kNtOrth || MODE == kNtMuon;   // B = X, MN-major
  static constexpr int kBK = MODE == kNtI8 ? 128 : 64; // K per stage (128 bytes)
  static constexpr int kSmemA = 128 * 128;
  static constexpr int kSmemB = (BN / 2) * 128;
  static constexpr int kStageBytes = kSmemA + kSmemB;
  static constexpr int kStaging = kSym ? 2 : 1;        // staging tiles per epilogue warp (direct + mirrored)
  static constexpr int kFree = 232448 - 1024 - kNtBarBytes - kNtEpiWarps * kStaging * kNtTileBytes;
  static constexpr int kStages = kFree / kStageBytes < 8 ? kFree / kStageBytes : 8;
  static constexpr int kSmem = kStages * kStageBytes + kNtEpiWarps * kStaging * kNtTileBytes + kNtBarBytes + 1024;
  static constexpr int kChunks = BN / 32;
  static constexpr int kPerWarp = (kChunks + 1) / 2;
  static_assert(BN == 64 || BN == 128 || BN == 256, "tile widths");
  static_assert(!kBmn || BN >= 128, "MN-major B comes in atoms of 64 columns per CTA");
  static_assert(kStages >= 4 && kSmem <= 232448 && 2 * kStages + 6 <= kNtBarBytes / 8, "shared memory per CTA");
  static_assert(kStageBytes % 1024 == 0 && kSmemB % 1024 == 0, "128B-swizzled tiles need 1 KB aligned starts");
  static_assert(2 * BN <= kTmemCols, "two accumulators in tensor memory");
};

struct NtArgs {
  int M, N;                  // output rows (features / short side) and columns (tokens / long side)
  int num_kt;                // K stages
  int batch, tiles;          // matrices, tiles per matrix
  uint64_t wait_budget;
  float alpha;               // Gram: 1/s^2; Orth: 1/s; Muon: step/s
  float a, b, c;             // Poly
  const uint16_t *gram;      // Poly: G, [batch][M][ld]
  int64_t gram_ld;
  const float *row_scale;    // I8: sw [M]
  const float *col_scale;    // I8: sx [N]
  uint16_t *out16;           // Orth: [batch][rows][cols]; Muon: W16 of the same layout, or null
  float *w;                  // Muon: fp32 weight [batch][rows][cols]
  float keep;                // Muon: 1 - lr * weight_decay
  int tall;                  // Orth, Muon: rows = N, cols = M (the matrix was transposed on the way in)
  int vec;                   // Orth, Muon: not tall, N even and pointers aligned for two entries at a time
  int tma_out;               // Orth: rows of out are whole 16-byte units, so it is stored by TMA
};

__device__ __forceinline__ void tma_load_3d_pair(void *smem_dst, const CUtensorMap *map, uint64_t *bar, int x, int y,
                                                 int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar) & kPairLeaderMask)
      : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *smem_src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(smem_u32(smem_src))
               : "memory");
}

// Dense 8-bit integer MMA of the pair (kind::i8, K = 32, 32-bit integer accumulation).
__device__ __forceinline__ void tc_mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::i8: D 32-bit integer, A and B signed, both K-major.
__host__ __device__ constexpr uint32_t make_idesc_i8(int m, int n) {
  return (2u << 4)                      // D format s32
         | (1u << 7)                    // A signed
         | (1u << 10)                   // B signed
         | ((uint32_t)(n >> 3) << 17)   // N / 8
         | ((uint32_t)(m >> 4) << 24);  // M / 16
}

// Four 8x8 16-bit matrices, as held (no transpose): register j of thread t is row t/4,
// columns 2(t%4) and 2(t%4)+1 of matrix j; lane 8j + r gives the address of its row r.
__device__ __forceinline__ void stmatrix_x4(uint32_t saddr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

// Tiles of a symmetric product: rows in blocks of 256, columns in blocks of BN (R = 256/BN
// per row block); row block i has column blocks 0 .. R(i+1)-1, cut at the matrix's edge.
__host__ __device__ constexpr int64_t nt_sym_tiles(int64_t m, int bn) {
  const int64_t rb = (m + 255) / 256, r = 256 / bn, cb = (m + bn - 1) / bn;
  return r * rb * (rb - 1) / 2 + (cb < r * rb ? cb : r * rb);
}

template <int MODE, int BN>
__device__ __forceinline__ void nt_tile(int t, const NtArgs &p, int &b, int &m0, int &n0, bool &mirror) {
  b = t / p.tiles;
  t -= b * p.tiles;
  if (NtGeom<MODE, BN>::kSym) {
    constexpr int R = 256 / BN;
    int i = (int)((sqrtf(1.0f + 8.0f * (float)t / (float)R) - 1.0f) * 0.5f);
    while (R * i * (i + 1) / 2 > t) --i;
    while (R * (i + 1) * (i + 2) / 2 <= t) ++i;
    const int j = t - R * i * (i + 1) / 2;
    m0 = i * 256;
    n0 = j * BN;
    mirror = n0 < m0;
  } else {
    const int num_mt = (p.M + 255) / 256;
    m0 = (t % num_mt) * 256;
    n0 = (t / num_mt) * BN;
    mirror = false;
  }
}

template <int MODE, int BN, bool BF16, bool GELU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kNtThreads, 1)
    sp24_gemm_nt_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                        const __grid_constant__ CUtensorMap tm_out, const NtArgs p) {
  using G = NtGeom<MODE, BN>;
  constexpr int kStages = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *epi_smem = smem + kStages * G::kStageBytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + kNtEpiWarps * G::kStaging * kNtTileBytes);
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

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kNtEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
    prefetch_tensormap(&tm_out);
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

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------ producer (both CTAs)
    uint32_t g = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < num_tiles; tile += npairs) {
      int b, m0, n0;
      bool mirror;
      nt_tile<MODE, BN>(tile, p, b, m0, n0, mirror);
      const int a_row = m0 + (int)rank * 128, b_row = n0 + (int)rank * (BN / 2);
      for (int kt = 0; kt < p.num_kt; ++kt, ++g) {
        const int s = (int)(g % kStages);
        if (!mbar_wait_bounded(&empty[s], ((g / kStages) & 1u) ^ 1u, p.wait_budget, s_abort)) {
          ok = false;
          break;
        }
        uint8_t *st = smem + s * G::kStageBytes;
        if (is_leader) mbar_arrive_expect_tx(&full[s], 2 * G::kStageBytes);
        tma_load_3d_pair(st, &tm_a, &full[s], kt * G::kBK, a_row, b);
        if (G::kBmn) {   // 64-column atoms of 64 rows of X
#pragma unroll
          for (int a = 0; a < BN / 128; ++a)
            tma_load_3d_pair(st + G::kSmemA + a * 8192, &tm_b, &full[s], b_row + 64 * a, kt * G::kBK, b);
        } else {
          tma_load_3d_pair(st + G::kSmemA, &tm_b, &full[s], kt * G::kBK, b_row, b);
        }
      }
    }
    // The leader's `full` barriers count both CTAs' bytes: let every copy land.
    if (is_leader) {
      for (uint32_t i = g > kStages ? g - kStages : 0; i < g; ++i) {
        volatile int no_abort = 0;
        mbar_wait_bounded(&full[i % kStages], (i / kStages) & 1u, kDrainBudget, &no_abort);
      }
    }
  } else if (warp == 1 && lane == 0 && is_leader) {
    // ----------------------------------------------------- MMA issuer (leader)
    constexpr uint32_t idesc = MODE == kNtI8 ? make_idesc_i8(256, BN)
                                             : (make_idesc_dense(false, 256, BN) | (G::kBmn ? (1u << 16) : 0u));
    const uint64_t a_desc0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
    const uint64_t b_desc0 = smem_desc(smem_u32(smem + G::kSmemA), G::kBmn ? 8192 : 16, 1024, kSwizzle128B);
    uint32_t g = 0;
    bool ok = true;
    int j = 0;
    for (int tile = pair; ok && tile < num_tiles; tile += npairs, ++j) {
      const int buf = j & 1;
      if (!(ok = mbar_wait_bounded(&acc_empty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u, p.wait_budget, s_abort))) break;
      tc_fence_after();
      const uint32_t acc = tmem_base + (uint32_t)(buf * BN);
      for (int kt = 0; kt < p.num_kt; ++kt, ++g) {
        const int s = (int)(g % kStages);
        if (!(ok = mbar_wait_bounded(&full[s], (g / kStages) & 1u, p.wait_budget, s_abort))) break;
        tc_fence_after();
        const uint64_t so = (uint64_t)((s * G::kStageBytes) >> 4);
        const uint64_t ad = a_desc0 + so, bd = b_desc0 + so;
        // Four K steps of 32 bytes through A's 128-byte rows; B the same way, or, MN-major,
        // 16 rows of 128 bytes.
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t bk = bd + (uint64_t)(G::kBmn ? kk * (2048 >> 4) : 2 * kk);
          const uint32_t accum = (kt != 0 || kk != 0) ? 1u : 0u;
          if (MODE == kNtI8) tc_mma_i8_pair(acc, ad + 2 * kk, bk, idesc, accum);
          else tc_mma_f16_pair(acc, ad + 2 * kk, bk, idesc, accum);
        }
        tc_commit_pair(&empty[s], 0x3);
      }
      if (ok) tc_commit_pair(&acc_full[buf], 0x3);
    }
    if (!ok) {
      tc_commit_pair(drain, 0x1);
      volatile int no_abort = 0;
      mbar_wait_bounded(drain, 0, kDrainBudget, &no_abort);
    }
  } else if (warp >= 2) {
    // ---------------------------------------------------- epilogue (both CTAs)
    // Warp w drains lanes 32q..32q+31 (q = w%4) at the 32-column chunks grp, grp + 2, ...
    // Registers r[k][h][g][4i + 2 sub + e] of lane l: row 16h + 8 sub + l/4, column
    // 16g + 8i + 2(l%4) + e of chunk k.
    const int ew = warp - 2, grp = ew >> 2, q = warp & 3;
    uint8_t *stg = epi_smem + ew * G::kStaging * kNtTileBytes;
    const uint32_t stg_u32 = smem_u32(stg);
    const int lr = lane >> 2, lc = 2 * (lane & 3);
    bool alive = true;
    int j = 0;
    for (int tile = pair; alive && tile < num_tiles; tile += npairs, ++j) {
      int b, m0, n0;
      bool mirror;
      nt_tile<MODE, BN>(tile, p, b, m0, n0, mirror);
      m0 += (int)rank * 128 + 32 * q;
      const int nch = min(G::kChunks, (p.N - n0 + 31) / 32);
      const int nk = grp < nch ? (nch - 1 - grp) / 2 + 1 : 0;
      float sw[2][2];
      if (MODE == kNtI8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int f = m0 + 16 * (e >> 1) + 8 * (e & 1) + lr;
          sw[e >> 1][e & 1] = f < p.M ? __ldg(p.row_scale + f) : 0.0f;
        }
      }
      const int buf = j & 1;
      const bool got = mbar_wait_bounded(&acc_full[buf], (uint32_t)(j >> 1) & 1u, p.wait_budget, s_abort);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        alive = false;
        break;
      }
      tc_fence_after();
      uint32_t r[G::kPerWarp][2][2][8];
      const uint32_t t_base = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * BN);
#pragma unroll
      for (int k = 0; k < G::kPerWarp; ++k)
        if (k < nk)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < 2; ++g)
              tmem_ld_16x256b_x2(t_base + ((uint32_t)(16 * h) << 16) + (uint32_t)(32 * (grp + 2 * k) + 16 * g),
                                 r[k][h][g]);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < G::kPerWarp; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int g = 0; g < 2; ++g) reg_fence(r[k][h][g]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(&acc_empty[buf]);
#pragma unroll
      for (int k = 0; k < G::kPerWarp; ++k) {
        if (k >= nk) break;
        const int c0 = n0 + 32 * (grp + 2 * k);
        if (MODE == kNtMuon || (MODE == kNtOrth && !p.tma_out)) {
          // Straight to global memory: element (i, j) of the short x long product is entry
          // (i, j) of the matrix, or (j, i) of a tall one; 8 lanes share a 32-byte sector.
          const int64_t ld = p.tall ? p.M : p.N;
          const int64_t base = (int64_t)b * p.M * p.N;
          const bool vec = p.vec != 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float2 wv[2][2][2];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int row = m0 + 16 * h + 8 * (e & 1) + lr, col = c0 + 16 * (e >> 2) + 8 * ((e >> 1) & 1) + lc;
              float2 &v = wv[e >> 2][(e >> 1) & 1][e & 1];
              v = make_float2(0.0f, 0.0f);
              if (MODE == kNtMuon && row < p.M && col < p.N) {
                if (vec) {
                  v = *reinterpret_cast<const float2 *>(p.w + base + (int64_t)row * ld + col);
                } else {
                  const int64_t o0 = base + (p.tall ? (int64_t)col * ld + row : (int64_t)row * ld + col);
                  v.x = p.w[o0];
                  if (col + 1 < p.N) v.y = p.w[o0 + (p.tall ? ld : 1)];
                }
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int g = e >> 2, i = (e >> 1) & 1, sub = e & 1;
              const int row = m0 + 16 * h + 8 * sub + lr, col = c0 + 16 * g + 8 * i + lc;
              const float2 acc = make_float2(__uint_as_float(r[k][h][g][4 * i + 2 * sub]),
                                             __uint_as_float(r[k][h][g][4 * i + 2 * sub + 1]));
              float2 v = make_float2(p.alpha * acc.x, p.alpha * acc.y);
              if (MODE == kNtMuon) {
                const float2 w = wv[g][i][sub];
                v = make_float2(fmaf(-p.alpha, acc.x, p.keep * w.x), fmaf(-p.alpha, acc.y, p.keep * w.y));
              }
              if (row >= p.M || col >= p.N) continue;
              const uint32_t v16 = pack2<BF16>(v.x, v.y);
              if (vec) {
                const int64_t o = base + (int64_t)row * ld + col;
                if (MODE == kNtMuon) *reinterpret_cast<float2 *>(p.w + o) = v;
                if (p.out16) *reinterpret_cast<uint32_t *>(p.out16 + o) = v16;
              } else {
                const int64_t o0 = base + (p.tall ? (int64_t)col * ld + row : (int64_t)row * ld + col);
                const int64_t o1 = o0 + (p.tall ? ld : 1);
                const bool two = col + 1 < p.N;
                if (MODE == kNtMuon) {
                  p.w[o0] = v.x;
                  if (two) p.w[o1] = v.y;
                }
                if (p.out16) {
                  p.out16[o0] = (uint16_t)(v16 & 0xFFFFu);
                  if (two) p.out16[o1] = (uint16_t)(v16 >> 16);
                }
              }
            }
          }
          continue;
        }
        // 16-bit tiles through shared memory: direct [row][column] and/or transposed [column][row].
        const bool direct = MODE != kNtI8 && !(MODE == kNtOrth && p.tall);
        const bool trans = MODE == kNtI8 || (G::kSym && mirror) || (MODE == kNtOrth && p.tall);
        uint32_t pk[2][2][4];   // [h][g][2 i + sub]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int col = c0 + 16 * g + 8 * i + lc;
              float2 sx = make_float2(0.0f, 0.0f);
              if (MODE == kNtI8) {
                if (col < p.N) sx.x = __ldg(p.col_scale + col);
                if (col + 1 < p.N) sx.y = __ldg(p.col_scale + col + 1);
              }
#pragma unroll
              for (int sub = 0; sub < 2; ++sub) {
                const uint32_t u0 = r[k][h][g][4 * i + 2 * sub], u1 = r[k][h][g][4 * i + 2 * sub + 1];
                float2 v = make_float2(__uint_as_float(u0), __uint_as_float(u1));
                if (MODE == kNtI8) {
                  v = make_float2((__int2float_rn((int)u0) * sw[h][sub]) * sx.x,
                                  (__int2float_rn((int)u1) * sw[h][sub]) * sx.y);
                  if (GELU) v = gelu2(v);
                } else if (MODE == kNtGram || MODE == kNtOrth) {
                  v = make_float2(p.alpha * v.x, p.alpha * v.y);
                } else if (MODE == kNtPoly) {
                  const int row = m0 + 16 * h + 8 * sub + lr;
                  float gx = 0.0f, gy = 0.0f;
                  if (row < p.M && col < p.M)
                    unpack2<false>(*reinterpret_cast<const uint32_t *>(p.gram + ((int64_t)b * p.M + row) * p.gram_ld + col),
                                   gx, gy);
                  v.x = fmaf(p.c, v.x, p.b * gx) + (row == col ? p.a : 0.0f);
                  v.y = fmaf(p.c, v.y, p.b * gy) + (row == col + 1 ? p.a : 0.0f);
                }
                pk[h][g][2 * i + sub] = pack2<(MODE == kNtI8 || MODE == kNtOrth) ? BF16 : false>(v.x, v.y);
              }
            }
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        uint8_t *t_stg = stg + (G::kSym ? kNtTileBytes : 0);
        const uint32_t t_u32 = smem_u32(t_stg);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (direct) stmatrix_x4(stg_u32 + swz64(16 * h + 8 * ((lane >> 3) & 1) + (lane & 7), 2 * g + (lane >> 4)), pk[h][g]);
            if (trans) stmatrix_x4_trans(t_u32 + swz64(16 * g + 8 * (lane >> 4) + (lane & 7), 2 * h + ((lane >> 3) & 1)), pk[h][g]);
          }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && m0 < p.M) {   // the TMA unit clips rows and columns past the matrix
          if (direct) tma_store_3d(&tm_out, stg, c0, m0, b);
          if (trans) tma_store_3d(&tm_out, t_stg, m0, c0, b);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's MMAs, copies and arrivals into this CTA are over
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

}  // namespace sp24
