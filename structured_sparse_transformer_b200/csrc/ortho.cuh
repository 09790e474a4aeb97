// Pass of the optimiser step before the Newton-Schulz products (ortho_gemm.cuh): the momentum
// update, the norm of the update direction U, and the iterate's start in fp16, transposed when
// the matrix is tall, so that the products always work on its short side.
//
// X0 = U / (|U|_F + eps) cannot be formed before U has been read once, but a power of two can
// take its place: the pass stores U 2^-e, rounded to fp16 with the same relative error, and
// round 0's products take the factor that is left (gamma, one float a matrix) in their
// epilogues.  e comes from the gradient's size at a few places, which every block reads for
// itself; a matrix whose entries do not fit fp16 that way (momentum far from the gradient's
// size, a few huge entries) is found from its exact sum of squares and largest entry, and
// rewritten as s U / (|U|_F + eps) by the next kernel, which otherwise only forms gamma.  So
// gradient and momentum are read once: at 6400 x 1600 a Muon step's passes moved 225 MB in 37 us
// when the second one always ran.
//
// The sum of squares is held in fp64 (fp32 entries near 1e-25 or 1e25 square out of fp32's
// range): one partial per block, added in a fixed order, so the result does not depend on
// scheduling.
#pragma once
#include "sp24_common.cuh"

namespace sp24 {

constexpr int kOrthThreads = 256;
constexpr int kOrthMaxBlocks = 1024;   // partial sums per matrix
constexpr int kOrthTile = 64;          // tile of the scaling pass

struct OrthSrc {
  const float *g;            // gradient (Orth: the matrix itself)
  float *m;                  // momentum, or null (Orth)
  int64_t rows, cols, ld, stride;   // entries; momentum is contiguous, so ld = cols there
  float mu;
  int nesterov;
};

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s_part[kOrthThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kOrthThreads / 32; ++w) t += s_part[w];
  __syncthreads();
  return t;
}

// Update direction of one entry from the gradient and the new momentum.
__device__ __forceinline__ float orth_dir(const OrthSrc &p, float g, float m) {
  return p.nesterov ? fmaf(p.mu, m, g) : m;
}

struct OrthPart {   // of one block
  double sumsq;
  float amax;
  float scale;       // 2^-e
};

// 2^-e with e near log2 of the gradient's root mean square over 32 entries at each of 8 places
// (one load of a thread).
__device__ __forceinline__ float orth_guess(const OrthSrc &p, const float *g) {
  const int64_t i = p.rows * p.cols / 8 * (threadIdx.x >> 5) + (threadIdx.x & 31);
  const int64_t r = min(i / p.cols, p.rows - 1);
  const double v = (double)g[r * p.ld + i % p.cols];
  const double sum = block_sum(v * v);
  if (!(sum > 0.0) || !(sum < 1e300)) return 1.0f;
  int e;
  frexp(sqrt(sum / kOrthThreads), &e);
  return (float)ldexp(1.0, min(max(-e, -100), 100));
}

// The fp16 start of a 64 x 64 tile whose entries u[k] (thread (tx, ty): rows ty + 16 k, columns
// 4 tx .. 4 tx + 3) are scaled: x [short][ldx].  Stores of four entries may run into the padding
// of a row of x, never past it.  Transposed through shared memory (rows of 33 words, so that
// the column reads spread over the banks).
template <bool TALL>
__device__ __forceinline__ void orth_store_tile(const float4 (&u)[4], int64_t r0, int64_t c0, int64_t rows, int64_t cols,
                                                __half *x, int64_t ldx, __half (*s_t)[kOrthTile + 2]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 lo = __floats2half2_rn(u[k].x, u[k].y), hi = __floats2half2_rn(u[k].z, u[k].w);
    const int64_t r = r0 + ty + 16 * k, c = c0 + 4 * tx;
    if (TALL) {
      *reinterpret_cast<__half2 *>(&s_t[ty + 16 * k][4 * tx]) = lo;
      *reinterpret_cast<__half2 *>(&s_t[ty + 16 * k][4 * tx + 2]) = hi;
    } else if (r < rows && c < cols) {
      *reinterpret_cast<uint2 *>(x + r * ldx + c) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
  }
  if (TALL) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int cc = ty + 16 * k;
      const int64_t c = c0 + cc, r = r0 + 4 * tx;
      const __half2 lo = __halves2half2(s_t[4 * tx][cc], s_t[4 * tx + 1][cc]);
      const __half2 hi = __halves2half2(s_t[4 * tx + 2][cc], s_t[4 * tx + 3][cc]);
      if (c < cols && r < rows)
        *reinterpret_cast<uint2 *>(x + c * ldx + r) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
    __syncthreads();
  }
}

// Entries of row r from column c on (QUADS: rows of whole aligned float4s), 0 past the matrix.
template <bool QUADS>
__device__ __forceinline__ float4 orth_load4(const float *src, int64_t r, int64_t c, const OrthSrc &p) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r >= p.rows || c >= p.cols) return v;
  src += r * p.ld + c;
  if (QUADS) return *reinterpret_cast<const float4 *>(src);
  v.x = src[0];
  if (c + 1 < p.cols) v.y = src[1];
  if (c + 2 < p.cols) v.z = src[2];
  if (c + 3 < p.cols) v.w = src[3];
  return v;
}

// Grid (blocks, matrices); a block takes every gridDim.x-th 64 x 64 tile of its matrix: momentum
// <- mu momentum + g in place (when given), U 2^-e to x [matrices][short][ldx], and the
// block's sum of squares and largest |U|.  Bound by memory: 14 bytes per entry (6 without
// momentum).
template <bool TALL, bool QUADS>
__global__ void __launch_bounds__(kOrthThreads)
    orth_start_kernel(const OrthSrc p, OrthPart *__restrict__ part, __half *__restrict__ x, int64_t ldx, int64_t col_tiles,
                      int64_t tiles) {
  __shared__ __align__(16) __half s_t[kOrthTile][kOrthTile + 2];
  __shared__ float s_max[kOrthThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t b = blockIdx.y;
  const float *g = p.g + b * p.stride;
  float *m = p.m ? p.m + b * p.stride : nullptr;
  x += b * (TALL ? p.cols : p.rows) * ldx;
  const float scale = orth_guess(p, g);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  double sum = 0.0;
  float amax = 0.0f;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = tile / col_tiles * kOrthTile, c0 = tile % col_tiles * kOrthTile;
    const int64_t c = c0 + 4 * tx;
    float4 u[4], mv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = orth_load4<QUADS>(g, r0 + ty + 16 * k, c, p);
    if (m) {
#pragma unroll
      for (int k = 0; k < 4; ++k) mv[k] = orth_load4<QUADS>(m, r0 + ty + 16 * k, c, p);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t r = r0 + ty + 16 * k;
        float *ue = reinterpret_cast<float *>(&u[k]), *me = reinterpret_cast<float *>(&mv[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          me[e] = fmaf(p.mu, me[e], ue[e]);
          ue[e] = orth_dir(p, ue[e], me[e]);
        }
        if (r < p.rows && c < p.cols) {
          float *dst = m + r * p.ld + c;
          if (QUADS) {
            *reinterpret_cast<float4 *>(dst) = mv[k];
          } else {
            dst[0] = me[0];
            if (c + 1 < p.cols) dst[1] = me[1];
            if (c + 2 < p.cols) dst[2] = me[2];
            if (c + 3 < p.cols) dst[3] = me[3];
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float *ue = reinterpret_cast<const float *>(&u[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum += (double)ue[e] * (double)ue[e];
        amax = fmaxf(amax, fabsf(ue[e]));
      }
      u[k] = make_float4(ue[0] * scale, ue[1] * scale, ue[2] * scale, ue[3] * scale);
    }
    orth_store_tile<TALL>(u, r0, c0, p.rows, p.cols, x, ldx, s_t);
  }
  sum = block_sum(sum);
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kOrthThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
    part[b * gridDim.x + blockIdx.x] = OrthPart{sum, amax, scale};
  }
}

// s / (|U| + eps) as a product of two floats (one alone could leave fp32's range): 0 for a
// zero matrix, NaN for one with a NaN or an infinity.
__device__ __forceinline__ float2 orth_factor(double sumsq, float s, float eps) {
  const double norm = sqrt(sumsq) + (double)eps;
  if (norm == 0.0) return make_float2(0.0f, 0.0f);
  const double f = (double)s / norm;
  if (!(f > 0.0)) return make_float2(__int_as_float(0x7FC00000), 1.0f);
  int e;
  frexp(f, &e);
  const double f1 = ldexp(1.0, e / 2);
  return make_float2((float)f1, (float)(f / f1));
}

// Grid (blocks, matrices): gamma[b] with gamma x = s X0, and where orth_start_kernel's x does not serve, x itself
// as s X0 (gamma 1).  It serves if x's root mean square is at least 2^-4 (entries down to 2^-10
// of it are normal numbers) and its largest entry at most 2^15.  Block (0, 0) also zeroes the
// products' counters.
template <bool TALL, bool QUADS>
__global__ void __launch_bounds__(kOrthThreads)
    orth_finish_start_kernel(const OrthSrc p, const OrthPart *__restrict__ part, int nparts, float s, float eps,
                             __half *__restrict__ x, int64_t ldx, int64_t col_tiles, int64_t tiles,
                             float *__restrict__ gamma, unsigned *__restrict__ counters, int ncounters) {
  __shared__ __align__(16) __half s_t[kOrthTile][kOrthTile + 2];
  __shared__ float2 s_f;
  __shared__ int s_redo;
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < ncounters; i += kOrthThreads) counters[i] = 0u;
  const int64_t b = blockIdx.y;
  const float *g = p.g + b * p.stride;
  const float scale = part[b * nparts].scale;
  double t = 0.0;
  float amax = 0.0f;
  for (int i = threadIdx.x; i < nparts; i += kOrthThreads) {
    t += part[b * nparts + i].sumsq;
    amax = fmaxf(amax, part[b * nparts + i].amax);
  }
  t = block_sum(t);
  const int too_big = __syncthreads_or(!(amax * scale <= 32768.0f));
  if (threadIdx.x == 0) {
    const double rms = sqrt(t / ((double)p.rows * (double)p.cols)) * (double)scale;
    s_redo = too_big || !(rms >= 0.0625);
    s_f = orth_factor(t, s, eps);
    if (blockIdx.x == 0) gamma[b] = s_redo ? 1.0f : (float)((double)s / (sqrt(t) + (double)eps) / (double)scale);
  }
  __syncthreads();
  if (!s_redo) return;
  const float2 f = s_f;
  const float *m = p.m ? p.m + b * p.stride : nullptr;
  x += b * (TALL ? p.cols : p.rows) * ldx;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = tile / col_tiles * kOrthTile, c0 = tile % col_tiles * kOrthTile;
    const int64_t c = c0 + 4 * tx;
    float4 u[4], mv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = orth_load4<QUADS>(g, r0 + ty + 16 * k, c, p);
    if (m) {
#pragma unroll
      for (int k = 0; k < 4; ++k) mv[k] = orth_load4<QUADS>(m, r0 + ty + 16 * k, c, p);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float *ue = reinterpret_cast<float *>(&u[k]);
      const float *me = reinterpret_cast<const float *>(&mv[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) ue[e] = (m ? orth_dir(p, ue[e], me[e]) : ue[e]) * f.x * f.y;
    }
    orth_store_tile<TALL>(u, r0, c0, p.rows, p.cols, x, ldx, s_t);
  }
}

}  // namespace sp24
