// Passes of the optimiser step around the Newton-Schulz products (ortho_gemm.cuh): the
// momentum update with the sum of squares, and the scaling of the update direction to the
// fp16 iterate X0 = s U / (|U|_F + eps), transposed when the matrix is tall, so that the
// products always work on its short side.
//
// The sum of squares is held in fp64 (fp32 entries near 1e-25 or 1e25 square out of fp32's
// range): one partial per block, added in block order by every block of the next pass, so
// the result does not depend on scheduling.
#pragma once
#include "sp24_common.cuh"

namespace sp24 {

constexpr int kOrthThreads = 256;
constexpr int kOrthMaxBlocks = 512;    // partial sums per matrix
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

// Grid (blocks, matrices): momentum <- mu momentum + g in place (when given) and the
// block's partial sum of squares of the update direction.
template <bool VEC>
__global__ void __launch_bounds__(kOrthThreads) orth_sumsq_kernel(const OrthSrc p, double *__restrict__ part) {
  pdl_launch_dependents();
  pdl_wait();
  const float *g = p.g + (int64_t)blockIdx.y * p.stride;
  float *m = p.m ? p.m + (int64_t)blockIdx.y * p.stride : nullptr;
  double sum = 0.0;
  auto one = [&](float gv, float &mv) {
    float u = gv;
    if (m) {
      mv = fmaf(p.mu, mv, gv);
      u = orth_dir(p, gv, mv);
    }
    sum += (double)u * (double)u;
  };
  const int64_t nthreads = (int64_t)gridDim.x * kOrthThreads;
  const int64_t tid = (int64_t)blockIdx.x * kOrthThreads + threadIdx.x;
  if (VEC) {   // contiguous, 16-byte aligned matrices of a multiple of 4 entries
    const int64_t n4 = p.rows * p.cols / 4;
    for (int64_t i = tid; i < n4; i += nthreads) {
      const float4 gv = reinterpret_cast<const float4 *>(g)[i];
      float4 mv = m ? reinterpret_cast<float4 *>(m)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
      one(gv.x, mv.x);
      one(gv.y, mv.y);
      one(gv.z, mv.z);
      one(gv.w, mv.w);
      if (m) reinterpret_cast<float4 *>(m)[i] = mv;
    }
  } else {     // a warp per row
    for (int64_t r = tid >> 5; r < p.rows; r += nthreads >> 5)
      for (int64_t c = threadIdx.x & 31; c < p.cols; c += 32) {
        float mv = m ? m[r * p.ld + c] : 0.0f;
        one(g[r * p.ld + c], mv);
        if (m) m[r * p.ld + c] = mv;
      }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
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

// Grid (blocks, matrices); a block takes every gridDim.x-th 64 x 64 tile of its matrix.  x is
// [matrices][short][ldx] fp16.  QUADS: rows of whole aligned float4s.  A tall matrix is
// transposed through shared memory (rows of 33 words, so that the column reads spread over
// the banks); stores of four entries may run into the padding of a row of x, never past it.
template <bool TALL, bool QUADS>
__global__ void __launch_bounds__(kOrthThreads)
    orth_scale_kernel(const OrthSrc p, const double *__restrict__ part, int nparts, float s, float eps,
                      __half *__restrict__ x, int64_t ldx, int64_t col_tiles, int64_t tiles,
                      unsigned *__restrict__ counters, int ncounters) {
  __shared__ __align__(16) __half s_t[kOrthTile][kOrthTile + 2];
  __shared__ float2 s_f;
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0)   // the products' counters (ortho_gemm.cuh)
    for (int i = threadIdx.x; i < ncounters; i += kOrthThreads) counters[i] = 0u;
  const int64_t b = blockIdx.y;
  double t = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kOrthThreads) t += part[b * nparts + i];
  t = block_sum(t);
  if (threadIdx.x == 0) s_f = orth_factor(t, s, eps);
  __syncthreads();
  const float2 f = s_f;
  const float *g = p.g + b * p.stride;
  const float *m = p.m ? p.m + b * p.stride : nullptr;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  // From the end of the matrix: what the pass before touched last is what the cache still holds.
  for (int64_t tile = tiles - 1 - blockIdx.x; tile >= 0; tile -= gridDim.x) {
    const int64_t r0 = tile / col_tiles * kOrthTile, c0 = tile % col_tiles * kOrthTile;
    float4 gv[4], mv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t r = r0 + ty + 16 * k, c = c0 + 4 * tx;
      float *ge = reinterpret_cast<float *>(&gv[k]), *me = reinterpret_cast<float *>(&mv[k]);
      gv[k] = mv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r >= p.rows) continue;
      if (QUADS) {
        if (c < p.cols) {
          gv[k] = *reinterpret_cast<const float4 *>(g + r * p.ld + c);
          if (m) mv[k] = *reinterpret_cast<const float4 *>(m + r * p.ld + c);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < p.cols) {
            ge[e] = g[r * p.ld + c + e];
            if (m) me[e] = m[r * p.ld + c + e];
          }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float *ge = reinterpret_cast<const float *>(&gv[k]), *me = reinterpret_cast<const float *>(&mv[k]);
      __align__(8) __half h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = __float2half_rn((m ? orth_dir(p, ge[e], me[e]) : ge[e]) * f.x * f.y);
      const int64_t r = r0 + ty + 16 * k, c = c0 + 4 * tx;
      if (TALL) {
        *reinterpret_cast<__half2 *>(&s_t[ty + 16 * k][4 * tx]) = __halves2half2(h[0], h[1]);
        *reinterpret_cast<__half2 *>(&s_t[ty + 16 * k][4 * tx + 2]) = __halves2half2(h[2], h[3]);
      } else if (r < p.rows && c < p.cols) {
        *reinterpret_cast<uint2 *>(x + (b * p.rows + r) * ldx + c) = *reinterpret_cast<const uint2 *>(h);
      }
    }
    if (TALL) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int cc = ty + 16 * k;
        const int64_t c = c0 + cc, r = r0 + 4 * tx;
        __align__(8) __half h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = s_t[4 * tx + e][cc];
        if (c < p.cols && r < p.rows)
          *reinterpret_cast<uint2 *>(x + (b * p.cols + c) * ldx + r) = *reinterpret_cast<const uint2 *>(h);
      }
      __syncthreads();
    }
  }
}

}  // namespace sp24
