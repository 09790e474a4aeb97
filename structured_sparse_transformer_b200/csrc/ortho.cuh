// Passes of the optimiser step around the Newton-Schulz products (gemm_nt.cuh): the
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
constexpr int kOrthTile = 64;          // transposing pass: 64 x 64 entries per block

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

// Grid (column tiles, row tiles, matrices) of 64 x 64 entries.  x [matrices][short][ldx] fp16.
template <bool TALL>
__global__ void __launch_bounds__(kOrthThreads)
    orth_scale_kernel(const OrthSrc p, const double *__restrict__ part, int nparts, float s, float eps,
                      __half *__restrict__ x, int64_t ldx, int64_t row_tiles) {
  __shared__ __half s_t[kOrthTile][kOrthTile + 2];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t b = blockIdx.z;
  double t = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kOrthThreads) t += part[b * nparts + i];
  const float2 f = orth_factor(block_sum(t), s, eps);
  const float *g = p.g + b * p.stride;
  const float *m = p.m ? p.m + b * p.stride : nullptr;
  const int64_t c0 = (int64_t)blockIdx.x * kOrthTile;
  const int tc = threadIdx.x & 63, tr = threadIdx.x >> 6;
  for (int64_t rt = blockIdx.y; rt < row_tiles; rt += gridDim.y) {
    const int64_t r0 = rt * kOrthTile;
#pragma unroll
    for (int k = 0; k < kOrthTile / 4; ++k) {
      const int64_t r = r0 + tr + 4 * k, c = c0 + tc;
      if (r < p.rows && c < p.cols) {
        const float gv = g[r * p.ld + c];
        const float u = m ? orth_dir(p, gv, m[r * p.ld + c]) : gv;
        const __half h = __float2half_rn(u * f.x * f.y);
        if (TALL) s_t[tr + 4 * k][tc] = h;
        else x[(b * p.rows + r) * ldx + c] = h;
      }
    }
    if (TALL) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kOrthTile / 4; ++k) {
        const int64_t c = c0 + tr + 4 * k, r = r0 + tc;
        if (r < p.rows && c < p.cols) x[(b * p.cols + c) * ldx + r] = s_t[tc][tr + 4 * k];
      }
      __syncthreads();
    }
  }
}

}  // namespace sp24
