// Row-wise 8-bit quantisation: scale[r] = amax_r / 127, q[r][c] = rint(x[r][c] (127 (1 / amax_r))),
// amax_r over the row's kept entries (all of them without a mask); a pruned entry counts as
// 0 whatever it holds.  Divisions and products are IEEE fp32, rounding to nearest even, so
// the integers are the same on every call.  |x| <= amax gives |q| <= 127 (the factor is
// within 2^-22 of 127 / amax), so nothing needs clamping.  A row of zeros gives scale 0 and
// q 0; a row whose amax is below 2^-100 counts as one (the factor would near the end of
// fp32's range); a row with a NaN or an infinity gives scale NaN and q 0.
//
// The maximum is taken on the bit patterns of |x| (monotone for both types, and NaN above
// infinity above every number).  Bound by memory: 2 bytes read and 1 written per entry
// (16384 x 5120 in 39 us, 98% of the copy rate; a masked 6400 x 1600 in 8.6).
#pragma once
#include "gemm_sp.cuh"

namespace sp24 {

constexpr int kQuantThreads = 256;

template <bool BF16>
__device__ __forceinline__ float2 quant_scales(uint32_t amax_bits) {   // (scale, 127 (1 / amax))
  const uint32_t inf = BF16 ? 0x7F80u : 0x7C00u;
  if (amax_bits >= inf) return make_float2(__int_as_float(0x7FC00000), 0.0f);
  const float amax = bits_to_f32<BF16>(amax_bits);
  if (amax < 7.888609052210118e-31f) return make_float2(0.0f, 0.0f);   // 2^-100
  return make_float2(__fdiv_rn(amax, 127.0f), __fmul_rn(__frcp_rn(amax), 127.0f));
}

template <bool BF16>
__device__ __forceinline__ int quant_one(uint32_t bits, float inv) {
  return inv == 0.0f ? 0 : __float2int_rn(__fmul_rn(bits_to_f32<BF16>(bits), inv));
}

__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  __shared__ uint32_t s_max[kQuantThreads / 32];
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t t = 0;
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) t = max(t, s_max[w]);
  __syncthreads();
  return t;
}

// Rows of whole aligned 16-byte units, held in registers between the two passes: TPR threads
// (a warp, or the block) per row, NV units of 8 entries per thread, so each entry is read
// once and a thread has NV independent loads in flight.  rint(p) for |p| <= 2^22 is the low
// byte of p + 1.5 2^23 (one fp32 addition rounding to even; the conversion instruction runs at
// an eighth of its rate).
template <bool BF16, bool MASKED, int TPR, int NV>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_vec_kernel(const uint16_t *__restrict__ X, int64_t rows, int64_t cols, int64_t ldx,
                        const uint8_t *__restrict__ idx, int8_t *__restrict__ q, float *__restrict__ scale) {
  // Patterns' bits in shared memory before the wait: a look-up is off the path from idx to the
  // values then.
  __shared__ uint16_t s_bits[MASKED ? 256 : 1];
  if (MASKED) s_bits[threadIdx.x] = g_tables.bits[threadIdx.x];
  pdl_launch_dependents();
  if (MASKED) __syncthreads();
  pdl_wait();
  constexpr int kRows = kQuantThreads / TPR;
  const int t = threadIdx.x % TPR;
  const int nvec = (int)(cols >> 3);
  for (int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR; r < rows; r += (int64_t)gridDim.x * kRows) {
    const uint4 *x = reinterpret_cast<const uint4 *>(X + r * ldx);
    uint32_t two[MASKED ? NV : 1];   // the patterns of each unit's two blocks
    if (MASKED) {
      const uint16_t *id = reinterpret_cast<const uint16_t *>(idx + (r >> 2) * (cols >> 2));
#pragma unroll
      for (int k = 0; k < NV; ++k) two[k] = t + k * TPR < nvec ? (uint32_t)__ldg(id + t + k * TPR) : 0u;
    }
    uint4 v[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = t + k * TPR < nvec ? __ldcs(x + t + k * TPR) : make_uint4(0u, 0u, 0u, 0u);
    if (MASKED) {
      const int sh = 4 * (int)(r & 3);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        uint32_t *e = reinterpret_cast<uint32_t *>(&v[k]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t keep = (uint32_t)s_bits[(two[k] >> (8 * h)) & 0xFFu] >> sh;
          e[2 * h] &= ((keep & 1u) ? 0xFFFFu : 0u) | ((keep & 2u) ? 0xFFFF0000u : 0u);
          e[2 * h + 1] &= ((keep & 4u) ? 0xFFFFu : 0u) | ((keep & 8u) ? 0xFFFF0000u : 0u);
        }
      }
    }
    uint32_t am = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint32_t *e = reinterpret_cast<const uint32_t *>(&v[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) am = __vmaxu2(am, e[i] & 0x7FFF7FFFu);
    }
    am = max(am & 0xFFFFu, am >> 16);
    am = TPR == 32 ? __reduce_max_sync(0xFFFFFFFFu, am) : block_max(am);
    const float2 s = quant_scales<BF16>(am);
    uint2 *out = reinterpret_cast<uint2 *>(q + r * cols);
    const bool zero = s.y == 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint32_t *e = reinterpret_cast<const uint32_t *>(&v[k]);
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2<BF16>(e[i], lo, hi);
        b[2 * i] = __float_as_uint(__fadd_rn(__fmul_rn(lo, s.y), 12582912.0f));
        b[2 * i + 1] = __float_as_uint(__fadd_rn(__fmul_rn(hi, s.y), 12582912.0f));
      }
      const uint32_t w0 = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
      const uint32_t w1 = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
      if (t + k * TPR < nvec) __stcs(out + t + k * TPR, zero ? make_uint2(0u, 0u) : make_uint2(w0, w1));
    }
    if (t == 0) scale[r] = s.x;
  }
}

// A block per row, any sizes and pitches.
template <bool BF16, bool MASKED>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows_kernel(const uint16_t *__restrict__ X, int64_t rows, int64_t cols, int64_t ldx,
                         const uint8_t *__restrict__ idx, int8_t *__restrict__ q, float *__restrict__ scale) {
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const uint16_t *x = X + r * ldx;
    auto value = [&](int64_t c) -> uint32_t {
      if (MASKED) {
        const uint32_t pat = g_tables.bits[__ldg(idx + (r >> 2) * (cols >> 2) + (c >> 2))];
        if (!((pat >> (4 * (int)(r & 3) + (int)(c & 3))) & 1u)) return 0u;
      }
      return x[c];
    };
    uint32_t amax = 0;
    for (int64_t c = threadIdx.x; c < cols; c += kQuantThreads) amax = max(amax, value(c) & 0x7FFFu);
    const float2 s = quant_scales<BF16>(block_max(amax));
    for (int64_t c = threadIdx.x; c < cols; c += kQuantThreads) q[r * cols + c] = (int8_t)quant_one<BF16>(value(c), s.y);
    if (threadIdx.x == 0) scale[r] = s.x;
  }
}

}  // namespace sp24
