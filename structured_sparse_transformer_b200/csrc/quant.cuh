// Row-wise 8-bit quantisation: scale[r] = amax_r / 127, q[r][c] = rint(x[r][c] (127 (1 / amax_r))),
// amax_r over the row's kept entries (all of them without a mask); a pruned entry counts as
// 0 whatever it holds.  Divisions and products are IEEE fp32, rounding to nearest even, so
// the integers are the same on every call.  |x| <= amax gives |q| <= 127 (the factor is
// within 2^-22 of 127 / amax), so nothing needs clamping.  A row of zeros gives scale 0 and
// q 0; a row whose amax is below 2^-100 counts as one (the factor would near the end of
// fp32's range); a row with a NaN or an infinity gives scale NaN and q 0.
//
// The maximum is taken on the bit patterns of |x| (monotone for both types, and NaN above
// infinity above every number).  Bound by memory: 2 bytes read and 1 written per entry.
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
