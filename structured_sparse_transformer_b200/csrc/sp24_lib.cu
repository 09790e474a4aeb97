// libsp24: host side of the C ABI declared in include/sp24.h.
//
// Every entry point validates its arguments on the host first (nothing is
// launched when a check fails), then enqueues its kernels on the caller's
// stream.  Device memory is allocated only for the weight gradient's split-tail workspace.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <cmath>
#include <map>
#include <mutex>
#include <utility>

#include "sp24.h"
#include "gemm_i8.cuh"
#include "gemm_sp.cuh"
#include "mask_kernels.cuh"
#include "mvue.cuh"
#include "ortho.cuh"
#include "ortho_gemm.cuh"
#include "quant.cuh"

namespace {

using namespace sp24;

std::atomic<uint64_t> g_wait_budget{1ull << 32};

inline cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool valid_dtype(sp24_dtype d) { return d == SP24_F16 || d == SP24_BF16; }

sp24_status check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return SP24_ERR_NO_DEVICE; }
  int major = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) {
    cudaGetLastError();
    return SP24_ERR_NO_DEVICE;
  }
  return major == 10 ? SP24_OK : SP24_ERR_NO_DEVICE;
}

// Launch with programmatic stream serialisation: the kernel may be scheduled
// while its predecessor in the stream drains; each kernel here calls
// griddepcontrol.wait before its first global-memory access.
template <typename... KArgs, typename... Args>
sp24_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return SP24_ERR_CUDA;
  }
  return SP24_OK;
}

constexpr int kMaxDevices = 64;

// A value computed once per device (under std::call_once, so concurrent host
// threads and several devices in one process each see their own).
struct PerDevice {
  std::once_flag once[kMaxDevices];
  int value[kMaxDevices] = {};
};

int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return -1;
  }
  return dev;
}

int sm_count() {
  static PerDevice cache;
  const int dev = current_device();
  if (dev < 0) return 148;
  std::call_once(cache.once[dev], [dev] {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 148;
    }
    cache.value[dev] = n;
  });
  return cache.value[dev];
}

// --------------------------------------------------------- tensor maps (TMA)

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D map over a row-major [outer x inner] array of 16-bit (or `type`) elements.
bool make_map_2d(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer, uint64_t pitch_bytes,
                 uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle,
                 CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {pitch_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, type, 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- GEMM launch

// CTA-pair kernel: clusters of two CTAs, tiles of 256 rows x 240 or 224 tokens (see gemm_sp.cuh).
// SPARSE: A = kept values [M x Kd/2] + metadata chunks; dense: A = [M x Kd].
// Weight gradient (kEpiWgrad): B = the layer input [Kd tokens x T columns]
// read MN-major, out = fp32 [M x T]; tiles of 256 x 256.
// Per device, once: the shared-memory opt-in of an instantiation and the number
// of its CTA pairs that fit at once (0: the set-up failed; -1: no device).
template <bool BF16, int EPI, bool SPARSE, bool WIDE = false>
int gemm_pairs() {
  constexpr int smem_bytes = pair_smem_bytes<SPARSE, EPI, WIDE>();
  auto kernel = sp24_gemm_pair_kernel<BF16, EPI, SPARSE, WIDE>;
  static PerDevice pairs_cache;
  const int dev = current_device();
  if (dev < 0) return -1;
  std::call_once(pairs_cache.once[dev], [&] {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes) != cudaSuccess) {
      cudaGetLastError();
      pairs_cache.value[dev] = 0;
      return;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)(sm_count() / 2));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = smem_bytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = sm_count() / 2;
    }
    pairs_cache.value[dev] = n;
  });
  return pairs_cache.value[dev];
}

// Split-tail workspace of the weight gradient, one per (device, stream), so that
// launches on different streams never share one (launches on one stream run
// one after another): the partial accumulators and ready counters of every
// CTA of a full-width launch.  Allocated on first use and kept for the life of
// the process.  The counters start at zero and every launch that completes
// leaves them at zero; after a kernel gives up waiting, sp24_device_status
// clears them.
struct SkWorkspace {
  float *part = nullptr;
  unsigned *flags = nullptr;
  int ctas = 0;
};
std::mutex g_sk_mutex;
std::map<std::pair<int, cudaStream_t>, SkWorkspace> g_sk_workspaces;

sp24_status sk_workspace(cudaStream_t stream, int ctas, SkWorkspace *out) {
  const int dev = current_device();
  if (dev < 0) return SP24_ERR_NO_DEVICE;
  std::lock_guard<std::mutex> lock(g_sk_mutex);
  SkWorkspace &w = g_sk_workspaces[std::make_pair(dev, stream)];
  if (w.ctas < ctas) {
    // cudaFree waits for the device, so no earlier launch still uses the old buffers.
    if (w.part) cudaFree(w.part);
    if (w.flags) cudaFree(w.flags);
    w = SkWorkspace{};
    float *part = nullptr;
    unsigned *flags = nullptr;
    if (cudaMalloc(&part, (size_t)ctas * kSkPartFloatsPerCta * sizeof(float)) != cudaSuccess ||
        cudaMalloc(&flags, (size_t)ctas * kEpiWarps * sizeof(unsigned)) != cudaSuccess ||
        cudaMemsetAsync(flags, 0, (size_t)ctas * kEpiWarps * sizeof(unsigned), stream) != cudaSuccess) {
      cudaGetLastError();
      if (part) cudaFree(part);
      if (flags) cudaFree(flags);
      return SP24_ERR_CUDA;
    }
    w.part = part;
    w.flags = flags;
    w.ctas = ctas;
  }
  *out = w;
  return SP24_OK;
}

// Zero the ready counters of every split-tail workspace of the current device
// (after a kernel gave up waiting, one may have been left raised).
sp24_status sk_clear_flags() {
  const int dev = current_device();
  if (dev < 0) return SP24_ERR_NO_DEVICE;
  std::lock_guard<std::mutex> lock(g_sk_mutex);
  if (cudaDeviceSynchronize() != cudaSuccess) return SP24_ERR_CUDA;
  for (auto &kv : g_sk_workspaces)
    if (kv.first.first == dev && cudaMemset(kv.second.flags, 0, (size_t)kv.second.ctas * kEpiWarps * sizeof(unsigned)) !=
                                     cudaSuccess)
      return SP24_ERR_CUDA;
  return SP24_OK;
}

// Fixed scratch of sp24_gemm_wgrad_noalloc, in the module's static device
// memory (zero at load): the split-tail partial sums of kNoAllocCtas CTAs, then
// their ready counters.
constexpr int kNoAllocCtas = 128;
constexpr size_t kNoAllocPartBytes = (size_t)kNoAllocCtas * kSkPartFloatsPerCta * sizeof(float);
constexpr size_t kNoAllocBytes = kNoAllocPartBytes + (size_t)kNoAllocCtas * kEpiWarps * sizeof(unsigned);
static_assert(kNoAllocPartBytes % 256 == 0, "counters start 256-byte aligned");
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocBytes];

// Its address on the current device, looked up once per device (with that
// device current) and checked.
sp24_status noalloc_scratch(SkWorkspace *out) {
  static std::once_flag once[kMaxDevices];
  static void *addr[kMaxDevices];
  static cudaError_t err[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return SP24_ERR_NO_DEVICE;
  std::call_once(once[dev], [dev] {
    void *p = nullptr;
    err[dev] = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (err[dev] != cudaSuccess) cudaGetLastError();
    addr[dev] = p;
  });
  if (err[dev] != cudaSuccess || addr[dev] == nullptr) return SP24_ERR_CUDA;
  out->part = static_cast<float *>(addr[dev]);
  out->flags = reinterpret_cast<unsigned *>(static_cast<unsigned char *>(addr[dev]) + kNoAllocPartBytes);
  out->ctas = kNoAllocCtas;
  return SP24_OK;
}

// Weight gradient with decay: dec_w/dec_idx/dec_lambda (the masked decay of dW in
// the epilogue); null dec_w elsewhere.  `fixed`: a caller-given split-tail
// scratch (its counters are zeroed here before the launch) instead of the
// per-stream workspace; null for every entry point but sp24_gemm_wgrad_noalloc.
template <bool BF16, int EPI, bool SPARSE, bool WIDE>
sp24_status launch_gemm_pair_w(const void *B, int64_t T, int64_t Kd, const void *vals, const void *meta, int64_t M,
                               void *out, void *aux, cudaStream_t stream, const void *dec_w, const uint8_t *dec_idx,
                               float dec_lambda, const SkWorkspace *fixed, bool a_mn) {
  using G = PairGeom<SPARSE, EPI, WIDE>;
  const int num_kt = (int)((Kd + G::kBK - 1) / G::kBK);
  const int64_t row_tiles = (M + kPairRows - 1) / kPairRows;
  const uint64_t a_cols = SPARSE ? (uint64_t)(Kd / 2) : (uint64_t)Kd;
  CUtensorMap ta, tb, tm;
  const bool b_ok = G::kWg ? make_map_2d(&tb, B, (uint64_t)T, (uint64_t)Kd, (uint64_t)T * 2, 64, (uint32_t)G::kBK,
                                         CU_TENSOR_MAP_SWIZZLE_128B)
                           : make_map_2d(&tb, B, (uint64_t)Kd, (uint64_t)T, (uint64_t)Kd * 2, 64, (uint32_t)(G::kBN / 2),
                                         CU_TENSOR_MAP_SWIZZLE_128B);
  // Dense weight gradient (A = dY [Kd tokens x M]) and dense input gradient with
  // a_mn (A = W [Kd x M]): A read MN-major in 64 x kBK boxes.
  a_mn = a_mn && !SPARSE && !G::kWg;
  const bool a_ok = (G::kWg && !SPARSE) || a_mn
                        ? make_map_2d(&ta, vals, (uint64_t)M, (uint64_t)Kd, (uint64_t)M * 2, 64, (uint32_t)G::kBK,
                                      CU_TENSOR_MAP_SWIZZLE_128B)
                        : make_map_2d(&ta, vals, a_cols, (uint64_t)M, a_cols * 2, G::kAcols, kPairRows,
                                      CU_TENSOR_MAP_SWIZZLE_128B);
  if (!a_ok || !b_ok) return SP24_ERR_CUDA;
  if (SPARSE) {
    if (!make_map_2d(&tm, meta, kSmemE / 8, (uint64_t)(row_tiles * num_kt), kSmemE, kSmemE / 8, 1,
                     CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_DATA_TYPE_UINT64))
      return SP24_ERR_CUDA;
  } else {
    tm = ta;  // unused by the dense kernel
  }
  // Epilogue staging tiles of row-major out / aux, 16 tokens high: 32 features
  // (64B swizzle); gated: out 16 features (no swizzle), aux 32; gated
  // gradient: out and aux 64 columns (128B swizzle) over twice the width.
  CUtensorMap to, tx;
  bool maps_ok;
  if (G::kWg) {   // direct fp32 stores: no staging maps
    to = ta;
    tx = ta;
    maps_ok = true;
  } else if (EPI == kEpiGeglu) {
    maps_ok = make_map_2d(&to, out, (uint64_t)M / 2, (uint64_t)T, (uint64_t)M, 16, kEpiTokens, CU_TENSOR_MAP_SWIZZLE_NONE) &&
              make_map_2d(&tx, aux, (uint64_t)M, (uint64_t)T, (uint64_t)M * 2, 32, kEpiTokens, CU_TENSOR_MAP_SWIZZLE_64B);
  } else if (EPI == kEpiDgeglu) {
    maps_ok = make_map_2d(&to, out, (uint64_t)M * 2, (uint64_t)T, (uint64_t)M * 4, 64, kEpiTokens, CU_TENSOR_MAP_SWIZZLE_128B) &&
              make_map_2d(&tx, aux, (uint64_t)M * 2, (uint64_t)T, (uint64_t)M * 4, 64, kEpiTokens, CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    maps_ok = make_map_2d(&to, out, (uint64_t)M, (uint64_t)T, (uint64_t)M * 2, 32, kEpiTokens, CU_TENSOR_MAP_SWIZZLE_64B) &&
              make_map_2d(&tx, (EPI == kEpiNone || EPI == kEpiGeluDerivPacked || EPI == kEpiMulAuxPacked) ? out : aux,
                          (uint64_t)M, (uint64_t)T, (uint64_t)M * 2, 32, kEpiTokens, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  if (!maps_ok) return SP24_ERR_CUDA;
  constexpr int smem_bytes = pair_smem_bytes<SPARSE, EPI, WIDE>();
  auto kernel = sp24_gemm_pair_kernel<BF16, EPI, SPARSE, WIDE>;
  const int max_pairs = gemm_pairs<BF16, EPI, SPARSE, WIDE>();
  if (max_pairs <= 0) return max_pairs == 0 ? SP24_ERR_CUDA : SP24_ERR_NO_DEVICE;
  const int64_t tiles = ((M + 2 * kPairRows - 1) / (2 * kPairRows)) * ((T + G::kBN - 1) / G::kBN);
  const int pairs = (int)(tiles < max_pairs ? tiles : max_pairs);
  // Weight gradient: number the tiles along dW's columns first when the A
  // operand is the larger one (each wave of pairs then reads it once).
  const double a_bytes = (double)M * (double)Kd * (SPARSE ? 1.0 + 1.0 / 8 : 2.0);
  const double b_bytes = (double)Kd * (double)T * 2.0;
  const int cols_fastest = (G::kWg && a_bytes > b_bytes) ? 1 : 0;
  // Weight gradient: when the last wave would leave pairs idle, split its r
  // tiles along K into min(P / r, 8, num_kt) parts on all P pairs.
  SkWorkspace ws;
  int split = 1, grid_pairs = pairs;
  const int64_t tail = tiles % max_pairs;
  if (G::kWg && tail != 0) {
    int64_t s = max_pairs / tail < num_kt ? max_pairs / tail : num_kt;
    if (s > kMaxSplit) s = kMaxSplit;
    if (s > 1) {
      if (fixed) {   // CTAs 0 .. 2 tail s - 1 use their partial slots and counters
        const int64_t used = 2 * tail * s;
        if (used > fixed->ctas) return SP24_ERR_SCRATCH_TOO_SMALL;
        ws = *fixed;
        if (cudaMemsetAsync(ws.flags, 0, (size_t)used * kEpiWarps * sizeof(unsigned), stream) != cudaSuccess) {
          cudaGetLastError();
          return SP24_ERR_CUDA;
        }
      } else {
        const sp24_status st = sk_workspace(stream, 2 * max_pairs, &ws);
        if (st != SP24_OK) return st;
      }
      split = (int)s;
      grid_pairs = max_pairs;
    }
  }
  return launch_pdl(kernel, dim3(2 * grid_pairs), dim3(kGemmThreads), smem_bytes, stream, ta, tb, tm, to, tx, (int)M,
                    (int)T, num_kt, (uint64_t)g_wait_budget.load(), G::kWg ? static_cast<float *>(out) : nullptr,
                    (int64_t)(G::kWg ? T : 0), static_cast<const uint16_t *>(dec_w), dec_idx, dec_lambda, ws.part,
                    ws.flags, split, cols_fastest, a_mn ? 1 : 0,
                    (EPI == kEpiGeluDerivPacked || EPI == kEpiMulAuxPacked) ? static_cast<uint16_t *>(aux) : nullptr,
                    (int)((M + 31) / 32));
}

// Tile width per call, for the variants that have both: the busiest pair's token
// columns, ceil(tiles / pairs) x width, with the 240-token tile counted 5% cheaper
// per token (measured on the 1.5B FFN launches, where its waves are as full);
// where waves quantise differently (e.g. 148 tiles of 224 tokens on 74 pairs
// against 140 of 240) the narrower tile is kept.
template <bool BF16, int EPI, bool SPARSE>
sp24_status launch_gemm_pair_t(const void *B, int64_t T, int64_t Kd, const void *vals, const void *meta, int64_t M,
                               void *out, void *aux, cudaStream_t stream, const void *dec_w = nullptr,
                               const uint8_t *dec_idx = nullptr, float dec_lambda = 0.0f,
                               const SkWorkspace *fixed = nullptr, bool a_mn = false) {
  constexpr int kWideBN = PairGeom<SPARSE, EPI, true>::kBN, kNarrowBN = PairGeom<SPARSE, EPI, false>::kBN;
  if constexpr (kWideBN != kNarrowBN) {
    const int P = gemm_pairs<BF16, EPI, SPARSE, false>();
    if (P > 0) {
      const int64_t mt = (M + 2 * kPairRows - 1) / (2 * kPairRows);
      auto busiest = [&](int bn) {
        const int64_t tiles = mt * ((T + bn - 1) / bn);
        return (double)((tiles + P - 1) / P) * (double)bn;
      };
      if (busiest(kWideBN) * 0.95 < busiest(kNarrowBN))
        return launch_gemm_pair_w<BF16, EPI, SPARSE, true>(B, T, Kd, vals, meta, M, out, aux, stream, dec_w, dec_idx,
                                                           dec_lambda, fixed, a_mn);
    }
  }
  return launch_gemm_pair_w<BF16, EPI, SPARSE, false>(B, T, Kd, vals, meta, M, out, aux, stream, dec_w, dec_idx,
                                                      dec_lambda, fixed, a_mn);
}

template <bool SPARSE>
sp24_status launch_gemm(const void *B, int64_t T, int64_t Kd, const void *vals, const void *meta, int64_t M,
                        sp24_dtype dt, void *out, int epi, void *aux, cudaStream_t s, bool a_mn = false) {
  const bool bf = dt == SP24_BF16;
  switch (epi) {
    case kEpiNone: return bf ? launch_gemm_pair_t<true, kEpiNone, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn)
                             : launch_gemm_pair_t<false, kEpiNone, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn);
    case kEpiGelu: return bf ? launch_gemm_pair_t<true, kEpiGelu, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn)
                             : launch_gemm_pair_t<false, kEpiGelu, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn);
    case kEpiDgelu: return bf ? launch_gemm_pair_t<true, kEpiDgelu, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn)
                              : launch_gemm_pair_t<false, kEpiDgelu, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn);
    case kEpiGeluDeriv:
      return bf ? launch_gemm_pair_t<true, kEpiGeluDeriv, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn)
                : launch_gemm_pair_t<false, kEpiGeluDeriv, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn);
    case kEpiMulAux:
      return bf ? launch_gemm_pair_t<true, kEpiMulAux, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn)
                : launch_gemm_pair_t<false, kEpiMulAux, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn);
    case kEpiGeluDerivPacked:
      return bf ? launch_gemm_pair_t<true, kEpiGeluDerivPacked, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn)
                : launch_gemm_pair_t<false, kEpiGeluDerivPacked, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn);
    case kEpiMulAuxPacked:
      return bf ? launch_gemm_pair_t<true, kEpiMulAuxPacked, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn)
                : launch_gemm_pair_t<false, kEpiMulAuxPacked, SPARSE>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn);
    default: break;
  }
  if (SPARSE) {   // the gated epilogues serve the 2:4 GEMMs
    switch (epi) {
      case kEpiGeglu: return bf ? launch_gemm_pair_t<true, kEpiGeglu, true>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn)
                                : launch_gemm_pair_t<false, kEpiGeglu, true>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn);
      case kEpiDgeglu: return bf ? launch_gemm_pair_t<true, kEpiDgeglu, true>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn)
                                 : launch_gemm_pair_t<false, kEpiDgeglu, true>(B, T, Kd, vals, meta, M, out, aux, s, nullptr, nullptr, 0.0f, nullptr, a_mn);
      default: break;
    }
  }
  return SP24_ERR_INVALID_ARG;
}

// The epilogues each product takes (bit e of the mask allows epilogue e).
constexpr unsigned kFwdEpis = (1u << SP24_EPI_NONE) | (1u << SP24_EPI_GELU) | (1u << SP24_EPI_GEGLU) |
                              (1u << SP24_EPI_GELU_DERIV) | (1u << SP24_EPI_GELU_DERIV_PACKED);
constexpr unsigned kDgradEpis = (1u << SP24_EPI_NONE) | (1u << SP24_EPI_DGELU) | (1u << SP24_EPI_DGEGLU) |
                                (1u << SP24_EPI_MUL_AUX) | (1u << SP24_EPI_MUL_AUX_PACKED);
constexpr unsigned kDenseEpis = (1u << SP24_EPI_NONE) | (1u << SP24_EPI_GELU) | (1u << SP24_EPI_DGELU) |
                                (1u << SP24_EPI_GELU_DERIV) | (1u << SP24_EPI_MUL_AUX) |
                                (1u << SP24_EPI_GELU_DERIV_PACKED) | (1u << SP24_EPI_MUL_AUX_PACKED);
constexpr unsigned kDenseDgradEpis = (1u << SP24_EPI_NONE) | (1u << SP24_EPI_DGELU) | (1u << SP24_EPI_MUL_AUX) |
                                     (1u << SP24_EPI_MUL_AUX_PACKED);
static_assert((int)SP24_EPI_GELU_DERIV_PACKED == (int)kEpiGeluDerivPacked &&
                  (int)SP24_EPI_MUL_AUX_PACKED == (int)kEpiMulAuxPacked &&
                  (int)SP24_EPI_GELU_DERIV == (int)kEpiGeluDeriv && (int)SP24_EPI_MUL_AUX == (int)kEpiMulAux,
              "public and kernel epilogue numbers");

sp24_status validate_gemm(const void *B, int64_t T, int64_t Kd, const void *vals, const void *meta, int64_t M,
                          sp24_dtype dt, const void *out, int epi, const void *aux, unsigned allowed_epis) {
  if (!B && T > 0) return SP24_ERR_INVALID_ARG;
  if (!vals || !meta || (!out && T > 0)) return SP24_ERR_INVALID_ARG;
  if (T < 0 || Kd <= 0 || M <= 0) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dt)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (epi < 0 || epi > 31 || !((allowed_epis >> epi) & 1u)) return SP24_ERR_INVALID_ARG;
  if (epi == SP24_EPI_GEGLU && M % (2 * kGegluGroup)) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (epi != SP24_EPI_NONE && !aux && T > 0) return SP24_ERR_INVALID_ARG;   // T == 0 touches nothing
  if (Kd % 16 || M % 16) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (T > INT32_MAX || M > INT32_MAX || Kd > INT32_MAX) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(B) || !aligned16(vals) || !aligned16(meta) || !aligned16(out) ||
      (epi != SP24_EPI_NONE && !aligned16(aux)))
    return SP24_ERR_MISALIGNED;
  return SP24_OK;
}

// ------------------------------------------------------------ mask launches

template <bool BF16, bool SEARCH, bool COMPRESS, bool FLIP>
sp24_status launch_mask_t(const void *W, int64_t R, int64_t C, int64_t ldw, uint8_t *idx, const uint8_t *prev,
                          unsigned long long *flip, void *vr, void *mr, void *vc, void *mc, cudaStream_t s) {
  // CTA tiles cover whole 128x128 regions (one metadata chunk of each orientation).
  const int64_t chunks_x = (C + kChunk - 1) / kChunk, chunks_y = (R + kChunk - 1) / kChunk;
  if (chunks_y > 65535 || chunks_x * (kChunk / kMaskCtaCols) > INT32_MAX) return SP24_ERR_UNSUPPORTED_SHAPE;
  const int64_t ntiles = chunks_x * chunks_y * (kChunk / kMaskCtaCols);
  CUtensorMap tm;
  // Persistent form with tensor-memory-accelerator loads of W (row pitch a multiple of 16 bytes).
  if (ldw % 8 == 0 && C <= INT32_MAX && R <= INT32_MAX &&
      make_map_2d(&tm, W, (uint64_t)C, (uint64_t)R, (uint64_t)ldw * 2, kMaskCtaCols, kChunk,
                  CU_TENSOR_MAP_SWIZZLE_NONE)) {
    const int64_t ctas = (int64_t)sm_count() * mask_ctas_per_sm<COMPRESS>();
    const unsigned grid = (unsigned)(ntiles < ctas ? ntiles : ctas);
    // The previous mask travels with each W tile by TMA ([R/4][C/4] bytes, a 16 x 32
    // box per tile) when its row pitch is a multiple of 16 bytes; else plain loads.
    CUtensorMap tp = tm;
    const int prev_tma = (FLIP && prev && (C / 4) % 16 == 0 && aligned16(prev) &&
                          make_map_2d(&tp, prev, (uint64_t)(C / 4), (uint64_t)(R / 4), (uint64_t)(C / 4), kMaskCtaCols / 4,
                                      kChunk / 4, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_DATA_TYPE_UINT8))
                             ? 1
                             : 0;
    return launch_pdl(mask_stream_kernel<BF16, SEARCH, COMPRESS, FLIP>, dim3(grid), dim3(kMaskThreads), 0, s, tm, R,
                      C, idx, prev, flip, static_cast<uint16_t *>(vr), static_cast<uint8_t *>(mr),
                      static_cast<uint16_t *>(vc), static_cast<uint8_t *>(mc), (uint64_t)g_wait_budget.load(), tp,
                      prev_tma);
  }
  dim3 grid((unsigned)(chunks_x * (kChunk / kMaskCtaCols)), (unsigned)chunks_y);
  return launch_pdl(mask_tile_kernel<BF16, SEARCH, COMPRESS, FLIP>, grid, dim3(kMaskThreads), 0, s,
                    static_cast<const uint16_t *>(W), R, C, ldw, idx, prev, flip, static_cast<uint16_t *>(vr),
                    static_cast<uint8_t *>(mr), static_cast<uint16_t *>(vc), static_cast<uint8_t *>(mc));
}

template <bool SEARCH, bool COMPRESS, bool FLIP>
sp24_status launch_mask_d(bool bf, const void *W, int64_t R, int64_t C, int64_t ldw, uint8_t *idx,
                          const uint8_t *prev, unsigned long long *flip, void *vr, void *mr, void *vc, void *mc,
                          cudaStream_t s) {
  return bf ? launch_mask_t<true, SEARCH, COMPRESS, FLIP>(W, R, C, ldw, idx, prev, flip, vr, mr, vc, mc, s)
            : launch_mask_t<false, SEARCH, COMPRESS, FLIP>(W, R, C, ldw, idx, prev, flip, vr, mr, vc, mc, s);
}

sp24_status validate_w(const void *W, sp24_dtype dt, int64_t rows, int64_t cols, int64_t ldw) {
  if (rows < 0 || cols < 0 || ldw < cols) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dt)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (rows % 4 || cols % 4) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (rows > 0 && cols > 0) {
    if (!W) return SP24_ERR_INVALID_ARG;
    if (!aligned16(W) || ldw % 4) return SP24_ERR_MISALIGNED;
  }
  return SP24_OK;
}

size_t meta_bytes_of(int64_t rows, int64_t cols) {
  return (size_t)((rows + 127) / 128) * (size_t)((cols + 127) / 128) * 2048u;
}

// Byte offset, inside the device metadata of a [rows x cols] matrix, of the
// nibble for row r, group g (columns 4g..4g+3), and the nibble's bit shift.
inline size_t meta_nibble_pos(int64_t r, int64_t g, int64_t cols, int *shift) {
  const int64_t kt_count = (cols + 127) / 128;
  const int64_t mt = r / 128, m = r % 128;
  const int64_t kt = g / 32, gk = g % 32;           // 32 groups per 128-column chunk
  const int64_t kk = gk / 8, gg = gk % 8;           // 8 groups per 32-column K step
  const int64_t lane = (m % 8) + 8 * (gg / 4) + 16 * (m / 16);
  const int bit = 4 * (int)(gg % 4) + 16 * (int)((m / 8) % 2);
  *shift = bit % 8;
  return (size_t)(mt * kt_count + kt) * 2048 + (size_t)lane * 16 + (size_t)kk * 4 + (size_t)(bit / 8);
}

// Weight gradient: tiles of 256 rows x 256 columns of dW (see PairGeom).
template <bool BF16, bool SPARSE>
sp24_status launch_wgrad(const void *X, int64_t T, int64_t K, const void *A, const void *meta, int64_t N, float *dW,
                         cudaStream_t s, const void *dec_w = nullptr, const uint8_t *dec_idx = nullptr,
                         float dec_lambda = 0.0f, const SkWorkspace *fixed = nullptr) {
  return launch_gemm_pair_t<BF16, kEpiWgrad, SPARSE>(X, K, T, A, meta, N, dW, nullptr, s, dec_w, dec_idx, dec_lambda,
                                                     fixed);
}

// ------------------------------------------- orthogonalisation and 8-bit products

// 3-D map over [batch][outer][inner] (pitches in bytes).
bool make_map_3d(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer, uint64_t batch,
                 uint64_t pitch_bytes, uint64_t batch_bytes, uint32_t box_inner, uint32_t box_outer,
                 CUtensorMapSwizzle swizzle, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {inner, outer, batch};
  cuuint64_t strides[2] = {pitch_bytes, batch_bytes};
  cuuint32_t box[3] = {box_inner, box_outer, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, type, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs of a kernel that fit at once (and, once per device, its shared-memory opt-in);
// 0: the set-up failed, -1: no device.
template <auto KERNEL, int THREADS, int SMEM>
int pairs_of() {
  static PerDevice cache;
  const int dev = current_device();
  if (dev < 0) return -1;
  std::call_once(cache.once[dev], [&] {
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) {
      cudaGetLastError();
      cache.value[dev] = 0;
      return;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)(sm_count() / 2));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 0;
    }
    cache.value[dev] = n;
  });
  return cache.value[dev];
}

// Newton-Schulz on the short side m of every matrix, n the long side.  The workspace holds
// counters, the norm's partial sums, two iterates [count][m][ldx], G and P [count][m][ldm]
// (fp16), and the split tiles' partial sums.
struct OrthPlan {
  int64_t count, rows, cols, m, n, ldx, ldm;
  int64_t tiles;                            // 256 x 256 tiles of P X, per matrix
  size_t counters, norm, gamma, x0, x1, gram, poly, part, total;   // byte offsets
  bool tall;
};

// SP24_ERR_INVALID_ARG / UNSUPPORTED_SHAPE for sizes the call does not take.
sp24_status orth_plan(int64_t count, int64_t rows, int64_t cols, OrthPlan *p) {
  if (count < 0 || rows < 0 || cols < 0) return SP24_ERR_INVALID_ARG;
  if (count > 65535 || rows > (1 << 24) || cols > (1 << 24)) return SP24_ERR_UNSUPPORTED_SHAPE;
  p->count = count;
  p->rows = rows;
  p->cols = cols;
  p->tall = rows > cols;
  p->m = p->tall ? cols : rows;
  p->n = p->tall ? rows : cols;
  if (p->m > 65536) return SP24_ERR_UNSUPPORTED_SHAPE;
  p->ldx = (p->n + 7) / 8 * 8;
  p->ldm = (p->m + 7) / 8 * 8;
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t bx = (size_t)count * p->m * p->ldx * 2, bm = (size_t)count * p->m * p->ldm * 2;
  const int64_t mb = (p->m + 255) / 256, nb = (p->n + 255) / 256;
  p->tiles = mb * nb;
  if (2 * count * p->tiles > INT32_MAX) return SP24_ERR_UNSUPPORTED_SHAPE;
  // A launch has at most kOgMaxSplit pairs per tile (of 128 columns, twice as many), and at
  // most kOgMaxPairs.
  const int64_t want = kOgMaxSplit * 2 * count * p->tiles;
  const int64_t slots = want < kOgMaxPairs ? want : kOgMaxPairs;
  p->counters = take(kOgCounters * sizeof(unsigned));
  p->norm = take((size_t)count * kOrthMaxBlocks * sizeof(OrthPart));
  p->gamma = take((size_t)count * sizeof(float));
  p->x0 = take(bx);
  p->x1 = take(bx);
  p->gram = take(bm);
  p->poly = take(bm);
  p->part = take((size_t)(2 * slots * kOgPartFloats) * sizeof(float));
  p->total = count == 0 || p->m == 0 ? 0 : at;
  return SP24_OK;
}

// The quintic Newton-Schulz coefficients of the Muon optimiser (K. Jordan et al., 2024).
constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;

struct OrthOut {
  uint16_t *out16;   // Orth: the result; Muon: the 16-bit weight, or null
  float *w;          // Muon: the fp32 weight
  float keep, step;
  bool bf16;
};

// Width of a phase's tiles and parts of its tail, by the least time in microseconds, from
// phases of the FFN-sized and small cases measured alone: a K stage of a tile of 256 columns
// (0.31 alone, 0.38 beside all other pairs, 0.45 with X read MN-major) and of 128 columns (0.25
// to 0.35: bound by shared memory, so more than half), a tile's epilogue, and the exchange of
// a split tile.  At 777 x 1333 narrow tiles take 9 us for P X where wide ones took 13; at
// 1600 x 6400 they take 40 where wide ones take 32.
struct OrthShape {
  int bn, split;
  int64_t use;      // pairs with work
  double us;
};

double orth_stage_us(int bn, bool apply, int64_t use) {
  const double share = (double)use / 74.0;
  return bn == 128 ? 0.25 + 0.10 * share : 0.31 + (apply ? 0.14 : 0.07) * share;
}

OrthShape orth_shape(int64_t tiles, int64_t kt, int64_t P, int bn, bool apply, int most) {
  OrthShape o = {bn, 1, tiles < P ? tiles : P, 0.0};
  o.us = orth_stage_us(bn, apply, P) * (double)(tiles / P * kt) + (bn == 256 ? 2.4 : 1.4);
  const int64_t tail = tiles % P;
  if (tail) {
    double least = orth_stage_us(bn, apply, tail) * (double)kt;
    for (int64_t s = 2; s <= most && s <= kt && tail * s <= P; ++s) {
      const double t = orth_stage_us(bn, apply, tail * s) * (double)((kt + s - 1) / s) + (bn == 256 ? 3.5 : 2.8) +
                       0.4 * (double)(s - 2);
      if (t < least) {
        least = t;
        o.split = (int)s;
      }
    }
    o.us += least;
    if (tiles < P) o.use = tail * o.split;
  }
  return o;
}

// Shapes of the three phases on P pairs for `batch` matrices; their time in sum, with what a
// phase costs besides (waiting, first loads, counting: 4.5 us, or 3.4 us in a cluster).
double orth_plan_phases(OrthProducts *p, int batch, int64_t P, bool cluster, int64_t *grid) {
  const int64_t mb = (p->m + 255) / 256;
  double us = 0.0;
  *grid = 0;   // pairs: as many as the phase that uses most
  for (int k = 0; k < 3; ++k) {
    const bool apply = k == kOrthApply;
    const int64_t kt = ((k == kOrthGram ? p->n : p->m) + 63) / 64;
    OrthShape best = {};
    for (int bn = 128; bn <= 256; bn += 128) {
      const int64_t per = apply ? mb * (((int64_t)p->n + bn - 1) / bn) : orth_sym_tiles(p->m, bn);
      const OrthShape o = orth_shape(batch * per, kt, P, bn, apply, cluster ? 1 : kOgMaxSplit);
      if (best.bn == 0 || o.us <= best.us) {
        best = o;
        p->tiles[k] = (int)per;
      }
    }
    p->bn[k] = best.bn;
    us += best.us + (cluster ? 3.4 : 4.5);
    if (best.use > *grid) *grid = best.use;
  }
  for (int k = 0; k < 3; ++k) {   // the splits on that many pairs
    const int64_t kt = ((k == kOrthGram ? p->n : p->m) + 63) / 64;
    p->split[k] = orth_shape((int64_t)batch * p->tiles[k], kt, *grid, p->bn[k], k == kOrthApply, cluster ? 1 : kOgMaxSplit).split;
  }
  return us;
}

// Clusters of C CTAs of a products kernel that fit at once (and its shared-memory opt-in).
template <auto kernel, int SMEM, int C>
int orth_clusters() {
  static PerDevice cache;
  const int dev = current_device();
  if (dev < 0) return -1;
  std::call_once(cache.once[dev], [&] {
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kOgThreads);
    cfg.dynamicSmemBytes = SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = C;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    cache.value[dev] = n;
  });
  return cache.value[dev];
}

template <auto kernel, int SMEM>
int orth_clusters_of(int c) {
  return c == 2 ? orth_clusters<kernel, SMEM, 2>() : (c == 4 ? orth_clusters<kernel, SMEM, 4>() : orth_clusters<kernel, SMEM, 8>());
}

// A round of orth_small_kernel with P X on `pairs` pairs: Gram on each pair, Poly, P X, hand-over.
double orth_small_round(OrthProducts *p, int pairs) {
  const int kt_n = (p->n + 63) / 64, kt_m = (p->m + 63) / 64;
  p->bn[kOrthApply] = p->n > 128 * pairs ? 256 : 128;
  p->tiles[kOrthApply] = (p->n + p->bn[kOrthApply] - 1) / p->bn[kOrthApply];
  const int turns = (p->tiles[kOrthApply] + pairs - 1) / pairs;
  return 2.6 + 0.35 * kt_n + 2.0 + 0.30 * kt_m + turns * (0.30 * kt_m + 0.3) + 1.8 + 2.0;
}

// What orth_products_kernel or orth_small_kernel is launched with (and the kernels' set-up on this device).
struct OrthProductsPlan {
  OrthProducts p;
  int matrices;
  int64_t grid;   // pairs, without clusters per matrix
  bool small;
};

sp24_status plan_orth_products(const OrthProducts &of, OrthProductsPlan *plan) {
  OrthProducts p = of;
  int64_t P = pairs_of<orth_products_kernel<false>, kOgThreads, kOgSmem>();
  if (P <= 0) return P == 0 ? SP24_ERR_CUDA : SP24_ERR_NO_DEVICE;
  if (P > kOgMaxPairs) P = kOgMaxPairs;
  const int matrices = p.batch;
  int64_t grid = 0;
  double least = orth_plan_phases(&p, matrices, P, false, &grid);
  // A cluster per matrix, of as many pairs as its phases use, where that is expected to be faster.
  for (int c = 2; c <= 8; c *= 2) {
    const int fit = orth_clusters_of<orth_products_kernel<true>, kOgSmem>(c);
    if (fit <= 0) continue;
    OrthProducts q = p;
    int64_t use = 0;
    const double us = orth_plan_phases(&q, 1, c / 2, true, &use) * (double)((matrices + fit - 1) / fit);
    if (us < least) {
      least = us;
      p = q;
      p.cluster = c;
    }
  }
  // Short sides up to 256: G and P in every pair's shared memory.
  bool small = false;
  for (int c = 2; c <= 8 && p.m <= 256; c *= 2) {
    const int fit = orth_clusters_of<orth_small_kernel, kOsSmem>(c);
    if (fit <= 0) continue;
    OrthProducts q = p;
    const double us = orth_small_round(&q, c / 2) * (double)((matrices + fit - 1) / fit);
    if (us < least || (small && us <= least)) {   // (as good by the model: the larger cluster)
      least = us;
      p = q;
      p.cluster = c;
      small = true;
    }
  }
  if (p.cluster) p.batch = 1;
  *plan = {p, matrices, grid, small};
  return SP24_OK;
}

sp24_status launch_orth_products(const OrthMaps &maps, const CUtensorMap &p_st128, const OrthProductsPlan &plan,
                                 cudaStream_t stream) {
  const OrthProducts &p = plan.p;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kOgThreads);
  cfg.dynamicSmemBytes = plan.small ? kOsSmem : kOgSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t err;
  if (p.cluster) {
    cfg.gridDim = dim3((unsigned)(p.cluster * plan.matrices));
    attr[0].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    err = plan.small ? cudaLaunchKernelEx(&cfg, orth_small_kernel, maps, p_st128, p)
                     : cudaLaunchKernelEx(&cfg, orth_products_kernel<true>, maps, p);
  } else {
    cfg.gridDim = dim3(2 * (unsigned)plan.grid);
    attr[0].val.clusterDim.x = 2;
    attr[1].id = cudaLaunchAttributeCooperative;   // its CTAs wait for one another: all are resident, or none starts
    attr[1].val.cooperative = 1;
    err = cudaLaunchKernelEx(&cfg, orth_products_kernel<false>, maps, p);
  }
  if (err != cudaSuccess) {
    cudaGetLastError();
    return SP24_ERR_CUDA;
  }
  return SP24_OK;
}

// x_cols: X in boxes of 64 columns x 64 rows; p_rows, p_half: P in boxes of 128 and 64 rows.
struct OrthLastMaps {
  CUtensorMap x_cols, p_rows, p_half;
};

// launch false: the kernel's set-up on this device only.
template <bool BF16, bool UPDATE, bool TALL, int BN>
sp24_status orth_last_t(const OrthLastMaps &m, OrthLast p, cudaStream_t s, bool launch) {
  constexpr auto kernel = orth_last_kernel<BF16, UPDATE, TALL, BN>;
  const int pairs = pairs_of<kernel, kOlThreads, kOlSmem>();
  if (pairs <= 0) return pairs == 0 ? SP24_ERR_CUDA : SP24_ERR_NO_DEVICE;
  if (!launch) return SP24_OK;
  p.tiles = (p.cols + 255) / 256 * ((p.rows + BN - 1) / BN);
  const int64_t tiles = (int64_t)p.batch * p.tiles;
  const int grid = (int)(tiles < pairs ? tiles : pairs);
  return launch_pdl(kernel, dim3(2 * grid), dim3(kOlThreads), kOlSmem, s, TALL ? m.p_rows : m.x_cols,
                    TALL ? m.x_cols : (BN == 256 ? m.p_rows : m.p_half), p);
}

// Narrow tiles while all of them run at once (512 x 256: 11.4 us of the step with wide ones).
template <bool BF16, bool UPDATE>
sp24_status orth_last(const OrthLastMaps &m, bool tall, const OrthLast &p, cudaStream_t s, bool launch) {
  const bool narrow = 2 * (int64_t)p.batch * p.tiles <= sm_count() / 2;
  if (narrow) return tall ? orth_last_t<BF16, UPDATE, true, 128>(m, p, s, launch) : orth_last_t<BF16, UPDATE, false, 128>(m, p, s, launch);
  return tall ? orth_last_t<BF16, UPDATE, true, 256>(m, p, s, launch) : orth_last_t<BF16, UPDATE, false, 256>(m, p, s, launch);
}

sp24_status run_orth(const OrthPlan &pl, OrthSrc src, const OrthOut &o, int steps, float eps, void *workspace,
                     cudaStream_t stream) {
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  unsigned *counters = reinterpret_cast<unsigned *>(ws + pl.counters);
  OrthPart *part = reinterpret_cast<OrthPart *>(ws + pl.norm);
  float *gamma = reinterpret_cast<float *>(ws + pl.gamma);
  __half *xb[2] = {reinterpret_cast<__half *>(ws + pl.x0), reinterpret_cast<__half *>(ws + pl.x1)};
  void *gram = ws + pl.gram, *poly = ws + pl.poly;
  const uint64_t px = (uint64_t)pl.ldx * 2, pm = (uint64_t)pl.ldm * 2;
  const uint64_t m = (uint64_t)pl.m, n = (uint64_t)pl.n, bt = (uint64_t)pl.count;
  const CUtensorMapSwizzle s128 = CU_TENSOR_MAP_SWIZZLE_128B, s64 = CU_TENSOR_MAP_SWIZZLE_64B;
  OrthMaps maps;
  bool ok = true;
  for (int i = 0; i < 2; ++i)
    ok = ok && make_map_3d(&maps.x_rows[i], xb[i], n, m, bt, px, m * px, 64, 128, s128) &&
         make_map_3d(&maps.x_half[i], xb[i], n, m, bt, px, m * px, 64, 64, s128) &&
         make_map_3d(&maps.x_st[i], xb[i], n, m, bt, px, m * px, 32, 32, s64);
  ok = ok && make_map_3d(&maps.g_rows, gram, m, m, bt, pm, m * pm, 64, 128, s128) &&
       make_map_3d(&maps.g_half, gram, m, m, bt, pm, m * pm, 64, 64, s128) &&
       make_map_3d(&maps.g_st, gram, m, m, bt, pm, m * pm, 32, 32, s64) &&
       make_map_3d(&maps.p_rows, poly, m, m, bt, pm, m * pm, 64, 128, s128) &&
       make_map_3d(&maps.p_st, poly, m, m, bt, pm, m * pm, 32, 32, s64);
  CUtensorMap p_st128 = maps.p_st;   // orth_small_kernel's last P: 64 columns x 32 rows
  if (pl.m <= 256) ok = ok && make_map_3d(&p_st128, poly, m, m, bt, pm, m * pm, 64, 32, s128);
  OrthLastMaps lm = {maps.x_half[(steps - 1) & 1], maps.p_rows, maps.p_rows};
  if (!pl.tall) ok = ok && make_map_3d(&lm.p_half, poly, m, m, bt, pm, m * pm, 64, 64, s128);
  if (!ok) return SP24_ERR_CUDA;

  // Scale of the iterate: a power of two near sqrt(n) (ortho_gemm.cuh).
  int e = 0;
  while ((int64_t(1) << (2 * (e + 1))) <= pl.n) ++e;
  const float s = (float)(1 << e);

  OrthProducts p = {};
  p.m = (int)pl.m;
  p.n = (int)pl.n;
  p.batch = (int)pl.count;
  p.phases = 3 * steps - 1;
  p.wait_budget = g_wait_budget.load();
  p.gram_alpha = 1.0f / (s * s);
  p.gamma = gamma;
  p.a = kNsA;
  p.b = kNsB;
  p.c = kNsC;
  p.part = reinterpret_cast<float *>(ws + pl.part);
  p.counters = counters;
  OrthLast l = {};
  l.rows = (int)pl.rows;
  l.cols = (int)pl.cols;
  l.num_kt = (int)((pl.m + 63) / 64);
  l.batch = (int)pl.count;
  l.tiles = (int)pl.tiles;
  l.wait_budget = p.wait_budget;
  l.alpha = (o.w ? o.step : 1.0f) / s;
  l.gamma = steps == 1 ? gamma : nullptr;
  l.keep = o.keep;
  l.w = o.w;
  l.out16 = o.out16;
  auto last = [&](bool launch) {
    if (o.bf16) return o.w ? orth_last<true, true>(lm, pl.tall, l, stream, launch) : orth_last<true, false>(lm, pl.tall, l, stream, launch);
    return o.w ? orth_last<false, true>(lm, pl.tall, l, stream, launch) : orth_last<false, false>(lm, pl.tall, l, stream, launch);
  };
  // Every kernel's set-up comes before the first launch, which advances the momentum: only a launch itself
  // can fail after that.
  OrthProductsPlan plan;
  sp24_status st = plan_orth_products(p, &plan);
  if (st != SP24_OK || (st = last(false)) != SP24_OK) return st;

  const int64_t col_tiles = (pl.cols + kOrthTile - 1) / kOrthTile;
  const int64_t tiles = col_tiles * ((pl.rows + kOrthTile - 1) / kOrthTile);
  int64_t blocks = (6 * (int64_t)sm_count() + pl.count - 1) / pl.count;   // six blocks of 256 threads an SM
  if (blocks > tiles) blocks = tiles;
  if (blocks > kOrthMaxBlocks) blocks = kOrthMaxBlocks;
  const dim3 grid((unsigned)blocks, (unsigned)pl.count);
  const bool quads = src.cols % 4 == 0 && src.ld % 4 == 0 && src.stride % 4 == 0 && aligned16(src.g) &&
                     (!src.m || aligned16(src.m));
  auto start = pl.tall ? (quads ? orth_start_kernel<true, true> : orth_start_kernel<true, false>)
                       : (quads ? orth_start_kernel<false, true> : orth_start_kernel<false, false>);
  st = launch_pdl(start, grid, dim3(kOrthThreads), 0, stream, src, part, xb[0], pl.ldx, col_tiles, tiles);
  if (st != SP24_OK) return st;
  auto finish = pl.tall ? (quads ? orth_finish_start_kernel<true, true> : orth_finish_start_kernel<true, false>)
                        : (quads ? orth_finish_start_kernel<false, true> : orth_finish_start_kernel<false, false>);
  const int64_t few = (2 * (int64_t)sm_count() + pl.count - 1) / pl.count;
  const dim3 grid2((unsigned)(blocks < few ? blocks : few), (unsigned)pl.count);
  st = launch_pdl(finish, grid2, dim3(kOrthThreads), 0, stream, src, part, (int)blocks, s, eps, xb[0], pl.ldx, col_tiles,
                  tiles, gamma, counters, kOgCounters);
  if (st != SP24_OK) return st;

  if ((st = launch_orth_products(maps, p_st128, plan, stream)) != SP24_OK) return st;
  return last(true);
}

// Buffers as a call sees them, and whether any that it writes shares memory with another.
struct Span {
  const void *p;
  size_t bytes;
};

bool overlap(const Span &a, const Span &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && a.bytes && b.bytes && (x < y ? y - x < a.bytes : x - y < b.bytes);
}

template <size_t N>
bool overlaps_any(const Span &a, const Span (&others)[N]) {
  for (const Span &o : others)
    if (overlap(a, o)) return true;
  return false;
}

sp24_status validate_orth(const OrthPlan &pl, int steps, float eps, const void *workspace, size_t workspace_bytes) {
  if (steps < 1 || steps > 16 || !(eps >= 0.0f) || std::isinf(eps)) return SP24_ERR_INVALID_ARG;
  if (pl.count == 0 || pl.m == 0) return SP24_OK;
  if (!workspace) return SP24_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return SP24_ERR_MISALIGNED;
  if (workspace_bytes < pl.total) return SP24_ERR_SCRATCH_TOO_SMALL;
  return SP24_OK;
}

// Longest contraction whose 32-bit integer sum cannot overflow: K 128 128 <= 2^31 - 1, K a
// multiple of 16.
constexpr int64_t kMaxI8K = 131056;

template <bool BF16, bool GELU>
sp24_status launch_i8_pair(const int8_t *Xq, int64_t T, int64_t K, const int8_t *Wq, int64_t N, void *Y,
                           const float *sx, const float *sw, cudaStream_t s) {
  using G = I8Geom;
  constexpr int BN = G::BN;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap tw, tx, ty;
  if (!make_map_2d(&tw, Wq, (uint64_t)K, (uint64_t)N, (uint64_t)K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B, u8) ||
      !make_map_2d(&tx, Xq, (uint64_t)K, (uint64_t)T, (uint64_t)K, 128, BN / 2, CU_TENSOR_MAP_SWIZZLE_128B, u8) ||
      !make_map_2d(&ty, Y, (uint64_t)N, (uint64_t)T, (uint64_t)N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
    return SP24_ERR_CUDA;
  constexpr auto kernel = gemm_i8_kernel<BF16, GELU>;
  const int pairs = pairs_of<kernel, kI8Threads, G::kSmem>();
  if (pairs <= 0) return pairs == 0 ? SP24_ERR_CUDA : SP24_ERR_NO_DEVICE;
  const int64_t tiles = ((N + 255) / 256) * ((T + BN - 1) / BN);
  if (tiles > INT32_MAX) return SP24_ERR_UNSUPPORTED_SHAPE;
  const int grid = (int)(tiles < pairs ? tiles : pairs);
  return launch_pdl(kernel, dim3(2 * grid), dim3(kI8Threads), G::kSmem, s, tw, tx, ty, (int)N, (int)T,
                    (int)((K + 127) / 128), (uint64_t)g_wait_budget.load(), sw, sx);
}

// Parts of K: doubled while the CTAs stay within one per SM and each keeps two stages.
int i8_split(int64_t tiles, int64_t kt) {
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sm_count() && kt >= 4 * split) split *= 2;
  return split;
}

// Whether gemm_i8_few_kernel is expected to be faster than the pairs' 256 x 256 tiles, from fits of
// both over 9-1024 tokens, 640-25600 features and K from 640 to 12800 with weights from memory (mean
// errors 5% and 3%): microseconds of launch and epilogue, then of each stage of 128 along K, more
// as more SMs read.  At 100 tokens: K 1600, N 6400 7.5 on pairs, 10.0 here; K 6400, N 1600 17.9 and 9.4.
bool i8_few_pays(int64_t T, int64_t K, int64_t N) {
  const int64_t tp = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  const int64_t sms = sm_count(), kt = (K + 127) / 128;
  const int64_t tiles = (N + 127) / 128 * ((T + tp - 1) / tp), wide = (N + 255) / 256 * ((T + 255) / 256);
  if (T > 128 && tiles > sms) return false;
  const int split = i8_split(tiles, kt);
  const int64_t mine = (kt + split - 1) / split, ctas = tiles * split;
  const int64_t smem = (mine < 8 ? mine : 8) * (16384 + 128 * tp) + 1280;
  const int64_t at_once = sms * (2 * smem <= 232448 ? 2 : 1);
  const double stages = (double)(mine * ((ctas + at_once - 1) / at_once));
  const double few = 2.8 + 0.018 * (double)tp + (split > 1 ? 0.4 + 0.017 * (double)tp : 0.0) +
                     stages * (0.09 + 0.275 * (double)(ctas < sms ? ctas : sms) / (double)sms);
  const int64_t pairs = sms / 2, used = wide < pairs ? wide : pairs;
  const double pair = 3.35 + 0.0044 * (double)(T < 256 ? T : 256) +
                      (double)(kt * ((wide + pairs - 1) / pairs)) * (0.26 + 0.136 * (double)used / (double)pairs);
  return few < pair;
}

template <int TP, bool BF16, bool GELU>
sp24_status launch_i8_few(const int8_t *Xq, int64_t T, int64_t K, const int8_t *Wq, int64_t N, void *Y, const float *sx,
                          const float *sw, cudaStream_t s) {
  using G = I8sGeom<TP>;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap tw, tx;
  if (!make_map_2d(&tw, Wq, (uint64_t)K, (uint64_t)N, (uint64_t)K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B, u8) ||
      !make_map_2d(&tx, Xq, (uint64_t)K, (uint64_t)T, (uint64_t)K, 128, TP, CU_TENSOR_MAP_SWIZZLE_128B, u8))
    return SP24_ERR_CUDA;
  constexpr auto kernel = gemm_i8_few_kernel<TP, BF16, GELU>;
  static PerDevice opt_in;   // 1: shared memory granted
  const int dev = current_device();
  if (dev < 0) return SP24_ERR_NO_DEVICE;
  std::call_once(opt_in.once[dev], [&] {
    opt_in.value[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             G::smem_for(G::kStagesMost)) == cudaSuccess;
    if (!opt_in.value[dev]) cudaGetLastError();
  });
  if (!opt_in.value[dev]) return SP24_ERR_CUDA;
  const int64_t ft = (N + 127) / 128, tt = (T + TP - 1) / TP, kt = (K + 127) / 128;
  const int split = i8_split(ft * tt, kt);
  const int64_t mine = (kt + split - 1) / split;
  const int stages = (int)(mine < G::kStagesMost ? mine : G::kStagesMost);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ft * split), (unsigned)tt);
  cfg.blockDim = dim3(kI8sThreads);
  cfg.dynamicSmemBytes = G::smem_for(stages);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, tw, tx, (int)N, (int)T, (int)kt, split, stages, (uint64_t)g_wait_budget.load(), sw,
                         sx, static_cast<uint16_t *>(Y)) != cudaSuccess) {
    cudaGetLastError();
    return SP24_ERR_CUDA;
  }
  return SP24_OK;
}

template <bool BF16, bool GELU>
sp24_status launch_i8(const int8_t *Xq, int64_t T, int64_t K, const int8_t *Wq, int64_t N, void *Y, const float *sx,
                      const float *sw, cudaStream_t s) {
  // Dot products while one pass of short blocks covers them (cold weights): 4 x 1600 x 6400 5.0 us
  // against 5.5 on tensor cores, 8 x 6400 x 6400 17 against 10.3.
  if (T <= 2 ? N <= 8192 || K >= 1024 : T <= 8 && T * N * ((K + 2047) / 2048) <= 25600) {
    const dim3 grid((unsigned)(N / kI8vRows));
    uint16_t *y = static_cast<uint16_t *>(Y);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kI8vThreads), 0, s, Xq, sx, (int)T, (int)K, Wq, sw, (int)N, y); };
    if (K <= 16 * kI8vThreads)
      return T == 1   ? go(gemv_i8_kernel<1, 1, BF16, GELU>)
             : T == 2 ? go(gemv_i8_kernel<2, 1, BF16, GELU>)
             : T <= 4 ? go(gemv_i8_kernel<4, 1, BF16, GELU>)
                      : go(gemv_i8_kernel<8, 1, BF16, GELU>);
    return T == 1   ? go(gemv_i8_kernel<1, 2, BF16, GELU>)
           : T == 2 ? go(gemv_i8_kernel<2, 2, BF16, GELU>)
           : T <= 4 ? go(gemv_i8_kernel<4, 2, BF16, GELU>)
                    : go(gemv_i8_kernel<8, 2, BF16, GELU>);
  }
  if (!i8_few_pays(T, K, N)) return launch_i8_pair<BF16, GELU>(Xq, T, K, Wq, N, Y, sx, sw, s);
  if (T <= 16) return launch_i8_few<16, BF16, GELU>(Xq, T, K, Wq, N, Y, sx, sw, s);
  if (T <= 32) return launch_i8_few<32, BF16, GELU>(Xq, T, K, Wq, N, Y, sx, sw, s);
  if (T <= 64) return launch_i8_few<64, BF16, GELU>(Xq, T, K, Wq, N, Y, sx, sw, s);
  return launch_i8_few<128, BF16, GELU>(Xq, T, K, Wq, N, Y, sx, sw, s);
}

// A warp per row holds the row in registers (up to 6144 entries); longer rows, and a matrix
// of few rows, take a block per row (up to 8192 in registers); the rest re-reads its rows.
template <bool BF16, bool MASKED>
sp24_status launch_quant_t(const uint16_t *X, int64_t rows, int64_t cols, int64_t ldx, const uint8_t *idx, int8_t *q,
                           float *scale, cudaStream_t s) {
  const int64_t vecs = cols / 8;
  const bool vec = cols % 8 == 0 && ldx % 8 == 0 && aligned_to(idx, 2);
  const int64_t warp_blocks = (rows + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
  auto go = [&](auto kernel, int64_t blocks) {
    return launch_pdl(kernel, dim3((unsigned)(blocks < INT32_MAX ? blocks : INT32_MAX)), dim3(kQuantThreads), 0, s, X,
                      rows, cols, ldx, idx, q, scale);
  };
  if (vec && vecs > 0 && vecs <= 4 * kQuantThreads && (rows < 4 * (int64_t)sm_count() || vecs > 24 * 32))
    return vecs <= kQuantThreads ? go(quantize_vec_kernel<BF16, MASKED, kQuantThreads, 1>, rows)
                                 : go(quantize_vec_kernel<BF16, MASKED, kQuantThreads, 4>, rows);
  if (vec && vecs > 0 && vecs <= 24 * 32) {
    if (vecs <= 4 * 32) return go(quantize_vec_kernel<BF16, MASKED, 32, 4>, warp_blocks);
    if (vecs <= 8 * 32) return go(quantize_vec_kernel<BF16, MASKED, 32, 8>, warp_blocks);
    if (vecs <= 16 * 32) return go(quantize_vec_kernel<BF16, MASKED, 32, 16>, warp_blocks);
    return go(quantize_vec_kernel<BF16, MASKED, 32, 24>, warp_blocks);
  }
  return go(quantize_rows_kernel<BF16, MASKED>, rows);
}

template <bool BF16>
sp24_status launch_quant(const uint16_t *X, int64_t rows, int64_t cols, int64_t ldx, const uint8_t *idx, int8_t *q,
                         float *scale, cudaStream_t s) {
  return idx ? launch_quant_t<BF16, true>(X, rows, cols, ldx, idx, q, scale, s)
             : launch_quant_t<BF16, false>(X, rows, cols, ldx, idx, q, scale, s);
}

}  // namespace

namespace {
// (packed chunk layout of the derivative-saving epilogues; see gemm_sp.cuh)
// Element offset, in the packed chunk layout of a [T x M] matrix, of (t, m).
size_t aux_packed_offset(int64_t t, int64_t m, int64_t M) {
  const int64_t tin = t & 15, fin = m & 31, h = fin >> 4, ff = fin & 15;
  const int64_t lane = 4 * (ff & 7) + ((tin & 7) >> 1), reg = 2 * (tin >> 3) + (ff >> 3);
  const int64_t block = (t >> 4) * ((M + 31) / 32) + (m >> 5);
  return (size_t)(block * 512 + h * 256 + lane * 8 + reg * 2 + (tin & 1));
}
}  // namespace

extern "C" {

const char *sp24_status_string(sp24_status st) {
  switch (st) {
    case SP24_OK: return "SP24_OK";
    case SP24_ERR_INVALID_ARG: return "SP24_ERR_INVALID_ARG";
    case SP24_ERR_UNSUPPORTED_SHAPE: return "SP24_ERR_UNSUPPORTED_SHAPE";
    case SP24_ERR_UNSUPPORTED_DTYPE: return "SP24_ERR_UNSUPPORTED_DTYPE";
    case SP24_ERR_MISALIGNED: return "SP24_ERR_MISALIGNED";
    case SP24_ERR_CUDA: return "SP24_ERR_CUDA";
    case SP24_ERR_TIMEOUT: return "SP24_ERR_TIMEOUT";
    case SP24_ERR_NO_DEVICE: return "SP24_ERR_NO_DEVICE";
    case SP24_ERR_SCRATCH_TOO_SMALL: return "SP24_ERR_SCRATCH_TOO_SMALL";
  }
  return "SP24_UNKNOWN_STATUS";
}

sp24_status sp24_pattern_table(uint16_t *out) {
  if (!out) return SP24_ERR_INVALID_ARG;
  constexpr PatternTables t = make_pattern_tables();
  for (int p = 0; p < kNumPatterns; ++p) out[p] = t.bits[p];
  return SP24_OK;
}

sp24_status sp24_compressed_size(int64_t rows, int64_t cols, sp24_dtype dtype, size_t *vals_bytes,
                                 size_t *meta_bytes) {
  if (!vals_bytes || !meta_bytes || rows < 0 || cols < 0) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (rows % 4 || cols % 4) return SP24_ERR_UNSUPPORTED_SHAPE;
  *vals_bytes = (size_t)rows * (size_t)(cols / 2) * 2u;
  *meta_bytes = meta_bytes_of(rows, cols);
  return SP24_OK;
}

sp24_status sp24_mask_step(const void *W, sp24_dtype dtype, int64_t rows, int64_t cols, int64_t ldw, uint8_t *idx,
                           const uint8_t *idx_prev, unsigned long long *d_flip_count, void *vals_row,
                           void *meta_row, void *vals_col, void *meta_col, void *stream) {
  sp24_status st = validate_w(W, dtype, rows, cols, ldw);
  if (st != SP24_OK) return st;
  const bool flip = idx_prev != nullptr;
  if ((idx_prev == nullptr) != (d_flip_count == nullptr)) return SP24_ERR_INVALID_ARG;
  const bool any_c = vals_row || meta_row || vals_col || meta_col;
  const bool all_c = vals_row && meta_row && vals_col && meta_col;
  if (any_c && !all_c) return SP24_ERR_INVALID_ARG;
  if (!idx && rows > 0 && cols > 0) return SP24_ERR_INVALID_ARG;
  if (all_c) {
    if (rows % 16 || cols % 16) return SP24_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(vals_row) || !aligned16(meta_row) || !aligned16(vals_col) || !aligned16(meta_col))
      return SP24_ERR_MISALIGNED;
  }
  if ((st = check_device()) != SP24_OK) return st;
  cudaStream_t s = as_stream(stream);
  if (flip && cudaMemsetAsync(d_flip_count, 0, sizeof(unsigned long long), s) != cudaSuccess)
    return SP24_ERR_CUDA;
  if (rows == 0 || cols == 0) return SP24_OK;
  const bool bf = dtype == SP24_BF16;
  if (all_c && flip)
    return launch_mask_d<true, true, true>(bf, W, rows, cols, ldw, idx, idx_prev, d_flip_count, vals_row, meta_row,
                                           vals_col, meta_col, s);
  if (all_c)
    return launch_mask_d<true, true, false>(bf, W, rows, cols, ldw, idx, nullptr, nullptr, vals_row, meta_row,
                                            vals_col, meta_col, s);
  if (flip)
    return launch_mask_d<true, false, true>(bf, W, rows, cols, ldw, idx, idx_prev, d_flip_count, nullptr, nullptr,
                                            nullptr, nullptr, s);
  return launch_mask_d<true, false, false>(bf, W, rows, cols, ldw, idx, nullptr, nullptr, nullptr, nullptr,
                                           nullptr, nullptr, s);
}

sp24_status sp24_mask_search(const void *W, sp24_dtype dtype, int64_t rows, int64_t cols, int64_t ldw, uint8_t *idx,
                             void *stream) {
  return sp24_mask_step(W, dtype, rows, cols, ldw, idx, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                        stream);
}

sp24_status sp24_prune_compress(const void *W, sp24_dtype dtype, int64_t rows, int64_t cols, int64_t ldw,
                                const uint8_t *idx, void *vals_row, void *meta_row, void *vals_col, void *meta_col,
                                void *stream) {
  sp24_status st = validate_w(W, dtype, rows, cols, ldw);
  if (st != SP24_OK) return st;
  if ((vals_row == nullptr) != (meta_row == nullptr) || (vals_col == nullptr) != (meta_col == nullptr))
    return SP24_ERR_INVALID_ARG;
  if (rows % 16 || cols % 16) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (rows > 0 && cols > 0 && !idx) return SP24_ERR_INVALID_ARG;
  if ((vals_row && (!aligned16(vals_row) || !aligned16(meta_row))) ||
      (vals_col && (!aligned16(vals_col) || !aligned16(meta_col))))
    return SP24_ERR_MISALIGNED;
  if ((st = check_device()) != SP24_OK) return st;
  if (rows == 0 || cols == 0 || (!vals_row && !vals_col)) return SP24_OK;
  return launch_mask_d<false, true, false>(dtype == SP24_BF16, W, rows, cols, ldw, const_cast<uint8_t *>(idx),
                                           nullptr, nullptr, vals_row, meta_row, vals_col, meta_col,
                                           as_stream(stream));
}

sp24_status sp24_gemm_fwd(const void *X, int64_t T, int64_t K, const void *vals_row, const void *meta_row, int64_t N,
                          sp24_dtype dtype, void *Y, sp24_epilogue epi, void *aux, void *stream) {
  sp24_status st = validate_gemm(X, T, K, vals_row, meta_row, N, dtype, Y, epi, aux, kFwdEpis);
  if (st != SP24_OK) return st;
  if ((st = check_device()) != SP24_OK) return st;
  if (T == 0) return SP24_OK;
  return launch_gemm<true>(X, T, K, vals_row, meta_row, N, dtype, Y, epi, aux, as_stream(stream));
}

sp24_status sp24_gemm_dgrad(const void *dY, int64_t T, int64_t N, const void *vals_col, const void *meta_col,
                            int64_t K, sp24_dtype dtype, void *dX, sp24_epilogue epi, const void *aux,
                            void *stream) {
  sp24_status st = validate_gemm(dY, T, N, vals_col, meta_col, K, dtype, dX, epi, aux, kDgradEpis);
  if (st != SP24_OK) return st;
  if ((st = check_device()) != SP24_OK) return st;
  if (T == 0) return SP24_OK;
  return launch_gemm<true>(dY, T, N, vals_col, meta_col, K, dtype, dX, epi, const_cast<void *>(aux),
                          as_stream(stream));
}

sp24_status sp24_gemm_dense(const void *B, int64_t T, int64_t Kd, const void *A, int64_t M, sp24_dtype dtype,
                            void *out, sp24_epilogue epi, void *aux, void *stream) {
  sp24_status st = validate_gemm(B, T, Kd, A, A, M, dtype, out, epi, aux, kDenseEpis);
  if (st != SP24_OK) return st;
  if ((st = check_device()) != SP24_OK) return st;
  if (T == 0) return SP24_OK;
  return launch_gemm<false>(B, T, Kd, A, nullptr, M, dtype, out, epi, aux, as_stream(stream));
}

sp24_status sp24_gemm_dgrad_dense(const void *dY, int64_t T, int64_t N, const void *W, int64_t K, sp24_dtype dtype,
                                  void *dX, sp24_epilogue epi, const void *aux, void *stream) {
  sp24_status st = validate_gemm(dY, T, N, W, W, K, dtype, dX, epi, aux, kDenseDgradEpis);
  if (st != SP24_OK) return st;
  if ((st = check_device()) != SP24_OK) return st;
  if (T == 0) return SP24_OK;
  return launch_gemm<false>(dY, T, N, W, nullptr, K, dtype, dX, epi, const_cast<void *>(aux), as_stream(stream),
                            /*a_mn=*/true);
}

sp24_status sp24_transpose(const void *in, int64_t rows, int64_t cols, sp24_dtype dtype, void *out, void *stream) {
  if (rows < 0 || cols < 0) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (rows == 0 || cols == 0) return SP24_OK;
  if (!in || !out) return SP24_ERR_INVALID_ARG;
  if (!aligned16(in) || !aligned16(out)) return SP24_ERR_MISALIGNED;
  if (rows > INT32_MAX || cols > INT32_MAX) return SP24_ERR_UNSUPPORTED_SHAPE;
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  const dim3 grid((unsigned)((cols + kTransTile - 1) / kTransTile),
                  (unsigned)((rows + kTransTile - 1) / kTransTile < 65535 ? (rows + kTransTile - 1) / kTransTile
                                                                            : 65535));
  return launch_pdl(transpose16_kernel, grid, dim3(256), 0, as_stream(stream),
                    static_cast<const uint16_t *>(in), static_cast<uint16_t *>(out), rows, cols);
}

sp24_status sp24_mvue_sparsify(const void *dY, int64_t T, int64_t N, int64_t ldy, sp24_dtype dtype, uint64_t seed,
                               uint64_t offset, void *vals, void *meta, void *stream) {
  if (T < 0 || N < 0 || ldy < N) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (T % 16 || N % 8) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (T > INT32_MAX || N > (int64_t)65535 / 2 * 128) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || N == 0) return SP24_OK;
  if (!dY || !vals || !meta) return SP24_ERR_INVALID_ARG;
  if (!aligned16(dY) || !aligned16(vals) || !aligned16(meta) || ldy % 8) return SP24_ERR_MISALIGNED;
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  // Whole metadata chunks: 128 tokens x 128 columns, two CTAs per chunk.
  const dim3 grid((unsigned)((T + kMvueTokens - 1) / kMvueTokens), (unsigned)(2 * ((N + 127) / 128)));
  cudaStream_t s = as_stream(stream);
  const uint16_t *d16 = static_cast<const uint16_t *>(dY);
  uint16_t *v16 = static_cast<uint16_t *>(vals);
  uint8_t *m8 = static_cast<uint8_t *>(meta);
  const PhiloxKeys keys = philox4x64_keys(seed, offset);
  return dtype == SP24_BF16
             ? launch_pdl(mvue_sparsify_kernel<true>, grid, dim3(kMvueThreads), 0, s, d16, T, N, ldy, keys, v16, m8)
             : launch_pdl(mvue_sparsify_kernel<false>, grid, dim3(kMvueThreads), 0, s, d16, T, N, ldy, keys, v16, m8);
}

sp24_status sp24_gemm_wgrad(const void *X, int64_t T, int64_t K, const void *vals, const void *meta, int64_t N,
                            sp24_dtype dtype, float *dW, void *stream) {
  if (T < 0 || K < 0 || N < 0) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (T % 16 || N % 16 || K % 8) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (T > INT32_MAX || K > INT32_MAX || N > INT32_MAX) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (N == 0 || K == 0) return SP24_OK;
  if (!dW || (T > 0 && (!X || !vals || !meta))) return SP24_ERR_INVALID_ARG;
  if (!aligned16(dW) || (T > 0 && (!aligned16(X) || !aligned16(vals) || !aligned16(meta)))) return SP24_ERR_MISALIGNED;
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  cudaStream_t s = as_stream(stream);
  if (T == 0) {   // an empty sum over tokens
    return cudaMemsetAsync(dW, 0, (size_t)N * (size_t)K * sizeof(float), s) == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
  }
  return dtype == SP24_BF16 ? launch_wgrad<true, true>(X, T, K, vals, meta, N, dW, s)
                            : launch_wgrad<false, true>(X, T, K, vals, meta, N, dW, s);
}

sp24_status sp24_gemm_wgrad_noalloc(const void *X, int64_t T, int64_t K, const void *vals, const void *meta,
                                    int64_t N, sp24_dtype dtype, float *dW, void *stream) {
  if (T < 0 || K < 0 || N < 0) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (T % 16 || N % 16 || K % 8) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (T > INT32_MAX || K > INT32_MAX || N > INT32_MAX) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (N == 0 || K == 0) return SP24_OK;
  if (!dW || (T > 0 && (!X || !vals || !meta))) return SP24_ERR_INVALID_ARG;
  if (!aligned16(dW) || (T > 0 && (!aligned16(X) || !aligned16(vals) || !aligned16(meta)))) return SP24_ERR_MISALIGNED;
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  cudaStream_t s = as_stream(stream);
  if (T == 0) {   // an empty sum over tokens
    return cudaMemsetAsync(dW, 0, (size_t)N * (size_t)K * sizeof(float), s) == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
  }
  SkWorkspace fixed;
  st = noalloc_scratch(&fixed);
  if (st != SP24_OK) return st;
  return dtype == SP24_BF16 ? launch_wgrad<true, true>(X, T, K, vals, meta, N, dW, s, nullptr, nullptr, 0.0f, &fixed)
                            : launch_wgrad<false, true>(X, T, K, vals, meta, N, dW, s, nullptr, nullptr, 0.0f, &fixed);
}

sp24_status sp24_gemm_wgrad_decay(const void *X, int64_t T, int64_t K, const void *vals, const void *meta,
                                  int64_t N, sp24_dtype dtype, const void *W, const uint8_t *idx, float lambda,
                                  float *dW, void *stream) {
  if (T < 0 || K < 0 || N < 0) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (T % 16 || N % 16 || K % 8) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (T > INT32_MAX || K > INT32_MAX || N > INT32_MAX) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (N == 0 || K == 0) return SP24_OK;
  if (!dW || !W || !idx || (T > 0 && (!X || !vals || !meta))) return SP24_ERR_INVALID_ARG;
  if (!aligned16(dW) || !aligned16(W) || (T > 0 && (!aligned16(X) || !aligned16(vals) || !aligned16(meta))))
    return SP24_ERR_MISALIGNED;
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  cudaStream_t s = as_stream(stream);
  if (T == 0) {   // an empty sum over tokens, then the decay of the zero gradient
    if (cudaMemsetAsync(dW, 0, (size_t)N * (size_t)K * sizeof(float), s) != cudaSuccess) return SP24_ERR_CUDA;
    return sp24_masked_decay(dW, W, dtype, N, K, idx, lambda, stream);
  }
  return dtype == SP24_BF16 ? launch_wgrad<true, true>(X, T, K, vals, meta, N, dW, s, W, idx, lambda)
                            : launch_wgrad<false, true>(X, T, K, vals, meta, N, dW, s, W, idx, lambda);
}

sp24_status sp24_gemm_wgrad_dense(const void *X, int64_t T, int64_t K, const void *dY, int64_t N, sp24_dtype dtype,
                                  float *dW, void *stream) {
  if (T < 0 || K < 0 || N < 0) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (T % 16 || N % 16 || K % 8) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (T > INT32_MAX || K > INT32_MAX || N > INT32_MAX) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (N == 0 || K == 0) return SP24_OK;
  if (!dW || (T > 0 && (!X || !dY))) return SP24_ERR_INVALID_ARG;
  if (!aligned16(dW) || (T > 0 && (!aligned16(X) || !aligned16(dY)))) return SP24_ERR_MISALIGNED;
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  cudaStream_t s = as_stream(stream);
  if (T == 0) {   // an empty sum over tokens
    return cudaMemsetAsync(dW, 0, (size_t)N * (size_t)K * sizeof(float), s) == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
  }
  return dtype == SP24_BF16 ? launch_wgrad<true, false>(X, T, K, dY, nullptr, N, dW, s)
                            : launch_wgrad<false, false>(X, T, K, dY, nullptr, N, dW, s);
}

sp24_status sp24_masked_decay(float *grad, const void *W, sp24_dtype dtype, int64_t rows, int64_t cols,
                              const uint8_t *idx, float lambda, void *stream) {
  sp24_status st = validate_w(W, dtype, rows, cols, cols);
  if (st != SP24_OK) return st;
  if (rows > 0 && cols > 0 && (!grad || !idx)) return SP24_ERR_INVALID_ARG;
  if (rows > 0 && cols > 0 && !aligned16(grad)) return SP24_ERR_MISALIGNED;
  if ((st = check_device()) != SP24_OK) return st;
  if (rows == 0 || cols == 0) return SP24_OK;
  const int64_t strips = (cols / 4 + 255) / 256;
  const int64_t brows = rows / 4;
  const dim3 grid((unsigned)strips, (unsigned)(brows < 65535 ? brows : 65535));
  cudaStream_t s = as_stream(stream);
  const uint16_t *w16 = static_cast<const uint16_t *>(W);
  return dtype == SP24_BF16 ? launch_pdl(masked_decay_kernel<true>, grid, dim3(256), 0, s, grad, w16, idx, rows, cols, lambda)
                            : launch_pdl(masked_decay_kernel<false>, grid, dim3(256), 0, s, grad, w16, idx, rows, cols, lambda);
}

sp24_status sp24_flip_rate(const uint8_t *idx_prev, const uint8_t *idx_cur, int64_t nblocks,
                           unsigned long long *d_count, void *stream) {
  if (nblocks < 0 || !d_count || (nblocks > 0 && (!idx_prev || !idx_cur))) return SP24_ERR_INVALID_ARG;
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  cudaStream_t s = as_stream(stream);
  if (cudaMemsetAsync(d_count, 0, sizeof(unsigned long long), s) != cudaSuccess) return SP24_ERR_CUDA;
  if (nblocks == 0) return SP24_OK;
  const int64_t want = (nblocks / 16 + 255) / 256 + 1;
  const int grid = (int)(want < (int64_t)sm_count() * 8 ? want : (int64_t)sm_count() * 8);
  return launch_pdl(flip_count_kernel, dim3(grid), dim3(256), 0, s, idx_prev, idx_cur, nblocks, d_count);
}

sp24_status sp24_orthogonalize_size(int64_t count, int64_t rows, int64_t cols, size_t *workspace_bytes) {
  if (!workspace_bytes) return SP24_ERR_INVALID_ARG;
  OrthPlan pl;
  const sp24_status st = orth_plan(count, rows, cols, &pl);
  if (st != SP24_OK) return st;
  *workspace_bytes = pl.total;
  return SP24_OK;
}

sp24_status sp24_orthogonalize(const float *G, int64_t count, int64_t rows, int64_t cols, int64_t ldg,
                               int64_t batch_stride, int steps, float eps, void *out, sp24_dtype dtype,
                               void *workspace, size_t workspace_bytes, void *stream) {
  OrthPlan pl;
  sp24_status st = orth_plan(count, rows, cols, &pl);
  if (st != SP24_OK) return st;
  if (ldg < cols || batch_stride < 0) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if ((st = validate_orth(pl, steps, eps, workspace, workspace_bytes)) != SP24_OK) return st;
  const bool empty = count == 0 || pl.m == 0;
  if (!empty && (!G || !out)) return SP24_ERR_INVALID_ARG;
  if (!empty && (!aligned_to(G, 4) || !aligned_to(out, 2))) return SP24_ERR_MISALIGNED;
  if ((st = check_device()) != SP24_OK) return st;
  if (empty) return SP24_OK;
  const Span sg = {G, 4 * (size_t)((count - 1) * batch_stride + (rows - 1) * ldg + cols)};
  if (overlaps_any(Span{workspace, pl.total}, {sg, Span{out, 2 * (size_t)(count * rows * cols)}})) return SP24_ERR_INVALID_ARG;
  OrthSrc src = {};
  src.g = G;
  src.rows = rows;
  src.cols = cols;
  src.ld = ldg;
  src.stride = batch_stride;
  OrthOut o = {};
  o.out16 = static_cast<uint16_t *>(out);
  o.bf16 = dtype == SP24_BF16;
  return run_orth(pl, src, o, steps, eps, workspace, as_stream(stream));
}

sp24_status sp24_muon_step(const float *grad, float *momentum, float *W, void *W16, sp24_dtype dtype, int64_t count,
                           int64_t rows, int64_t cols, float mu, int nesterov, float lr, float weight_decay, float scale,
                           int steps, float eps, void *workspace, size_t workspace_bytes, void *stream) {
  OrthPlan pl;
  sp24_status st = orth_plan(count, rows, cols, &pl);
  if (st != SP24_OK) return st;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if ((st = validate_orth(pl, steps, eps, workspace, workspace_bytes)) != SP24_OK) return st;
  const bool empty = count == 0 || pl.m == 0;
  if (!empty && (!grad || !momentum || !W)) return SP24_ERR_INVALID_ARG;
  if (!empty && (!aligned_to(grad, 4) || !aligned_to(momentum, 4) || !aligned_to(W, 4) || !aligned_to(W16, 2)))
    return SP24_ERR_MISALIGNED;
  if ((st = check_device()) != SP24_OK) return st;
  if (empty) return SP24_OK;
  // The momentum is written while the gradient may have to be read once more; W16 while other tiles of W still
  // wait for their update.
  const size_t n = (size_t)count * rows * cols;
  const Span sg = {grad, 4 * n}, sm = {momentum, 4 * n}, sw = {W, 4 * n}, s16 = {W16, 2 * n};
  if (overlaps_any(sm, {sg, sw, s16}) || overlaps_any(s16, {sg, sw}) ||
      overlaps_any(Span{workspace, pl.total}, {sg, sm, sw, s16}))
    return SP24_ERR_INVALID_ARG;
  OrthSrc src = {};
  src.g = grad;
  src.m = momentum;
  src.rows = rows;
  src.cols = cols;
  src.ld = cols;
  src.stride = rows * cols;
  src.mu = mu;
  src.nesterov = nesterov ? 1 : 0;
  OrthOut o = {};
  o.out16 = static_cast<uint16_t *>(W16);
  o.w = W;
  o.keep = (float)(1.0 - (double)lr * (double)weight_decay);
  o.step = (float)((double)lr * (double)scale);
  o.bf16 = dtype == SP24_BF16;
  return run_orth(pl, src, o, steps, eps, workspace, as_stream(stream));
}

sp24_status sp24_quantize_rows(const void *X, sp24_dtype dtype, int64_t rows, int64_t cols, int64_t ldx,
                               const uint8_t *idx, int8_t *q, float *scale, void *stream) {
  if (rows < 0 || cols < 0 || ldx < cols) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (idx && (rows % 4 || cols % 4)) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (rows > 0 && (!scale || (cols > 0 && (!X || !q)))) return SP24_ERR_INVALID_ARG;
  if (rows > 0 && (!aligned_to(scale, 4) || (cols > 0 && (!aligned16(X) || !aligned16(q))))) return SP24_ERR_MISALIGNED;
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  if (rows == 0) return SP24_OK;
  const Span sx = {X, cols ? 2 * (size_t)((rows - 1) * ldx + cols) : 0}, si = {idx, (size_t)(rows / 4) * (size_t)(cols / 4)};
  const Span sq = {q, (size_t)(rows * cols)}, ss = {scale, 4 * (size_t)rows};
  if (overlaps_any(sq, {sx, si, ss}) || overlaps_any(ss, {sx, si})) return SP24_ERR_INVALID_ARG;
  const uint16_t *x = static_cast<const uint16_t *>(X);
  return dtype == SP24_BF16 ? launch_quant<true>(x, rows, cols, ldx, idx, q, scale, as_stream(stream))
                            : launch_quant<false>(x, rows, cols, ldx, idx, q, scale, as_stream(stream));
}

sp24_status sp24_gemm_i8(const int8_t *Xq, const float *sx, int64_t T, int64_t K, const int8_t *Wq, const float *sw,
                         int64_t N, sp24_dtype dtype, void *Y, sp24_epilogue epi, void *stream) {
  if (T < 0 || K <= 0 || N <= 0) return SP24_ERR_INVALID_ARG;
  if (!Wq || !sw || (T > 0 && (!Xq || !sx || !Y))) return SP24_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return SP24_ERR_UNSUPPORTED_DTYPE;
  if (epi != SP24_EPI_NONE && epi != SP24_EPI_GELU) return SP24_ERR_INVALID_ARG;
  if (K % 16 || N % 16 || K > kMaxI8K || T > INT32_MAX - 256 || N > INT32_MAX - 256) return SP24_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(Xq) || !aligned16(Wq) || !aligned16(Y) || !aligned_to(sx, 4) || !aligned_to(sw, 4)) return SP24_ERR_MISALIGNED;
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  if (T == 0) return SP24_OK;
  if (overlaps_any(Span{Y, 2 * (size_t)(T * N)}, {Span{Xq, (size_t)(T * K)}, Span{Wq, (size_t)(N * K)}, Span{sx, 4 * (size_t)T},
                                                  Span{sw, 4 * (size_t)N}}))
    return SP24_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  if (dtype == SP24_BF16)
    return epi == SP24_EPI_GELU ? launch_i8<true, true>(Xq, T, K, Wq, N, Y, sx, sw, s)
                                : launch_i8<true, false>(Xq, T, K, Wq, N, Y, sx, sw, s);
  return epi == SP24_EPI_GELU ? launch_i8<false, true>(Xq, T, K, Wq, N, Y, sx, sw, s)
                              : launch_i8<false, false>(Xq, T, K, Wq, N, Y, sx, sw, s);
}

sp24_status sp24_aux_packed_size(int64_t T, int64_t M, size_t *bytes) {
  if (T < 0 || M < 0 || !bytes) return SP24_ERR_INVALID_ARG;
  *bytes = (size_t)((T + 15) / 16) * (size_t)((M + 31) / 32) * 1024u;
  return SP24_OK;
}

sp24_status sp24_aux_pack(const void *rowmajor, int64_t T, int64_t M, void *packed) {
  if (T < 0 || M < 0 || (T > 0 && M > 0 && (!rowmajor || !packed))) return SP24_ERR_INVALID_ARG;
  const uint16_t *src = static_cast<const uint16_t *>(rowmajor);
  uint16_t *dst = static_cast<uint16_t *>(packed);
  size_t bytes = 0;
  sp24_aux_packed_size(T, M, &bytes);
  if (bytes) memset(dst, 0, bytes);
  for (int64_t t = 0; t < T; ++t)
    for (int64_t m = 0; m < M; ++m) dst[aux_packed_offset(t, m, M)] = src[t * M + m];
  return SP24_OK;
}

sp24_status sp24_aux_unpack(const void *packed, int64_t T, int64_t M, void *rowmajor) {
  if (T < 0 || M < 0 || (T > 0 && M > 0 && (!rowmajor || !packed))) return SP24_ERR_INVALID_ARG;
  const uint16_t *src = static_cast<const uint16_t *>(packed);
  uint16_t *dst = static_cast<uint16_t *>(rowmajor);
  for (int64_t t = 0; t < T; ++t)
    for (int64_t m = 0; m < M; ++m) dst[t * M + m] = src[aux_packed_offset(t, m, M)];
  return SP24_OK;
}

sp24_status sp24_meta_to_canonical(const void *meta_dev_layout_host, int64_t rows, int64_t cols, uint16_t *canon) {
  if (!meta_dev_layout_host || !canon || rows < 0 || cols < 0) return SP24_ERR_INVALID_ARG;
  if (rows % 4 || cols % 16) return SP24_ERR_UNSUPPORTED_SHAPE;
  const uint8_t *dev = static_cast<const uint8_t *>(meta_dev_layout_host);
  const int64_t words = cols / 16;
  for (int64_t r = 0; r < rows; ++r)
    for (int64_t w = 0; w < words; ++w) {
      uint16_t v = 0;
      for (int e = 0; e < 4; ++e) {
        int shift = 0;
        const size_t pos = meta_nibble_pos(r, 4 * w + e, cols, &shift);
        v |= (uint16_t)(((dev[pos] >> shift) & 0xF) << (4 * e));
      }
      canon[r * words + w] = v;
    }
  return SP24_OK;
}

sp24_status sp24_meta_from_canonical(const uint16_t *canon, int64_t rows, int64_t cols, void *meta_dev_layout_host) {
  if (!meta_dev_layout_host || !canon || rows < 0 || cols < 0) return SP24_ERR_INVALID_ARG;
  if (rows % 4 || cols % 16) return SP24_ERR_UNSUPPORTED_SHAPE;
  uint8_t *dev = static_cast<uint8_t *>(meta_dev_layout_host);
  memset(dev, 0x44, meta_bytes_of(rows, cols));
  const int64_t words = cols / 16;
  for (int64_t r = 0; r < rows; ++r)
    for (int64_t w = 0; w < words; ++w)
      for (int e = 0; e < 4; ++e) {
        int shift = 0;
        const size_t pos = meta_nibble_pos(r, 4 * w + e, cols, &shift);
        const uint8_t nib = (uint8_t)((canon[r * words + w] >> (4 * e)) & 0xF);
        dev[pos] = (uint8_t)((dev[pos] & ~(0xF << shift)) | (nib << shift));
      }
  return SP24_OK;
}

sp24_status sp24_device_status(void *stream) {
  sp24_status st = check_device();
  if (st != SP24_OK) return st;
  if (cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) return SP24_ERR_CUDA;
  unsigned int word = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&word, g_device_error, sizeof(word)) != cudaSuccess) return SP24_ERR_CUDA;
  if (word && cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero)) != cudaSuccess) return SP24_ERR_CUDA;
  if (word && sk_clear_flags() != SP24_OK) return SP24_ERR_CUDA;
  return (word & kDevErrTimeout) ? SP24_ERR_TIMEOUT : SP24_OK;
}

sp24_status sp24_set_wait_budget(uint64_t cycles) {
  g_wait_budget.store(cycles);
  return SP24_OK;
}

}  // extern "C"
