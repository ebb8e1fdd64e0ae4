// C ABI of the 8-bit integer matrix product and its quantiser: host checks and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/moe.h"
#include "linear8.cuh"

namespace {

using namespace moe;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }  // (null: yes)
inline bool aligned16(const void* p) { return aligned(p, 16); }

moe_status launched() { return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int64_t row_bytes(int32_t n) { return (static_cast<int64_t>(n) + 15) / 16 * 16; }

bool dim_ok(int32_t n) { return n >= 1 && n <= MOE_I8_MAX_IN; }

// Launch with leave to start while the kernel before it in the stream runs, if that one allows it (the quantiser
// does): the kernels here set themselves up meanwhile and touch memory after waiting for it.
template <class... P, class... A>
moe_status launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st, A... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = at;
  c.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&c, kern, static_cast<P>(args)...) == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

template <int R, int NT>
moe_status launch_rows(const l8::LinArgs& a, int nsm, cudaStream_t st) {
  const int groups = (a.N + R - 1) / R;
  // split K over warps until there are 32 warps a multiprocessor, with a chunk for every lane at least; and as long as a
  // lane has 16 chunks of a row: fewer rows of many pages are read at once (one and two tokens x 65,536 -> 20,000 191 and
  // 207 us against 228 and 285, 16,384 -> 16,384 37.9 against 39.5; with 4 chunks 2,048 -> 65,536 21.8 against 20.3)
  int kw = 1;
  while (kw < l8::kRowWarps && (groups * kw < nsm * 32 || a.K16 >= 512 * kw) && a.K16 >= 64 * kw) kw *= 2;
  const int per = l8::kRowWarps / kw;
  return launch_after(l8::rows_kernel<R, NT>, dim3((groups + per - 1) / per), 32 * l8::kRowWarps, 0, 1, st, a, kw);
}

constexpr int kMaxDev = 64;

// Multiprocessors of the current device (0 on failure) and its number.
int multiprocessors(int* dev) {
  static std::atomic<int> known[kMaxDev];
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDev) return 0;
  int n = known[*dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) return 0;
    known[*dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// A matrix of `rows` rows of `cols` bytes, ld bytes apart, in boxes of 128 bytes x box_rows, 128-byte swizzle; what a
// box has past the edges is zero.
bool codes_map(CUtensorMap* m, const void* base, int cols, int rows, int64_t ld, int box_rows) {
  const EncodeTiledFn f = encode_tiled();
  if (!f) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {l8::kGK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int MODE>
moe_status launch_gemm_mode(const l8::GemmMaps& maps, const l8::GemmArgs& a, int nsm, int dev, cudaStream_t st) {
  auto kern = l8::gemm_kernel<BN, MODE>;
  static std::atomic<bool> allowed[kMaxDev];
  if (!allowed[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, l8::GemmCfg<BN>::kSmem) != cudaSuccess)
      return MOE_ERR_CUDA;
    allowed[dev].store(true, std::memory_order_relaxed);
  }
  const int tiles = a.m_tiles * a.n_tiles;
  const int pairs = tiles < nsm / 2 ? tiles : nsm / 2;
  return launch_after(kern, dim3(2 * pairs), l8::kGThreads, l8::GemmCfg<BN>::kSmem, 1, st, maps, a);
}

template <int BN, int MODE>
moe_status launch_split_mode(const l8::GemmMaps& maps, const l8::GemmArgs& a, int S, int dev, cudaStream_t st) {
  auto kern = l8::split_kernel<BN, MODE>;
  static std::atomic<bool> allowed[kMaxDev];
  if (!allowed[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, l8::SplitCfg<BN>::kSmem) != cudaSuccess)
      return MOE_ERR_CUDA;
    allowed[dev].store(true, std::memory_order_relaxed);
  }
  return launch_after(kern, dim3(a.m_tiles * S, a.n_tiles), l8::kSplitThreads, l8::SplitCfg<BN>::kSmem, S, st, maps, a, S);
}

// m_rows, box: weight rows of a tile, tokens of one copy
bool make_args(l8::GemmMaps* maps, l8::GemmArgs* a, const l8::LinArgs& lin, int in_dim, int m_rows, int bn, int box, int* err) {
  a->lin = lin;
  a->KT = (in_dim + l8::kGK - 1) / l8::kGK;
  a->m_tiles = (lin.N + m_rows - 1) / m_rows;
  a->n_tiles = (lin.T + bn - 1) / bn;
  a->err = err;
  a->timeout_ns = 2000000000LL;
  return codes_map(&maps->w, lin.W, in_dim, lin.N, lin.ldw, l8::kGM) &&
         codes_map(&maps->q, lin.q, in_dim, lin.T, lin.ldq, box);
}

template <int BN>
moe_status launch_split(const l8::LinArgs& lin, int in_dim, int* err, int nsm, int dev, cudaStream_t st) {
  l8::GemmMaps maps;
  l8::GemmArgs a{};
  if (!make_args(&maps, &a, lin, in_dim, l8::kGM, BN, BN, err)) return MOE_ERR_CUDA;
  int S = 1;
  while (S < 8 && a.m_tiles * a.n_tiles * S * 2 <= nsm && a.KT >= 2 * S) S *= 2;
  switch (lin.out_mode) {
    case 0: return launch_split_mode<BN, 0>(maps, a, S, dev, st);
    case 1: return launch_split_mode<BN, 1>(maps, a, S, dev, st);
    default: return launch_split_mode<BN, 2>(maps, a, S, dev, st);
  }
}

template <int BN>
moe_status launch_gemm(const l8::LinArgs& lin, int in_dim, int* err, int nsm, int dev, cudaStream_t st) {
  l8::GemmMaps maps;
  l8::GemmArgs a{};
  if (!make_args(&maps, &a, lin, in_dim, 2 * l8::kGM, BN, BN / 2, err)) return MOE_ERR_CUDA;
  switch (lin.out_mode) {
    case 0: return launch_gemm_mode<BN, 0>(maps, a, nsm, dev, st);
    case 1: return launch_gemm_mode<BN, 1>(maps, a, nsm, dev, st);
    default: return launch_gemm_mode<BN, 2>(maps, a, nsm, dev, st);
  }
}

}  // namespace

extern "C" {

size_t moe_i8_row_bytes(int32_t n) { return dim_ok(n) ? static_cast<size_t>(row_bytes(n)) : 0; }

moe_status moe_quant_i8(const void* x, int32_t x_type, int32_t T, int32_t H, float eps, int8_t* q, int64_t ldq,
                        float* scale, void* stream) {
  if ((x_type != 0 && x_type != 1) || std::isnan(eps)) return MOE_ERR_INVALID_ARG;
  if (T < 0 || T > MOE_MAX_TOKENS || !dim_ok(H)) return MOE_ERR_UNSUPPORTED;
  if (ldq < row_bytes(H) || ldq % 16) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !q || !scale || !aligned16(q) || !aligned(x, x_type == 1 ? 2 : 4) || !aligned(scale, 4))
    return MOE_ERR_INVALID_ARG;
  l8::QuantArgs a{x, T, H, eps, q, ldq, scale};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // whole 8-value pieces: rows that begin on 16 bytes (and their codes on 8)
  const bool vec = H % 8 == 0 && aligned16(x);
  if (x_type == 1)
    (vec ? l8::quant_kernel<true, true> : l8::quant_kernel<true, false>)<<<T, l8::kQThreads, 0, st>>>(a);
  else
    (vec ? l8::quant_kernel<false, true> : l8::quant_kernel<false, false>)<<<T, l8::kQThreads, 0, st>>>(a);
  return launched();
}

moe_status moe_linear_i8(const moe_linear8* W, const int8_t* q, int64_t ldq, const float* qscale, int32_t T, void* out,
                         int32_t out_mode, int32_t* err_word, void* stream) {
  if (!W || out_mode < 0 || out_mode > 2) return MOE_ERR_INVALID_ARG;
  if (T < 0 || T > MOE_MAX_TOKENS || !dim_ok(W->in_dim) || W->out_dim < 1 || W->out_dim > MOE_I8_MAX_OUT)
    return MOE_ERR_UNSUPPORTED;
  const int64_t need = row_bytes(W->in_dim);
  if (W->ld < need || W->ld % 16 || ldq < need || ldq % 16) return MOE_ERR_INVALID_ARG;
  if (!W->codes || !W->scale || !aligned16(W->codes) || !aligned(W->scale, 4) || !aligned(W->bias, 4))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!q || !qscale || !out || !aligned16(q) || !aligned(qscale, 4) || !aligned(out, out_mode == 1 ? 2 : 4) ||
      !aligned(err_word, 4))
    return MOE_ERR_INVALID_ARG;
  l8::LinArgs a{};
  a.W = W->codes;
  a.ldw = W->ld;
  a.sw = W->scale;
  a.bias = W->bias;
  a.q = q;
  a.ldq = ldq;
  a.sx = qscale;
  a.T = T;
  a.N = W->out_dim;
  a.K16 = static_cast<int>(need / 16);
  a.out = out;
  a.out_mode = out_mode;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0;
  const int nsm = multiprocessors(&dev), in = W->in_dim;
  if (nsm < 1) return MOE_ERR_CUDA;
  // Few tokens: dp4a over the weight rows where that is done before a tensor-core kernel has begun (2^24 products take
  // it 3 to 4 us; the cluster split takes 4.3 for anything small: 3 x 1,008 -> 2,051 2.6 against 5.0 us, 8 x 1,024 ->
  // 2,048 3.9 against 4.8, but 5 x 2,048 -> 2,048 6.0 against 5.5 and 8 x 2,048 -> 65,536 41 against 29), and for one or
  // two tokens with rows long enough to keep a warp's loads going (2,048 -> 65,536: 18.6 against 29.2 us, two tokens 21.7
  // against 29.3; 400 -> 200,000 22.3 against 32.4, two tokens 512 -> 200,000 24.9 against 30.7; short rows, 64 ->
  // 1,000,000: 104 against 93, two tokens 256 -> 300,000 36.3 against 32.8).
  if (T <= 8) {
    const int nt = T <= 2 ? T : T <= 4 ? 4 : 8;
    if (static_cast<long long>(a.N) * a.K16 * nt <= 1 << 20 || (T <= 2 && a.K16 >= 24)) {
      if (nt == 1) return launch_rows<4, 1>(a, nsm, st);
      if (nt == 2) return launch_rows<4, 2>(a, nsm, st);
      if (nt == 4) return launch_rows<4, 4>(a, nsm, st);
      return launch_rows<2, 8>(a, nsm, st);
    }
  }
  const long long m = (a.N + l8::kGM - 1) / l8::kGM, m2 = (m + 1) / 2;
  auto tiles = [&](long long rows, int bn) { return rows * ((T + bn - 1) / bn); };
  // K split over clusters while the tiles find a multiprocessor each; for up to 16 tokens, two (16 x 2,048 -> 30,000:
  // 16.5 us against 16.9 with CTA pairs; 32 tokens 18.4 against 16.7, 16 x 2,048 -> 65,536 31.4 against 29.4)
  if (tiles(m, 32) <= nsm || (T <= 16 && m <= 2 * nsm)) return launch_split<32>(a, in, err_word, nsm, dev, st);
  if (tiles(m, 64) <= nsm) return launch_split<64>(a, in, err_word, nsm, dev, st);
  // the token tile whose waves of tiles take the least time: a tile costs its columns, and 16 more for its turn
  auto cost = [&](int bn) { return (tiles(m2, bn) + nsm / 2 - 1) / (nsm / 2) * (bn + 16); };
  const long long c256 = cost(256), c192 = cost(192), c128 = cost(128), c64 = cost(64);
  if (c256 <= c192 && c256 <= c128 && c256 <= c64) return launch_gemm<256>(a, in, err_word, nsm, dev, st);
  if (c192 <= c128 && c192 <= c64) return launch_gemm<192>(a, in, err_word, nsm, dev, st);
  if (c128 <= c64) return launch_gemm<128>(a, in, err_word, nsm, dev, st);
  return launch_gemm<64>(a, in, err_word, nsm, dev, st);
}

}  // extern "C"
