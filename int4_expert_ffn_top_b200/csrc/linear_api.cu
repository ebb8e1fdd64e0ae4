// C ABI of the 8-bit integer matrix product and its quantiser: host checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/moe.h"
#include "linear8.cuh"

namespace {

using namespace moe;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status launched() { return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int64_t row_bytes(int32_t n) { return (static_cast<int64_t>(n) + 15) / 16 * 16; }

bool dim_ok(int32_t n) { return n >= 1 && n <= MOE_I8_MAX_IN; }

template <int NT>
void launch_rows(const l8::LinArgs& a, cudaStream_t st) {
  const int tiles = (a.N + 15) / 16, steps = (a.K16 + 3) / 4;
  // split K over warps until there are 16 warps a multiprocessor, with four 64-byte steps a warp at least
  int kw = 1;
  while (kw < l8::kRowWarps && tiles * kw < 148 * 16 && steps >= 8 * kw) kw *= 2;
  const int per = l8::kRowWarps / kw;
  dim3 grid((tiles + per - 1) / per, (a.T + NT * 8 - 1) / (NT * 8));
  l8::rows_kernel<NT><<<grid, 32 * l8::kRowWarps, 0, st>>>(a, kw);
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
  if (!x || !q || !scale || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  l8::QuantArgs a{x, T, H, eps, q, ldq, scale};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (x_type == 1)
    l8::quant_kernel<true><<<T, l8::kQThreads, 0, st>>>(a);
  else
    l8::quant_kernel<false><<<T, l8::kQThreads, 0, st>>>(a);
  return launched();
}

moe_status moe_linear_i8(const moe_linear8* W, const int8_t* q, int64_t ldq, const float* qscale, int32_t T, void* out,
                         int32_t out_mode, int32_t* err_word, void* stream) {
  if (!W || out_mode < 0 || out_mode > 2) return MOE_ERR_INVALID_ARG;
  if (T < 0 || T > MOE_MAX_TOKENS || !dim_ok(W->in_dim) || W->out_dim < 1 || W->out_dim > MOE_I8_MAX_OUT)
    return MOE_ERR_UNSUPPORTED;
  const int64_t need = row_bytes(W->in_dim);
  if (W->ld < need || W->ld % 16 || ldq < need || ldq % 16) return MOE_ERR_INVALID_ARG;
  if (!W->codes || !W->scale || !aligned16(W->codes)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!q || !qscale || !out || !aligned16(q)) return MOE_ERR_INVALID_ARG;
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
  if (T <= 8)
    launch_rows<1>(a, st);
  else if (T <= 16)
    launch_rows<2>(a, st);
  else if (T <= 32)
    launch_rows<4>(a, st);
  else
    launch_rows<8>(a, st);
  (void)err_word;
  return launched();
}

}  // extern "C"
