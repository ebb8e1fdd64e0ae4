// 8-bit integer matrix product with one scale per token and one per output
// channel, and the per-token quantiser that feeds it.
//
//   q[t][k] = round(127 x[t][k] / max_k |x[t][k]|),  sx[t] = max_k |x[t][k]| rstd_t / 127
//   y[t][n] = sx[t] sw[n] sum_k q[t][k] W[n][k] + bias[n]
//
// RMSNorm scales a whole row by rstd, which leaves the codes as they are and
// goes into the scale alone, so the quantiser never forms the normed row.
#pragma once

#include "common.cuh"

namespace moe {
namespace l8 {

// ----------------------------------------------------------------------------- quantiser
constexpr int kQThreads = 256;

MOE_DEV float max_bits(float a, float b) {  // of non-negative floats by their bits: a NaN ranks above infinity and stays
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// The integer nearest to 127 x / m (ties to even), exactly.  x k, with k = 127/m rounded, is within 127 * 2^-22 of
// it; only where that does not settle the rounding is 127 |x| compared with (n + 1/2) m, both exact in 64 bits.
MOE_DEV int code_of(float x, float m, float k) {
  const float t = x * k, r = rintf(t);
  if (fabsf(t - r) < 0.4999f) return static_cast<int>(r);
  const float n = floorf(fabsf(t));
  const double a = 127.0 * fabs(static_cast<double>(x)), b = (static_cast<double>(n) + 0.5) * static_cast<double>(m);
  const int i = static_cast<int>(n), c = a > b ? i + 1 : (a < b ? i : i + (i & 1));
  return x < 0.f ? -c : c;
}

struct QuantArgs {
  const void* x;
  int T, H;
  float eps;  // < 0: no RMSNorm
  int8_t* q;
  int64_t ldq;
  float* scale;
};

template <bool BF16>
MOE_DEV float load1(const void* x, size_t i) {
  if (BF16) return bf16_bits_to_float(static_cast<const uint16_t*>(x)[i]);
  return static_cast<const float*>(x)[i];
}

// One block per token.
template <bool BF16>
__global__ void __launch_bounds__(kQThreads) quant_kernel(const QuantArgs a) {
  __shared__ float red[2][kQThreads / 32];
  const int t = blockIdx.x, tid = threadIdx.x;
  const size_t row = static_cast<size_t>(t) * a.H;
  float m = 0.f, ss = 0.f;
  for (int i = tid; i < a.H; i += kQThreads) {
    const float v = load1<BF16>(a.x, row + i);
    m = max_bits(m, fabsf(v));
    ss = fmaf(v, v, ss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = max_bits(m, __shfl_xor_sync(0xffffffffu, m, o));
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  if ((tid & 31) == 0) red[0][tid >> 5] = m, red[1][tid >> 5] = ss;
  __syncthreads();
  m = red[0][0], ss = red[1][0];
#pragma unroll
  for (int w = 1; w < kQThreads / 32; ++w) m = max_bits(m, red[0][w]), ss += red[1][w];
  const bool fine = m <= 3.402823466e38f;  // false for infinity and NaN
  const float c = m < 1e-20f ? 0x1p64f : (m > 1e20f ? 0x1p-64f : 1.f);  // exact; keeps 127/m and x k in range
  const float mc = m * c, k = m > 0.f ? 127.f / mc : 0.f;
  int8_t* out = a.q + static_cast<size_t>(t) * a.ldq;
  for (int i = tid; i < a.H; i += kQThreads)
    out[i] = static_cast<int8_t>(fine && m > 0.f ? code_of(load1<BF16>(a.x, row + i) * c, mc, k) : 0);
  if (tid == 0) {
    float s = m / 127.f;
    if (a.eps >= 0.f && m > 0.f) s = m * (1.f / sqrtf(ss / static_cast<float>(a.H) + a.eps)) / 127.f;
    a.scale[t] = fine ? s : __uint_as_float(0x7fc00000u);
  }
}

// ----------------------------------------------------------------------------- product
struct LinArgs {
  const int8_t* W;  // [N][ldw], zero from in_dim to the next multiple of 16
  int64_t ldw;
  const float* sw;
  const float* bias;
  const int8_t* q;  // [T][ldq]
  int64_t ldq;
  const float* sx;
  int T, N, K16;  // K16: row length in 16-byte units
  void* out;      // [T][N]
  int out_mode;
};

MOE_DEV void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

MOE_DEV void store_out(const LinArgs& a, int t, int n, int acc) {
  float y = static_cast<float>(acc) * a.sx[t] * a.sw[n];
  if (a.bias) y += a.bias[n];
  const size_t o = static_cast<size_t>(t) * a.N + n;
  if (a.out_mode == 1) {
    static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(y);
  } else {
    float* p = static_cast<float*>(a.out) + o;
    *p = a.out_mode == 2 ? *p + y : y;
  }
}

constexpr int kRowWarps = 8;

// Few tokens: the weight rows are the MMA's M side (16 rows a warp, read once from memory straight into the
// fragments), 8 NT tokens its N side.  A lane's 16 bytes of a row are two k32 slices' fragments: K is permuted
// the same way in both operands, which leaves the integer sum as it is.  KW warps split K and add up in shared
// memory, so that enough loads are in flight when there are few rows.
template <int NT>
__global__ void __launch_bounds__(32 * kRowWarps) rows_kernel(const LinArgs a, int KW) {
  __shared__ int part[kRowWarps][NT * 8][17];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, tig = lane & 3;
  const int tiles = kRowWarps / KW, tile = warp / KW, kw = warp % KW;
  const int n0 = (blockIdx.x * tiles + tile) * 16, t0 = blockIdx.y * NT * 8;
  int acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0;
  if (n0 < a.N) {
    const int8_t* w0 = a.W + static_cast<size_t>(min(n0 + g, a.N - 1)) * a.ldw;
    const int8_t* w1 = a.W + static_cast<size_t>(min(n0 + g + 8, a.N - 1)) * a.ldw;
    const int8_t* x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] = a.q + static_cast<size_t>(min(t0 + j * 8 + g, a.T - 1)) * a.ldq;
    const int steps = (a.K16 + 3) / 4;  // of 64 bytes
#pragma unroll 4
    for (int s = kw; s < steps; s += KW) {
      const int c = s * 4 + tig;
      const bool in = c < a.K16;
      const uint4 z = make_uint4(0, 0, 0, 0);
      const uint4 p = in ? ldg_stream(w0 + 16 * c) : z, q = in ? ldg_stream(w1 + 16 * c) : z;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4 b = in ? *reinterpret_cast<const uint4*>(x[j] + 16 * c) : z;
        mma_s8(acc[j], p.x, q.x, p.y, q.y, b.x, b.y);
        mma_s8(acc[j], p.z, q.z, p.w, q.w, b.z, b.w);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][j * 8 + 2 * tig + (i & 1)][g + 8 * (i >> 1)] = acc[j][i];
  __syncthreads();
  for (int i = threadIdx.x; i < tiles * NT * 8 * 16; i += 32 * kRowWarps) {
    const int r = i & 15, t = (i >> 4) % (NT * 8), tl = i / (16 * NT * 8);
    const int n = (blockIdx.x * tiles + tl) * 16 + r;
    if (n >= a.N || t0 + t >= a.T) continue;
    int v = 0;
    for (int w = 0; w < KW; ++w) v += part[tl * KW + w][t][r];
    store_out(a, t0 + t, n, v);
  }
}

}  // namespace l8
}  // namespace moe
