// 8-bit integer matrix product with one scale per token and one per output
// channel, and the per-token quantiser that feeds it.
//
//   q[t][k] = round(127 x[t][k] / max_k |x[t][k]|),  sx[t] = max_k |x[t][k]| rstd_t / 127
//   y[t][n] = sx[t] sw[n] sum_k q[t][k] W[n][k] + bias[n]
//
// RMSNorm scales a whole row by rstd, which leaves the codes as they are and
// goes into the scale alone, so the quantiser never forms the normed row.
#pragma once

#include "tc_primitives.cuh"

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

// A kernel that runs after the quantiser in a stream may start while it runs (programmatic launch): it sets itself up and
// asks for its first weights in L2, and reads or writes memory only after dependency_wait().  That holds for the weights
// too: the quantiser's output is what a matrix is made of, so the kernel before may be writing them.  (A prefetch to L2
// returns nothing, and L2 is where that kernel's writes arrive.)
MOE_DEV void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
MOE_DEV void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Loads of what that kernel may have written.  Not through the read-only path (ld.global.nc, __ldg): it is for memory that
// nothing writes while the kernel runs, and its loads need not stay behind the wait.
MOE_DEV uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
MOE_DEV float load_f32(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
MOE_DEV void prefetch_to_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Eight neighbouring values of a row, or (VEC false: rows that are not aligned or not whole blocks) one.
template <bool BF16, bool VEC>
struct Piece {
  static constexpr int kN = VEC ? 8 : 1;
  float v[kN];
  MOE_DEV void load(const void* x, size_t i) {
    if (VEC && BF16) {
      const uint4 p = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
      const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] = __uint_as_float((j & 1) ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
    } else if (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 p = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i + 4 * h);
        const float q[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[(4 * h + j) % kN] = q[j];
      }
    } else {
      v[0] = BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(x)[i]) : static_cast<const float*>(x)[i];
    }
  }
};

// A block per token; a thread keeps its first pieces in registers between the two passes.  Bound by memory: 3,328 x
// 2,048 fp32 (34 MB in and out) takes 10.2 us, one token 2.1 us.  (A warp per token without barriers, 64 values a lane,
// took 15.6 us: all of its loads come before all of its stores, and nothing else fills the gap.)
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kQThreads) quant_kernel(const QuantArgs a) {
  using P = Piece<BF16, VEC>;
  constexpr int kKeep = VEC ? 2 : 4, kStep = kQThreads;
  __shared__ float red[2][kQThreads / 32];
  dependents_may_start();
  const int tid = threadIdx.x, i0 = tid, n = a.H / P::kN, t = blockIdx.x;
  const size_t row = static_cast<size_t>(t) * a.H;
  P keep[kKeep];
  float m = 0.f, ss = 0.f;
  auto take = [&](const P& p) {
#pragma unroll
    for (int j = 0; j < P::kN; ++j) {
      m = max_bits(m, fabsf(p.v[j]));
      ss = fmaf(p.v[j], p.v[j], ss);
    }
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (i0 + i * kStep < n) keep[i].load(a.x, row + static_cast<size_t>(i0 + i * kStep) * P::kN);
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (i0 + i * kStep < n) take(keep[i]);
#pragma unroll 2
  for (int i = i0 + kKeep * kStep; i < n; i += kStep) {
    P p;
    p.load(a.x, row + static_cast<size_t>(i) * P::kN);
    take(p);
  }
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((tid & 31) == 0) red[0][tid >> 5] = m, red[1][tid >> 5] = ss;
  __syncthreads();
  m = red[0][0], ss = red[1][0];
#pragma unroll
  for (int w = 1; w < kQThreads / 32; ++w) m = max_bits(m, red[0][w]), ss += red[1][w];
  const bool fine = m <= 3.402823466e38f;  // false for infinity and NaN
  const float c = m < 1e-20f ? 0x1p64f : (m > 1e20f ? 0x1p-64f : 1.f);  // exact; keeps 127/m and x k in range
  const float mc = m * c, k = m > 0.f ? 127.f / mc : 0.f;
  const bool zero = !fine || m == 0.f;
  int8_t* out = a.q + static_cast<size_t>(t) * a.ldq;
  auto put = [&](const P& p, int i) {
    uint32_t w[2] = {0u, 0u};
    if (!zero) {
#pragma unroll
      for (int j = 0; j < P::kN; ++j)
        w[j >> 2] |= (static_cast<uint32_t>(code_of(p.v[j] * c, mc, k)) & 0xffu) << (8 * (j & 3));
    }
    if (VEC)
      *reinterpret_cast<uint2*>(out + static_cast<size_t>(i) * 8) = make_uint2(w[0], w[1]);
    else
      out[i] = static_cast<int8_t>(w[0]);
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (i0 + i * kStep < n) put(keep[i], i0 + i * kStep);
#pragma unroll 1
  for (int i = i0 + kKeep * kStep; i < n; i += kStep) {
    P p;
    p.load(a.x, row + static_cast<size_t>(i) * P::kN);
    put(p, i);
  }
  // squares that fp32 may not hold (the same in the whole block): summed of values scaled by a power of two that keeps the
  // largest's square, times 65,536, in range
  const bool far = a.eps >= 0.f && !zero && (m > 1e16f || m < 1e-15f);
  if (far) {
    const float sc = m > 1.f ? 0x1p-96f : 0x1p96f;
    ss = 0.f;
#pragma unroll 1
    for (int i = tid; i < a.H; i += kStep) {
      Piece<BF16, false> p;
      p.load(a.x, row + i);
      ss = fmaf(p.v[0] * sc, p.v[0] * sc, ss);
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    __syncthreads();
    if ((tid & 31) == 0) red[1][tid >> 5] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll 1
    for (int w = 0; w < kQThreads / 32; ++w) ss += red[1][w];
  }
  if (tid == 0) {
    float s = m / 127.f;
    if (far)
      s = static_cast<float>(m / sqrt(static_cast<double>(ss) / a.H * (m > 1.f ? 0x1p192 : 0x1p-192) + a.eps) / 127.0);
    else if (a.eps >= 0.f && m > 0.f)
      s = m * (1.f / sqrtf(ss / static_cast<float>(a.H) + a.eps)) / 127.f;
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

MOE_DEV void store_out(const LinArgs& a, int t, int n, int acc) {
  const float y = fmaf(static_cast<float>(acc) * load_f32(a.sx + t), load_f32(a.sw + n), a.bias ? load_f32(a.bias + n) : 0.f);
  const size_t o = static_cast<size_t>(t) * a.N + n;
  if (a.out_mode == 1) {
    static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(y);
  } else {
    float* p = static_cast<float*>(a.out) + o;
    *p = a.out_mode == 2 ? *p + y : y;
  }
}

constexpr int kRowWarps = 8;

// Few tokens: a warp takes R weight rows, a lane every 32nd 16-byte chunk of them (of its part of K: KW warps split it
// and add up in shared memory, so that enough loads are in flight when there are few rows), four dp4a a chunk, row and
// token.  Bound by the weights' bytes; the tensor cores would add nothing to them (mma.sync s8, tried first, has its own
// limit here: 27.7 us against 19.0 for one token x 2,048 -> 65,536, which is 7.1 TB/s).  Eight loads of a lane go together,
// where 16 leave room for half as many warps (22.3 us; behind the quantiser, 2,048 -> 4,096 6.1 against 4.7).  Without the
// prefetch to L2 ahead of the wait the two take 21.8 and 5.3 us.
template <int R, int NT>
__global__ void __launch_bounds__(32 * kRowWarps) rows_kernel(const LinArgs a, int KW) {
  __shared__ int part[kRowWarps][R * NT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = kRowWarps / KW, grp = warp / KW, kw = warp % KW;
  const int n0 = (blockIdx.x * groups + grp) * R;
  const int8_t* w[R];
#pragma unroll
  for (int i = 0; i < R; ++i) w[i] = a.W + static_cast<size_t>(min(n0 + i, a.N - 1)) * a.ldw;
  int acc[R][NT];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = 0;
  constexpr int kAhead = 8 / R;  // chunks whose weights are loaded together
#pragma unroll
  for (int j = 0; j < kAhead; ++j)  // the first of them into L2, a lane per 128 bytes
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (j * KW + kw) * 32 + lane;
      if ((lane & 7) == 0 && c < a.K16) prefetch_to_l2(w[i] + 16 * static_cast<size_t>(c));
    }
  dependency_wait();
#pragma unroll 1
  for (int c0 = kw * 32 + lane; c0 - lane < a.K16; c0 += 32 * KW * kAhead) {
    uint4 q[kAhead][R];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = c0 + j * 32 * KW;
        q[j][i] = c < a.K16 ? load_stream(w[i] + 16 * static_cast<size_t>(c)) : make_uint4(0, 0, 0, 0);
      }
    // one token: all of these loads before the codes' (mixed, 20.9 us for 2,048 -> 65,536 in place of 19.2); with more the
    // codes' are as many, and best among them (two tokens, 2,048 -> 4,096: 5.0 us against 6.2)
    if (NT == 1) __syncwarp();
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = min(c0 + j * 32 * KW, a.K16 - 1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 x = *reinterpret_cast<const uint4*>(a.q + static_cast<size_t>(min(t, a.T - 1)) * a.ldq + 16 * static_cast<size_t>(c));
#pragma unroll
        for (int i = 0; i < R; ++i) {
          int s = acc[i][t];
          s = __dp4a(static_cast<int>(q[j][i].x), static_cast<int>(x.x), s);
          s = __dp4a(static_cast<int>(q[j][i].y), static_cast<int>(x.y), s);
          s = __dp4a(static_cast<int>(q[j][i].z), static_cast<int>(x.z), s);
          acc[i][t] = __dp4a(static_cast<int>(q[j][i].w), static_cast<int>(x.w), s);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int v = __reduce_add_sync(0xffffffffu, acc[i][t]);
      if (lane == (i * NT + t) % 32) part[warp][i * NT + t] = v;
    }
  if (KW > 1)
    __syncthreads();
  else
    __syncwarp();
  if (kw == 0 && lane < R * NT) {
    const int i = lane / NT, t = lane % NT, n = n0 + i;
    int v = 0;
    for (int k = 0; k < KW; ++k) v += part[warp + k][lane];
    if (n < a.N && t < a.T) store_out(a, t, n, v);
  }
}

// ----------------------------------------------------------------------------- many tokens: tcgen05 kind::i8
// D[n][t] = sum_k W[n][k] q[t][k]: weight rows are the MMA's M side, tokens its N side, 32-bit integer accumulators in
// tensor memory.  A pair of CTAs (cta_group::2) works on 256 weight rows x BN tokens: each holds 128 of the rows and
// half of the tokens in its shared memory and the tensor cores of both read both halves of the tokens.  An 8-bit tile of
// one CTA (128 x 256) asks its shared memory for 192 bytes a cycle (operands in by TMA, out to the MMA), more than the
// 128 it has; the pair's share is 128: 8,192 x 4,096 -> 4,096 takes 92.7 to 95.7 us against 98.7 with
// tiles of one CTA (2.9 POPS; back to back for seconds the power limit holds it at 107 to 110 us).
// Persistent and warp-specialised: warp 0 brings 128-byte K slices of both operands by TMA (128-byte swizzle, zero-filled
// past the matrices' edges), both CTAs' slices counted by the first CTA's barrier; warp 1 of the first CTA issues the
// MMAs (four k32 steps a slice) and its commits free the stages of both; eight epilogue warps (TMEM lane quadrant =
// warp % 4, two warps per quadrant splitting the columns) drain one accumulator while the next tile's MMAs fill the
// other.  A lane is a weight row and a column a token, so the 32 lanes of a store write 32 neighbouring outputs of one
// token.
// Every wait is bounded: a role whose wait runs out stops and records MOE_ERR_TIMEOUT; copies and MMAs under way are
// waited for (bounded) by the MMAs' thread before the CTAs leave.  (A producer that gives up starves that thread, so it
// alone sees every copy's end.)
constexpr int kGM = 128, kGK = 128;
constexpr int kGEpiWarps = 8, kGThreads = 64 + 32 * kGEpiWarps;

template <int BN>
struct GemmCfg {  // per CTA
  static constexpr int kStage = (kGM + BN / 2) * kGK;
  static constexpr int kStages = BN >= 256 ? 6 : (BN >= 192 ? 6 : 8);
  static constexpr int kSxBytes = 2 * BN * 4;
  static constexpr int kSmem = 1024 + kStages * kStage + kSxBytes + 256;
  static constexpr uint32_t kCols = 2 * BN <= 128 ? 128 : (2 * BN <= 256 ? 256 : 512);
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct GemmMaps {
  CUtensorMap w, q;
};

struct GemmArgs {
  LinArgs lin;
  int KT, m_tiles, n_tiles;  // K slices; tiles of weight rows, of tokens
  int* err;
  long long timeout_ns;
};

// Instruction descriptor, kind::i8: signed 8-bit A and B (K-major), 32-bit integer accumulator.
MOE_DEV uint32_t instr_desc_i8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <int CTAS>
MOE_DEV void mma_i8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (CTAS == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

// Arrive on the barrier at this offset in both CTAs of the pair when the MMAs issued so far are done.
MOE_DEV void commit_pair(uint64_t* b) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(tc::sa(b)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Address of CTA `rank`'s counterpart of a shared-memory address of this CTA.
MOE_DEV uint32_t peer_addr(const void* p, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::sa(p)), "r"(rank));
  return at;
}

// 2-D TMA load into this CTA's shared memory, counted by a barrier of either CTA of the pair (cluster address).
MOE_DEV void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(tc::sa(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// The tile of a 2-D TMA load into L2 only.
MOE_DEV void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

MOE_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

// OR of v over the 256 epilogue threads (named barrier 1).
MOE_DEV bool epi_any(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

template <int BN, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
    gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs a) {
  using C = GemmCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sxs = reinterpret_cast<float*>(sm + C::kStages * C::kStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::kStages * C::kStage + C::kSxBytes);  // the first CTA's count both
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + 2;  // the first CTA's count both CTAs' epilogue warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = a.m_tiles * a.n_tiles;
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      tc::bar_init(full + s, 1);
      tc::bar_init(empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::bar_init(acc_full + s, 1);
      tc::bar_init(acc_empty + s, 2 * kGEpiWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::sa(tmem_slot)),
                 "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  int fail = 0;
  auto parity = [](int i, int n) { return static_cast<uint32_t>(i / n) & 1u; };

  if (warp == 0) {
    if (lane == 0) {
      dependency_wait();
      int n = 0;
#pragma unroll 1
      for (int t = pair; t < tiles && !fail; t += pairs) {
        const int m0 = (t % a.m_tiles) * 2 * kGM + rank * kGM, t0 = (t / a.m_tiles) * BN + rank * (BN / 2);
#pragma unroll 1
        for (int k = 0; k < a.KT; ++k, ++n) {
          const int s = n % C::kStages;
          if (!tc::bar_wait(empty + s, parity(n, C::kStages) ^ 1u, a.timeout_ns)) {
            fail = 1;
            break;
          }
          if (rank == 0) tc::bar_expect_tx(full + s, 2 * C::kStage);
          const uint32_t bar = peer_addr(full + s, 0);
          tma_load_pair(sm + s * C::kStage, &maps.w, k * kGK, m0, bar);
          tma_load_pair(sm + s * C::kStage + kGM * kGK, &maps.q, k * kGK, t0, bar);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = instr_desc_i8(2 * kGM, BN);
      int n = 0, it = 0;
#pragma unroll 1
      for (int t = pair; t < tiles && !fail; t += pairs, ++it) {
        const int ab = it & 1;
        if (!tc::bar_wait(acc_empty + ab, parity(it, 2) ^ 1u, a.timeout_ns)) {
          fail = 1;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + ab * BN;
#pragma unroll 1
        for (int k = 0; k < a.KT; ++k, ++n) {
          const int s = n % C::kStages;
          if (!tc::bar_wait(full + s, parity(n, C::kStages), a.timeout_ns)) {
            fail = 1;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint64_t da = tc::smem_desc(tc::sa(sm + s * C::kStage)), db = tc::smem_desc(tc::sa(sm + s * C::kStage + kGM * kGK));
#pragma unroll
          for (int i = 0; i < kGK / 32; ++i) mma_i8<2>(d, da + 2 * i, db + 2 * i, idesc, k > 0 || i > 0);
          commit_pair(empty + s);
        }
        if (!fail) commit_pair(acc_full + ab);
      }
      // Nothing of the pair's is under way when it leaves: both CTAs' copies are counted here (after a failure at most one
      // for each stage beyond the slices used), and `empty` says that the MMAs are done with their operands.
#pragma unroll 1
      for (int q = n; fail && q < n + C::kStages; ++q) tc::bar_wait(full + q % C::kStages, parity(q, C::kStages), a.timeout_ns / 8);
      if (n > 0) tc::bar_wait(empty + (n - 1) % C::kStages, parity(n - 1, C::kStages), a.timeout_ns);
    }
  } else {
    const int ew = warp - 2, quad = warp & 3, half = ew >> 2, et = tid - 64;
    const uint32_t release[2] = {peer_addr(acc_empty, 0), peer_addr(acc_empty + 1, 0)};
    dependency_wait();
    int it = 0;
#pragma unroll 1
    for (int t = pair; t < tiles && !fail; t += pairs, ++it) {
      const int ab = it & 1, m0 = (t % a.m_tiles) * 2 * kGM + rank * kGM, t0 = (t / a.m_tiles) * BN;
      const int n = m0 + quad * 32 + lane;
      const bool row = n < a.lin.N;
      const float sw = row ? load_f32(a.lin.sw + n) : 0.f, bias = row && a.lin.bias ? load_f32(a.lin.bias + n) : 0.f;
      float* sx = sxs + ab * BN;
#pragma unroll 1
      for (int i = et; i < BN; i += 32 * kGEpiWarps) sx[i] = t0 + i < a.lin.T ? load_f32(a.lin.sx + t0 + i) : 0.f;
      // the eight warps go on together or not at all (and see the scales)
      if (epi_any(!tc::bar_wait(acc_full + ab, parity(it, 2), a.timeout_ns))) {
        fail = 1;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      auto let_go = [&]() {  // this warp has read its part of the accumulator
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(release[ab]) : "memory");
      };
#pragma unroll 1
      for (int c = half * 32; c < BN && t0 + c < a.lin.T; c += 64) {
        float v[32];
        tc::tmem_ld32(tmem + ab * BN + c + (static_cast<uint32_t>(quad * 32) << 16), v);
        if (c + 64 >= BN || t0 + c + 64 >= a.lin.T) let_go();
        const size_t base = static_cast<size_t>(t0 + c) * a.lin.N + n;
        const int cols = min(32, a.lin.T - t0 - c);
        if (row) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (i < cols) {
              const float y = fmaf(static_cast<float>(__float_as_int(v[i])) * sx[c + i], sw, bias);
              const size_t o = base + static_cast<size_t>(i) * a.lin.N;
              if (MODE == 1) {
                static_cast<__nv_bfloat16*>(a.lin.out)[o] = __float2bfloat16_rn(y);
              } else {
                float* p = static_cast<float*>(a.lin.out) + o;
                *p = MODE == 2 ? *p + y : y;
              }
            }
          }
        }
      }
      if (!(half * 32 < BN && t0 + half * 32 < a.lin.T)) let_go();  // nothing to read for this warp
    }
  }
  if (fail) report(a.err, 5 /* MOE_ERR_TIMEOUT */);
  __syncthreads();
  cluster_sync();  // neither CTA's memory or barriers are in use by the other
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols));
  }
}

// ----------------------------------------------------------------------------- a medium number of tokens: K split over a cluster
// The same product where the tiles are too few for the device: the CTAs of a cluster take a run of K slices each (all of
// a CTA's slices, or kSplitStages of them, are under way at once), leave their integer sums in shared memory, and each
// CTA adds up and writes its part of the columns, reading its neighbours' sums through distributed shared memory.
// Integer sums: the split leaves no trace in the result.  Bound by latency (launch, first bytes of the weights, one join):
// quantiser and 64 tokens x 2,048 -> 2,048 take 8.2 us, 10 with the tiles of gemm_kernel; 13 x 1,000 -> 2,051 5.2 against
// 7.0 us.
constexpr int kSplitStages = 4, kSplitThreads = 192;

template <int BN>
struct SplitCfg {
  static constexpr int kStage = (kGM + BN) * kGK;
  static constexpr int kSmem = 1024 + kSplitStages * kStage + 256;
  static_assert(kSplitStages * kStage >= BN * kGM * 4, "the sums fit where the operands were");
};

template <int BN, int MODE>
__global__ void __launch_bounds__(kSplitThreads, 1) split_kernel(const __grid_constant__ GemmMaps maps,
                                                                 const __grid_constant__ GemmArgs a, int S) {
  using C = SplitCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kSplitStages * C::kStage);
  uint64_t* empty = full + kSplitStages;
  uint64_t* done = empty + kSplitStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % S, m0 = (blockIdx.x / S) * kGM, t0 = blockIdx.y * BN;  // clusters run along x
  const int k0 = rank * a.KT / S, k1 = (rank + 1) * a.KT / S;
  if (tid == 0) {
    for (int s = 0; s < kSplitStages; ++s) {
      tc::bar_init(full + s, 1);
      tc::bar_init(empty + s, 1);
    }
    tc::bar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::sa(tmem_slot)), "r"(BN));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  int fail = 0;
  auto parity = [](int i) { return static_cast<uint32_t>(i / kSplitStages) & 1u; };
  if (warp == 0 && lane == 0) {
    // the first weights into L2 (32 tokens x 4,096 -> 4,096, weights out of cache: 10.4 us, 10.8 without)
#pragma unroll 1
    for (int n = 0; n < min(k1 - k0, kSplitStages); ++n) tma_prefetch_2d(&maps.w, (k0 + n) * kGK, m0);
    dependency_wait();
    int n = 0;
#pragma unroll 1
    for (; n < k1 - k0; ++n) {
      const int s = n % kSplitStages;
      if (n >= kSplitStages && !tc::bar_wait(empty + s, parity(n) ^ 1u, a.timeout_ns)) {
        fail = 1;
        break;
      }
      tc::bar_expect_tx(full + s, C::kStage);
      tc::tma_load_2d(sm + s * C::kStage, &maps.w, (k0 + n) * kGK, m0, full + s);
      tc::tma_load_2d(sm + s * C::kStage + kGM * kGK, &maps.q, (k0 + n) * kGK, t0, full + s);
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = instr_desc_i8(kGM, BN);
#pragma unroll 1
    for (int n = 0; n < k1 - k0; ++n) {
      const int s = n % kSplitStages;
      if (!tc::bar_wait(full + s, parity(n), a.timeout_ns)) {
        fail = 1;
        for (int q = n; q < k1 - k0 && q < n + kSplitStages; ++q)  // copies under way
          tc::bar_wait(full + q % kSplitStages, parity(q), a.timeout_ns / 8);
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint64_t da = tc::smem_desc(tc::sa(sm + s * C::kStage)), db = tc::smem_desc(tc::sa(sm + s * C::kStage + kGM * kGK));
#pragma unroll
      for (int i = 0; i < kGK / 32; ++i) mma_i8<1>(tmem, da + 2 * i, db + 2 * i, idesc, n > 0 || i > 0);
      tc::mma_commit(empty + s);
    }
    tc::mma_commit(done);  // (of what was issued, where a wait ran out)
  }
  __syncwarp();
  dependency_wait();
  float sw[2], bias[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = min(m0 + (tid & 63) + 64 * h, a.lin.N - 1);
    sw[h] = load_f32(a.lin.sw + n);
    bias[h] = a.lin.bias ? load_f32(a.lin.bias + n) : 0.f;
  }
  if (!tc::bar_wait(done, 0, 2 * a.timeout_ns)) fail = 1;
  if (fail) report(a.err, 5 /* MOE_ERR_TIMEOUT */);
  __syncwarp();
  int* sums = reinterpret_cast<int*>(sm);  // [BN][128]; the MMAs have read their operands
  __syncthreads();
  if (warp >= 2) {
    const int quad = warp & 3;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
    for (int c = 0; c < BN && t0 + c < a.lin.T; c += 32) {
      float v[32];
      tc::tmem_ld32(tmem + c + (static_cast<uint32_t>(quad * 32) << 16), v);
#pragma unroll
      for (int i = 0; i < 32; ++i) sums[(c + i) * kGM + quad * 32 + lane] = __float_as_int(v[i]);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  cluster_sync();
  {
    // a thread per (row, column): rank takes every S-th column; 192 threads: row = tid % 64 (+ 64), column = tid / 64
#pragma unroll 1
    for (int c = rank + S * (tid >> 6); c < BN && t0 + c < a.lin.T; c += 3 * S) {
      const float sx = load_f32(a.lin.sx + t0 + c);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = (tid & 63) + 64 * h, n = m0 + row;
        if (n >= a.lin.N) continue;
        int x[8], v = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          x[p] = 0;
          if (p < S) {
            const uint32_t at = peer_addr(sums + c * kGM + row, p);
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x[p]) : "r"(at) : "memory");
          }
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) v += x[p];
        const float y = fmaf(static_cast<float>(v) * sx, sw[h], bias[h]);
        const size_t o = static_cast<size_t>(t0 + c) * a.lin.N + n;
        if (MODE == 1) {
          static_cast<__nv_bfloat16*>(a.lin.out)[o] = __float2bfloat16_rn(y);
        } else {
          float* q = static_cast<float*>(a.lin.out) + o;
          *q = MODE == 2 ? *q + y : y;
        }
      }
    }
  }
  cluster_sync();  // nobody reads this CTA's sums any more
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(BN));
  }
}

}  // namespace l8
}  // namespace moe
