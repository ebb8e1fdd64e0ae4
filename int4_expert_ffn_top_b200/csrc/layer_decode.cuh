// The whole routed-expert layer for a few tokens in one cooperative launch:
// RMSNorm (optional), router, top-K gating, the chosen int4 experts, the shared
// expert, LoRA and the combine.  One CTA per SM; the steps that need every CTA's
// result are separated by grid barriers (logits | hidden values, plus one before
// the router when the tokens' images are formed once for all CTAs, and one each
// for routed adapters).
//
// Mathematics.  A quantised row is w_k = s_g q_k + b_g for k in group g (64
// inputs), so per group
//   sum_k w_k u_k = s_g sum_k q_k u_k + b_g sum_k u_k.
// The sums over q u run on mma.sync m16n8k16 with the weight rows as M and the
// tokens (or slots) of an expert as N: an expert has one to a few of them, so N = 8
// is what there is, and the fp16 operand comes straight out of the packed codes in
// registers.  fp16 numbers with a zero exponent field are m 2^-24, so a masked
// nibble IS the code times 2^-24, exactly, without a conversion: bits 0..3 of each
// half after (w & 0x000F000F), and 16 times the code after (w & 0x00F000F0), which
// the other operand makes up for (its entries for k % 4 odd are stored / 16).  A
// word's four half pairs are (q_j, q_{j+4}), "pair order", and the other operand is
// stored in the same order.
//
// Precision.  u (bf16, 8 significant bits) is exact in fp16 after scaling each token
// by a power of two that puts its largest entry in [2^9, 2^10); hidden values h are
// stored as two fp16 numbers, hi and 2^11 (h - hi), 22 bits together, in two columns
// of the N side.  Products are exact, group sums and everything after are fp32.
#pragma once

#include "common.cuh"
#include "tc_primitives.cuh"

namespace moe {
namespace ld {

using tc::bar_arrive;
using tc::bar_expect_tx;
using tc::bar_init;
using tc::bar_test;
using tc::gtime;
using tc::sa;

constexpr int kWarps = 16;
constexpr int kComp = 32 * kWarps;   // compute threads
constexpr int kThreads = kComp + 32;  // and the warp that issues the weight copies
constexpr int kMaxT = 32, kMaxK = 8, kMaxSlots = kMaxT * kMaxK, kMaxE = 256, kMaxR = 32;
constexpr int kTileRows = 16;        // gate/up: 8 (gate, up) pairs
constexpr int kDownRows = 15;        // down: row 15 of the MMA tile sums the hidden values
constexpr int kSlotBlock = 4;        // down: slots per MMA (hi and lo columns)
constexpr int kMaxStagesG = 16, kMaxStagesD = 32;
constexpr int kMaxEls = kMaxSlots + kMaxT / kSlotBlock;
constexpr int kHeaderBytes = 256;

enum Bar { B_IMAGE = 0, B_LOGITS = 1, B_EXGU = 2, B_HIDDEN = 3, B_EXDOWN = 4, kBars = 5 };

struct Smem {  // byte offsets
  int img, us, ic, scratch, sraw, sel, w, dist, start, slots, els, gate, td, red, bars, ring, total;
  int sg, nsg, stage_g;  // gate/up: row stride, stages, stage bytes
  int sd, nsd, stage_d;  // down
};

struct Args {
  int T, K, E, H, I, logI, r;
  const uint16_t* u;  // bf16 [T][H], or null: the normed x
  const float* x;     // fp32 [T][H] to norm, or null
  float eps;
  uint16_t* u_out;
  const int32_t* exec_idx;
  float* logits;
  int32_t* idx;
  float* w;
  void* out;
  int out_mode;
  const uint8_t* router;
  const float* rbias;
  const uint8_t* sgate;
  const uint8_t* shared;
  const uint16_t* shA[3];
  const uint16_t* shB[3];
  float lora_scale;
  const uint8_t* pool;
  int64_t stride;
  const uint16_t *exA, *exB, *exAgu, *exBgu;
  // workspace
  uint32_t* bar;      // kBars counters, zero on entry
  uint8_t* img;       // [T][2H + 16]
  float* us;          // [T][G]
  float* ic;          // [T]
  float* aux;         // [1 + 2r][T]: shared gate logit, gate and up LoRA-A products
  uint16_t* h;        // [T K + T][2][I]
  float* tgu;         // [T K][2][r]
  float* tex;         // [T K][r]
  int* err;
  long long timeout_ns;
  int smem_image;     // the tokens' images are in shared memory
  int shared_build;   // the images are formed once, by CTA t for token t, and passed through memory
  Smem sm;
};

// Row stride in shared memory: 32 or 96 bytes past a multiple of 128, so that the 8-byte reads of 4 rows x 32
// bytes (one phase of a warp's fragment load) fall on different banks.
__host__ __device__ constexpr int padded_row(int rec) {
  int s = rec;
  while (s % 128 != 32 && s % 128 != 96) s += 16;
  return s;
}

// Barriers of the compute threads, of all threads, and of a team of warps.  Warps are reconverged first and the
// barriers are the non-aligned form: lanes may come from loops of different trip counts.
MOE_DEV void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
MOE_DEV void cta_sync() { named_sync(15, kComp); }
MOE_DEV void all_sync() { named_sync(14, kThreads); }
MOE_DEV void team_sync(int team, int warps) {
  if (warps == 1)
    __syncwarp();
  else
    named_sync(1 + team, 32 * warps);
}

MOE_DEV void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(sa(dst)),
               "l"(src), "r"(bytes), "r"(sa(bar))
               : "memory");
}

MOE_DEV void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

MOE_DEV float half_at(const uint8_t* p) { return half_bits_to_float(*reinterpret_cast<const uint16_t*>(p)); }

// Bounded wait on an mbarrier phase; after a first failure of this CTA no wait blocks any more (the call's outputs
// are undefined then, but every index read below stays in range).
struct Waiter {
  volatile int* failed;
  int* err;
  long long timeout_ns;
  MOE_DEV void fail() const {
    *failed = 1;
    report(err, 5 /* MOE_ERR_TIMEOUT */);
  }
  MOE_DEV void wait(uint64_t* b, uint32_t parity, bool even_if_failed = false) const {
    if (bar_test(b, parity)) return;
    const long long end = gtime() + timeout_ns;
    while (!bar_test(b, parity)) {
      if (*failed && !even_if_failed) return;
      if (gtime() > end) return fail();
    }
  }
};

// Wait for the copy that is number i in a ring of n stages.  Teams of warps take the ring's copies in turn, and a
// parity tells a phase from its neighbours only, while the copy before this one in the stage is another team's and may
// still be under way.  So the copying warp writes down which copy a stage holds next (`turn`) once the one before is
// used up, and a consumer looks at the phase only after that.
MOE_DEV void ring_open(uint32_t* turn, int i, int n) {
  asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(sa(turn + i % n)), "r"(i) : "memory");
}
MOE_DEV void ring_wait(const Waiter& wt, const uint32_t* turn, uint64_t* full, int i, int n) {
  if (i >= n) {
    const long long end = gtime() + wt.timeout_ns;
    for (;;) {
      int v;
      asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(v) : "r"(sa(turn + i % n)) : "memory");
      if (v == i || *wt.failed) break;
      if (gtime() > end) {
        wt.fail();
        break;
      }
    }
  }
  wt.wait(full + i % n, static_cast<uint32_t>(i / n) & 1u);
}

// ----------------------------------------------------------------------------- grid barrier
// Each CTA adds one to the barrier's counter when its part is written; a CTA goes on when the counter has reached
// the grid's size.  All CTAs are resident (cooperative launch).
MOE_DEV void grid_arrive(const Args& a, int b) {
  cta_sync();
  if (threadIdx.x == 0) {
    __threadfence();
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.bar + b) : "memory");
  }
}

MOE_DEV void grid_wait(const Args& a, int b, const Waiter& wt) {
  if (threadIdx.x == 0) {
    const long long end = gtime() + a.timeout_ns;
    for (;;) {
      uint32_t v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.bar + b) : "memory");
      if (v >= gridDim.x || *wt.failed) break;
      if (gtime() > end) {
        wt.fail();
        break;
      }
    }
    __threadfence();
  }
  cta_sync();
}

// ----------------------------------------------------------------------------- token images
// bf16 of the fp32 quotient x / sqrt(mean + eps): the fp32 product is off by at most two units of its last place, so
// only where that could change the bf16 rounding is the quotient formed in 64 bits and rounded to fp32 first.
MOE_DEV uint16_t normed_bf16(float x, float rstd, double rstd64) {
  const float p = x * rstd;
  const uint32_t low = __float_as_uint(p) & 0xffffu;
  const float q = (low - 0x7ff8u) <= 0x10u ? static_cast<float>(static_cast<double>(x) * rstd64) : p;
  return __bfloat16_as_ushort(__float2bfloat16_rn(q));
}

MOE_DEV float max_bits(float a, float b) {  // non-negative floats by their bits (a NaN stays)
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

MOE_DEV void load8(const Args& a, size_t at, float (&v)[8]) {
  if (a.x) {
    const float4 p = *reinterpret_cast<const float4*>(a.x + at), q = *reinterpret_cast<const float4*>(a.x + at + 4);
    v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
  } else {
    const uint4 p = *reinterpret_cast<const uint4*>(a.u + at);
    const uint32_t s[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(s[i] << 16);
      v[2 * i + 1] = __uint_as_float(s[i] & 0xffff0000u);
    }
  }
}

// Token t's image by `warps` warps (this one is number wi): u scaled by a power of two c, fp16, pair order, odd pairs
// / 16; per group 2^-24 sum of c u; 1/c.
MOE_DEV void build_image(const Args& a, int t, int wi, int warps, int team, double* red, uint8_t* row, float* us,
                         float* ic, bool write_u) {
  const int lane = threadIdx.x & 31, nb = a.H / 8;
  const size_t base = static_cast<size_t>(t) * a.H;
  float m = 0.f;
  double ss = 0.0;
  for (int b = wi * 32 + lane; b < nb; b += 32 * warps) {
    float v[8];
    load8(a, base + 8 * b, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_bits(m, fabsf(v[i]));
    if (a.x) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), ss);
    }
  }
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  if (a.x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  if (warps > 1) {
    double* r = red + 2 * warps * team;
    if (lane == 0) r[2 * wi] = ss, r[2 * wi + 1] = static_cast<double>(m);
    team_sync(team, warps);
    ss = 0.0;
    for (int w = 0; w < warps; ++w) {
      ss += r[2 * w];
      m = max_bits(m, static_cast<float>(r[2 * w + 1]));
    }
    team_sync(team, warps);
  }
  double rstd64 = 1.0;
  float rstd = 1.f;
  if (a.x) {
    rstd64 = 1.0 / sqrt(ss / a.H + static_cast<double>(a.eps));
    rstd = static_cast<float>(rstd64);
    m *= rstd;
  }
  // c = 2^(9 - e) for m in [2^e, 2^(e+1)); 1 where m is zero or not finite
  const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
  const int ce = (m > 0.f && e < 128) ? min(max(9 - e, -126), 126) : 0;
  const float c = __uint_as_float(static_cast<uint32_t>(127 + ce) << 23);
  if (wi == 0 && lane == 0) *ic = __uint_as_float(static_cast<uint32_t>(127 - ce) << 23);
  for (int b = wi * 32 + lane; b < nb; b += 32 * warps) {
    float v[8];
    load8(a, base + 8 * b, v);
    if (a.x) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint16_t q = normed_bf16(v[i], rstd, rstd64);
        v[i] = bf16_bits_to_float(q);
        if (i & 1)
          o[i >> 1] |= static_cast<uint32_t>(q) << 16;
        else
          o[i >> 1] = q;
      }
      if (write_u && a.u_out) *reinterpret_cast<uint4*>(a.u_out + base + 8 * b) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] *= c;
      sum += v[i];
    }
    uint32_t p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = (j & 1) ? 0.0625f : 1.f;
      p[j] = h2_bits(__floats2half2_rn(v[j] * f, v[j + 4] * f));
    }
    *reinterpret_cast<uint4*>(row + 16 * b) = make_uint4(p[0], p[1], p[2], p[3]);
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
    if ((b & 7) == 0) us[b >> 3] = sum * 0x1p-24f;
  }
}

// Two B registers quads of a lane's 8-blocks 2 tig and 2 tig + 1 of group gi (image rows, shared or global memory).
struct BFrag {
  uint4 x, y;
};
MOE_DEV BFrag b_frag(const uint8_t* row, int gi, int tig) {
  const uint4* p = reinterpret_cast<const uint4*>(row + gi * 128 + tig * 32);
  return {p[0], p[1]};
}
MOE_DEV BFrag b_frag_l2(const uint8_t* row, int gi, int tig) {
  const uint4* p = reinterpret_cast<const uint4*>(row + gi * 128 + tig * 32);
  return {__ldcg(p), __ldcg(p + 1)};
}

// ----------------------------------------------------------------------------- int4 rows: gate/up
// acc += rows g and g + 8 of the stage over groups [g0, g1) times NB column blocks of 8.
template <int NB>
MOE_DEV void int4_tile(const uint8_t* stage, int sg, int code_bytes, int G, int g0, int g1, const uint8_t* const (&col)[NB],
                       const float* const (&ua)[NB], const float* const (&ub)[NB], float (&acc)[NB][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const uint8_t* ra = stage + g * sg;
  const uint8_t* rb = ra + 8 * sg;
#pragma unroll 2
  for (int gi = g0; gi < g1; ++gi) {
    const uint2 wa = *reinterpret_cast<const uint2*>(ra + gi * 32 + tig * 8);
    const uint2 wb = *reinterpret_cast<const uint2*>(rb + gi * 32 + tig * 8);
    const float s0 = half_at(ra + code_bytes + 2 * gi), b0 = half_at(ra + code_bytes + 2 * (G + gi));
    const float s1 = half_at(rb + code_bytes + 2 * gi), b1 = half_at(rb + code_bytes + 2 * (G + gi));
    BFrag f[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) f[n] = b_frag(col[n], gi, tig);
    const uint32_t wa8 = wa.x >> 8, wb8 = wb.x >> 8, va8 = wa.y >> 8, vb8 = wb.y >> 8;
    const uint32_t lo = 0x000F000Fu, hi = 0x00F000F0u;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma16(d, wa.x & lo, wb.x & lo, wa.x & hi, wb.x & hi, f[n].x.x, f[n].x.y);
      mma16(d, wa8 & lo, wb8 & lo, wa8 & hi, wb8 & hi, f[n].x.z, f[n].x.w);
      mma16(d, wa.y & lo, wb.y & lo, wa.y & hi, wb.y & hi, f[n].y.x, f[n].y.y);
      mma16(d, va8 & lo, vb8 & lo, va8 & hi, vb8 & hi, f[n].y.z, f[n].y.w);
      const float u0 = ua[n][gi], u1 = ub[n][gi];
      acc[n][0] = fmaf(b0, u0, fmaf(s0, d[0], acc[n][0]));
      acc[n][1] = fmaf(b0, u1, fmaf(s0, d[1], acc[n][1]));
      acc[n][2] = fmaf(b1, u0, fmaf(s1, d[2], acc[n][2]));
      acc[n][3] = fmaf(b1, u1, fmaf(s1, d[3], acc[n][3]));
    }
  }
}

// One (tile, block of 8 NB columns) by a team of W warps: partial sums of the warps' groups to part[w][16][8 NB].
// token(c): token of column c.
template <int NB, class TokenFn>
MOE_DEV void gate_up_block(const Args& a, const uint8_t* img, const float* us, const uint8_t* stage, int wi, int W,
                           float* part, TokenFn token) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3, G = a.H / 64, ldu = 2 * a.H + 16;
  const uint8_t* col[NB];
  const float *ua[NB], *ub[NB];
  float acc[NB][4];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    col[n] = img + static_cast<size_t>(token(8 * n + g)) * ldu;
    ua[n] = us + token(8 * n + 2 * tig) * G;
    ub[n] = us + token(8 * n + 2 * tig + 1) * G;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  }
  int4_tile<NB>(stage, a.sm.sg, a.H / 2, G, wi * G / W, (wi + 1) * G / W, col, ua, ub, acc);
  float* p = part + wi * (16 * 8 * NB);
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    *reinterpret_cast<float2*>(p + g * (8 * NB) + 8 * n + 2 * tig) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(p + (g + 8) * (8 * NB) + 8 * n + 2 * tig) = make_float2(acc[n][2], acc[n][3]);
  }
}

// (a, b) of pair pr, column c: the warps' partial sums in order, scaled back.
template <int NB>
MOE_DEV float2 pair_sum(const float* part, int W, int pr, int c) {
  float x = 0.f, y = 0.f;
  for (int w = 0; w < W; ++w) {
    x += part[w * (16 * 8 * NB) + (2 * pr) * (8 * NB) + c];
    y += part[w * (16 * 8 * NB) + (2 * pr + 1) * (8 * NB) + c];
  }
  return make_float2(x * 0x1p24f, y * 0x1p24f);
}

// Hidden value j of row `row` of the hidden buffer, as hi and lo.
MOE_DEV void store_h(const Args& a, int row, int j, float x, float y) {
  const float v = silu(x) * y;
  if (fabsf(v) > kF16Max && fabsf(v) <= 3.402823466e38f) report(a.err, 6 /* MOE_ERR_RANGE */);
  const float s = (j & 1) ? v * 0.0625f : v;
  const __half hi = __float2half_rn(s);
  const __half lo = __float2half_rn((s - __half2float(hi)) * 2048.f);
  uint16_t* p = a.h + static_cast<size_t>(row) * 2 * a.I + pair_pos(j);
  p[0] = __half_as_ushort(hi);
  p[a.I] = __half_as_ushort(lo);
}

MOE_DEV float dot_r(const uint16_t* B, const float* t, int r) {
  float v = 0.f;
  for (int i = 0; i < r; ++i) v = fmaf(half_bits_to_float(B[i]), __ldcg(t + i), v);
  return v;
}

// ----------------------------------------------------------------------------- fp16 rows (LoRA A)
// even/odd accumulators of rows g and g + 8 (row pointers, in halves) over groups [g0, g1) times one column block.
template <bool L2, class Col>
MOE_DEV void f16_rows(const uint16_t* ra, const uint16_t* rb, int g0, int g1, Col col, float (&ev)[4], float (&od)[4]) {
  const int tig = threadIdx.x & 3;
#pragma unroll 2
  for (int gi = g0; gi < g1; ++gi) {
    const BFrag f = L2 ? b_frag_l2(col, gi, tig) : b_frag(col, gi, tig);
    const uint4* pa = reinterpret_cast<const uint4*>(ra + gi * 64 + tig * 16);
    const uint4* pb = reinterpret_cast<const uint4*>(rb + gi * 64 + tig * 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 x = __ldg(pa + h), y = __ldg(pb + h), b = h ? f.y : f.x;
      mma16(ev, prmt(x.x, x.z, 0x5410), prmt(y.x, y.z, 0x5410), prmt(x.y, x.w, 0x5410), prmt(y.y, y.w, 0x5410), b.x, b.z);
      mma16(od, prmt(x.x, x.z, 0x7632), prmt(y.x, y.z, 0x7632), prmt(x.y, x.w, 0x7632), prmt(y.y, y.w, 0x7632), b.y, b.w);
    }
  }
}

// ----------------------------------------------------------------------------- the kernel
struct Tile {  // 8 or fewer (gate, up) pairs of one chosen expert
  int d, p0, n;
};
MOE_DEV Tile next_tile(int pos, int hi, int logI) {
  const int d = pos >> logI, p0 = pos & ((1 << logI) - 1);
  const int end = min(hi, (d + 1) << logI);
  return {d, p0, min(kTileRows / 2, end - pos)};
}

MOE_DEV uint32_t fparity(int i, int n) { return static_cast<uint32_t>(i / n) & 1u; }

// Lanes of the copy warp bring `rows` records of `rec` bytes to `dst` (row stride `ld`).
MOE_DEV void copy_rows(uint8_t* dst, int ld, const uint8_t* src, int rec, int rows, uint64_t* bar) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) bar_expect_tx(bar, static_cast<uint32_t>(rec * rows));
  __syncwarp();
  if (ld == rec) {
    if (lane == 0) bulk_copy(dst, src, static_cast<uint32_t>(rec * rows), bar);
  } else if (lane < rows) {
    bulk_copy(dst + lane * ld, src + static_cast<size_t>(lane) * rec, static_cast<uint32_t>(rec), bar);
  }
}

__global__ void __launch_bounds__(kThreads, 1) layer_decode_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) uint8_t sm[];
  const Smem& S = a.sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tig = lane & 3;
  const int cta = blockIdx.x, grid = gridDim.x;
  const int T = a.T, K = a.K, TK = T * K, G = a.H / 64, G2 = a.I / 64, ldu = 2 * a.H + 16, r = a.r;
  uint64_t* full_g = reinterpret_cast<uint64_t*>(sm + S.bars);
  uint64_t* empty_g = full_g + kMaxStagesG;
  uint64_t* full_d = empty_g + kMaxStagesG;
  uint64_t* empty_d = full_d + kMaxStagesD;
  int* misc = reinterpret_cast<int*>(empty_d + kMaxStagesD);  // [0] failed, [1] distinct experts, [2] down elements
  uint32_t* turn_g = reinterpret_cast<uint32_t*>(misc + 24);
  uint32_t* turn_d = turn_g + kMaxStagesG;
  const Waiter wt{misc, a.err, a.timeout_ns};
  int* sel = reinterpret_cast<int*>(sm + S.sel);
  float* sw = reinterpret_cast<float*>(sm + S.w);
  int* dist = reinterpret_cast<int*>(sm + S.dist);
  int* start = reinterpret_cast<int*>(sm + S.start);
  int* slots = reinterpret_cast<int*>(sm + S.slots);
  int* els = reinterpret_cast<int*>(sm + S.els);
  float* scratch = reinterpret_cast<float*>(sm + S.scratch);
  float* sraw = reinterpret_cast<float*>(sm + S.sraw);
  uint8_t* ring = sm + S.ring;

  // this CTA's shares: pairs of the shared expert, rows of the down projections
  const int sp0 = cta * a.I / grid, sp1 = (cta + 1) * a.I / grid, nsp = sp1 - sp0;
  const int nst = (nsp + 7) / 8;  // shared tiles
  const int dr0 = cta * a.H / grid, ndr = (cta + 1) * a.H / grid - dr0;
  const int nrt = (ndr + kDownRows - 1) / kDownRows, rt_rows = nrt ? (ndr + nrt - 1) / nrt : 0;
  const int RGU = qrow_bytes(a.H, 4), RDN = qrow_bytes(a.I, 4);
  const size_t dn_off = static_cast<size_t>(2 * a.I) * RGU;
  const int sh_blocks = (T + kSlotBlock - 1) / kSlotBlock;

  if (tid == 0) {
    for (int i = 0; i < kMaxStagesG; ++i) bar_init(full_g + i, 1), bar_init(empty_g + i, 1);
    for (int i = 0; i < kMaxStagesD; ++i) bar_init(full_d + i, 1), bar_init(empty_d + i, 1);
    for (int i = 0; i < kMaxStagesG + kMaxStagesD; ++i) turn_g[i] = 0;
    misc[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------------------- weight copies
    for (int i = 0; i < nst; ++i)
      copy_rows(ring + i * S.stage_g, S.sg, a.shared + static_cast<size_t>(2 * (sp0 + 8 * i)) * RGU, RGU,
                2 * min(8, nsp - 8 * i), full_g + i);
    all_sync();  // the expert list stands
    const int D = misc[1], nel = misc[2];
    const int lo = static_cast<int>(static_cast<long long>(cta) * (D << a.logI) / grid);
    const int hi = static_cast<int>(static_cast<long long>(cta + 1) * (D << a.logI) / grid);
    int n = nst;
    for (int pos = lo; pos < hi; ++n) {
      const Tile t = next_tile(pos, hi, a.logI);
      const int s = n % S.nsg;
      if (n >= S.nsg) {
        wt.wait(empty_g + s, fparity(n - S.nsg, S.nsg));
        if (lane == 0) ring_open(turn_g, n, S.nsg);
      }
      copy_rows(ring + s * S.stage_g, S.sg, a.pool + dist[t.d] * a.stride + static_cast<size_t>(2 * t.p0) * RGU, RGU,
                2 * t.n, full_g + s);
      pos += t.n;
    }
    for (int i = max(0, n - S.nsg); i < n; ++i) wt.wait(empty_g + i % S.nsg, fparity(i, S.nsg));  // the ring is free
    const int total = nrt * nel;
    for (int i = 0; i < total; ++i) {
      const int rt = i / nel, el = els[i - rt * nel], d = el & 511, s = i % S.nsd;
      const uint8_t* block = d == 511 ? a.shared : a.pool + dist[d] * a.stride;
      if (i >= S.nsd) {
        wt.wait(empty_d + s, fparity(i - S.nsd, S.nsd));
        if (lane == 0) ring_open(turn_d, i, S.nsd);
      }
      copy_rows(ring + s * S.stage_d, S.sd, block + dn_off + static_cast<size_t>(dr0 + rt * rt_rows) * RDN, RDN,
                min(rt_rows, ndr - rt * rt_rows), full_d + s);
    }
    // no copy may be in flight when the CTA leaves
    for (int i = max(0, n - S.nsg); i < n; ++i) wt.wait(full_g + i % S.nsg, fparity(i, S.nsg), true);
    for (int i = max(0, total - S.nsd); i < total; ++i) wt.wait(full_d + i % S.nsd, fparity(i, S.nsd), true);
    return;
  }

  // --------------------------------------------------------------------------- token images
  const uint8_t* img = a.smem_image ? sm + S.img : a.img;
  float* us = reinterpret_cast<float*>(sm + S.us);
  float* ic = reinterpret_cast<float*>(sm + S.ic);
  double* red = reinterpret_cast<double*>(sm + S.red);
  if (a.shared_build) {
    for (int t = cta; t < T; t += grid)
      build_image(a, t, warp, kWarps, 0, red, a.img + static_cast<size_t>(t) * ldu, a.us + t * G, a.ic + t, true);
    grid_arrive(a, B_IMAGE);
    grid_wait(a, B_IMAGE, wt);
    if (a.smem_image)
      for (int i = tid; i < T * ldu / 16; i += kComp)
        reinterpret_cast<uint4*>(sm + S.img)[i] = __ldcg(reinterpret_cast<const uint4*>(a.img) + i);
    for (int i = tid; i < T * G; i += kComp) us[i] = __ldcg(a.us + i);
    if (tid < T) ic[tid] = __ldcg(a.ic + tid);
  } else {
    int W = kWarps;
    while (W > 1 && W * T > kWarps) W >>= 1;
    const int teams = kWarps / W, team = warp / W;
    for (int t = team; t < T; t += teams)
      build_image(a, t, warp % W, W, team, red, sm + S.img + t * ldu, us + t * G, ic + t, t % grid == cta);
  }
  cta_sync();

  // --------------------------------------------------------------------------- rows over all tokens: router, shared
  // gate (8 bits), the shared expert's gate and up LoRA A (fp16)
  const int nA = (a.shA[0] ? r : 0) + (a.shA[1] ? r : 0);
  {
    const int nrows = a.E + 1 + nA, r0 = cta * nrows / grid, r1 = (cta + 1) * nrows / grid;
    const int g0 = warp * G / kWarps, g1 = (warp + 1) * G / kWarps;
    const int n8 = max(0, min(r1, a.E + 1) - r0);  // 8-bit rows r0 .. r0 + n8 - 1, then fp16 rows
    const int R8 = qrow_bytes(a.H, 8);
    for (int t0 = 0; t0 < T; t0 += 8) {
      const uint8_t* col = img + static_cast<size_t>(min(t0 + g, T - 1)) * ldu;
      const float* ua = us + min(t0 + 2 * tig, T - 1) * G;
      const float* ub = us + min(t0 + 2 * tig + 1, T - 1) * G;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      if (n8 > 0) {
        const int row = r0 + min(g, n8 - 1);
        const uint8_t* rec = row < a.E ? a.router + static_cast<size_t>(row) * R8 : a.sgate;
#pragma unroll 2
        for (int gi = g0; gi < g1; ++gi) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(rec + gi * 64 + tig * 16));
          const BFrag f = b_frag(col, gi, tig);
          float ev[4] = {0.f, 0.f, 0.f, 0.f}, od[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t m = 0x00FF00FFu;
          mma16(ev, prmt(q.x, q.y, 0x4400) & m, 0, prmt(q.x, q.y, 0x6622) & m, 0, f.x.x, f.x.z);
          mma16(od, prmt(q.x, q.y, 0x5511) & m, 0, prmt(q.x, q.y, 0x7733) & m, 0, f.x.y, f.x.w);
          mma16(ev, prmt(q.z, q.w, 0x4400) & m, 0, prmt(q.z, q.w, 0x6622) & m, 0, f.y.x, f.y.z);
          mma16(od, prmt(q.z, q.w, 0x5511) & m, 0, prmt(q.z, q.w, 0x7733) & m, 0, f.y.y, f.y.w);
          const float s = half_at(rec + a.H + 2 * gi), b = half_at(rec + a.H + 2 * (G + gi));
          acc[0] = fmaf(b, ua[gi], fmaf(s, fmaf(16.f, od[0], ev[0]), acc[0]));
          acc[1] = fmaf(b, ub[gi], fmaf(s, fmaf(16.f, od[1], ev[1]), acc[1]));
        }
      }
      if (g < n8) *reinterpret_cast<float2*>(scratch + (warp * 16 + g) * 8 + 2 * tig) = make_float2(acc[0], acc[1]);
      const int nf = r1 - r0 - n8;
      if (nf > 0) {
        const int j = r0 + n8 + min(g, nf - 1) - (a.E + 1);  // LoRA row: gate's rows, then up's
        const uint16_t* A = (a.shA[0] && j < r) ? a.shA[0] + static_cast<size_t>(j) * a.H
                                                : a.shA[1] + static_cast<size_t>(a.shA[0] ? j - r : j) * a.H;
        float ev[4] = {0.f, 0.f, 0.f, 0.f}, od[4] = {0.f, 0.f, 0.f, 0.f};
        f16_rows<false>(A, A, g0, g1, col, ev, od);
        if (g < nf)
          *reinterpret_cast<float2*>(scratch + (warp * 16 + n8 + g) * 8 + 2 * tig) =
              make_float2(fmaf(16.f, od[0], ev[0]), fmaf(16.f, od[1], ev[1]));
      }
      cta_sync();
      for (int i = tid; i < (r1 - r0) * 8; i += kComp) {
        const int row = i >> 3, t = t0 + (i & 7);
        if (t < T) {
          float v = 0.f;
          for (int w = 0; w < kWarps; ++w) v += scratch[(w * 16 + row) * 8 + (i & 7)];
          v *= ic[t];
          const int j = r0 + row;
          if (j < a.E)
            a.logits[static_cast<size_t>(t) * a.E + j] = v * 0x1p24f + (a.rbias ? a.rbias[j] : 0.f);
          else
            a.aux[(j - a.E) * T + t] = j == a.E ? v * 0x1p24f : v;
        }
      }
      cta_sync();
    }
  }
  grid_arrive(a, B_LOGITS);

  // --------------------------------------------------------------------------- shared expert's gate/up, raw
  if (nst > 0) {
    const int nb = (T + 15) / 16, units = nst * nb, W = units > 1 ? 8 : 16, teams = kWarps / W, team = warp / W;
    float* part = scratch + team * (W * 16 * 16);
    for (int un = 0; un < units; un += teams) {
      const int q = un + team, ti = q / nb, t0 = (q % nb) * 16;
      const bool on = q < units;
      if (on) {
        wt.wait(full_g + ti, 0);
        gate_up_block<2>(a, img, us, ring + ti * S.stage_g, warp % W, W, part, [&](int c) { return min(t0 + c, T - 1); });
      }
      cta_sync();
      if (on) {
        for (int i = tid - team * W * 32; i < 8 * 16; i += W * 32) {
          const int pr = i & 7, c = i >> 3, t = t0 + c;
          if (8 * ti + pr < nsp && t < T) {
            const float2 v = pair_sum<2>(part, W, pr, c);
            sraw[t * 2 * nsp + 2 * (8 * ti + pr)] = v.x * ic[t];
            sraw[t * 2 * nsp + 2 * (8 * ti + pr) + 1] = v.y * ic[t];
          }
        }
      }
      cta_sync();
    }
    if (tid == 0)
      for (int i = 0; i < nst; ++i) bar_arrive(empty_g + i);
  }

  // --------------------------------------------------------------------------- top-K, gating, the expert list
  grid_wait(a, B_LOGITS, wt);
  uint32_t* mask = reinterpret_cast<uint32_t*>(scratch);  // [256 experts][8 words]: the slots that chose an expert
  for (int i = tid; i < kMaxE * 8; i += kComp) mask[i] = 0;
  cta_sync();
  for (int t = warp; t < T; t += kWarps) {
    const float* lg = a.logits + static_cast<size_t>(t) * a.E;
    uint32_t key[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      uint32_t k = 0;
      if (e < a.E) {
        const float v = __ldcg(lg + e);
        const uint32_t b = __float_as_uint(v);
        k = v != v ? 1u : b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);  // order of the floats; NaN last
      }
      key[i] = k;
    }
    int my_e = 0;
    float my_l = -INFINITY;
    for (int k = 0; k < K; ++k) {
      uint32_t best = key[0];
      int bi = 0;
#pragma unroll
      for (int i = 1; i < 8; ++i)
        if (key[i] > best) best = key[i], bi = i;
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const int e = static_cast<int>(
          __reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(lane + 32 * bi) : 0xffffu));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e == lane + 32 * i) key[i] = 0;
      if (lane == k) my_e = min(e, a.E - 1);
    }
    if (lane < K && cta == 0) a.idx[t * K + lane] = my_e;
    if (a.exec_idx && lane < K) my_e = min(max(a.exec_idx[t * K + lane], 0), a.E - 1);
    if (lane < K) my_l = __ldcg(lg + my_e);
    float mx = my_l;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float ex = lane < K ? expf(my_l - mx) : 0.f;
    float den = ex;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (lane < K) {
      const int s = t * K + lane;
      sel[s] = my_e;
      sw[s] = ex / den;
      atomicOr(mask + my_e * 8 + (s >> 5), 1u << (s & 31));
      if (cta == 0) a.w[s] = ex / den;
    }
  }
  float* gate = reinterpret_cast<float*>(sm + S.gate);
  if (tid < T) gate[tid] = sigmoid(__ldcg(a.aux + tid));
  cta_sync();
  if (warp < 8) {  // chosen experts in ascending order, their slots in ascending order, the down elements
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) cnt += __popc(mask[tid * 8 + i]);
    const uint32_t bal = __ballot_sync(0xffffffffu, cnt > 0);
    int v = cnt | ((cnt + kSlotBlock - 1) / kSlotBlock) << 16;
    const int own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    int* tot = misc + 4;  // [8][2]
    if (lane == 31) tot[2 * warp] = v, tot[2 * warp + 1] = __popc(bal);
    named_sync(1, 256);
    int off = v - own, d = __popc(bal & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) off += tot[2 * w], d += tot[2 * w + 1];
    int so = off & 0xffff, eo = sh_blocks + (off >> 16);
    if (cnt > 0) {
      dist[d] = tid;
      start[d] = so;
      for (int b = 0; b < cnt; b += kSlotBlock) els[eo++] = d | (so + b) << 9 | min(kSlotBlock, cnt - b) << 20;
      for (int i = 0; i < 8; ++i)
        for (uint32_t m = mask[tid * 8 + i]; m; m &= m - 1) slots[so++] = 32 * i + __ffs(m) - 1;
    }
    if (tid == 255) {
      const int D = d + (cnt > 0);
      misc[1] = D;
      misc[2] = sh_blocks + (off >> 16) + (own >> 16);
      start[D] = TK;
    }
    if (tid < sh_blocks) els[tid] = 511 | (tid * kSlotBlock) << 9 | min(kSlotBlock, T - tid * kSlotBlock) << 20;
  }
  all_sync();
  const int D = misc[1], nel = misc[2];

  // --------------------------------------------------------------------------- routed gate/up adapters: A u
  if (a.exAgu) {
    const int rows = 2 * r, total = D * rows;
    for (int q = cta * kWarps + warp; q < total; q += grid * kWarps) {
      const int d = q / rows, i = q - d * rows, e = dist[d];
      const uint16_t* A = a.exAgu + (static_cast<size_t>(e) * rows + i) * a.H;
      for (int s = start[d]; s < start[d + 1]; ++s) {
        const int t = slots[s] / K;
        const uint8_t* row = img + static_cast<size_t>(t) * ldu;
        float v = 0.f;
        for (int b = lane; b < a.H / 8; b += 32) {
          const uint4 p = __ldg(reinterpret_cast<const uint4*>(A) + b), x = *reinterpret_cast<const uint4*>(row + 16 * b);
          v = dot2_mix(prmt(p.x, p.z, 0x5410), x.x, v);
          v = dot2_mix(prmt(p.y, p.w, 0x5410), x.z, v);
          float o = dot2_mix(prmt(p.x, p.z, 0x7632), x.y, 0.f);
          o = dot2_mix(prmt(p.y, p.w, 0x7632), x.w, o);
          v = fmaf(16.f, o, v);
        }
        v = warp_reduce(v);
        if (lane == 0) a.tgu[(static_cast<size_t>(slots[s]) * 2 + i / r) * r + i % r] = v * ic[t];
      }
    }
    grid_arrive(a, B_EXGU);
    grid_wait(a, B_EXGU, wt);
  }

  // --------------------------------------------------------------------------- shared expert's hidden values
  for (int i = tid; i < T * nsp; i += kComp) {
    const int t = i / nsp, j = sp0 + i - t * nsp;
    float x = sraw[2 * i], y = sraw[2 * i + 1];
    const float* ta = a.aux + T + t;
    if (a.shA[0]) {
      float v = 0.f;
      for (int k = 0; k < r; ++k) v = fmaf(half_bits_to_float(a.shB[0][static_cast<size_t>(j) * r + k]), __ldcg(ta + k * T), v);
      x = fmaf(a.lora_scale, v, x);
      ta += r * T;
    }
    if (a.shA[1]) {
      float v = 0.f;
      for (int k = 0; k < r; ++k) v = fmaf(half_bits_to_float(a.shB[1][static_cast<size_t>(j) * r + k]), __ldcg(ta + k * T), v);
      y = fmaf(a.lora_scale, v, y);
    }
    store_h(a, TK + t, j, x, y);
  }

  // --------------------------------------------------------------------------- chosen experts' gate/up
  {
    const int lo = static_cast<int>(static_cast<long long>(cta) * (D << a.logI) / grid);
    const int hi = static_cast<int>(static_cast<long long>(cta + 1) * (D << a.logI) / grid);
    int nt = 0;
    for (int pos = lo; pos < hi; ++nt) pos += next_tile(pos, hi, a.logI).n;
    int W = nt >= 8 ? 4 : (nt >= 2 ? 8 : 16);
    const int teams = kWarps / W, team = warp / W, wi = warp % W, ltid = tid - team * W * 32;
    float* part = scratch + team * (W * 16 * 16);
    int n = nst, q = 0;
    for (int pos = lo; pos < hi; ++n, ++q) {
      const Tile tl = next_tile(pos, hi, a.logI);
      pos += tl.n;
      if (q % teams != team) continue;
      const int s = n % S.nsg, e = dist[tl.d], s0 = start[tl.d], cnt = start[tl.d + 1] - s0;
      const uint8_t* stage = ring + s * S.stage_g;
      ring_wait(wt, turn_g, full_g, n, S.nsg);
      for (int b = 0; b < cnt;) {
        const bool one = cnt - b <= 8;
        auto token = [&](int c) { return slots[s0 + min(b + c, cnt - 1)] / K; };
        if (one)
          gate_up_block<1>(a, img, us, stage, wi, W, part, token);
        else
          gate_up_block<2>(a, img, us, stage, wi, W, part, token);
        team_sync(team, W);
        const int cols = one ? 8 : 16;
        for (int i = ltid; i < 8 * cols; i += 32 * W) {
          const int pr = i & 7, c = i >> 3;
          if (pr < tl.n && b + c < cnt) {
            const int slot = slots[s0 + b + c], j = tl.p0 + pr;
            float2 v = one ? pair_sum<1>(part, W, pr, c) : pair_sum<2>(part, W, pr, c);
            const float f = ic[slot / K];
            v.x *= f;
            v.y *= f;
            if (a.exAgu) {
              const uint16_t* B = a.exBgu + (static_cast<size_t>(e) * 2 * a.I + 2 * j) * r;
              const float* t = a.tgu + static_cast<size_t>(slot) * 2 * r;
              v.x = fmaf(a.lora_scale, dot_r(B, t, r), v.x);
              v.y = fmaf(a.lora_scale, dot_r(B + r, t + r, r), v.y);
            }
            store_h(a, slot, j, v.x, v.y);
          }
        }
        b += cols;
        team_sync(team, W);
      }
      if (ltid == 0) bar_arrive(empty_g + s);
    }
  }
  grid_arrive(a, B_HIDDEN);
  grid_wait(a, B_HIDDEN, wt);

  // --------------------------------------------------------------------------- LoRA A on the hidden values
  const uint8_t* hb = reinterpret_cast<const uint8_t*>(a.h);
  const size_t hrow = static_cast<size_t>(a.I) * 2;  // bytes of one hi or lo row
  auto lora_h = [&](const uint16_t* A, int m0, int pos_of_col, float (&v)[2]) {  // rows m0 + g, m0 + g + 8
    const uint16_t* ra = A + static_cast<size_t>(min(m0 + g, r - 1)) * a.I;
    const uint16_t* rb = A + static_cast<size_t>(min(m0 + g + 8, r - 1)) * a.I;
    float ev[4] = {0.f, 0.f, 0.f, 0.f}, od[4] = {0.f, 0.f, 0.f, 0.f};
    f16_rows<true>(ra, rb, 0, G2, hb + (static_cast<size_t>(pos_of_col) * 2 + (g & 1)) * hrow, ev, od);
    v[0] = fmaf(fmaf(16.f, od[1], ev[1]), 0x1p-11f, fmaf(16.f, od[0], ev[0]));
    v[1] = fmaf(fmaf(16.f, od[3], ev[3]), 0x1p-11f, fmaf(16.f, od[2], ev[2]));
  };
  const int mts = (r + 15) / 16;
  if (a.exA) {  // each (block of slots, 16 rows of A) once in the grid
    for (int q = cta + grid * warp; q < (nel - sh_blocks) * mts; q += grid * kWarps) {
      const int el = els[sh_blocks + q / mts], m0 = (q % mts) * 16, d = el & 511, s0 = (el >> 9) & 511, n = el >> 20;
      float v[2];
      lora_h(a.exA + static_cast<size_t>(dist[d]) * r * a.I, m0, slots[s0 + min(g >> 1, n - 1)], v);
      if (tig < n) {
        float* t = a.tex + static_cast<size_t>(slots[s0 + tig]) * r;
        if (m0 + g < r) t[m0 + g] = v[0];
        if (m0 + g + 8 < r) t[m0 + g + 8] = v[1];
      }
    }
    grid_arrive(a, B_EXDOWN);
  }
  float* td = reinterpret_cast<float*>(sm + S.td);
  if (a.shA[2]) {
    for (int q = kWarps - 1 - warp; q < sh_blocks * mts; q += kWarps) {
      const int t0 = (q / mts) * kSlotBlock, m0 = (q % mts) * 16;
      float v[2];
      lora_h(a.shA[2], m0, TK + min(t0 + (g >> 1), T - 1), v);
      if (t0 + tig < T) {
        if (m0 + g < r) td[(t0 + tig) * kMaxR + m0 + g] = v[0];
        if (m0 + g + 8 < r) td[(t0 + tig) * kMaxR + m0 + g + 8] = v[1];
      }
    }
  }

  // --------------------------------------------------------------------------- down projections
  const int NS = TK + T, RS = nrt * kTileRows;  // y [W][slot][RS]
  int Wd = 1;
  while (Wd < 8 && nrt * nel * Wd * 2 <= kWarps && G2 >= 2 * Wd) Wd *= 2;
  {
    const int teams = kWarps / Wd, team = warp / Wd, wi = warp % Wd;
    const int g0 = wi * G2 / Wd, g1 = (wi + 1) * G2 / Wd;
    for (int i = team; i < nrt * nel; i += teams) {
      const int rt = i / nel, el = els[i - rt * nel], d = el & 511, s0 = (el >> 9) & 511, n = el >> 20, s = i % S.nsd;
      const int cs = min(g >> 1, n - 1);
      const int pos = d == 511 ? TK + s0 + cs : slots[s0 + cs];
      const uint8_t* col = hb + (static_cast<size_t>(pos) * 2 + (g & 1)) * hrow;
      const uint8_t* ra = ring + s * S.stage_d + g * S.sd;
      const uint8_t* rb = ra + 8 * S.sd;
      const bool ones = g == 7;  // row 15
      if (ones) rb = ra;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      ring_wait(wt, turn_d, full_d, i, S.nsd);
#pragma unroll 4
      for (int gi = g0; gi < g1; ++gi) {
        const BFrag f = b_frag_l2(col, gi, tig);
        const uint2 wa = *reinterpret_cast<const uint2*>(ra + gi * 32 + tig * 8);
        const uint2 wb = *reinterpret_cast<const uint2*>(rb + gi * 32 + tig * 8);
        const float sc0 = half_at(ra + a.I / 2 + 2 * gi), b0 = half_at(ra + a.I / 2 + 2 * (G2 + gi));
        const float sc1 = half_at(rb + a.I / 2 + 2 * gi), b1 = half_at(rb + a.I / 2 + 2 * (G2 + gi));
        // codes times 2^-22 (and 16 of that).  The MMA aligns its products by their exponents, and a subnormal counts
        // with the smallest one, so two more of the mantissa's bits in use keep two more of h's 11 in the sum
        // (u's 8 fit either way): 3e-6 of the result against 7e-7.
        const uint32_t lo = 0x003C003Cu, hi = 0x03C003C0u;
        const uint32_t p0 = wa.x << 2, p1 = wa.x >> 6, p2 = wa.y << 2, p3 = wa.y >> 6;
        const uint32_t q0 = wb.x << 2, q1 = wb.x >> 6, q2 = wb.y << 2, q3 = wb.y >> 6;
        const uint32_t one = 0x3C003C00u, sixteen = 0x4C004C00u;  // row 15: the plain sum (odd entries are / 16)
        float dd[4] = {0.f, 0.f, 0.f, 0.f};
        mma16(dd, p0 & lo, ones ? one : q0 & lo, p0 & hi, ones ? sixteen : q0 & hi, f.x.x, f.x.y);
        mma16(dd, p1 & lo, ones ? one : q1 & lo, p1 & hi, ones ? sixteen : q1 & hi, f.x.z, f.x.w);
        mma16(dd, p2 & lo, ones ? one : q2 & lo, p2 & hi, ones ? sixteen : q2 & hi, f.y.x, f.y.y);
        mma16(dd, p3 & lo, ones ? one : q3 & lo, p3 & hi, ones ? sixteen : q3 & hi, f.y.z, f.y.w);
        const float u0 = __shfl_sync(0xffffffffu, dd[2], 28 + tig) * 0x1p-22f;
        const float u1 = __shfl_sync(0xffffffffu, dd[3], 28 + tig) * 0x1p-22f;
        acc[0] = fmaf(b0, u0, fmaf(sc0, dd[0], acc[0]));
        acc[1] = fmaf(b0, u1, fmaf(sc0, dd[1], acc[1]));
        acc[2] = fmaf(b1, u0, fmaf(sc1, dd[2], acc[2]));
        acc[3] = fmaf(b1, u1, fmaf(sc1, dd[3], acc[3]));
      }
      if (tig < n) {
        const int p = d == 511 ? TK + s0 + tig : slots[s0 + tig];
        float* y = scratch + (wi * NS + p) * RS + rt * kTileRows;
        y[g] = fmaf(acc[1], 0x1p-11f, acc[0]) * 0x1p22f;
        if (!ones) y[g + 8] = fmaf(acc[3], 0x1p-11f, acc[2]) * 0x1p22f;
      }
      team_sync(team, Wd);
      if (wi == 0 && lane == 0) bar_arrive(empty_d + s);
    }
  }
  if (a.exA)
    grid_wait(a, B_EXDOWN, wt);
  else
    cta_sync();

  // --------------------------------------------------------------------------- combine
  for (int i = tid; i < T * ndr; i += kComp) {
    const int t = i / ndr, row = i - t * ndr, rt = row / rt_rows, o = rt * kTileRows + row - rt * rt_rows;
    const int hr = dr0 + row;
    auto y_of = [&](int pos) {
      float v = 0.f;
      for (int w = 0; w < Wd; ++w) v += scratch[(w * NS + pos) * RS + o];
      return v;
    };
    float v = 0.f;
    for (int k = 0; k < K; ++k) {
      const int s = t * K + k;
      float y = y_of(s);
      if (a.exA)
        y = fmaf(a.lora_scale, dot_r(a.exB + (static_cast<size_t>(sel[s]) * a.H + hr) * r, a.tex + static_cast<size_t>(s) * r, r), y);
      v = fmaf(sw[s], y, v);
    }
    float y = y_of(TK + t);
    if (a.shA[2]) {
      float l = 0.f;
      for (int k = 0; k < r; ++k) l = fmaf(half_bits_to_float(a.shB[2][static_cast<size_t>(hr) * r + k]), td[t * kMaxR + k], l);
      y = fmaf(a.lora_scale, l, y);
    }
    v = fmaf(gate[t], y, v);
    const size_t at = static_cast<size_t>(t) * a.H + hr;
    if (a.out_mode == 1)
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    else if (a.out_mode == 2)
      static_cast<float*>(a.out)[at] += v;
    else
      static_cast<float*>(a.out)[at] = v;
  }
}

}  // namespace ld
}  // namespace moe
