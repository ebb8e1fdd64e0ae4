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
// nibble IS the code times a power of two, exactly, without a conversion: times
// 2^-22 in bits 2..5 of each half, times 2^-18 in bits 6..9.  A word's four half
// pairs are (q_j, q_{j+4}), "pair order", and the other operand is stored in the
// same order.
//
// Where in the mantissa matters: the MMA aligns its products by their exponents and
// a subnormal counts with the smallest one, so a code's leading zeros are bits lost at
// the other end of the sum.  Gate/up takes a word's even pairs at 2^-22 and its odd
// ones at 2^-18 (two shifts and four masks for 8 codes; the images' odd pairs are stored
// / 16); down, whose columns have 11 bits and not 8, takes all four at 2^-18 (four
// shifts).  Gate/up at 2^-24 and 2^-20 (one shift) and down as gate/up is now leave the
// layer's output off by 6e-7 to 1.1e-6 of its size instead of 3e-7 to 6e-7, and are 0 to
// 3 % faster (35B shape, 1 / 16 / 32 tokens in a graph: 21.9 / 51.3 / 93 us, 22.2 / 51.8 / 94).
//
// Precision.  u (bf16, 8 significant bits) is exact in fp16 after scaling each token
// by a power of two that puts its largest entry in [2^9, 2^10) (entries under 2^-22 of
// it lose bits: 2^-30 of it at most); hidden values h are stored as two fp16 numbers, hi
// and 2^11 (h - hi), 22 bits together, in two columns of the N side.  They are stored
// unscaled: below 2^-14 what stays is an absolute 2^-36.  A power of two for each row
// would need the row's largest value, which only another exchange between all CTAs gives
// (1.1 us and more of 22), and normed tokens have no hidden vectors that small (unless
// mean(x^2) is far below eps).
// Products are exact, group sums and everything after are fp32.
//
// What bounds it (B200, 35B shape): waiting.  One token, 22 us: the chain of steps; 9.7 MB of weights take 1.5 us.  Up to
// 4 tokens without routed adapters pass two grid barriers (logits, hidden values), each 1.1 us from arrival to departure
// and a trip to L2 for the data behind it; images 2.5, router rows 1.6, shared gate/up 0.9, top-K with its barrier 3.2,
// gate/up 3.6, down with its barrier 4.1, combine 1.8.  16 tokens, 52 us (103 MB, 16 us at copy speed), and 32, 93 us:
// gate/up 18 and down 15 us of 16 tokens' 52.  Eight codes take six to eight half-rate integer operations and two MMAs of
// which one to three of eight columns are used, but no pipe is full: issue slots 42 % busy, the integer pipe 38 %, shared
// memory and L1 29 %, the tensor pipe 11 %, DRAM a third.  Warps wait for instruction fetch, fixed latencies, barriers and
// loads about alike.  With the columns' loads left out (wrong results) the down loop is a fifth shorter (3.2 of 14.9 us),
// with the copies left out a tenth (1.3), without the decoding or the shuffles as long; bringing the weights to L2 ahead
// of time, or the columns to L1 or registers, moves it by less than a tenth each.  What would take the columns' loads
// away, hidden values read once for several row tiles, is not built.  16 warps: 8, 12, 20 and 24 take 62, 55, 54 and 55 us
// for 16 tokens.
#pragma once

#include "common.cuh"
#include "tc_primitives.cuh"

namespace moe {
namespace ld {

using tc::gtime;
using tc::sa;

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxT = 32, kMaxK = 8, kMaxSlots = kMaxT * kMaxK, kMaxE = 256, kMaxR = 32;
constexpr int kDownRows = 15;  // down: row 15 of the MMA tile sums the hidden values
constexpr int kSlotBlock = 4;  // down: slots per MMA (hi and lo columns)
constexpr int kMaxEls = kMaxSlots + kMaxT / kSlotBlock;
constexpr int kRowGroups = (4096 / 64 + kWarps - 1) / kWarps;  // groups of a row over all tokens a warp takes
constexpr int kMaxSharedPairs = 16;  // pairs of the shared expert a CTA takes
constexpr int kHeaderBytes = 256;
constexpr int kUnitBytes = 16 * 128, kSetsBytes = 1024;  // see UnitPlan
constexpr int kWarpRing = 2 * kUnitBytes + kSetsBytes;

enum Bar { B_IMAGE = 0, B_LOGITS = 1, B_EXGU = 2, B_HIDDEN = 3, B_EXDOWN = 4, kBars = 5 };

struct Smem {  // byte offsets
  int img, us, ic, scratch, sraw, sel, w, dist, start, slots, els, gate, td, red, misc, ring, total;
};

struct Header;

struct Args {
  int T, K, E, H, I, logI, logU, r;  // I = 2^logI, H / 256 = 2^logU
  uint32_t gmul, kmul;  // 2^32 / grid and 2^16 / K, rounded up
  const uint16_t* u;  // bf16 [T][H], or null: the normed x
  const float* x;     // fp32 [T][H] to norm, or null
  float eps;
  double inv_h;  // 1 / H
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
  Header* bar;
  uint8_t* img;       // [T][2H + 16]
  float* us;          // [T][G]
  float* ic;          // [T]
  float* aux;         // [T][4 + 2r]: shared gate logit, (3 unused), gate and up LoRA-A products
  uint16_t* h;        // [T K + T][2][I]
  float* tgu;         // [T K][2][r]
  float* tex;         // [T K][r]
  int* err;
  long long timeout_ns;
  int late_cta;       // test hook: this CTA starts four limits late (-1: none)
  int smem_image;     // every CTA forms the tokens' images in shared memory; else CTA t forms token t's, in img
  Smem sm;
};

MOE_DEV void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
MOE_DEV void team_sync(int team, int warps) {
  if (warps == 1)
    __syncwarp();
  else
    named_sync(1 + team, 32 * warps);
}

MOE_DEV void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a b
MOE_DEV void mma16_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

MOE_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MOE_DEV void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}
MOE_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

MOE_DEV float lo_half(uint32_t v) { return half_bits_to_float(static_cast<uint16_t>(v)); }
MOE_DEV float hi_half(uint32_t v) { return half_bits_to_float(static_cast<uint16_t>(v >> 16)); }

// ----------------------------------------------------------------------------- grid barrier
// The header of the workspace: a word per barrier, one for the CTAs that are through with every barrier, and a mark.  A
// word is a tag (48 bits, of its place and the workspace's address) over a count (16 bits).  The last CTA of a call
// leaves every count at zero, so a header whose tags all hold is ready; where one does not (a new workspace, or one that
// something else has written to) CTA 0 sets the header up: it zeroes the words whose tags hold, then writes the others, so
// that a CTA that finds every tag good, in whatever order it reads them, counts on zeros.
// A CTA that gave up waiting for the tags leaves without counting.  One whose wait at a barrier ran out goes on, makes its
// counts and takes the mark away.  If CTA 0 sets the header up after that (it was late), it wipes out counts at a barrier
// (the mark and the CTAs that are through it writes before the barriers, and a CTA counts there last), its own wait there
// runs out, and the mark goes after everything else.  The next call finds no mark and sets the header up again.
struct Header {
  unsigned long long word[kBars + 2];  // [kBars]: CTAs that are through, [kBars + 1]: the mark
};
static_assert(sizeof(Header) <= kHeaderBytes, "header");

MOE_DEV unsigned long long header_word(const Header* h, int i, unsigned count) {
  return ((0x6c617965725full ^ (reinterpret_cast<unsigned long long>(h) >> 8)) + static_cast<unsigned>(i)) << 16 | count;
}

MOE_DEV uint32_t header_holds(const Header* h) {  // a bit per word
  const volatile Header* v = h;
  unsigned long long w[kBars + 2];
#pragma unroll
  for (int i = 0; i < kBars + 2; ++i) w[i] = v->word[i];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kBars + 2; ++i) m |= static_cast<uint32_t>(w[i] >> 16 == header_word(h, i, 0) >> 16) << i;
  return m;
}

// False: this CTA gave up.
__device__ __noinline__ bool header_ready(Header* h, int* err, long long timeout_ns) {
  constexpr uint32_t kAll = (1u << (kBars + 2)) - 1;
  const uint32_t m = header_holds(h);
  if (m != kAll) {
    if (blockIdx.x == 0) {
      volatile Header* v = h;
      for (int pass = 0; pass < 2; ++pass)
        for (int i = kBars + 1; i >= 0; --i)
          if (((m >> i) & 1) == static_cast<uint32_t>(1 - pass)) {
            v->word[i] = header_word(h, i, 0);
            __threadfence();
          }
    } else {
      const long long end = gtime() + timeout_ns;
      while (header_holds(h) != kAll) {
        if (gtime() > end) {
          report(err, 5 /* MOE_ERR_TIMEOUT */);
          return false;
        }
      }
    }
  }
  return true;  // (the release with which the CTA counts keeps its counts behind these reads, so behind CTA 0's zeros)
}

// Each CTA adds one to a barrier's counter when its part is written and goes on when the counter has reached the
// grid's size.  All CTAs are resident (cooperative launch).  After a wait that ran out no wait of this CTA blocks any
// more: the call's outputs are undefined then, but every index read stays in range.
// The release on the counter covers the whole CTA's writes (they come before it by the CTA's own barrier), and the
// polls are plain reads with one acquire at the end: 1.1 us from arrival to departure on 148 CTAs, against 1.7 us with
// a full fence on either side.
MOE_DEV void grid_arrive(Header* h, int b) {
  named_sync(15, kThreads);
  if (threadIdx.x == 0)
    asm volatile("red.release.gpu.global.add.u64 [%0], 1;" ::"l"(h->word + b) : "memory");
}

__device__ __noinline__ void grid_wait(Header* h, int b, bool last, volatile int* failed, int* err,
                                       long long timeout_ns) {
  if (threadIdx.x == 0) {
    const unsigned long long *c = h->word + b, full = header_word(h, b, gridDim.x);
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(c) : "memory");
    if (v < full) {
      const long long end = gtime() + timeout_ns;
      for (;;) {
        asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(c) : "memory");
        if (v >= full || *failed) break;
        if (gtime() > end) {
          *failed = 1;
          report(err, 5 /* MOE_ERR_TIMEOUT */);
        }
      }
    }
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(c) : "memory");
    if (last) {
      volatile Header* w = h;
      if (*failed) __threadfence();
      if (atomicAdd(h->word + kBars, 1ull) == header_word(h, kBars, gridDim.x - 1)) {  // no CTA reads the counts any more
        for (int i = 0; i <= kBars; ++i) w->word[i] = header_word(h, i, 0);
      }
      if (*failed) {
        __threadfence();
        w->word[kBars + 1] = 0;
      }
    }
  }
  named_sync(15, kThreads);
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

// Eight values of a token as they are in memory: fp32, or bf16 pairs.
template <bool F32>
struct Raw8;
template <>
struct Raw8<true> {
  float4 p, q;
  MOE_DEV void load(const Args& a, size_t at) {
    p = *reinterpret_cast<const float4*>(a.x + at);
    q = *reinterpret_cast<const float4*>(a.x + at + 4);
  }
  MOE_DEV void get(float (&v)[8]) const {
    v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
  }
};
template <>
struct Raw8<false> {
  uint4 p;
  MOE_DEV void load(const Args& a, size_t at) { p = *reinterpret_cast<const uint4*>(a.u + at); }
  MOE_DEV void get(float (&v)[8]) const {
    const uint32_t s[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(s[i] << 16);
      v[2 * i + 1] = __uint_as_float(s[i] & 0xffff0000u);
    }
  }
};

// Token t's image by `warps` warps (this one is number wi): u scaled by a power of two c, fp16, pair order, odd pairs
// / 16; per group 2^-24 sum of c u; 1/c.  The squares are summed with their rounding errors (two fp32 numbers per lane),
// then in 64 bits: fp64 runs at a few lanes a cycle, and a token's 2,048 squares in it cost more than the rest of the
// image.
template <bool F32>
__device__ __noinline__ void build_image(const Args& a, int t, int wi, int warps, int team, double* red, uint8_t* row,
                                         float* us, float* ic, bool write_u) {
  const int lane = threadIdx.x & 31, nb = a.H / 8, b0 = wi * 32 + lane, step = 32 * warps;
  const size_t base = static_cast<size_t>(t) * a.H;
  constexpr int kChunk = 4;  // blocks whose loads are issued together
  float m = 0.f, s = 0.f, e2 = 0.f;
#pragma unroll 1
  for (int c0 = b0; c0 < nb; c0 += kChunk * step) {
    Raw8<F32> raw[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (c0 + i * step < nb) raw[i].load(a, base + 8 * (c0 + i * step));
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (c0 + i * step < nb) {
        float v[8];
        raw[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m = max_bits(m, fabsf(v[j]));
          if (F32) {
            const float p = v[j] * v[j], sum = s + p, z = sum - s;
            e2 += ((s - (sum - z)) + (p - z)) + fmaf(v[j], v[j], -p);
            s = sum;
          }
        }
      }
  }
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  double ss = 0.0;
  if (F32) {
    ss = static_cast<double>(s) + static_cast<double>(e2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  double* r = red + 2 * warps * team;
  if (warps > 1) {
    if (lane == 0) r[2 * wi] = ss, r[2 * wi + 1] = static_cast<double>(m);
    team_sync(team, warps);
    const bool on = lane < warps;  // each warp adds up the others' sums, a lane per warp
    m = on ? static_cast<float>(r[2 * lane + 1]) : 0.f;
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    if (F32) {
      ss = on ? r[2 * lane] : 0.0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
  }
  float rstd = 1.f;
  double rstd64 = 1.0;
  if (F32) {
    if (m > 1e15f || m < 1e-15f) {  // squares that fp32 may not hold (uniform over the team): in 64 bits
      ss = 0.0;
#pragma unroll 1
      for (int b = b0; b < nb; b += step)
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
          const double v = a.x[base + 8 * b + j];
          ss = fma(v, v, ss);
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (warps > 1) {
        team_sync(team, warps);
        if (lane == 0) r[2 * wi] = ss;
        team_sync(team, warps);
        ss = 0.0;
#pragma unroll 1
        for (int w = 0; w < warps; ++w) ss += r[2 * w];
      }
    }
    const double v = ss * a.inv_h + static_cast<double>(a.eps);  // H is a power of two
    if (v > 1e-30 && v < 1e30) {  // 1/sqrt(v): Newton's iteration from the fp32 value, 23 -> 46 -> 52 bits
      double y = rsqrtf(static_cast<float>(v));
      y = fma(0.5 * y, fma(-v * y, y, 1.0), y);
      rstd64 = fma(0.5 * y, fma(-v * y, y, 1.0), y);
    } else {
      rstd64 = 1.0 / sqrt(v);
    }
    rstd = static_cast<float>(rstd64);
    m = static_cast<float>(m * rstd64);
  }
  // c = 2^(9 - e) for m in [2^e, 2^(e+1)); 1 where m is zero or not finite
  const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
  const int ce = (m > 0.f && e < 128) ? min(max(9 - e, -126), 126) : 0;
  const float c = __uint_as_float(static_cast<uint32_t>(127 + ce) << 23);
  if (wi == 0 && lane == 0) *ic = __uint_as_float(static_cast<uint32_t>(127 - ce) << 23);
#pragma unroll 2
  for (int b = b0; b < nb; b += step) {
    {
      float v[8];
      Raw8<F32> raw;
      raw.load(a, base + 8 * b);
      raw.get(v);
      if (F32) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint16_t q = normed_bf16(v[j], rstd, rstd64);
          v[j] = bf16_bits_to_float(q);
          if (j & 1)
            o[j >> 1] |= static_cast<uint32_t>(q) << 16;
          else
            o[j >> 1] = q;
        }
        if (write_u && a.u_out)
          *reinterpret_cast<uint4*>(a.u_out + base + 8 * b) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] *= c;
        sum += v[j];
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
}

// ----------------------------------------------------------------------------- int4 units
// The unit of weight traffic and of work: the codes of 16 rows x 4 groups (2 where a row has only 2), brought by one
// warp into its own buffers with cp.async and used by that warp alone: no barrier is needed between copy and use, and
// each warp has two units of 2 KB, one in use and one in flight (a third takes L1 away from the token images: 62 us
// against 57 for 16 tokens of the 35B shape, when there were 24 warps).  16-byte chunk c of row m lies at place
// c ^ 2 (m % 4) of the row's 128 bytes, so that the 8-byte fragment reads of 4 rows fall on different banks.  The scales
// and biases come for two units at a time (16 bytes each of a row) into sets of their own, [16 rows][scales, biases].
// Row m of a unit is record (m % 8) * step_lo + (m / 8) * step_hi: gate rows over up rows for gate/up (2, 1), rows in
// order for down (1, 8).
struct UnitPlan {  // a lane's places: bytes from the unit's first record (its chunk of row lane/8; its scales)
  uint32_t c0, c4, c8, c12, s;
  int piece;  // bytes of scales (as of biases) of a row in a set, 16 or 8 places apart
  bool on;
  MOE_DEV int half() const { return piece == 16 ? 16 : 8; }
  MOE_DEV int set_bytes() const { return 32 * half(); }
  MOE_DEV void make(int rec, int G, int step_lo, int step_hi) {
    const int lane = threadIdx.x & 31, q = lane >> 3, ch = lane & 7, m = lane >> 1;
    on = ch < (G >= 4 ? 8 : 2 * G);
    c0 = q * step_lo * rec + 16 * ch;
    c4 = c0 + 4 * step_lo * rec;
    c8 = c0 + step_hi * rec;
    c12 = c4 + step_hi * rec;
    piece = G >= 8 ? 16 : 2 * G;
    s = ((m & 7) * step_lo + (m >> 3) * step_hi) * rec + G * 32 + 2 * G * (lane & 1);
  }
};

// The codes of unit u of the records at base; lo and hi rows of each half exist.
MOE_DEV void issue_codes(uint32_t buf, const UnitPlan& p, const uint8_t* base, int u, int lo, int hi) {
  const int lane = threadIdx.x & 31, q = lane >> 3;
  auto cp16 = [](uint32_t d, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  };
  const uint32_t d = buf + q * 128 + 16 * ((lane & 7) ^ 2 * q);  // q + 4, + 8, + 12: the same places
  base += 128 * u;
  if (p.on) {
    if (q < lo) cp16(d, base + p.c0);
    if (q + 4 < lo) cp16(d + 4 * 128, base + p.c4);
    if (q < hi) cp16(d + 8 * 128, base + p.c8);
    if (q + 4 < hi) cp16(d + 12 * 128, base + p.c12);
  }
}

// The scales and biases of units u and u ^ 1.
MOE_DEV void issue_scales(uint32_t set, const UnitPlan& p, const uint8_t* base, int u, int lo, int hi) {
  const int lane = threadIdx.x & 31, m = lane >> 1;
  const uint32_t d = set + p.half() * lane;
  base += p.s + 16 * (u >> 1);
  if ((m & 7) < (m < 8 ? lo : hi)) {
    if (p.piece == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(base) : "memory");
    else if (p.piece == 8)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(base) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(base) : "memory");
  }
}

struct Frag {  // the N side of one group: a lane's 8-blocks 2 tig and 2 tig + 1
  uint4 x, y;
};

MOE_DEV Frag load_frag(const uint8_t* col, int i) {
  const uint4* p = reinterpret_cast<const uint4*>(col + i * 128 + (threadIdx.x & 3) * 32);
  return {p[0], p[1]};
}

// acc += 2^-22 of one unit of gate/up rows times 8 columns (ua, ub: 2^-24 of the groups' sums), two groups at a time (four
// would take half as many warps again in registers).
MOE_DEV void gate_up_unit(const uint8_t* buf, const uint8_t* set, int half, const uint8_t* col, const float* ua, const float* ub,
                          float (&acc)[4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  // chunk 2 i + tig / 2 of row g (and g + 8)
  const uint8_t* ra = buf + g * 128 + 8 * (tig & 1);
  const int ch = (tig >> 1) ^ 2 * (g & 3);
  const uint32_t lo = 0x003C003Cu, hi = 0x03C003C0u;
  const uint8_t* sp = set + 2 * half * g;
  const uint2 sa2 = *reinterpret_cast<const uint2*>(sp), ba2 = *reinterpret_cast<const uint2*>(sp + half);
  const uint2 sb2 = *reinterpret_cast<const uint2*>(sp + 16 * half), bb2 = *reinterpret_cast<const uint2*>(sp + 17 * half);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float d[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Frag f = load_frag(col, 2 * h + i);
      const uint8_t* w = ra + 16 * (ch ^ (4 * h + 2 * i));
      const uint2 wa = *reinterpret_cast<const uint2*>(w), wb = *reinterpret_cast<const uint2*>(w + 1024);
      const uint32_t p0 = wa.x << 2, p1 = wa.x >> 6, p2 = wa.y << 2, p3 = wa.y >> 6;
      const uint32_t q0 = wb.x << 2, q1 = wb.x >> 6, q2 = wb.y << 2, q3 = wb.y >> 6;
      mma16_0(d[i], p0 & lo, q0 & lo, p0 & hi, q0 & hi, f.x.x, f.x.y);
      mma16(d[i], p1 & lo, q1 & lo, p1 & hi, q1 & hi, f.x.z, f.x.w);
      mma16(d[i], p2 & lo, q2 & lo, p2 & hi, q2 & hi, f.y.x, f.y.y);
      mma16(d[i], p3 & lo, q3 & lo, p3 & hi, q3 & hi, f.y.z, f.y.w);
    }
    const uint32_t s0 = h ? sa2.y : sa2.x, b0 = h ? ba2.y : ba2.x, s1 = h ? sb2.y : sb2.x, b1 = h ? bb2.y : bb2.x;
    const float2 u = *reinterpret_cast<const float2*>(ua + 2 * h), v = *reinterpret_cast<const float2*>(ub + 2 * h);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float p = i ? hi_half(s0) : lo_half(s0), q = i ? hi_half(b0) : lo_half(b0);
      const float r = i ? hi_half(s1) : lo_half(s1), t = i ? hi_half(b1) : lo_half(b1), ui = 4.f * (i ? u.y : u.x), vi = 4.f * (i ? v.y : v.x);
      acc[0] = fmaf(q, ui, fmaf(p, d[i][0], acc[0]));
      acc[1] = fmaf(q, vi, fmaf(p, d[i][1], acc[1]));
      acc[2] = fmaf(t, ui, fmaf(r, d[i][2], acc[2]));
      acc[3] = fmaf(t, vi, fmaf(r, d[i][3], acc[3]));
    }
  }
}

// acc += one unit of down rows (15 of them; row 15 holds code 15 everywhere: 15 times the columns' sums) times the 8
// columns (hi and lo of 4 slots).
MOE_DEV void down_unit(const uint8_t* buf, const uint8_t* set, int half, Frag f0, Frag f1, const uint8_t* col, bool whole,
                       float (&acc)[4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const uint8_t* ra = buf + g * 128 + 8 * (tig & 1);
  const int ch = (tig >> 1) ^ 2 * (g & 3);
  const uint32_t top = 0x03C003C0u;
  Frag f2 = f0, f3 = f1;
  if (whole) f2 = load_frag(col, 2), f3 = load_frag(col, 3);
  const uint8_t *sp = set + 2 * half * g, *sq = sp + 16 * half;
  const uint2 sa2 = *reinterpret_cast<const uint2*>(sp), ba2 = *reinterpret_cast<const uint2*>(sp + half);
  const uint2 sb2 = *reinterpret_cast<const uint2*>(sq), bb2 = *reinterpret_cast<const uint2*>(sq + half);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h && !whole) break;  // a row of two groups
    float d[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Frag& f = h ? (i ? f3 : f2) : (i ? f1 : f0);
      const uint8_t* w = ra + 16 * (ch ^ (4 * h + 2 * i));
      const uint2 wa = *reinterpret_cast<const uint2*>(w), wb = *reinterpret_cast<const uint2*>(w + 1024);
      auto four = [&](float (&o)[4], bool first, uint32_t x, uint32_t y, uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
        const uint32_t a0 = (x << 6) & top, a1 = (y << 6) & top, a2 = (x << 2) & top, a3 = (y << 2) & top;
        if (first)
          mma16_0(o, a0, a1, a2, a3, b0, b1);
        else
          mma16(o, a0, a1, a2, a3, b0, b1);
        mma16(o, (x >> 2) & top, (y >> 2) & top, (x >> 6) & top, (y >> 6) & top, b2, b3);
      };
      four(d[i], true, wa.x, wb.x, f.x.x, f.x.y, f.x.z, f.x.w);
      four(d[i], false, wa.y, wb.y, f.y.x, f.y.y, f.y.z, f.y.w);
    }
    const uint32_t s0 = h ? sa2.y : sa2.x, b0 = h ? ba2.y : ba2.x, s1 = h ? sb2.y : sb2.x, b1 = h ? bb2.y : bb2.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float u = __shfl_sync(0xffffffffu, d[i][2], 28 + tig) * (1.f / 15.f);
      const float v = __shfl_sync(0xffffffffu, d[i][3], 28 + tig) * (1.f / 15.f);
      const float p = i ? hi_half(s0) : lo_half(s0), q = i ? hi_half(b0) : lo_half(b0);
      const float r = i ? hi_half(s1) : lo_half(s1), t = i ? hi_half(b1) : lo_half(b1);
      acc[0] = fmaf(q, u, fmaf(p, d[i][0], acc[0]));
      acc[1] = fmaf(q, v, fmaf(p, d[i][1], acc[1]));
      acc[2] = fmaf(t, u, fmaf(r, d[i][2], acc[2]));
      acc[3] = fmaf(t, v, fmaf(r, d[i][3], acc[3]));
    }
  }
}

// ----------------------------------------------------------------------------- hidden values, adapters
// Hidden value j of row `row` of the hidden buffer, as hi and lo.
MOE_DEV void store_h(const Args& a, int row, int j, float x, float y) {
  const float v = silu(x) * y;
  if (fabsf(v) > kF16Max && fabsf(v) <= 3.402823466e38f) report(a.err, 6 /* MOE_ERR_RANGE */);
  const __half hi = __float2half_rn(v);
  const __half lo = __float2half_rn((v - __half2float(hi)) * 2048.f);
  uint16_t* p = a.h + static_cast<size_t>(row) * 2 * a.I + pair_pos(j);
  p[0] = __half_as_ushort(hi);
  p[a.I] = __half_as_ushort(lo);
}

// sum_i B[i] t[i], r a multiple of 8, both 16-byte aligned.
__device__ __noinline__ float dot_r(const uint16_t* B, const float* t, int r) {
  float v = 0.f;
#pragma unroll 2
  for (int i = 0; i < r; i += 8) {
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(B + i));
    const float4 p = *reinterpret_cast<const float4*>(t + i), q = *reinterpret_cast<const float4*>(t + i + 4);
    v = fmaf(lo_half(b.x), p.x, v);
    v = fmaf(hi_half(b.x), p.y, v);
    v = fmaf(lo_half(b.y), p.z, v);
    v = fmaf(hi_half(b.y), p.w, v);
    v = fmaf(lo_half(b.z), q.x, v);
    v = fmaf(hi_half(b.z), q.y, v);
    v = fmaf(lo_half(b.w), q.z, v);
    v = fmaf(hi_half(b.w), q.w, v);
  }
  return v;
}

// Rows g and g + 8 of an fp16 matrix (row pointers) over groups [g0, g1) times 8 columns in pair order; what the odd
// pairs of a column are stored divided by (images: 16, hidden values: 1).
MOE_DEV void f16_rows(const uint16_t* ra, const uint16_t* rb, int g0, int g1, const uint8_t* col, float odd, float (&v)[4]) {
  const int tig = threadIdx.x & 3;
  float ev[4] = {0.f, 0.f, 0.f, 0.f}, od[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int gi = g0; gi < g1; ++gi) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4* bp = reinterpret_cast<const uint4*>(col + gi * 128 + tig * 32) + h;
      const uint4 b = *bp;
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(ra + gi * 64 + tig * 16) + h);
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(rb + gi * 64 + tig * 16) + h);
      mma16(ev, prmt(x.x, x.z, 0x5410), prmt(y.x, y.z, 0x5410), prmt(x.y, x.w, 0x5410), prmt(y.y, y.w, 0x5410), b.x, b.z);
      mma16(od, prmt(x.x, x.z, 0x7632), prmt(y.x, y.z, 0x7632), prmt(x.y, x.w, 0x7632), prmt(y.y, y.w, 0x7632), b.y, b.w);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = fmaf(odd, od[i], ev[i]);
}

// ----------------------------------------------------------------------------- top-K and gating of one token (a warp)
__device__ __noinline__ void route_token(const Args& a, int t, int* sel, float* sw, uint32_t* mask) {
  const int lane = threadIdx.x & 31, K = a.K;
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
  uint32_t my_k = 0;
#pragma unroll 1
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (key[i] > best) best = key[i], bi = i;
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int e =
        static_cast<int>(__reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(lane + 32 * bi) : 0xffffu));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e == lane + 32 * i) key[i] = 0;
    if (lane == k) my_e = min(e, a.E - 1), my_k = top;
  }
  const bool write = blockIdx.x == 0;
  if (lane < K && write) a.idx[t * K + lane] = my_e;
  if (a.exec_idx && lane < K) my_e = min(max(a.exec_idx[t * K + lane], 0), a.E - 1);
  float l = -INFINITY;
  if (lane < K) {
    if (a.exec_idx)
      l = __ldcg(lg + my_e);
    else  // the logit back from its key
      l = my_k == 1u ? __uint_as_float(0x7fc00000u) : __uint_as_float(my_k ^ ((my_k >> 31) ? 0x80000000u : 0xffffffffu));
  }
  float mx = l;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ex = lane < K ? expf(l - mx) : 0.f;
  float den = ex;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  if (lane < K) {
    const int s = t * K + lane;
    sel[s] = my_e;
    sw[s] = ex / den;
    atomicOr(mask + (s >> 5) * kMaxE + my_e, 1u << (s & 31));
    if (write) a.w[s] = ex / den;
  }
}

// Where the part of CTA c of n things split over the grid begins: c n / grid, with gmul = 2^32 / grid rounded up.
// (Neighbours agree on the border whatever the rounding; at c = grid it is n for every n up to 2^19.)
MOE_DEV int share(int c, int n, uint32_t gmul) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(c) * static_cast<uint32_t>(n)) * gmul) >> 32);
}

// ----------------------------------------------------------------------------- the kernel
__global__ void __launch_bounds__(kThreads, 1) layer_decode_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) uint8_t sm[];
  const Smem& S = a.sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tig = lane & 3;
  const int cta = blockIdx.x, grid = gridDim.x;
  const int T = a.T, K = a.K, TK = T * K, G = a.H / 64, ldu = 2 * a.H + 16, r = a.r;
  const int U = G / 4, G2 = a.I / 64, U2 = G2 < 4 ? 1 : G2 / 4;
  int* misc = reinterpret_cast<int*>(sm + S.misc);  // [0] failed, [1] distinct experts, [2] down elements, [4..19] sums
  int* sel = reinterpret_cast<int*>(sm + S.sel);
  float* sw = reinterpret_cast<float*>(sm + S.w);
  int* dist = reinterpret_cast<int*>(sm + S.dist);
  int* start = reinterpret_cast<int*>(sm + S.start);
  int* slots = reinterpret_cast<int*>(sm + S.slots);  // slot | token << 16
  int* els = reinterpret_cast<int*>(sm + S.els);
  float* scratch = reinterpret_cast<float*>(sm + S.scratch);
  float* sraw = reinterpret_cast<float*>(sm + S.sraw);
  uint8_t* ring = sm + S.ring + warp * kWarpRing;  // codes, then sets of scales
  uint8_t* sets = ring + 2 * kUnitBytes;

  // this CTA's shares: pairs of the shared expert, rows of the down projections, rows over all tokens
  const int sp0 = share(cta, a.I, a.gmul), nsp = share(cta + 1, a.I, a.gmul) - sp0, nst = (nsp + 7) / 8;
  const int dr0 = share(cta, a.H, a.gmul), ndr = share(cta + 1, a.H, a.gmul) - dr0;
  const int nrt = (ndr > 0) + (ndr > kDownRows), rt_rows = nrt > 1 ? (ndr + 1) / 2 : ndr;  // row tiles, rows of one
  const int RGU = qrow_bytes(a.H, 4), RDN = qrow_bytes(a.I, 4), R8 = qrow_bytes(a.H, 8);
  const size_t dn_off = static_cast<size_t>(2 * a.I) * RGU;
  const int sh_blocks = (T + kSlotBlock - 1) / kSlotBlock;
  const int nA = (a.shA[0] ? r : 0) + (a.shA[1] ? r : 0);
  const int nrows = a.E + 1 + nA, r0 = share(cta, nrows, a.gmul), r1 = share(cta + 1, nrows, a.gmul);
  const int n8 = max(0, min(r1, a.E + 1) - r0);  // 8-bit rows r0 .. r0 + n8 - 1, then fp16 rows
  const int nblk = (T + 7) / 8;

  if (tid == kThreads - 32) {
    if (cta == a.late_cta)
      for (const long long end = gtime() + 4 * a.timeout_ns; gtime() < end;) __nanosleep(1000);
    misc[0] = header_ready(a.bar, a.err, a.timeout_ns) ? 0 : 1;
  }
  // --------------------------------------------------------------------------- weights that no token decides
  // The first shared tile's units: unit warp % U for token blocks warp / U, + sh_n, ...
  const uint32_t ring32 = sa(ring), sets32 = sa(sets);
  const int sh_ways = max(1, min(nblk, kWarps >> a.logU));
  UnitPlan plan;
  plan.make(RGU, G, 2, 1);
  {
    const uint8_t* src = a.shared + static_cast<size_t>(2 * sp0) * RGU;
    const int u = warp & (U - 1), n = min(8, nsp);
    if (nst > 0 && warp < U * sh_ways) {
      issue_codes(ring32, plan, src, u, n, n);
      issue_scales(sets32, plan, src, u, n, n);
    }
    cp_commit();
  }
  const int g0 = warp * G / kWarps, g1 = (warp + 1) * G / kWarps;  // groups of the rows over all tokens
  uint4 q8[kRowGroups];
  uint32_t sb8[kRowGroups];  // scale and bias
  if (n8 > 0) {
    const int row = r0 + min(g, n8 - 1);
    const uint8_t* rec = row < a.E ? a.router + static_cast<size_t>(row) * R8 : a.sgate;
#pragma unroll
    for (int i = 0; i < kRowGroups; ++i)
      if (g0 + i < g1) {
        q8[i] = __ldg(reinterpret_cast<const uint4*>(rec + (g0 + i) * 64 + tig * 16));
        const uint16_t* p = reinterpret_cast<const uint16_t*>(rec + a.H) + g0 + i;
        sb8[i] = __ldg(p) | static_cast<uint32_t>(__ldg(p + G)) << 16;
      }
  }
  // adapters read later: into L2
  if (a.shA[2] && tid < r * G2) prefetch_l2(a.shA[2] + tid * 64);
  if (tid < nsp) {
    if (a.shA[0]) prefetch_l2(a.shB[0] + static_cast<size_t>(sp0 + tid) * r);
    if (a.shA[1]) prefetch_l2(a.shB[1] + static_cast<size_t>(sp0 + tid) * r);
  }
  if (a.shA[2] && tid >= 32 && tid < 32 + ndr) prefetch_l2(a.shB[2] + static_cast<size_t>(dr0 + tid - 32) * r);
  const float bias = a.rbias && r0 + warp < min(r1, a.E) ? __ldg(a.rbias + r0 + warp) : 0.f;  // of row r0 + warp
  // --------------------------------------------------------------------------- token images
  const uint8_t* img = a.smem_image ? sm + S.img : a.img;
  float* us = reinterpret_cast<float*>(sm + S.us);
  float* ic = reinterpret_cast<float*>(sm + S.ic);
  double* red = reinterpret_cast<double*>(sm + S.red);
  volatile int* failed = misc;
  auto build = [&](int t, int wi, int warps, int team, uint8_t* row, float* u, float* c, bool write_u) {
    if (a.x)
      build_image<true>(a, t, wi, warps, team, red, row, u, c, write_u);
    else
      build_image<false>(a, t, wi, warps, team, red, row, u, c, write_u);
  };
  auto gave_up = [&]() {  // on the header (the whole CTA)
    named_sync(15, kThreads);
    if (!*failed) return false;
    cp_wait<0>();
    return true;
  };
  if (!a.smem_image) {
    if (cta < T)
      build(cta, warp, kWarps, 0, a.img + static_cast<size_t>(cta) * ldu, a.us + cta * G, a.ic + cta, true);
    if (gave_up()) return;
    grid_arrive(a.bar, B_IMAGE);
    grid_wait(a.bar, B_IMAGE, false, failed, a.err, a.timeout_ns);
#pragma unroll 1
    for (int i = tid; i < T * G; i += kThreads) us[i] = __ldcg(a.us + i);
    if (tid < T) ic[tid] = __ldcg(a.ic + tid);
    named_sync(15, kThreads);
  } else {
    int logW = 0;  // at most 4 tokens
    while (T << (logW + 1) <= kWarps) ++logW;
    const int W = 1 << logW, team = warp >> logW;
    if (team < T)
      build(team, warp & (W - 1), W, team, sm + S.img + team * ldu, us + team * G, ic + team, team == cta);
    if (gave_up()) return;
  }

  // --------------------------------------------------------------------------- rows over all tokens: router, shared
  // gate (8 bits), the shared expert's gate and up LoRA A (fp16)
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const int first = kind ? r0 + n8 : r0, n = kind ? r1 - first : n8;
    if (n <= 0) continue;
    const int row = first + min(g, n - 1);
#pragma unroll 2
    for (int b = 0; b < nblk; ++b) {
      const uint8_t* col = img + static_cast<size_t>(min(8 * b + g, T - 1)) * ldu;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (kind == 0) {
        const float* ua = us + min(8 * b + 2 * tig, T - 1) * G;
        const float* ub = us + min(8 * b + 2 * tig + 1, T - 1) * G;
#pragma unroll
        for (int i = 0; i < kRowGroups; ++i) {
          const int gi = g0 + i;
          if (gi < g1) {
            const uint4* p = reinterpret_cast<const uint4*>(col + gi * 128 + tig * 32);
            const uint4 x = p[0], y = p[1], q = q8[i];
            float ev[4] = {0.f, 0.f, 0.f, 0.f}, od[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t m = 0x00FF00FFu;
            mma16(ev, prmt(q.x, q.y, 0x4400) & m, 0, prmt(q.x, q.y, 0x6622) & m, 0, x.x, x.z);
            mma16(od, prmt(q.x, q.y, 0x5511) & m, 0, prmt(q.x, q.y, 0x7733) & m, 0, x.y, x.w);
            mma16(ev, prmt(q.z, q.w, 0x4400) & m, 0, prmt(q.z, q.w, 0x6622) & m, 0, y.x, y.z);
            mma16(od, prmt(q.z, q.w, 0x5511) & m, 0, prmt(q.z, q.w, 0x7733) & m, 0, y.y, y.w);
            const float s = lo_half(sb8[i]), o = hi_half(sb8[i]);
            v[0] = fmaf(o, ua[gi], fmaf(s, fmaf(16.f, od[0], ev[0]), v[0]));
            v[1] = fmaf(o, ub[gi], fmaf(s, fmaf(16.f, od[1], ev[1]), v[1]));
          }
        }
      } else {
        const int j = row - (a.E + 1);  // gate's rows, then up's
        const uint16_t* A = (a.shA[0] && j < r) ? a.shA[0] + static_cast<size_t>(j) * a.H
                                                : a.shA[1] + static_cast<size_t>(a.shA[0] ? j - r : j) * a.H;
        f16_rows(A, A, g0, g1, col, 16.f, v);
      }
      if (g < n) *reinterpret_cast<float2*>(scratch + ((warp * 4 + b) * 8 + g) * 8 + 2 * tig) = make_float2(v[0], v[1]);
    }
    named_sync(15, kThreads);
    {  // one thread per (row, token): up to 8 rows x 32 tokens
      const int q = tid >> 5, t = tid & 31;
      if (q < n && t < T) {
        float v = 0.f;
#pragma unroll 4
        for (int w = 0; w < kWarps; ++w) v += scratch[((w * 4 + (t >> 3)) * 8 + q) * 8 + (t & 7)];
        v *= ic[t];
        const int j = first + q;
        if (j < a.E)
          a.logits[static_cast<size_t>(t) * a.E + j] = v * 0x1p24f + bias;  // kind 0: row r0 + warp
        else if (j == a.E)
          a.aux[t * (4 + 2 * r)] = v * 0x1p24f;
        else
          a.aux[t * (4 + 2 * r) + 4 + j - (a.E + 1)] = v;
      }
    }
    named_sync(15, kThreads);
  }
  grid_arrive(a.bar, B_LOGITS);

  // --------------------------------------------------------------------------- shared expert's gate/up, raw
#pragma unroll 1
  for (int ti = 0; ti < nst; ++ti) {
#pragma unroll 1
    for (int task = warp; task < U * sh_ways; task += kWarps) {
      const int u = task & (U - 1);
      if (ti > 0 || task >= kWarps) {
        const uint8_t* src = a.shared + static_cast<size_t>(2 * (sp0 + 8 * ti)) * RGU;
        const int n = min(8, nsp - 8 * ti);
        issue_codes(ring32, plan, src, u, n, n);
        issue_scales(sets32, plan, src, u, n, n);
        cp_commit();
      }
      cp_wait<0>();
#pragma unroll 1
      for (int b = task >> a.logU; b < nblk; b += sh_ways) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        gate_up_unit(ring, sets + (U > 1 ? 8 * (u & 1) : 0), plan.half(), img + static_cast<size_t>(min(8 * b + g, T - 1)) * ldu + u * 512,
                     us + min(8 * b + 2 * tig, T - 1) * G + 4 * u, us + min(8 * b + 2 * tig + 1, T - 1) * G + 4 * u, acc);
        *reinterpret_cast<float4*>(scratch + ((b * U + u) * 32 + lane) * 4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      }
      __syncwarp();
    }
    named_sync(15, kThreads);
    if (warp < nblk) {  // block `warp`: (pair g, tokens 2 tig and 2 tig + 1)
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int u = 0; u < U; ++u) {
        const float4 p = *reinterpret_cast<const float4*>(scratch + ((warp * U + u) * 32 + lane) * 4);
        v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
      }
      const int t = 8 * warp + 2 * tig, pr = 8 * ti + g;
      if (pr < nsp) {
        float2* o = reinterpret_cast<float2*>(sraw) + pr;
        if (t < T) o[t * 16] = make_float2(v.x * 0x1p22f * ic[t], v.z * 0x1p22f * ic[t]);
        if (t + 1 < T) o[(t + 1) * 16] = make_float2(v.y * 0x1p22f * ic[t + 1], v.w * 0x1p22f * ic[t + 1]);
      }
    }
    named_sync(15, kThreads);
  }

  // --------------------------------------------------------------------------- top-K, gating, the expert list
  uint32_t* mask = reinterpret_cast<uint32_t*>(scratch);  // [8 words][256 experts]: the slots that chose an expert
  for (int i = tid; i < kMaxE * 2; i += kThreads) reinterpret_cast<uint4*>(mask)[i] = make_uint4(0, 0, 0, 0);
  grid_wait(a.bar, B_LOGITS, false, failed, a.err, a.timeout_ns);
#pragma unroll 1
  for (int t = warp; t < T; t += kWarps) route_token(a, t, sel, sw, mask);
  float* gate = reinterpret_cast<float*>(sm + S.gate);
  if (tid >= kThreads - 32 && lane < T) gate[lane] = sigmoid(__ldcg(a.aux + lane * (4 + 2 * r)));
  named_sync(15, kThreads);
  if (warp < 8) {  // chosen experts in ascending order, their slots in ascending order, the down elements
    uint32_t m[8];
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = 32 * i < TK ? mask[i * kMaxE + tid] : 0u;
      cnt += __popc(m[i]);
    }
    const uint32_t bal = __ballot_sync(0xffffffffu, cnt > 0);
    // slots | elements << 10 | experts << 20, summed over the experts before
    const int own = cnt | ((cnt + kSlotBlock - 1) / kSlotBlock) << 10;
    int v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    int* tot = misc + 4;  // [8]
    if (lane == 31) tot[warp] = v + (__popc(bal) << 20);
    named_sync(1, 256);
    int off = v - own + (__popc(bal & ((1u << lane) - 1)) << 20);
#pragma unroll
    for (int w = 0; w < 7; ++w) off += w < warp ? tot[w] : 0;
    const int d = off >> 20;
    int so = off & 1023, eo = sh_blocks + ((off >> 10) & 1023);
    if (cnt > 0) {
      dist[d] = tid;
      start[d] = so;
#pragma unroll 1
      for (int b = 0; b < cnt; b += kSlotBlock) els[eo++] = d | (so + b) << 9 | min(kSlotBlock, cnt - b) << 20;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll 1
        for (uint32_t q = m[i]; q; q &= q - 1) {
          const int s = 32 * i + __ffs(q) - 1;
          slots[so++] = s | static_cast<int>(s * a.kmul >> 16) << 16;
        }
    }
    if (tid == 255) {
      const int D = d + (cnt > 0);
      misc[1] = D;
      misc[2] = sh_blocks + ((off >> 10) & 1023) + (own >> 10);
      start[D] = TK;
    }
    if (tid < sh_blocks) els[tid] = 511 | (tid * kSlotBlock) << 9 | min(kSlotBlock, T - tid * kSlotBlock) << 20;
  }
  named_sync(15, kThreads);
  const int D = misc[1], nel = misc[2];
  if (a.exA) {  // the routed down adapters: this CTA's share of A, its rows of B for every slot, into L2 for later
    const int logm = r > 16, lines = G2 * 16;  // of 16 rows of A
#pragma unroll 1
    for (int q = cta; q < (nel - sh_blocks) << logm; q += grid) {
      const uint16_t* A = a.exA + (static_cast<size_t>(dist[els[sh_blocks + (q >> logm)] & 511]) * r + 16 * (q & logm)) * a.I;
      const int n = min(lines, (r - 16 * (q & logm)) * G2);
#pragma unroll 1
      for (int i = tid; i < n; i += kThreads) prefetch_l2(A + i * 64);
    }
#pragma unroll 1
    for (int s = warp; s < TK; s += kWarps)
      if (lane < ndr) prefetch_l2(a.exB + (static_cast<size_t>(sel[s]) * a.H + dr0 + lane) * r);
  }

  // --------------------------------------------------------------------------- routed gate/up adapters: A u
  if (a.exAgu) {
    const int rows = 2 * r, total = D * rows;
#pragma unroll 1
    for (int q = cta * kWarps + warp; q < total; q += grid * kWarps) {
      const int d = q / rows, i = q - d * rows, e = dist[d];
      const uint16_t* A = a.exAgu + (static_cast<size_t>(e) * rows + i) * a.H;
#pragma unroll 1
      for (int s = start[d]; s < start[d + 1]; ++s) {
        const int sl = slots[s] & 0xffff, t = slots[s] >> 16;
        const uint8_t* row = img + static_cast<size_t>(t) * ldu;
        float v = 0.f;
#pragma unroll 1
        for (int b = lane; b < a.H / 8; b += 32) {
          const uint4 p = __ldg(reinterpret_cast<const uint4*>(A) + b), x = *reinterpret_cast<const uint4*>(row + 16 * b);
          v = dot2_mix(prmt(p.x, p.z, 0x5410), x.x, v);
          v = dot2_mix(prmt(p.y, p.w, 0x5410), x.z, v);
          float o = dot2_mix(prmt(p.x, p.z, 0x7632), x.y, 0.f);
          o = dot2_mix(prmt(p.y, p.w, 0x7632), x.w, o);
          v = fmaf(16.f, o, v);
        }
        v = warp_reduce(v);
        if (lane == 0) a.tgu[static_cast<size_t>(sl) * 2 * r + i] = v * ic[t];
      }
    }
    grid_arrive(a.bar, B_EXGU);
    grid_wait(a.bar, B_EXGU, false, failed, a.err, a.timeout_ns);
  }

  // --------------------------------------------------------------------------- chosen experts' gate/up
  // The tiles (8 pairs) of all chosen experts, one after the other, are split evenly over the CTAs; a CTA's items (tile,
  // block of 8 slots) are runs of U units each, and all its units are split evenly over the warps.  An item whose
  // units fall to several warps is joined by the one that has its first unit, after a barrier: the others leave their
  // sums in scratch (a warp has at most one item that it did not begin).
  {
    const int logt = a.logI - 3, nt = D << logt, t0 = share(cta, nt, a.gmul), t1 = share(cta + 1, nt, a.gmul);
    const int tmask = (1 << logt) - 1;
    auto blocks = [&](int d) { return (start[d + 1] - start[d] + 7) >> 3; };
    int items = 0;  // of this CTA
#pragma unroll 1
    for (int t = t0; t < t1;) {
      const int d = t >> logt, e = min(t1, (d + 1) << logt);
      items += (e - t) * blocks(d);
      t = e;
    }
    const int total = items << a.logU;
    auto border = [&](int w) { return static_cast<int>(static_cast<uint32_t>(total * w) / kWarps); };
    const int ub = border(warp), ue = border(warp + 1);
    // the warp's item: tile t, block of slots b, units u .. end - 1 of it here; `left` units after them
    int t = t0, b = 0, u = ub & (U - 1), left = ue - ub;
    {
      int i = ub >> a.logU;  // item of the first unit
#pragma unroll 1
      while (t < t1) {
        const int d = t >> logt, e = min(t1, (d + 1) << logt), nb = blocks(d), n = (e - t) * nb;
        if (i < n) {
          const int q = nb == 1 ? i : i / nb;
          t += q;
          b = 8 * (i - q * nb);
          break;
        }
        i -= n;
        t = e;
      }
    }
    auto records = [&](int tile) {
      return a.pool + dist[tile >> logt] * a.stride + static_cast<size_t>(16 * (tile & tmask)) * RGU;
    };
    const uint8_t* base = a.pool;
    uint32_t flip = 0;           // buffer of the unit that comes next to be used
    uint32_t wset = sets32;      // set that comes next to be filled
    auto copy = [&](const uint8_t* from, int unit, bool scales, uint32_t buf) {
      issue_codes(ring32 + buf * kUnitBytes, plan, from, unit, 8, 8);
      if (scales) {
        issue_scales(wset, plan, from, unit, 8, 8);
        if ((wset += plan.set_bytes()) == sets32 + kSetsBytes) wset = sets32;
      }
    };
    if (left > 0) {
      base = records(t);
      copy(base, u, true, 0);
    }
    cp_commit();

    // the shared expert's hidden values while the first copies are under way: a pair of lanes per (token, pair)
#pragma unroll 1
    for (int tk = kWarps - 1 - warp; tk < T && nsp > 0; tk += kWarps) {
      const int pr = min(lane >> 1, nsp - 1), up = lane & 1;
      const float2 v = reinterpret_cast<const float2*>(sraw)[tk * 16 + pr];
      float x = up ? v.y : v.x;
      const uint16_t* B = up ? a.shB[1] : a.shB[0];
      if (up ? a.shA[1] != nullptr : a.shA[0] != nullptr)
        x = fmaf(a.lora_scale, dot_r(B + static_cast<size_t>(sp0 + pr) * r, a.aux + tk * (4 + 2 * r) + 4 + (up && a.shA[0] ? r : 0), r), x);
      __syncwarp();
      const float y = __shfl_xor_sync(0xffffffffu, x, 1);
      if (!up && lane < 2 * nsp) store_h(a, TK + tk, sp0 + pr, x, y);
    }

    const uint8_t* set = sets;
    float4* part = reinterpret_cast<float4*>(scratch);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    auto finish = [&]() {  // hidden values of item (t, b)
      const int d = t >> logt, q0 = start[d] + b + 2 * tig, q1 = min(q0 + 2, start[d + 1]), j = (t & tmask) * 8 + g;
#pragma unroll 1
      for (int q = q0; q < q1; ++q) {
        const int sl = slots[q] & 0xffff;
        const float k = ic[slots[q] >> 16] * 0x1p22f;
        float x = (q > q0 ? acc[1] : acc[0]) * k, y = (q > q0 ? acc[3] : acc[2]) * k;
        if (a.exAgu) {
          const uint16_t* B = a.exBgu + (static_cast<size_t>(dist[d]) * 2 * a.I + 2 * j) * r;
          const float* ta = a.tgu + static_cast<size_t>(sl) * 2 * r;
          x = fmaf(a.lora_scale, dot_r(B, ta, r), x);
          y = fmaf(a.lora_scale, dot_r(B + r, ta + r, r), y);
        }
        store_h(a, sl, j, x, y);
      }
      __syncwarp();
    };
    bool open = false;  // the warp began the item and others go on with it
#pragma unroll 1
    while (left > 0) {
      const int d = t >> logt, s0 = start[d], cl = start[d + 1] - 1, c0 = s0 + b;
      const uint8_t* col = img + static_cast<size_t>(slots[min(c0 + g, cl)] >> 16) * ldu;
      const float* ua = us + (slots[min(c0 + 2 * tig, cl)] >> 16) * G;
      const float* uc = us + (slots[min(c0 + 2 * tig + 1, cl)] >> 16) * G;
      const bool mine = u == 0;
      const int end = min(U, u + left);
      left -= end - u;
      // where the units after these come from
      const bool next_tile = c0 + 8 > cl;
      const uint8_t* after = left > 0 && next_tile ? records(t + 1) : base;
#pragma unroll 1
      for (; u < end; ++u) {
        const bool last = u + 1 == end;
        const int n = last ? 0 : u + 1;
        flip ^= 1;
        if (!last || left > 0) copy(last ? after : base, n, (n & 1) == 0, flip);
        cp_commit();
        cp_wait<1>();
        gate_up_unit(ring + (flip ^ 1) * kUnitBytes, set + 8 * (u & 1), plan.half(), col + u * 512, ua + 4 * u, uc + 4 * u, acc);
        if (((u & 1) || U == 1) && (set += plan.set_bytes()) == sets + kSetsBytes) set = sets;
        __syncwarp();
      }
      if (!mine) {
        part[warp * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      } else if (end < U) {
        open = true;
        break;
      } else {
        finish();
      }
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      u = 0;
      b = next_tile ? 0 : b + 8;
      t += next_tile;
      base = after;
    }
    if (ub == ue) part[warp * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    named_sync(15, kThreads);
    if (open) {
      const int end = ue + U - u;  // of the item
#pragma unroll 2
      for (int w = warp + 1; w < kWarps && border(w) < end; ++w) {
        const float4 v = part[w * 32 + lane];
        acc[0] += v.x, acc[1] += v.y, acc[2] += v.z, acc[3] += v.w;
      }
      finish();
    }
  }
  grid_arrive(a.bar, B_HIDDEN);

  // --------------------------------------------------------------------------- down projections
  // Elements: (row tile, a block of up to 4 slots of one expert), dealt out to teams of Wd warps that split the units.
  const int NS = TK + T, RS = nrt * 16, total = nrt * nel;  // y [Wd][slot][RS]
  int logWd = 0;
  while (logWd < 3 && total << (logWd + 1) <= kWarps && U2 >> (logWd + 1) > 0) ++logWd;
  const int Wd = 1 << logWd, teams = kWarps >> logWd, wi = warp & (Wd - 1);
  const int u0 = wi * (U2 >> logWd), u1 = u0 + (U2 >> logWd);
  plan.make(RDN, G2, 1, 8);
  // where the rows of element e (and how many of them) come from
  auto rows_of = [&](int e) {
    const int rt = e < nel ? 0 : 1, d = els[e - rt * nel] & 511;
    return (d == 511 ? a.shared : a.pool + dist[d] * a.stride) + dn_off + static_cast<size_t>(dr0 + rt * rt_rows) * RDN;
  };
  uint32_t wset = sets32, flip = 0;
  auto copy = [&](const uint8_t* from, int e, int unit, bool scales, uint32_t buf) {
    const int n = e < nel ? rt_rows : ndr - rt_rows;
    issue_codes(ring32 + buf * kUnitBytes, plan, from, unit, min(8, n), n - 8);
    if (scales) {
      issue_scales(wset, plan, from, unit, min(8, n), n - 8);
      if ((wset += plan.set_bytes()) == sets32 + kSetsBytes) wset = sets32;
    }
  };
  int ei = warp >> logWd;
  const uint8_t* base = a.shared;
  cp_wait<0>();
  for (int i = 0; i < 2; ++i)  // row 15 of the buffers
    *reinterpret_cast<uint32_t*>(ring + i * kUnitBytes + 15 * 128 + 4 * lane) = 0xffffffffu;
  __syncwarp();
  if (ei < total) {
    base = rows_of(ei);
    copy(base, ei, u0, true, 0);
  }
  cp_commit();
  if (a.shA[2] && warp < ndr && lane < (r * 2 + 127) / 128)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(a.shB[2] + static_cast<size_t>(dr0 + warp) * r + 64 * lane));
  grid_wait(a.bar, B_HIDDEN, !a.exA, failed, a.err, a.timeout_ns);

  const uint8_t* hb = reinterpret_cast<const uint8_t*>(a.h);
  const size_t hrow = static_cast<size_t>(a.I) * 2;  // bytes of one hi or lo row
  const int logm = r > 16 ? 1 : 0;  // 16-row tiles of A: 1 or 2
  float* td = reinterpret_cast<float*>(sm + S.td);
  // LoRA A on hidden values: routed, each (block of slots, 16 rows of A) once in the grid, its groups split over eight
  // warps of a CTA and joined there (a warp for the whole task waits for its loads several times over: 94 us against 88
  // for 32 tokens of the 35B shape); shared, in every CTA, with the groups split over as many warps as there are
  // (partial sums [part][token][kMaxR])
  int logp = 0;
  while (logp < 3 && (sh_blocks << logm) << (logp + 1) <= kWarps && G2 >> (logp + 1) > 0) ++logp;
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const uint16_t* A = kind ? a.shA[2] : a.exA;
    if (!A) continue;
    const int lp = kind ? logp : min(a.logI - 6, 3), mask = (1 << lp) - 1;
    const int tasks = (kind ? sh_blocks : nel - sh_blocks) << logm;
    const int w0 = kind ? kWarps - 1 - warp : warp, step = (kind ? 1 : grid) * (kWarps >> lp);
#pragma unroll 1
    for (int q0 = kind ? 0 : cta; q0 < tasks; q0 += step) {  // the same turns in every warp
      const int q = q0 + (kind ? 1 : grid) * (w0 >> lp), part = w0 & mask;
      const bool on = q < tasks;
      const int m0 = (q & ((1 << logm) - 1)) * 16, el = on ? els[(kind ? 0 : sh_blocks) + (q >> logm)] : 1 << 20;
      const int d = el & 511, s0 = (el >> 9) & 511, n = el >> 20, cs = s0 + min(g >> 1, n - 1);
      float v[4];
      if (on) {
        const uint16_t* M = A + (kind ? 0 : static_cast<size_t>(dist[d]) * r * a.I);
        const int pos = kind ? TK + cs : slots[cs] & 0xffff, span = G2 >> lp;
        f16_rows(M + static_cast<size_t>(min(m0 + g, r - 1)) * a.I, M + static_cast<size_t>(min(m0 + g + 8, r - 1)) * a.I,
                 part * span, (part + 1) * span, hb + (static_cast<size_t>(pos) * 2 + (g & 1)) * hrow, 1.f, v);
      }
      if (kind == 0) {  // join the parts
        float4* sums = reinterpret_cast<float4*>(scratch);
        if (on && part > 0) sums[warp * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
        named_sync(15, kThreads);
        if (on && part == 0) {
#pragma unroll 1
          for (int w = 1; w <= mask; ++w) {
            const float4 p = sums[(warp + w) * 32 + lane];
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
          }
        }
        named_sync(15, kThreads);
      }
      if (on && tig < n && (kind || part == 0)) {
        float* o = kind ? td + (part * T + s0 + tig) * kMaxR : a.tex + static_cast<size_t>(slots[s0 + tig] & 0xffff) * r;
        if (m0 + g < r) o[m0 + g] = fmaf(v[1], 0x1p-11f, v[0]);
        if (m0 + g + 8 < r) o[m0 + g + 8] = fmaf(v[3], 0x1p-11f, v[2]);
      }
    }
    if (kind == 0) grid_arrive(a.bar, B_EXDOWN);
  }

  {
    const uint8_t* set = sets;
#pragma unroll 1
    while (ei < total) {
      const int el = els[ei < nel ? ei : ei - nel], s0 = (el >> 9) & 511, n = el >> 20;
      const bool sh = (el & 511) == 511;
      const int cs = s0 + min(g >> 1, n - 1);
      const uint8_t* col = hb + (static_cast<size_t>(sh ? TK + cs : slots[cs] & 0xffff) * 2 + (g & 1)) * hrow;
      const int ne = ei + teams;
      const uint8_t* after = ne < total ? rows_of(ne) : base;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int u = u0; u < u1; ++u) {
        const Frag f0 = load_frag(col + u * 512, 0), f1 = load_frag(col + u * 512, 1);
        const bool last = u + 1 == u1;
        const int nu = last ? u0 : u + 1;
        flip ^= 1;
        if (!last || ne < total) copy(last ? after : base, last ? ne : ei, nu, last || (nu & 1) == 0, flip);
        cp_commit();
        cp_wait<1>();
        down_unit(ring + (flip ^ 1) * kUnitBytes, set + 8 * (u & 1), plan.half(), f0, f1, col + u * 512, G2 >= 4, acc);
        if (((u & 1) || last) && (set += plan.set_bytes()) == sets + kSetsBytes) set = sets;
        __syncwarp();
      }
      if (tig < n) {
        const int p = sh ? TK + s0 + tig : slots[s0 + tig] & 0xffff;
        float* y = scratch + (wi * NS + p) * RS + (ei < nel ? 0 : 16);
        y[g] = fmaf(acc[1], 0x1p-11f, acc[0]) * 0x1p18f;
        if (g < 7) y[g + 8] = fmaf(acc[3], 0x1p-11f, acc[2]) * 0x1p18f;
      }
      ei = ne;
      base = after;
    }
  }
  if (a.exA) {
#pragma unroll 1
    for (int s = warp; s < TK; s += kWarps)
      if (lane < ndr)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.exB + (static_cast<size_t>(sel[s]) * a.H + dr0 + lane) * r));
  }
  if (a.exA) {
    grid_wait(a.bar, B_EXDOWN, true, failed, a.err, a.timeout_ns);
    for (int i = tid; i < TK * r / 32; i += kThreads)  // every row of a slot reads its A h
      asm volatile("prefetch.global.L1 [%0];" ::"l"(a.tex + 32 * i));
  } else {
    named_sync(15, kThreads);
  }

  // --------------------------------------------------------------------------- combine
  if (a.shA[2] && logp > 0) {  // the parts of the shared down adapter's A h
#pragma unroll 1
    for (int i = tid; i < T * kMaxR; i += kThreads) {
      float v = td[i];
      for (int w = 1; w < 1 << logp; ++w) v += td[w * T * kMaxR + i];
      td[i] = v;
    }
    named_sync(15, kThreads);
  }
  // a thread per (token, row of a tile)
#pragma unroll 1
  for (int i = tid; i < T * nrt * 16; i += kThreads) {
    const int t = nrt > 1 ? i >> 5 : i >> 4, rt = nrt > 1 ? (i >> 4) & 1 : 0;
    const int row = rt * rt_rows + (i & 15), o = rt * 16 + (i & 15);
    if ((i & 15) >= rt_rows || row >= ndr) continue;
    const int hr = dr0 + row;
    float out = 0.f;
#pragma unroll 1
    for (int k = 0; k <= K; ++k) {  // the K experts in order, then the shared one
      const int s = k < K ? t * K + k : TK + t;
      float y = 0.f;
#pragma unroll 1
      for (int w = 0; w < Wd; ++w) y += scratch[(w * NS + s) * RS + o];
      if (k < K) {
        if (a.exA)
          y = fmaf(a.lora_scale, dot_r(a.exB + (static_cast<size_t>(sel[s]) * a.H + hr) * r, a.tex + static_cast<size_t>(s) * r, r), y);
        out = fmaf(sw[s], y, out);
      } else {
        if (a.shA[2]) {
          float l = 0.f;
#pragma unroll 1
          for (int k8 = 0; k8 < r; k8 += 8) {
            const uint4 b = __ldg(reinterpret_cast<const uint4*>(a.shB[2] + static_cast<size_t>(hr) * r + k8));
            const float* v = td + t * kMaxR + k8;
            l = fmaf(lo_half(b.x), v[0], l), l = fmaf(hi_half(b.x), v[1], l);
            l = fmaf(lo_half(b.y), v[2], l), l = fmaf(hi_half(b.y), v[3], l);
            l = fmaf(lo_half(b.z), v[4], l), l = fmaf(hi_half(b.z), v[5], l);
            l = fmaf(lo_half(b.w), v[6], l), l = fmaf(hi_half(b.w), v[7], l);
          }
          y = fmaf(a.lora_scale, l, y);
        }
        out = fmaf(gate[t], y, out);
      }
    }
    const size_t at = static_cast<size_t>(t) * a.H + hr;
    if (a.out_mode == 1)
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(out);
    else if (a.out_mode == 2)
      static_cast<float*>(a.out)[at] += out;
    else
      static_cast<float*>(a.out)[at] = out;
  }
}

}  // namespace ld
}  // namespace moe
