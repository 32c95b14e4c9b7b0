// Dense attention over the paged 8-bit or 4-bit K/V cache for requests of many rows (prompt pieces), on tcgen05 tensor
// cores.  (Compiled here for the 8-bit cache; kv4_prompt.cu compiles the same kernel for the 4-bit one.)
// Definition as in paged_attention.cu:
//   z_s = scale * q[r,h] . (k_code_s * ks),  out = softmax(z) (v_code * vs),  lse = ln sum exp(z)
//
// Here the products bound the call (4 * 128 flop per visible pair and head), so the tiles are square:
//   S [128 pairs x 128 keys]  = Q [128 x 128] K^T     K's codes as they are, Q in two e4m3 terms, from shared memory
//   O [128 pairs x 128 dims] += P [128 x 128] V       P in fp16 from TMEM, V widened to fp16 in shared memory
// Two e4m3 products take as long as one in fp16 or bf16 and K needs no widening.  Q = hi + lo in units of 2^-8 of
// the row's largest value: 8 bits of bf16 are kept down to 2^-9 of it, with an absolute error of at most 2^-17
// below (bf16 itself has 2^-9 of each value; one accumulator for both terms leaves no room for a scale
// of lo's own).  ks multiplies the scores of its page, one fp32 factor per 16 keys.  V as fp16 holds codes exactly;
// vs goes into it relative to the largest of the piece's pages, exactly for the powers of two that the append writes.
// P carries 2^8 times the probability (11 bits of it, with an absolute error of 2^-33 of the row's largest).
//
// Work: (request, 256 pairs, K/V head, tile of 128 keys) units split into one contiguous range per CTA
// (persistent, one CTA per SM), as in paged_attention.cu; a segment that is cut leaves fp32 pieces for a join.
// Segments count the tiles their last row sees, so causal rows are balanced over the CTAs.
//
// Per CTA (20 warps): warps 0-3 and 4-7 are the softmax of the two 128-pair halves, one pair a thread (no
// cross-lane work at all).  A half goes through a tile as two times 64 keys, each with its own 64 columns of TMEM
// for S and then P: while the softmax works on one, the tensor cores add the other to O and compute the next
// tile's S in its place.  One S of 128 keys a half, its softmax and its products taking turns, took 4,500
// cycles a tile (a quarter longer for 4,096 rows at 64K); the scores' products are a half slower at 64 keys, which
// this more than pays for.  Warp 16 issues the output products, warps 17 and 18 one half's scores each, as soon as
// the output product that read the P in their place is known to be done (products of different kinds are not
// promised to run in order; one warp a half for both kinds, waiting for that, took 8 % longer).
// Warps 8-11 and 12-15 widen the V tiles, even and odd ones; warp 19 loads K tiles by TMA and finds the CTA's
// segments for everyone (each role finding them for itself cost 30 registers, and spills).
//
// 4-bit cache: block scales in TMEM, as the kernel for few rows has them, need columns that S and O do not leave, so K's
// codes are widened too: to e5m2, which holds code * 2^e exactly for the exponents of the cache (-15 .. 13).  V's fp16
// values are code * scale in units that put the piece's largest scale at 2^12 (6 * 2^13 is the largest value, fp16's is 65,504): exact
// for scales down to 2^-26 of it, a step of 2^-36 of it below (rows of a prompt that see only such tokens).  Warps 8-11 widen K, 12-15 V.
// TMEM (all 512 columns): S of half q and key half h at 128 q + 64 h, with P over its first 32; O of half q at 256 + 128 q.
#include "paged_attention.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <type_traits>

namespace dsa {
using namespace sm100;

namespace pp {
constexpr int kTok = kPaTok;
constexpr int kHalfPairs = 128;
constexpr int kQTermBytes = kHalfPairs * kKvDim;     // 16 KB: one e4m3 term of one half's queries
constexpr int kKBytes = kTok * kKvDim;               // 16 KB of codes
constexpr int kVBytes = kTok * kKvDim * 2;           // 32 KB of fp16: two 64-wide column chunks of 128-byte rows
constexpr int kChunkBytes = kTok * 128;
template <bool k4>
constexpr int kKStages = k4 ? 3 : 4;
// 4-bit cache: a tile's codes and scales as they are in the cache, on their way to the widening warps
constexpr int kRawKBytes = kTok * (kKvDim / 2 + kKv4Blocks), kRawVBytes = kTok * (kKvDim / 2 + 2), kRawStages = 2;
constexpr int kThreads = 640;
constexpr int kConvWarp0 = 8, kOutWarp = 16, kScoreWarp0 = 17, kLoadWarp = 19;
constexpr uint32_t kRegsSoft = 128, kRegsConv = 80, kRegsRest = 64;   // 2 * 128 + 2 * 80 + 64 = 480 = 5 * 96, the launch's
constexpr uint32_t kTmemCols = 512, kColO = 256;
constexpr float kSlack = 6.f;                        // log2 by which a row's maximum may be exceeded
constexpr float kPLog2 = 8.f;                        // P = 2^8 p
constexpr float kV4Up = 4096.f;                      // 4 bits: the piece's largest scale of V in fp16, 2^12
constexpr uint32_t kPolls = 1u << 18;                // of 3.8 us each or more: a second
// Rolled: four polls written out at each of the many waits take 10 % longer (4,096 rows at 64K, 3.30 instead of 2.98 ms when
// measured).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t code, uint32_t polls) {
  return mbar_wait_warp<1>(bar, parity, err, code, polls);
}
// A segment counts as this many tiles beside its own: loading its queries and writing its outputs is not hidden.  (2
// prompts of 1,633 rows and 64 heads, 1 to 13 tiles a segment: 175 us; without, 358.)  Capped and biased tiles take
// longer, so their segments' ends weigh less.
constexpr int kSegUnits = 4, kModsSegUnits = 2;
constexpr int kRuns = 512;                           // runs of (request, pairs) entries that are summed
constexpr int kMetaBufs = 8;                         // tiles whose K scales are kept (a tile's outlive its K stage)
constexpr int kSegBufs = 4;
template <bool k4>
constexpr int kFixedSmem = 4 * kQTermBytes + kKStages<k4> * kKBytes + 2 * kVBytes + (k4 ? kRawStages * (kRawKBytes + kRawVBytes) : 0) + 1024;
}  // namespace pp

// (request, 256 pairs): its rows' last key, and the tiles that they see
struct PpEntry {
  int b, qt, tiles;
  PaShape shape;
  int start, prefix;               // position of row 0; positions that every row sees
};

__device__ __forceinline__ int pp_limit(const PpEntry& e, int row) {
  return min(max(e.start + row + 1, e.prefix), e.shape.len);
}

__device__ __forceinline__ int pp_entries(const PagedAttnArgs& a, const PaShape& s) {
  return (int)(((int64_t)s.rows * a.group + kPromptPairs - 1) / kPromptPairs);
}

__device__ __forceinline__ PpEntry pp_entry(const PagedAttnArgs& a, const PaShape& shape, int b, int qt) {
  PpEntry e;
  e.b = b;
  e.qt = qt;
  e.shape = shape;
  e.start = a.seq_lens[b] - e.shape.rows;
  e.prefix = a.prefix_lens ? min(a.prefix_lens[b], e.shape.len) : 0;
  const int last = min(e.shape.rows - 1, ((qt + 1) * kPromptPairs - 1) / a.group);
  e.tiles = max(1, (pp_limit(e, last) + pp::kTok - 1) / pp::kTok);
  return e;
}

// A run of tiles of one segment (entry and K/V head), as the scheduler warp leaves it in shared memory for the others
struct __align__(16) PpSeg {
  int n, tile, h, qt;              // its tiles and the first of them (n = 0: no further segment)
  int b, tiles, slot, rows;        // the segment's tiles; where a piece goes
  int row0, len, start, prefix;    // as in PaShape and PpEntry

  // Its t-th tile: the last keys come first.  A bias on distance makes scores grow towards a row's own position, and
  // with them the reference, tile by tile in rising order (a fifth of such a call's time); in falling order it stands.
  __device__ __forceinline__ int tile_at(int t) const { return tile + n - 1 - t; }
};

__device__ __forceinline__ int pp_limit(const PpSeg& s, int row) { return min(max(s.start + row + 1, s.prefix), s.len); }

// Where the scheduler stands: the entry and how many units before it
struct PpCursor {
  int b, qt;
  int64_t before;                  // units of the entries before this one
};

// The segment that unit u lies in (its first kEnds units stand for no tile, the others for one each), cut at u1; u
// moves to the next one and the cursor up to the entry.  n is 0 where no tile of the segment lies in [u, u1).
template <int kEnds>
__device__ __forceinline__ PpSeg pp_segment(const PagedAttnArgs& a, PpCursor& c, int64_t& u, int64_t u1, int cta) {
  PpEntry e;
  for (;;) {
    uint32_t none = 0;
    const PaShape sh = pa_shape(a, c.b, none);
    if (c.qt >= pp_entries(a, sh)) {
      ++c.b;
      c.qt = 0;
      continue;
    }
    e = pp_entry(a, sh, c.b, c.qt);
    const int64_t units = (int64_t)(e.tiles + kEnds) * a.kv_heads;
    if (u < c.before + units) break;
    c.before += units;
    ++c.qt;
  }
  PpSeg s;
  const int64_t in = u - c.before;
  const int per = e.tiles + kEnds;
  s.h = in < (int64_t(1) << 31) ? (int)((uint32_t)in / (uint32_t)per) : (int)(in / per);
  const int at = (int)(in - (int64_t)s.h * per), end = (int)min((int64_t)per, at + (u1 - u));
  s.tile = max(at - kEnds, 0);
  s.n = max(end - kEnds, 0) - s.tile;
  u += end - at;
  s.qt = e.qt;
  s.b = e.b;
  s.tiles = e.tiles;
  s.slot = s.tile > 0 ? 2 * cta : 2 * cta + 1;
  s.rows = e.shape.rows;
  s.row0 = e.shape.row0;
  s.len = e.shape.len;
  s.start = e.start;
  s.prefix = e.prefix;
  return s;
}

// four fp16 pairs of eight e4m3 codes
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = (i < 2 ? lo : hi) >> (16 * (i & 1));
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
    r[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// four fp16 pairs of eight e2m1 codes
__device__ __forceinline__ uint4 widen8(uint32_t w) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w >> (8 * i)), __NV_E2M1);
    r[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ uint32_t mul2(uint32_t x, __half2 f) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), f);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// two fp32 values in one 64-bit register pair (one instruction for both)
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16 consecutive 32-bit columns of the warp's lanes written from registers
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14,"
      " %15, %16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15},"
      " [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// A softmax thread's row: its reference m (log2 units), its sum l of P, and what masks and biases need.
struct PpRow {
  float m, l, cf, slope;
  int limit, pos;
};

// 64 keys of a row that sees them all, in one pass over their scores: 16 at a time they come out of TMEM (the next
// 16 in flight), and P = 2^(z - m + 8) is formed against the reference that the row has.  P stays in registers until
// the largest score (returned) is known to exceed it by no more than the slack, as for nearly every tile; else
// the pass is repeated.  (Two passes, as below, take 7 % longer for 4,096 rows at 64K.)
// k4: the scores need no factor of their keys.
template <bool k4>
__device__ __forceinline__ float pp_half(const PpRow& w, uint32_t tS, const float* ks, uint32_t (&p)[32], float& sum_out) {
  const float shift = pp::kPLog2 - (w.m == -INFINITY ? 0.f : w.m);
  const uint64_t shift2 = pack2(shift, shift);
  uint64_t sum[2] = {0, 0};
  uint32_t r[2][16];
  float top = -INFINITY;
  tmem_ld16(tS, r[0]);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    tmem_wait_ld();
    if (g < 3) tmem_ld16(tS + 16 * (g + 1), r[(g + 1) & 1]);
    const uint32_t* x = r[g & 1];
    const float kc = k4 ? w.cf : ks[g] * w.cf;
    float m = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
    const uint64_t kc2 = pack2(kc, kc);
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      if (c) m = fmaxf(m, fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
      float y0, y1;
      unpack2(fma2(pack2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), kc2, shift2), y0, y1);
      y0 = ex2_approx(y0);
      y1 = ex2_approx(y1);
      sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(y0, y1));
      const __half2 h = __floats2half2_rn(y0, y1);
      p[8 * g + (c >> 1)] = *reinterpret_cast<const uint32_t*>(&h);
    }
    top = fmaxf(top, k4 ? m : m * kc);
  }
  if (k4) top *= w.cf;
  float s0, s1, s2, s3;
  unpack2(sum[0], s0, s1);
  unpack2(sum[1], s2, s3);
  sum_out = (s0 + s1) + (s2 + s3);
  return top;
}

// 64 keys with masks, a cap or a bias, in two rolled passes (one body of each: unrolled like the plain form, the call
// with a cap and a bias took a fifth longer): the scores are made final and written back, with their largest ..
template <bool k4, PaMods kModSet, bool kMasked>
__device__ __forceinline__ float pp_max64(const PpRow& w, const PagedAttnArgs& a, uint32_t tS, int key0, uint32_t bad, const float* ks) {
  constexpr bool kMods = kModSet != kPaPlain;
  const float in = kMods && a.cap_log2 > 0.f ? 2.f * 1.4426950408889634f / a.cap_log2 : 0.f;
  float top = -INFINITY;
#pragma unroll 1
  for (int g = 0; g < 4; g += 2) {
    uint32_t r[32];
    tmem_ld32(tS + 16 * g, r);
    tmem_wait_ld();
#pragma unroll
    for (int gg = 0; gg < 2; ++gg) {
      uint32_t* x = r + 16 * gg;
      const float own = in != 0.f ? w.cf * in : w.cf, kc = k4 ? own : ks[g + gg] * own;
      const int left = ((bad >> (g + gg)) & 1u) ? 0 : w.limit - key0 - 16 * (g + gg);   // keys of the group that are seen
      const float away = kMods ? (float)(w.pos - key0 - 16 * (g + gg)) : 0.f;           // of the row from the first of them
      // a loop each: a choice made inside one of them would leave the values no instructions to overlap with
      float z[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) z[c] = __uint_as_float(x[c]) * kc;
      if (kMods && in != 0.f) {
#pragma unroll
        for (int c = 0; c < 16; ++c) z[c] = capped<kModSet>(z[c], a.cap_log2);
      }
      if (kMods) {
#pragma unroll
        for (int c = 0; c < 16; ++c) z[c] = fmaf(-w.slope, fabsf(away - (float)c), z[c]);
      }
      // a masked score is -inf whatever the factor (which may be 0)
#pragma unroll
      for (int c = 0; c < 16; ++c) x[c] = !kMasked || c < left ? __float_as_uint(z[c]) : 0xFF800000u;
#pragma unroll
      for (int c = 0; c < 16; c += 2) top = fmaxf(top, fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
    }
    tmem_st32(tS + 16 * g, r);
  }
  tmem_wait_st();
  return top;
}

// .. and P takes their place.  (Their factors are in them by now.)
__device__ __forceinline__ float pp_exp64(const PpRow& w, uint32_t tS) {
  const float shift = pp::kPLog2 - (w.m == -INFINITY ? 0.f : w.m);
  const uint64_t shift2 = pack2(shift, shift);
  uint64_t sum[2] = {0, 0};
#pragma unroll 1
  for (int g = 0; g < 4; g += 2) {
    uint32_t r[32], p[16];
    tmem_ld32(tS + 16 * g, r);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      float y0, y1;
      unpack2(add2(pack2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), shift2), y0, y1);
      y0 = ex2_approx(y0);
      y1 = ex2_approx(y1);
      sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(y0, y1));
      const __half2 h = __floats2half2_rn(y0, y1);
      p[c >> 1] = *reinterpret_cast<const uint32_t*>(&h);
    }
    tmem_st16(tS + 8 * g, p);
  }
  float s0, s1, s2, s3;
  unpack2(sum[0], s0, s1);
  unpack2(sum[1], s2, s3);
  return (s0 + s1) + (s2 + s3);
}

// The same for scores of the 4-bit cache without a cap or bias, which nothing but their row's factor separates from their final form:
// their largest, and P formed from the products as they are (written back in between, 4,096 rows at 64K took 3.18 ms instead of 3.12).
__device__ __forceinline__ float pp_max64(const PpRow& w, uint32_t tS, int key0, uint32_t bad) {
  float top = -INFINITY;
#pragma unroll 1
  for (int g = 0; g < 4; g += 2) {
    uint32_t r[32];
    tmem_ld32(tS + 16 * g, r);
    tmem_wait_ld();
#pragma unroll
    for (int gg = 0; gg < 2; ++gg) {
      const int left = ((bad >> (g + gg)) & 1u) ? 0 : w.limit - key0 - 16 * (g + gg);   // keys of the group that are seen
      float m = -INFINITY;
#pragma unroll
      for (int c = 0; c < 16; ++c) m = fmaxf(m, c < left ? __uint_as_float(r[16 * gg + c]) : -INFINITY);
      top = fmaxf(top, m);
    }
  }
  return top == -INFINITY ? top : top * w.cf;          // (-inf whatever the factor, which may be 0)
}

// .. and P in their place
__device__ __forceinline__ float pp_exp64(const PpRow& w, uint32_t tS, int key0, uint32_t bad) {
  const float shift = pp::kPLog2 - (w.m == -INFINITY ? 0.f : w.m);
  const uint64_t shift2 = pack2(shift, shift), kc2 = pack2(w.cf, w.cf);
  uint64_t sum[2] = {0, 0};
#pragma unroll 1
  for (int g = 0; g < 4; g += 2) {
    uint32_t r[32], p[16];
    tmem_ld32(tS + 16 * g, r);
    tmem_wait_ld();
#pragma unroll
    for (int gg = 0; gg < 2; ++gg) {
      const int left = ((bad >> (g + gg)) & 1u) ? 0 : w.limit - key0 - 16 * (g + gg);
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const uint32_t* x = r + 16 * gg + c;
        float y0, y1;
        unpack2(fma2(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])), kc2, shift2), y0, y1);
        y0 = c < left ? ex2_approx(y0) : 0.f;
        y1 = c + 1 < left ? ex2_approx(y1) : 0.f;
        sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(y0, y1));
        const __half2 h = __floats2half2_rn(y0, y1);
        p[8 * gg + (c >> 1)] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    tmem_st16(tS + 8 * g, p);
  }
  float s0, s1, s2, s3;
  unpack2(sum[0], s0, s1);
  unpack2(sum[1], s2, s3);
  return (s0 + s1) + (s2 + s3);
}

// 16 columns a step: the accumulator of a row whose reference moved
__device__ __forceinline__ void pp_shrink(uint32_t tO, float al) {
#pragma unroll 1
  for (int c = 0; c < kKvDim; c += 16) {
    uint32_t o[16];
    tmem_ld16(tO + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
    tmem_st16(tO + c, o);
  }
  tmem_wait_st();
}

// The queries of the warp's 32 pairs (first, first + 1, ..; there are none from `pairs` on) of one half, in two e4m3 terms
// from row `row0` of q_hi on; returns the factor of the lane's own row's scores.  16 lanes a row, so that loads are
// whole lines, two rows a step and four steps ahead; rolled, as it is run once a segment.
__device__ __forceinline__ float pp_queries(const PagedAttnArgs& a, const PpSeg& s, int first, int pairs, uint8_t* q_hi, int row0) {
  const int lane = threadIdx.x & 31, part = lane & 15, half = lane >> 4;
  // where the lane's own pair lies
  const int own_n = min(first + lane, pairs - 1), own_i = own_n / a.group;
  const int64_t from = (int64_t)(s.row0 + own_i) * a.q_stride + (int64_t)(s.h * a.group + own_n - own_i * a.group) * kKvDim;
  auto load = [&](int k) {
    const int64_t at = __shfl_sync(0xffffffffu, from, (2 * k + half) & 31);
    return k < 16 && first + 2 * k + half < pairs ? __ldg(reinterpret_cast<const uint4*>(a.q + at) + part) : make_uint4(0, 0, 0, 0);
  };
  float cf = 0.f;
  uint4 x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = load(j);
#pragma unroll 1
  for (int k0 = 0; k0 < 16; k0 += 4) {
    uint4 y[4];
    uint32_t tops[4];                                  // the largest |x| of each step's rows as bf16 bits, side by side
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = x[j];
      const uint32_t m = __vmaxu2(__vmaxu2(y[j].x & 0x7FFF7FFFu, y[j].y & 0x7FFF7FFFu), __vmaxu2(y[j].z & 0x7FFF7FFFu, y[j].w & 0x7FFF7FFFu));
      tops[j] = max(m & 0xFFFFu, m >> 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = load(k0 + j + 4);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) tops[j] = max(tops[j], __shfl_xor_sync(0xffffffffu, tops[j], o));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + j;
      const uint32_t w[4] = {y[j].x, y[j].y, y[j].z, y[j].w}, top = tops[j];
      const int E = pa_exponent(top);
      const __nv_bfloat162 up = pa_up(E);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pa_split<1>(w[e], up, hi[e], lo[e]);
      const uint32_t at = sw128_offset(row0 + 2 * k + half, part >> 1) + 8 * (part & 1);
      *reinterpret_cast<uint2*>(q_hi + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2*>(q_hi + pp::kQTermBytes + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      const float f = pa_factor(top, E, a.scale_log2);
      const float own = __shfl_sync(0xffffffffu, f, 16 * (lane & 1));
      if ((lane >> 1) == k) cf = own;
    }
  }
  return cf;
}

// ---- the 4-bit cache's widening warps.  The loader copies a tile's codes and scales into shared memory as they are; a thread takes
// 32 codes of a row (16 bytes, and for K one scale) a step: four lanes a row, eight rows a warp and 32 the four warps, in
// four steps a tile.  (Loads from the cache straight into registers, a tile ahead, took 5.7 ms for 4,096 rows at 64K: a fence
// waits for loads in flight, so they had only the time between two of them.)
struct PpRaw {
  uint8_t* bytes;                  // [stages] of codes, then scales
  uint64_t *full, *empty;          // [stages]
  const uint32_t* bad;             // [kMetaBufs] 16-key groups without a valid page
};

// The bytes of e5m2(code * 2^e) for e2m1 codes 0 .. 3 and 4 .. 7 without their sign, from a scale byte; NaN for the NaN scale.  With
// k = e + 14 >= 1 code c stands for exponent field k + (c >> 1) and mantissa bits c & 1, 0, but for 0 and for 1 = 2^-1,
// whose mantissa is 0; below, the small ones are subnormal numbers.
__device__ __forceinline__ void pp_e5m2_table(uint32_t scale, uint32_t& lo, uint32_t& hi) {
  static_assert(kKv4LowExp == -15 && kKv4HighExp == 13, "what e5m2 holds exactly");
  const int k = min(max((int)scale - 127, kKv4LowExp), kKv4HighExp) + 14;
  hi = 0x0E0C0A08u + (uint32_t)k * 0x04040404u;
  lo = k > 0 ? 0x06040000u + (uint32_t)k * 0x04040400u : k == 0 ? 0x06040200u : 0x03020100u;
  if (scale == 255u) lo = hi = 0x7F7F7F7Fu;
}

// Eight codes: magnitudes looked up four at a time by a byte permutation, whose other mode spreads the sign bits
__device__ __forceinline__ uint2 pp_e5m2(uint32_t w, uint32_t lo, uint32_t hi) {
  const uint32_t m = w & 0x77777777u, l = w << 4;
  uint32_t s0, s1;
  asm("prmt.b32 %0, %1, %2, 0xD9C8;" : "=r"(s0) : "r"(l), "r"(w));
  asm("prmt.b32 %0, %1, %2, 0xFBEA;" : "=r"(s1) : "r"(l), "r"(w));
  return make_uint2(__byte_perm(lo, hi, m) | (s0 & 0x80808080u), __byte_perm(lo, hi, m >> 16) | (s1 & 0x80808080u));
}

// K tiles: code * 2^e as e5m2
__device__ __forceinline__ void pp_widen_k4(const PpSeg* segs, uint64_t* seg_full, uint64_t* seg_empty, uint64_t* k_full, uint64_t* k_empty,
                                            uint8_t* sK, const PpRaw& raw, uint32_t* err) {
  using namespace pp;
  const int lane = threadIdx.x & 31, part = lane & 3, row0 = 8 * ((threadIdx.x >> 5) & 3) + (lane >> 2);
  int i = 0;
  for (int seg = 0;; ++seg) {
    if (!wait_warp(&seg_full[seg % kSegBufs], (seg / kSegBufs) & 1, err, kErrMmaTimeout, kPolls)) return;
    const int n = segs[seg % kSegBufs].n;
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[seg % kSegBufs]);
    if (n == 0) return;
    for (int t = 0; t < n; ++t, ++i) {
      const int st = i % kKStages<true>, use = i / kKStages<true>, rb = i % kRawStages;
      if (!wait_warp(&raw.full[rb], (i / kRawStages) & 1, err, kErrTmaTimeout, kPolls)) return;
      const uint8_t* const from = raw.bytes + rb * kRawKBytes;
      if (use > 0 && !wait_warp(&k_empty[st], (use - 1) & 1, err, kErrMmaTimeout, kPolls)) return;
      uint8_t* const to = sK + st * kKBytes;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        const uint4 x = reinterpret_cast<const uint4*>(from)[(32 * g + row0) * 4 + part];
        uint32_t lo, hi;
        pp_e5m2_table(from[kTok * kKvDim / 2 + (32 * g + row0) * kKv4Blocks + part], lo, hi);
        const uint2 a = pp_e5m2(x.x, lo, hi), b = pp_e5m2(x.y, lo, hi), c = pp_e5m2(x.z, lo, hi), d = pp_e5m2(x.w, lo, hi);
        *reinterpret_cast<uint4*>(to + sw128_offset(32 * g + row0, 2 * part)) = make_uint4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<uint4*>(to + sw128_offset(32 * g + row0, 2 * part + 1)) = make_uint4(c.x, c.y, d.x, d.y);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&k_full[st]);
        mbar_arrive(&raw.empty[rb]);
      }
    }
  }
}

// V tiles: code * scale in fp16, in units of 2^-12 of the power of two at or below the piece's largest scale
__device__ __forceinline__ void pp_widen_v4(const PagedAttnArgs& a, const PpSeg* segs, uint64_t* seg_full, uint64_t* seg_empty,
                                            uint64_t* v_full, uint64_t* v_empty, uint8_t* sV, const PpRaw& raw, int* nan_key,
                                            float* vmax_part, float* v_ref, uint32_t* err) {
  using namespace pp;
  const int lane = threadIdx.x & 31, cw = (threadIdx.x >> 5) & 3, part = lane & 3, row0 = 8 * cw + (lane >> 2), lp = a.log2_page;
  int i = 0;
  bool ok = true;
  for (int seg = 0; ok; ++seg) {
    const int sb = seg % kSegBufs;
    if (!wait_warp(&seg_full[sb], (seg / kSegBufs) & 1, err, kErrMmaTimeout, kPolls)) break;
    const PpSeg s = segs[sb];
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[sb]);
    if (s.n == 0) break;
    // the reference: eight tokens' scales a load, all in one page
    uint32_t top = 0;                                  // bf16 bits, sign off, finite ones
    const int c0 = s.tile * (kTok / 8), c1 = min((s.tile + s.n) * (kTok / 8), (s.len + 7) >> 3);
    const int32_t* const table = a.block_table + (int64_t)s.b * a.table_stride;
#pragma unroll 8
    for (int c = c0 + 32 * cw + lane; c < c1; c += 128) {
      const int id = table[(8 * c) >> lp];
      if (id >= 0 && id < a.num_pages) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.v_scales4 + (((int64_t)id * a.kv_heads + s.h) << lp) + ((8 * c) & ((1 << lp) - 1))));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t lo = u[q] & 0x7FFFu, hi = (u[q] >> 16) & 0x7FFFu;
          if (lo < 0x7F80u && 8 * c + 2 * q < s.len) top = max(top, lo);
          if (hi < 0x7F80u && 8 * c + 2 * q + 1 < s.len) top = max(top, hi);
        }
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) vmax_part[cw] = __uint_as_float(top);
    if (cw == 0 && lane == 0) nan_key[sb * kKvDim] = INT32_MAX;
    group_sync(2, 128);
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(vmax_part[k]));
    const uint32_t e_top = top & 0x7F80u;
    const float vref = e_top ? __uint_as_float(e_top << 16) : 1.f, vinv = 1.f / vref;
    if (cw == 0 && lane == 0) v_ref[sb] = vref;
    group_sync(2, 128);                                // before the next segment's maxima
    for (int t = 0; t < s.n; ++t, ++i) {
      const int key0 = s.tile_at(t) * kTok, rb = i % kRawStages;
      ok = wait_warp(&raw.full[rb], (i / kRawStages) & 1, err, kErrTmaTimeout, kPolls);
      if (!ok) break;
      const uint8_t* const from = raw.bytes + rb * kRawVBytes;
      const uint32_t bad = raw.bad[i % kMetaBufs];
      uint4 x[4];
      float scale[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int row = 32 * g + row0;
        x[g] = reinterpret_cast<const uint4*>(from)[row * 4 + part];
        scale[g] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(from + kTok * kKvDim / 2)[row]);
        // what lies behind the request's tokens, or in a page that was not loaded, is anything
        if (key0 + row >= s.len || ((bad >> (row >> 4)) & 1u)) scale[g] = 0.f;
      }
      if (i >= 2) ok = wait_warp(&v_empty[i & 1], ((i >> 1) - 1) & 1, err, kErrMmaTimeout, kPolls);
      if (!ok) break;
      uint8_t* const to = sV + (i & 1) * kVBytes + (part >> 1) * kChunkBytes;
      // dims 32 part .. + 31 are half a row of a 64-wide chunk; the two chunks' rows lie on the same banks, so lanes of the
      // second one write their units in another order
      const bool second = part >= 2;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float ratio = scale[g] * vinv * kV4Up;         // below 2^13
        if (!(fabsf(scale[g]) < INFINITY)) {           // a NaN for the rows that see the key, noted apart: 0 * NaN is NaN
          ratio = 0.f;
          atomicMin(&nan_key[sb * kKvDim], key0 + 32 * g + row0);
        }
        const __half2 f = __float2half2_rn(ratio);
        const uint32_t in[4] = {second ? x[g].z : x[g].x, second ? x[g].w : x[g].y, second ? x[g].x : x[g].z, second ? x[g].y : x[g].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 h = widen8(in[q]);
          h = make_uint4(mul2(h.x, f), mul2(h.y, f), mul2(h.z, f), mul2(h.w, f));
          *reinterpret_cast<uint4*>(to + sw128_offset(32 * g + row0, 4 * (part & 1) + (q ^ (second ? 2 : 0)))) = h;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&v_full[i & 1]);
        mbar_arrive(&raw.empty[rb]);
      }
    }
  }
  group_leave(2, 128);
}

template <bool k4, PaMods kModSet>
__global__ void __launch_bounds__(pp::kThreads, 1)
    paged_prompt_kernel(const __grid_constant__ CUtensorMap k_map, const uint8_t* __restrict__ v_codes,
                        const __grid_constant__ PagedAttnArgs a) {
  using namespace pp;
  constexpr bool kMods = kModSet != kPaPlain;
  constexpr int kEnds = kMods ? kModsSegUnits : kSegUnits;
  constexpr int kKStages = pp::kKStages<k4>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 4 * kQTermBytes;
  uint8_t* sV = sK + kKStages * kKBytes;
  uint8_t* sRaw = sV + 2 * kVBytes;                      // 4 bits: [raw stages] of K, then of V
  int32_t* entry_end = reinterpret_cast<int32_t*>(sV);   // [requests] entries of requests 0 .. b, before V is there

  __shared__ uint64_t k_full[kKStages], k_empty[kKStages], v_full[2], v_empty[2];
  __shared__ uint64_t rawk_full[kRawStages], rawk_empty[kRawStages], rawv_full[kRawStages], rawv_empty[kRawStages];
  __shared__ uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];   // by pairs' half and keys' half
  __shared__ uint64_t q_full[2], o_full[2], o_empty[2], mma_done;
  __shared__ __align__(16) float sks[kMetaBufs][8];   // K scale of each 16 keys of a tile
  __shared__ uint32_t sbad[kMetaBufs];                // 16-key groups without a valid page
  __shared__ int nan_key[kSegBufs][kKvDim];           // first key with a NaN code that only some rows see, by dim
  __shared__ int32_t run_units[kRuns];                // units (without heads) of the runs before
  __shared__ uint32_t scan[kThreads / 32];
  __shared__ float vmax_part[8], v_ref[kSegBufs];     // V's reference of a segment
  __shared__ PpSeg segs[kSegBufs];
  __shared__ uint64_t seg_full[kSegBufs], seg_empty[kSegBufs];
  __shared__ uint32_t tmem_base, bits_all;
  __shared__ bool rec_open;                           // thread 0's: its record has not been written yet

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&k_full[i], k4 ? 4 : 1);               // 4 bits: the widening warps
      mbar_init(&k_empty[i], 2);                       // both halves' scores
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&s_full[i][h], 2);                   // the products, and their issuer
        mbar_init(&p_full[i][h], 4);
        mbar_init(&pv_done[i][h], 1);
      }
      mbar_init(&q_full[i], 4);
      mbar_init(&o_full[i], 2);
      mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < kRawStages; ++i) {
      mbar_init(&rawk_full[i], 1);
      mbar_init(&rawv_full[i], 1);
      mbar_init(&rawk_empty[i], 4);
      mbar_init(&rawv_empty[i], 4);
    }
    for (int i = 0; i < kSegBufs; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 19);                    // every warp of the other roles
    }
    mbar_init(&mma_done, 3);
    prefetch_tmap(&k_map);
    bits_all = 0;
    rec_open = true;
    fence_mbar_init();
  }
  if (warp == kOutWarp) {
    tmem_alloc(&tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // No pdl_wait() yet: the kernel before this one is of the same call and lets this one start only once the call's inputs
  // are complete.  The first write waits for its end, so that this grid's end stands for both.
  const int B = a.num_requests;
  // block-wide inclusive sum of one value a thread
  auto block_sum = [&](uint32_t v) {
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += scan[w];
    return before + incl;
  };
  // Requests that share no rows have no more entries than this (2^22 + 4096 at most, so no sum below passes 32 bits, and by the
  // host's check no sum of their tiles does).  Starts that run back can name the same rows again and again: refused.
  const uint32_t most_entries = (uint32_t)((int64_t)a.num_rows * a.group / kPromptPairs) + B;
  {
    uint32_t bits = 0;
    const int per = (B + kThreads - 1) / kThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    uint32_t sum = 0;
    for (int b = b0; b < b1; ++b) {
      sum = min(sum + pp_entries(a, pa_shape(a, b, bits)), most_entries + 1);
      entry_end[b] = sum;
    }
    const uint32_t before = block_sum(sum) - sum;
    for (int b = b0; b < b1; ++b) entry_end[b] += before;
    if (b0 < b1 && b1 == B && (uint32_t)entry_end[B - 1] > most_entries) {
      entry_end[B - 1] = 0;                            // no entries: nothing is taken
      bits |= DSA_DEVICE_BAD_LENGTH;
    }
    if (bits) atomicOr(&bits_all, bits);
  }
  __syncthreads();
  const int entries = entry_end[B - 1];
  const int run = (entries + kRuns - 1) / kRuns;
  // the entry with index x
  auto find = [&](int x, PpCursor& c) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (entry_end[mid] > x) hi = mid;
      else lo = mid + 1;
    }
    c.b = lo;
    c.qt = x - (lo ? entry_end[lo - 1] : 0);
  };
  {
    int sum = 0;
    const int x0 = min(entries, min(tid, kRuns) * run), x1 = tid < kRuns ? min(entries, x0 + run) : x0;
    if (x0 < x1) {
      PpCursor c;
      find(x0, c);
      for (int x = x0; x < x1; ++x) {
        uint32_t none = 0;
        PaShape sh = pa_shape(a, c.b, none);
        while (c.qt >= pp_entries(a, sh)) {
          sh = pa_shape(a, ++c.b, none);
          c.qt = 0;
        }
        sum += pp_entry(a, sh, c.b, c.qt).tiles + kEnds;
        ++c.qt;
      }
    }
    const int incl = block_sum(sum);
    if (tid < kRuns) run_units[tid] = incl - sum;
    __syncthreads();
    if (tid == kThreads - 1) scan[0] = incl;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int64_t units = (int64_t)scan[0] * a.kv_heads;
  const int64_t u0 = pa_unit_start(cta, units, ctas), u1 = pa_unit_start(cta + 1, units, ctas);
  uint32_t* const err = &bits_all;
  // the scheduler starts at the run that holds u0
  PpCursor cur = {0, 0, 0};
  if (warp == kLoadWarp && u0 < u1) {
    int lo = 0, hi = kRuns - 1;                       // the last run whose units begin at or before u0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)run_units[mid] * a.kv_heads <= u0) lo = mid;
      else hi = mid - 1;
    }
    cur.before = (int64_t)run_units[lo] * a.kv_heads;
    find(min(lo * run, entries - 1), cur);
  }
  __syncthreads();                                     // V's tiles take the place of the entries' sums

  if (warp < kConvWarp0) {
    regs_inc<kRegsSoft>();
    // ---------------------------------------------------------------- softmax and outputs: one pair a thread
    const int q = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t tS = tmem + lanes + 128 * q, tO = tmem + lanes + kColO + 128 * q;
    uint8_t* const q_hi = sQ + 2 * q * kQTermBytes;
    // this thread's pair of a segment: its row and head (of the last pair where there are fewer)
    auto pair_of = [&](const PpSeg& s, int& r, int& head) {
      const int n = min(s.qt * kPromptPairs + kHalfPairs * q + row, s.rows * a.group - 1);
      r = n / a.group;
      head = s.h * a.group + (n - r * a.group);
      return s.qt * kPromptPairs + kHalfPairs * q + row == n;
    };
    // the queries of a segment, once the last segment's scores have been computed
    auto load_queries = [&](const PpSeg& s) {
      const float cf = pp_queries(a, s, s.qt * kPromptPairs + kHalfPairs * q + 32 * quarter, s.rows * a.group, q_hi, 32 * quarter);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[q]);
      return cf;
    };
    int i = 0;
    bool ok = wait_warp(&seg_full[0], 0, err, kErrMmaTimeout, kPolls);
    float cf = 0.f;
    if (ok && segs[0].n) cf = load_queries(segs[0]);
    for (int seg = 0; ok; ++seg) {
      const PpSeg& s = segs[seg % kSegBufs];
      const int tiles = s.n;
      if (tiles == 0) break;
      int r, head;
      const bool there = pair_of(s, r, head);
      PpRow w = {-INFINITY, 0.f, cf, kMods && a.slopes ? a.slopes[head] * 1.4426950408889634f : 0.f, pp_limit(s, r), s.start + r};
      // keys below it are seen by every pair of this half
      const int min_limit = pp_limit(s, min(s.qt * kPromptPairs + kHalfPairs * q, s.rows * a.group - 1) / a.group);
      // 64 keys of tile t.  The masked form is a separate body as a whole, not a variant of a part of it: with one
      // body and the scores' pass chosen inside it the unmasked tiles took 5,400 cycles instead of 3,400.
      auto keys64 = [&](auto masked, int t, int h, uint32_t bad) {
        const int key0 = s.tile_at(t) * kTok + 64 * h;
        const float* ks = sks[i % kMetaBufs] + 4 * h;
        // moves the rows' references where their scores ask for it; true where some did
        auto raise = [&](float top) {
          const bool grow = top > w.m + kSlack || (w.m == -INFINITY && top > w.m);
          if (!__any_sync(0xffffffffu, grow)) return false;
          const float m_new = grow ? top : w.m;
          const float al = m_new == w.m ? 1.f : w.m == -INFINITY ? 0.f : ex2_approx(w.m - m_new);
          w.m = m_new;
          if (t > 0 || h > 0) {
            // the accumulator is settled when the 64 keys before have been added
            ok = wait_warp(&pv_done[q][h ^ 1], (i - 1 + h) & 1, err, kErrMmaTimeout, kPolls);
            if (!ok) return false;
            tc_fence_after();
            pp_shrink(tO, al);
            w.l *= al;
          }
          return true;
        };
        if constexpr (k4 && !kMods && decltype(masked)::value) {
          raise(pp_max64(w, tS + 64 * h, key0, bad >> (4 * h)));
          if (!ok) return;
          w.l += pp_exp64(w, tS + 64 * h, key0, bad >> (4 * h));
        } else if constexpr (kMods || decltype(masked)::value) {
          raise(pp_max64<k4, kModSet, decltype(masked)::value>(w, a, tS + 64 * h, key0, bad >> (4 * h), ks));
          if (!ok) return;
          w.l += pp_exp64(w, tS + 64 * h);
        } else {
          uint32_t p[32];
          float sum;
          while (raise(pp_half<k4>(w, tS + 64 * h, ks, p, sum))) {
          }
          if (!ok) return;
          w.l += sum;
          tmem_st32(tS + 64 * h, p);                   // P takes the first half of the scores' columns
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[q][h]);
      };
      for (int t = 0; t < tiles && ok; ++t, ++i) {
        const int key_end = (s.tile_at(t) + 1) * kTok;
#pragma unroll 1
        for (int h = 0; h < 2 && ok; ++h) {
          // the scores' arrival also stands for the tile's scales: K's own barrier may be a phase further by now
          ok = wait_warp(&s_full[q][h], i & 1, err, kErrMmaTimeout, kPolls);
          if (!ok) break;
          tc_fence_after();
          const uint32_t bad = sbad[i % kMetaBufs];
          if (__any_sync(0xffffffffu, key_end > min_limit || bad)) keys64(std::true_type{}, t, h, bad);
          else keys64(std::false_type{}, t, h, 0);
        }
      }
      if (!ok) break;
      const int nx = (seg + 1) % kSegBufs;
      ok = wait_warp(&seg_full[nx], ((seg + 1) / kSegBufs) & 1, err, kErrMmaTimeout, kPolls);
      if (!ok) break;
      if (segs[nx].n) cf = load_queries(segs[nx]);
      if (seg == 0) {
        pdl_wait();
        if (tid == 0) {
          reinterpret_cast<PaRecord*>(a.rec)[cta].tile = -1;   // no piece to join until it has been written
          rec_open = false;
        }
      }
      // ---- the segment's end
      const bool whole = s.n == s.tiles;
      ok = wait_warp(&o_full[q], seg & 1, err, kErrMmaTimeout, kPolls);
      if (!ok) break;
      tc_fence_after();
      const float m = w.m, l = w.l;
      const bool any = l > 0.f || l != l;
      const int64_t at = (int64_t)(s.row0 + r) * a.kv_heads * a.group + head;
      const int slot = s.slot;
      const float vref = v_ref[seg % kSegBufs];
      // a mean of V before its scale comes in: sums over keys times the largest scales would leave fp32's range, and the smallest
      // scales divided by the sums, too
      const float inv = any ? (k4 ? 1.f / kV4Up : 1.f) / l : 0.f;
      const int* nk = nan_key[seg % kSegBufs];       // (4 bits: a key is NaN as a whole)
#pragma unroll 1
      for (int c = 0; c < kKvDim; c += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c, o);
        tmem_wait_ld();
        if (there) {
          float x[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            x[k] = __uint_as_float(o[k]) * inv * vref;
            if (nk[k4 ? 0 : c + k] < w.limit) x[k] = __int_as_float(0x7FC00000);
          }
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + at * kKvDim + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint4 v;
              uint32_t* vv = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
              for (int k2 = 0; k2 < 4; ++k2) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[8 * k + 2 * k2], x[8 * k + 2 * k2 + 1]);
                vv[k2] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              dst[k] = v;
            }
          } else {
            // [slot][dim / 4][pair] float4: a warp's stores are contiguous
            float4* dst = reinterpret_cast<float4*>(a.part_o) + ((int64_t)slot * (kKvDim / 4) + c / 4) * kPromptPairs + kHalfPairs * q + row;
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[k * kPromptPairs] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          }
        }
      }
      if (there) {
        if (!whole) {
          reinterpret_cast<float2*>(a.part_ml)[(int64_t)slot * kPromptPairs + kHalfPairs * q + row] = make_float2(m, l);
        } else if (a.lse) {
          a.lse[at] = any ? (m - kPLog2 + __log2f(l)) * 0.69314718055994530942f : -INFINITY;
        }
      }
      if (tid == 0 && seg == 0)                        // for the join: this CTA's first piece
        reinterpret_cast<PaRecord*>(a.rec)[cta] = {units, s.tile, s.tiles, s.row0, s.rows * a.group, s.qt * kPromptPairs, s.h};
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&o_empty[q]);
        mbar_arrive(&seg_empty[seg % kSegBufs]);
      }
    }
  } else if (warp < kOutWarp) {
    regs_dec<kRegsConv>();
    if constexpr (k4) {
      if (warp < kConvWarp0 + 4) {
        pp_widen_k4(segs, seg_full, seg_empty, k_full, k_empty, sK, PpRaw{sRaw, rawk_full, rawk_empty, sbad}, err);
      } else {
        pp_widen_v4(a, segs, seg_full, seg_empty, v_full, v_empty, sV,
                    PpRaw{sRaw + kRawStages * kRawKBytes, rawv_full, rawv_empty, sbad}, &nan_key[0][0], vmax_part, v_ref, err);
      }
    } else {
    // ---------------------------------------------------------------- V tiles: codes to fp16
    // Two groups of four warps take alternate tiles: eight lanes a row of 16-byte pieces, 16 rows a pass, so that a
    // pass is one 16-key group and lies in one page.  Eight neighbouring lanes hold half of two rows each, whose
    // units in the swizzled tile do not share a bank.  A tile's loads go out after the last tile's fence, which
    // would wait for loads in flight too.
    const int grp = (warp - kConvWarp0) >> 2, cw = warp & 3, lp = a.log2_page;
    const int part = (lane & 3) + 4 * (lane >> 4), sub = 4 * cw + ((lane >> 2) & 3);
    uint8_t* const tile = sV + grp * kVBytes + (part >> 2) * kChunkBytes + sub * 128;   // row 16 g + sub: 2048 g on
    const int at_lo = ((2 * (part & 3)) ^ (sub & 7)) << 4, at_hi = ((2 * (part & 3) + 1) ^ (sub & 7)) << 4;
    int i0 = 0;                                        // the CTA's tiles before this segment
    bool ok = true;
    for (int seg = 0;; ++seg) {
      ok = wait_warp(&seg_full[seg % kSegBufs], (seg / kSegBufs) & 1, err, kErrMmaTimeout, kPolls);
      if (!ok) break;
      const PpSeg s = segs[seg % kSegBufs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[seg % kSegBufs]);
      if (s.n == 0) break;
      const int len = s.len, pages = (len + (1 << lp) - 1) >> lp;
      const int32_t* table = a.block_table + (int64_t)s.b * a.table_stride;
      // this lane's 16 bytes of row 0 of page 0; a page further is page_step bytes on
      const uint8_t* const base = v_codes + ((int64_t)s.h << lp) * kKvDim + 16 * part;
      const int64_t page_step = ((int64_t)a.kv_heads << lp) * kKvDim;
      // the page of a key, -1 where there is none (the loader of K reports bad ids)
      auto id_of = [&](int key) {
        const int p = key >> lp;
        const int id = p < pages ? table[p] : -1;
        return id < a.num_pages ? id : -1;
      };
      // V's reference: the power of two at or below the piece's largest scale
      float top = 0.f;
      const int p0 = (s.tile * kTok) >> lp, p1 = min(pages, ((s.tile + s.n) * kTok) >> lp);
#pragma unroll 4
      for (int p = p0 + 32 * (warp - kConvWarp0) + lane; p < p1; p += 256) {
        const int id = table[p];
        if (id >= 0 && id < a.num_pages) top = fmaxf(top, fabsf(a.v_scales[(int64_t)id * a.kv_heads + s.h]));
      }
      top = warp_max_f32(top);
      if (lane == 0) vmax_part[warp - kConvWarp0] = top;
      if (grp == 0) nan_key[seg % kSegBufs][32 * cw + lane] = INT32_MAX;
      group_sync(1, 256);
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, vmax_part[k]);
      const uint32_t top_bits = __float_as_uint(top) & 0x7F800000u;
      const float vref = top_bits && top_bits < 0x7F800000u ? __uint_as_float(top_bits) : 1.f;
      if (warp == kConvWarp0 && lane == 0) v_ref[seg % kSegBufs] = vref;
      const float vinv = 1.f / vref;
      group_sync(1, 256);
      const int min_limit = pp_limit(s, min(s.qt * kPromptPairs, s.rows * a.group - 1) / a.group);

      uint4 x[8];
      float scale = 0.f;
      int t = (i0 + grp) & 1;
      // lane g (and g + 8, ..): the page of 16-key group g, of the tile to load and of this group's next one
      const int own = 16 * (lane & 7);
      int id = t < s.n ? id_of(s.tile_at(t) * kTok + own) : -1, id2 = t + 2 < s.n ? id_of(s.tile_at(t + 2) * kTok + own) : -1;
      auto load = [&](int key0) {
        scale = id >= 0 ? a.v_scales[(int64_t)id * a.kv_heads + s.h] : 0.f;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const int page = __shfl_sync(0xffffffffu, id, g), key = key0 + 16 * g + sub;
          x[g] = make_uint4(0, 0, 0, 0);
          if (page >= 0 && key < len)
            x[g] = __ldg(reinterpret_cast<const uint4*>(base + page * page_step + (key & ((1 << lp) - 1)) * kKvDim));
        }
      };
      if (t < s.n) load(s.tile_at(t) * kTok);
      for (; t < s.n; t += 2) {
        const int key0 = s.tile_at(t) * kTok, i = i0 + t;
        if (i >= 2) ok = wait_warp(&v_empty[grp], ((i >> 1) - 1) & 1, err, kErrMmaTimeout, kPolls);
        if (!ok) break;
        // NaN codes of a tile that only some rows see in full
        uint32_t any_nan = 0;
        if (key0 + kTok > min_limit) {
#pragma unroll
          for (int g = 0; g < 8; ++g)
            any_nan |= ((x[g].x & 0x7F7F7F7Fu) + 0x01010101u) | ((x[g].y & 0x7F7F7F7Fu) + 0x01010101u) |
                       ((x[g].z & 0x7F7F7F7Fu) + 0x01010101u) | ((x[g].w & 0x7F7F7F7Fu) + 0x01010101u);
          any_nan &= 0x80808080u;
        }
        const float ratio = scale * vinv;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const __half2 f = __float2half2_rn(__shfl_sync(0xffffffffu, ratio, g));
          uint4 lo = widen8(x[g].x, x[g].y), hi = widen8(x[g].z, x[g].w);
          lo = make_uint4(mul2(lo.x, f), mul2(lo.y, f), mul2(lo.z, f), mul2(lo.w, f));
          hi = make_uint4(mul2(hi.x, f), mul2(hi.y, f), mul2(hi.z, f), mul2(hi.w, f));
          *reinterpret_cast<uint4*>(tile + 2048 * g + at_lo) = lo;
          *reinterpret_cast<uint4*>(tile + 2048 * g + at_hi) = hi;
        }
        if (any_nan) {
          // out of the tile, and noted for the rows that see the key
#pragma unroll 1
          for (int k = 0; k < 8 * 16; ++k) {
            const int g = k >> 4, e = k & 15;
            uint16_t* v = reinterpret_cast<uint16_t*>(tile + 2048 * g + (e < 8 ? at_lo : at_hi)) + (e & 7);
            if ((*v & 0x7FFFu) > 0x7C00u) {
              *v = 0;
              atomicMin(&nan_key[seg % kSegBufs][16 * part + e], key0 + 16 * g + sub);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[grp]);
        if (t + 2 < s.n) {
          id = id2;
          id2 = t + 4 < s.n ? id_of(key0 - 4 * kTok + own) : -1;
          load(key0 - 2 * kTok);
        }
      }
      if (!ok) break;
      i0 += s.n;
    }
    }
    group_leave(1, 256);
  } else {
    regs_dec<kRegsRest>();
    if (warp == kOutWarp) {
      // ---------------------------------------------------------------- output products of both halves
      const bool leader = elect_one();
      const uint32_t id_o = idesc_f16(128, kKvDim, false, false, false, true);
      const uint64_t d_v = smem_desc(smem_u32(sV), kChunkBytes, 1024, kSwizzle128B);
      bool ok = true;
      int i = 0;
      for (int seg = 0;; ++seg) {
        ok = wait_warp(&seg_full[seg % kSegBufs], (seg / kSegBufs) & 1, err, kErrMmaTimeout, kPolls);
        if (!ok) break;
        const int n = segs[seg % kSegBufs].n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[seg % kSegBufs]);
        if (n == 0) break;
        for (int t = 0; t < n && ok; ++t, ++i) {
          const uint64_t v = d_v + (uint64_t)(((i & 1) * kVBytes) >> 4);
          ok = wait_warp(&v_full[i & 1], (i >> 1) & 1, err, kErrMmaTimeout, kPolls);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (t == 0 && h == 0 && seg > 0) ok = ok && wait_warp(&o_empty[q], (seg - 1) & 1, err, kErrMmaTimeout, kPolls);
              ok = ok && wait_warp(&p_full[q][h], i & 1, err, kErrMmaTimeout, kPolls);
              if (!ok) break;
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_ts(tmem + kColO + 128 * q, tmem + 128 * q + 64 * h + 8 * kk, v + (uint64_t)(((64 * h + 16 * kk) * 128) >> 4),
                         id_o, t > 0 || h > 0 || kk > 0);
                mma_commit(&pv_done[q][h]);
                if (h == 1 && q == 1) mma_commit(&v_empty[i & 1]);
                if (h == 1 && t + 1 == n) {
                  mma_commit(&o_full[q]);
                  mbar_arrive(&o_full[q]);
                }
              }
              __syncwarp();
            }
        }
        if (!ok) break;
      }
      if (leader) mma_commit(&mma_done);
      wait_warp(&mma_done, 0, err, kErrMmaTimeout, kPolls);
    } else if (warp < kLoadWarp) {
      // ---------------------------------------------------------------- score products of one half
      const int q = warp - kScoreWarp0;
      const bool leader = elect_one();
      const uint32_t id_s = idesc_e4m3(128, 64) | (k4 ? kFmtE5m2 << 10 : 0u);
      const uint64_t d_q = smem_desc(smem_u32(sQ + 2 * q * kQTermBytes), 16, 1024, kSwizzle128B);
      const uint64_t d_k = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
      bool ok = true;
      int i = 0;
      for (int seg = 0;; ++seg) {
        ok = wait_warp(&seg_full[seg % kSegBufs], (seg / kSegBufs) & 1, err, kErrMmaTimeout, kPolls);
        if (!ok) break;
        const int n = segs[seg % kSegBufs].n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[seg % kSegBufs]);
        if (n == 0) break;
        ok = wait_warp(&q_full[q], seg & 1, err, kErrMmaTimeout, kPolls);
        for (int t = 0; t < n && ok; ++t, ++i) {
          const int st = i % kKStages;
          ok = wait_warp(&k_full[st], (i / kKStages) & 1, err, kErrTmaTimeout, kPolls);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // S takes the place of the P of the tile before, once O has read it
            if (i > 0) ok = ok && wait_warp(&pv_done[q][h], (i - 1) & 1, err, kErrMmaTimeout, kPolls);
            if (!ok) break;
            tc_fence_after();
            const uint64_t k = d_k + (uint64_t)((st * kKBytes + 64 * h * kKvDim) >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)           // hi, then lo
                mma_ss_f8(tmem + 128 * q + 64 * h, d_q + (uint64_t)(((kk >> 2) * kQTermBytes + (kk & 3) * 32) >> 4), k + 2 * (kk & 3),
                          id_s, kk > 0);
              mma_commit(&s_full[q][h]);
              mbar_arrive(&s_full[q][h]);
              if (h == 1) mma_commit(&k_empty[st]);
            }
            __syncwarp();
          }
        }
        if (!ok) break;
      }
      if (leader) mma_commit(&mma_done);
      wait_warp(&mma_done, 0, err, kErrMmaTimeout, kPolls);
    } else {
      // ---------------------------------------------------------------- segments (and an end mark), and their K tiles
      const uint64_t policy = l2_evict_normal();
      const int lp = a.log2_page, ppt = kTok >> lp;
      const uint32_t page_bytes = (uint32_t)kKvDim << lp;
      int i = 0;
      int64_t u = u0;
      bool ok = true;
      // 4 bits: a page a lane of the tile whose V is to be copied next (its first row, or -1), and how many there are; tiles of K and
      // of V whose copies are under way or done
      int v_row = -1;
      uint32_t v_pages = 0;
      int k_tiles = 0, v_tiles = 0;
      // codes (lanes 0 .. ppt - 1, a page each) and scales (lanes 8 ..) of K or of V, of the rows from `row` on
      auto copy_raw = [&](int row, uint32_t loads, uint8_t* to, uint64_t* full, const uint8_t* codes, const void* scales, int scale_bytes) {
        if (lane == 0) mbar_arrive_expect_tx(full, loads * ((uint32_t)(kKvDim / 2 + scale_bytes) << lp));
        __syncwarp();
        if (lane < 16 && row >= 0) {
          const int mine = lane & 7;
          const uint32_t bytes = (uint32_t)(lane < 8 ? kKvDim / 2 : scale_bytes);
          bulk_load_hint(to + (lane < 8 ? 0 : kTok * kKvDim / 2) + mine * (bytes << lp),
                         (lane < 8 ? codes : static_cast<const uint8_t*>(scales)) + (int64_t)row * bytes, bytes << lp, full, policy);
        }
      };
      // V lags a tile: it is widened later than K, and its place comes free later
      auto copy_v = [&](int j) {
        const int rb = j % kRawStages;
        if (j >= kRawStages && !wait_warp(&rawv_empty[rb], (j / kRawStages - 1) & 1, err, kErrMmaTimeout, kPolls)) return false;
        copy_raw(v_row, v_pages, sRaw + kRawStages * kRawKBytes + rb * kRawVBytes, &rawv_full[rb], v_codes, a.v_scales4, 2);
        v_tiles = j + 1;
        return true;
      };
      for (int seg = 0;; ++seg) {
        if (seg >= kSegBufs) ok = wait_warp(&seg_empty[seg % kSegBufs], (seg / kSegBufs - 1) & 1, err, kErrMmaTimeout, kPolls);
        if (!ok) break;
        PpSeg s = {};
        // segments are cut where the range ends, or (short requests) belong as a whole to the range with their first tile
        while (u < u1 && s.n == 0) {
          s = pp_segment<kEnds>(a, cur, u, a.whole ? units : u1, cta);
          if (a.whole && (s.tile > 0 || u - s.n >= u1)) s.n = 0;
        }
        if (lane == 0) {
          segs[seg % kSegBufs] = s;
          mbar_arrive(&seg_full[seg % kSegBufs]);
        }
        __syncwarp();
        if (s.n == 0) break;
        // its queries on their way into L2: they are loaded when the segment before ends, with nothing to hide them
        if (seg > 0) {
          const int first = s.qt * kPromptPairs, last = min(first + kPromptPairs, s.rows * a.group);
          for (int n = first + (lane >> 1); n < last; n += 16) {
            const int r = n / a.group, g = n - r * a.group;
            const __nv_bfloat16* p = a.q + (int64_t)(s.row0 + r) * a.q_stride + (int64_t)(s.h * a.group + g) * kKvDim + 64 * (lane & 1);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
          }
        }
        const int pages = (s.len + (1 << lp) - 1) >> lp;
        int batch = -1, page = -1;                     // 32 pages at a time, one a lane
        float ks = 0.f;
        for (int t = 0; t < s.n; ++t, ++i) {
          const int p0 = s.tile_at(t) * ppt;
          if ((p0 >> 5) != batch) {
            batch = p0 >> 5;
            const int p = 32 * batch + lane;
            page = -1;
            if (p < pages) {
              page = a.block_table[(int64_t)s.b * a.table_stride + p];
              if (page < 0 || page >= a.num_pages) {
                if (p >= s.tile * ppt && p < p0 + ppt) atomicOr(err, kErrBadPage);
                page = -1;
              }
            }
            ks = !k4 && page >= 0 ? a.k_scales[(int64_t)page * a.kv_heads + s.h] : 0.f;
          }
          const int st = i % kKStages, use = i / kKStages, rb = i % kRawStages;
          if (k4) {
            if (i >= kRawStages) ok = wait_warp(&rawk_empty[rb], (i / kRawStages - 1) & 1, err, kErrMmaTimeout, kPolls);
          } else if (use > 0) {
            ok = wait_warp(&k_empty[st], (use - 1) & 1, err, kErrMmaTimeout, kPolls);
          }
          if (!ok) break;
          const int o = p0 & 31;
          if constexpr (k4) {
            const int mine = lane & 7;
            const int id = __shfl_sync(0xffffffffu, page, (o + mine) & 31);
            const int of_group = __shfl_sync(0xffffffffu, page, (o + ((16 * mine) >> lp)) & 31);
            const uint32_t bad = __ballot_sync(0xffffffffu, lane < 8 && of_group < 0);
            const int row = mine < ppt && id >= 0 ? (id * a.kv_heads + s.h) << lp : -1;   // (the host holds rows below 2^31)
            const uint32_t loads = __popc(__ballot_sync(0xffffffffu, lane < 8 && row >= 0));
            if (lane == 0) sbad[i % kMetaBufs] = bad;
            copy_raw(row, loads, sRaw + rb * kRawKBytes, &rawk_full[rb], a.k_codes4, a.k_scales4, kKv4Blocks);
            k_tiles = i + 1;
            if (i > 0) ok = copy_v(i - 1);
            if (!ok) break;
            v_row = row;
            v_pages = loads;
            continue;
          }
          const int pg = __shfl_sync(0xffffffffu, page, (o + lane) & 31);
          // 16-key group g lies in page g * 16 / page size of the tile
          const int of_group = (o + ((16 * (lane & 7)) >> lp)) & 31;
          const float kg = __shfl_sync(0xffffffffu, ks, of_group);
          const int pg_g = __shfl_sync(0xffffffffu, page, of_group);   // every lane takes part
          const uint32_t bad = __ballot_sync(0xffffffffu, lane < 8 && pg_g < 0);
          const bool load = lane < ppt && pg >= 0;
          const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
          if (lane < 8) sks[i % kMetaBufs][lane] = kg;
          if (lane == 0) sbad[i % kMetaBufs] = bad;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&k_full[st], loads * page_bytes);
          __syncwarp();
          if (load) tma_load_2d_hint(sK + st * kKBytes + lane * page_bytes, &k_map, 0, (pg * a.kv_heads + s.h) << lp, &k_full[st], policy);
        }
        if (!ok) break;
      }
      // nothing may still be landing in shared memory when the CTA exits
      if constexpr (k4) {
        if (i > 0 && ok) ok = copy_v(i - 1);
        auto landed = [&](uint64_t* full, int tiles) {   // the last of these tiles in each place
          for (int rb = 0; rb < kRawStages; ++rb)
            if (tiles > rb) wait_warp(&full[rb], ((tiles - rb + kRawStages - 1) / kRawStages - 1) & 1, err, kErrTmaTimeout, kPolls);
        };
        landed(rawk_full, k_tiles);
        landed(rawv_full, v_tiles);
      } else {
        for (int st = 0; st < kKStages; ++st)
          if (i > st) wait_warp(&k_full[st], ((i - st + kKStages - 1) / kKStages - 1) & 1, err, kErrTmaTimeout, kPolls);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kOutWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0) {
    pdl_wait();
    if (rec_open) reinterpret_cast<PaRecord*>(a.rec)[cta].tile = -1;
    a.err[kStatusCtaWords + cta] |= bits_all;          // beside what the first kernel reported
  }
}

template <bool k4>
cudaError_t launch_prompt(const PagedAttnArgs& a, const CUtensorMap& k_map, const uint8_t* v_codes, int ctas, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = once_per_device(ready, [] {
    const int most = pp::kFixedSmem<k4>;
    cudaError_t r = cudaFuncSetAttribute(paged_prompt_kernel<k4, kPaPlain>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(paged_prompt_kernel<k4, kPaCapBias>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(paged_prompt_kernel<k4, kPaLargeCap>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return r;
  });
  if (e != cudaSuccess) return e;
  const PaMods mods = pa_mods(a);
  auto kernel = mods == kPaPlain     ? paged_prompt_kernel<k4, kPaPlain>
                : mods == kPaCapBias ? paged_prompt_kernel<k4, kPaCapBias>
                                     : paged_prompt_kernel<k4, kPaLargeCap>;
  e = launch_pdl(kernel, dim3(ctas), dim3(pp::kThreads), pp::kFixedSmem<k4>, s, k_map, v_codes, a);
  count_launches(1);
  return e;
}

#ifndef DSA_PAGED_KERNEL_ONLY
// Joins the pieces of the segments that CTA boundaries cut, as pa_join: a thread a pair, 16 dims of it per y.
__device__ __forceinline__ void pp_join(const PagedAttnArgs& a, int ctas, int c, int y) {
  const PaRecord rec = pa_load_record(a, c);
  int first, last, first_slot;
  if (!pa_pieces(rec, c, ctas, first, last, first_slot)) return;
  const int n = rec.first_pair + threadIdx.x;
  if (n >= rec.pairs) return;
  const int64_t units = rec.units;
  float M = -INFINITY, L = 0.f;
  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  constexpr int kGroup = 2;                                // pieces whose loads are in flight together
  for (int p0 = first; p0 <= last; p0 += kGroup) {
    float2 ml[kGroup];
    float4 x[kGroup][4];
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      const int p = p0 + g;
      ml[g] = make_float2(-INFINITY, 0.f);
      if (p <= last && (units >= ctas || pa_unit_start(p, units, ctas) < pa_unit_start(p + 1, units, ctas))) {
        const int64_t slot = p == first ? first_slot : 2 * p;
        ml[g] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot * kPromptPairs + threadIdx.x);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[g][k] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (slot * (kKvDim / 4) + 4 * y + k) * kPromptPairs + threadIdx.x);
      }
    }
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      if (ml[g].y == 0.f) continue;                        // a piece that sees nothing (NaN counts as seen)
      const float Mn = fmaxf(M, ml[g].x);
      const float Lo = M == -INFINITY ? 0.f : L * exp2f(M - Mn), lg = ml[g].y * exp2f(ml[g].x - Mn);
      L = Lo + lg;
      const float inv = 1.f / L, sc = Lo * inv, w = lg * inv;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[4 * k] = fmaf(w, x[g][k].x, acc[4 * k] * sc);
        acc[4 * k + 1] = fmaf(w, x[g][k].y, acc[4 * k + 1] * sc);
        acc[4 * k + 2] = fmaf(w, x[g][k].z, acc[4 * k + 2] * sc);
        acc[4 * k + 3] = fmaf(w, x[g][k].w, acc[4 * k + 3] * sc);
      }
      M = Mn;
    }
  }
  const int i = n / a.group;
  const int64_t at = (int64_t)(rec.row0 + i) * a.kv_heads * a.group + rec.h * a.group + (n - i * a.group);
  uint4 v[2];
  __nv_bfloat162* xo = reinterpret_cast<__nv_bfloat162*>(v);
#pragma unroll
  for (int e = 0; e < 8; ++e) xo[e] = __floats2bfloat162_rn(acc[2 * e], acc[2 * e + 1]);
  uint4* dst = reinterpret_cast<uint4*>(a.out + at * kKvDim) + 2 * y;
  dst[0] = v[0];
  dst[1] = v[1];
  if (a.lse && y == 0) a.lse[at] = L == 0.f ? -INFINITY : (M - pp::kPLog2 + log2f(L)) * 0.69314718055994530942f;
}

// Both kernels' joins in one launch, so that nothing stands between the two kernels
__global__ void __launch_bounds__(kPromptPairs)
    paged_prompt_join_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ PagedAttnArgs few, int few_y, int ctas) {
  static_assert(kPromptPairs == 256, "pa_join's block");
  pdl_wait();
  pdl_trigger();
  const int y = blockIdx.y;
  if (y < few_y) pa_join(few, ctas, blockIdx.x + 1, y);
  else pp_join(a, ctas, blockIdx.x + 1, y - few_y);
}

cudaError_t launch_prompt_join(const PagedAttnArgs& a, const PagedAttnArgs& few, int few_y, int ctas, cudaStream_t s) {
  if (ctas < 2 || a.whole) return cudaSuccess;
  const cudaError_t e = launch_pdl(paged_prompt_join_kernel, dim3(ctas - 1, few_y + kKvDim / 16), dim3(kPromptPairs), 0, s, a, few, few_y, ctas);
  count_launches(1);
  return e;
}

cudaError_t launch_paged_prompt(const PagedAttnArgs& a, const PagedAttnArgs& few, int few_y, const CUtensorMap& k_map,
                                const uint8_t* v_codes, int ctas, cudaStream_t s) {
  const cudaError_t e = launch_prompt<false>(a, k_map, v_codes, ctas, s);
  return e != cudaSuccess ? e : launch_prompt_join(a, few, few_y, ctas, s);
}
#endif  // DSA_PAGED_KERNEL_ONLY

}  // namespace dsa
