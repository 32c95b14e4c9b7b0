// Shared by the two dense attention kernels: what a request brings, and the split of the units over CTAs.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_internal.cuh"

namespace dsa {

constexpr int kPaTok = 128;          // keys per tile

// Rows, first row and readable keys of request b.  rows is 0 where the call leaves the request alone: no rows, more than
// max_rows or rows that the batch does not have (reported), or a number of (row, head) pairs outside (lo, hi], which the
// other kernel takes.
struct PaShape {
  int rows, row0, len, tiles;        // tiles: of 128 keys, at least one
};

__device__ __forceinline__ PaShape pa_shape(const PagedAttnArgs& a, int b, uint32_t& bits) {
  PaShape s = {0, b, 0, 0};
  const int held = a.seq_lens[b];    // with the offsets, not after them: at the start every load is a trip to L2
  int n = 1;
  if (a.query_start_loc) {
    s.row0 = a.query_start_loc[b];
    const int64_t d = (int64_t)a.query_start_loc[b + 1] - s.row0;
    if (d == 0) return s;
    if (d < 0 || d > a.max_rows || s.row0 < 0 || s.row0 + d > a.num_rows) {
      bits |= DSA_DEVICE_BAD_LENGTH;
      return s;
    }
    n = (int)d;
  }
  const int64_t pairs = (int64_t)n * a.group;
  if (pairs <= a.lo_pairs || pairs > a.hi_pairs) return s;
  const int64_t room = (int64_t)a.table_stride << a.log2_page;
  int64_t len = max(held, 0);
  if (len > room) {
    bits |= DSA_DEVICE_BAD_PAGE;
    len = room;
  }
  s.rows = n;
  s.len = (int)len;
  s.tiles = max(1, (int)((len + kPaTok - 1) / kPaTok));
  return s;
}

// Two bf16 values as two e4m3 terms: hi = e4m3(x up), lo = e4m3(kLo (x up - hi)), with up a power of two that brings the
// row's largest value to [128, 256).  x up is exact in bf16, and in fp16 too but far below e4m3's smallest step; so are the
// difference and its product with kLo.  Half the instructions of the same steps in fp32.
template <int kLo>
__device__ __forceinline__ void pa_split(uint32_t w, __nv_bfloat162 up, uint32_t& hi, uint32_t& lo) {
  const float2 x = __bfloat1622float2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), up));
  const __half2 h = __floats2half2_rn(x.x, x.y);
  hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
  const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3);
  __half2 d = __hsub2(h, __half2(back));
  if (kLo != 1) d = __hmul2(d, __float2half2_rn((float)kLo));
  lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(d), __NV_SATFINITE, __NV_E4M3);
}

// The exponent of a row's largest value (its bf16 bits, sign off), held at -100: smaller rows score 0.
__device__ __forceinline__ int pa_exponent(uint32_t top) { return max((int)(top >> 7) - 127, -100); }
__device__ __forceinline__ __nv_bfloat162 pa_up(int E) {        // 2^(7 - E), twice
  const uint32_t b = (uint32_t)(7 - E + 127) << 7, bb = b | b << 16;
  return *reinterpret_cast<const __nv_bfloat162*>(&bb);
}
// What a row's scores are multiplied with: 2^(E - 7) (exact) times the scale.  A row with an infinity or NaN scores NaN,
// as the infinity's product with a key's zeros or mixed signs does.
__device__ __forceinline__ float pa_factor(uint32_t top, int E, float scale) {
  return top >= 0x7F80u ? __int_as_float(0x7FC00000) : __uint_as_float((uint32_t)(E - 7 + 127) << 23) * scale;
}

// Requests of many rows (paged_prompt.cu), and the join of both kernels' pieces (few: the first kernel's arguments, few_y
// groups of 8 columns); k_map: the K codes in boxes of a page.
cudaError_t launch_paged_prompt(const PagedAttnArgs& a, const PagedAttnArgs& few, int few_y, const CUtensorMap& k_map,
                                const uint8_t* v_codes, int ctas, cudaStream_t s);

// A capped score: cap * tanh(z / cap), with y = 2 log2(e) / cap * z and all in log2 units.
//   small caps: cap * (1 - 2 / (1 + 2^y)), exact to about 2^-22 of the cap (1.5e-5 of a score at a cap of 64); past the
//   range of 2^y the quotient is 0 or 2, and NaN stays.
//   large caps: an error of the cap's size would be one of 0.1 at a cap of 1e6, and past 1e8 every score would be 0.  Where
//   |z / cap| is below 0.3 the odd series takes over, t - t^3/3 + 2 t^5/15 - 17 t^7/315 + 62 t^9/2835 with t = z / cap =
//   ln(2) / 2 y: the next term is below 2^-24 of the score, and a score is held to 2^-21 of itself.
// The series' eight instructions a score cost the mixed capped batch 110 us instead of 95, and 6 % even where a branch steps
// around them, so kernels for large caps are compiled apart.
constexpr float kLargeCap = 64.f * 1.44269504f;         // log2 units
enum PaMods : int { kPaPlain, kPaCapBias, kPaLargeCap };   // plain scores; a cap, a distance bias or both; with a large cap
__host__ __device__ __forceinline__ PaMods pa_mods(const PagedAttnArgs& a) {
  return a.cap_log2 > kLargeCap ? kPaLargeCap : a.cap_log2 > 0.f || a.slopes ? kPaCapBias : kPaPlain;
}
template <PaMods kModSet>
__device__ __forceinline__ float capped(float y, float cap) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  const float quotient = fmaf(-2.f * cap, r, cap);
  if (kModSet != kPaLargeCap) return quotient;
  constexpr float kHalfLn2 = 0.34657359f, kSq = kHalfLn2 * kHalfLn2;
  const float s = y * y;
  float p = fmaf(62.f / 2835.f * kSq * kSq * kSq * kSq, s, -17.f / 315.f * kSq * kSq * kSq);
  p = fmaf(p, s, 2.f / 15.f * kSq * kSq);
  p = fmaf(p, s, -1.f / 3.f * kSq);
  p = fmaf(p, s, 1.f);
  return fabsf(y) < 0.86f ? kHalfLn2 * cap * y * p : quotient;
}

// Units [start(c), start(c + 1)) belong to CTA c: units * c / ctas.
__device__ __forceinline__ int64_t pa_unit_start(int c, int64_t units, int ctas) {
  if (units < (int64_t(1) << 31)) {                     // 32-bit divisions: (q ctas + r) c / ctas = q c + r c / ctas
    const uint32_t n = (uint32_t)units, q = n / (uint32_t)ctas, r = n - q * (uint32_t)ctas;
    return (int64_t)q * c + r * (uint32_t)c / (uint32_t)ctas;
  }
  return units * c / ctas;
}

__device__ __forceinline__ int pa_cta_of_unit(int64_t u, int64_t units, int ctas) {
  int c = units < (int64_t(1) << 31) / ctas ? (int)((uint32_t)u * (uint32_t)ctas / (uint32_t)units) : (int)(u * ctas / units);
  while (c + 1 < ctas && pa_unit_start(c + 1, units, ctas) <= u) ++c;
  while (c > 0 && pa_unit_start(c, units, ctas) > u) --c;
  return c;
}

// What a CTA leaves about the first segment of its range, for the join: all that it needs besides the pieces.
struct __align__(16) PaRecord {
  int64_t units;
  int32_t tile, tiles;             // the segment's tiles, and which of them the range begins with (-1: nothing written)
  int32_t row0, pairs;             // the request's first row, and its (row, head) pairs
  int32_t first_pair, h;           // the segment's first pair, and its K/V head
};
static_assert(sizeof(PaRecord) == 32, "two 16-byte loads");

__device__ __forceinline__ PaRecord pa_load_record(const PagedAttnArgs& a, int c) {
  union {
    int4 w[2];
    PaRecord r;
  } x;
  const int4* p = reinterpret_cast<const int4*>(a.rec) + 2 * c;
  x.w[0] = __ldcg(p);
  x.w[1] = __ldcg(p + 1);
  return x.r;
}

// The pieces of the segment that the boundary in front of range c cuts: CTAs first .. last, the first one's (which begins
// with the segment's first tile) in first_slot, the others' in slot 2 * CTA.  False where there is none, or an
// earlier boundary cuts it too.
__device__ __forceinline__ bool pa_pieces(const PaRecord& r, int c, int ctas, int& first, int& last, int& first_slot) {
  if (r.tile <= 0) return false;                          // nothing written, or the range begins with a segment
  const int64_t u = pa_unit_start(c, r.units, ctas);
  if (u == pa_unit_start(c + 1, r.units, ctas)) return false;
  const int64_t seg = u - r.tile;
  first = pa_cta_of_unit(u - 1, r.units, ctas);
  if (pa_unit_start(first, r.units, ctas) > seg) return false;
  last = pa_cta_of_unit(seg + r.tiles - 1, r.units, ctas);
  first_slot = 2 * first + 1;
  return true;
}

// Joins the pieces of the segments that CTA boundaries cut, each an output o_p of its own keys:
//   out = sum_p w_p o_p,  w_p = 2^{m_p - M} l_p / L,  L = sum_p 2^{m_p - M} l_p.
// Pieces and running sum are weighted means of V throughout: V's scales go up to 2^120, and a sum over keys before its
// division by L would leave fp32's range.
// A block (c, y) handles the boundary in front of range c if it is the first that cuts its segment, and
// columns 8 y .. 8 y + 7: a warp a column, four dims a lane.
__device__ __forceinline__ void pa_join(const PagedAttnArgs& a, int ctas, int c, int y) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PaRecord rec = pa_load_record(a, c);
  int first, last, first_slot;
  if (!pa_pieces(rec, c, ctas, first, last, first_slot)) return;
  const int col = 8 * y + warp, n = rec.first_pair + col;
  if (n >= rec.pairs) return;
  const int64_t units = rec.units;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kGroup = 4;                               // pieces whose loads are in flight together
  for (int p0 = first; p0 <= last; p0 += kGroup) {
    float mj[kGroup], lj[kGroup];
    float4 x[kGroup];
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      const int p = p0 + g;
      mj[g] = -INFINITY;
      lj[g] = 0.f;
      x[g] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p <= last && (units >= ctas || pa_unit_start(p, units, ctas) < pa_unit_start(p + 1, units, ctas))) {
        const int64_t at = (int64_t)(p == first ? first_slot : 2 * p) * kPagedAttnColumns + col;
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at);
        mj[g] = ml.x;
        lj[g] = ml.y;
        x[g] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * kKvDim) + lane);
      }
    }
    float Mn = M;
#pragma unroll
    for (int g = 0; g < kGroup; ++g) Mn = fmaxf(Mn, mj[g]);
    const float Lo = M == -INFINITY ? 0.f : L * exp2f(M - Mn);
    L = Lo;
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      lj[g] = lj[g] == 0.f ? 0.f : lj[g] * exp2f(mj[g] - Mn);
      L += lj[g];
    }
    const float inv = L == 0.f ? 0.f : 1.f / L, w0 = Lo * inv;
    acc.x *= w0;
    acc.y *= w0;
    acc.z *= w0;
    acc.w *= w0;
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      const float w = lj[g] * inv;
      acc.x = fmaf(w, x[g].x, acc.x);
      acc.y = fmaf(w, x[g].y, acc.y);
      acc.z = fmaf(w, x[g].z, acc.z);
      acc.w = fmaf(w, x[g].w, acc.w);
    }
    M = Mn;
  }
  const int i = n / a.group;
  const int64_t at = (int64_t)(rec.row0 + i) * a.kv_heads * a.group + rec.h * a.group + (n - i * a.group);
  const __nv_bfloat162 v0 = __floats2bfloat162_rn(acc.x, acc.y), v1 = __floats2bfloat162_rn(acc.z, acc.w);
  reinterpret_cast<uint2*>(a.out + at * kKvDim)[lane] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
  if (a.lse && lane == 0) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

}  // namespace dsa
