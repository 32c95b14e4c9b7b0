// Shared by the two dense attention kernels: what a request brings, and the split of the units over CTAs.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_internal.cuh"
#include "sm100.cuh"

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

__device__ __forceinline__ void tmem_ld_cols8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// What the query warp leaves about a segment's columns
struct __align__(16) PaColumns {      // (an array of them is read four floats at a time)
  float factor[kPagedAttnColumns];    // 2^k of the split query * softmax scale * log2 e
  int limit[kPagedAttnColumns];       // keys below it are seen
  float row[kPagedAttnColumns];       // of the request: its position is start + row
  float slope[kPagedAttnColumns];     // * log2 e
  int at[kPagedAttnColumns];          // row * query heads + head
  int min_limit;                      // over the columns
  int start;                          // position of the request's first row
};
static_assert(sizeof(PaColumns) % 16 == 0, "every one of an array is aligned");

// A segment's queries (requests' rows and heads from pair kCE * cg on), by one warp: their values in two e4m3 terms into the
// rows of q_hi (lo: kHalf rows on), and what the softmax has to know of them into cm.  ready(): waits until both may be written.
template <int kCE, int kHalf, bool kMods, class Seg, class Ready>
__device__ __forceinline__ bool pa_query_columns(const PagedAttnArgs& a, const Seg& s, uint8_t* q_hi, PaColumns& cm, Ready ready) {
  const int lane = threadIdx.x & 31;
  // first what a lane knows of a column of its own.  A column without a pair scores NaN whatever an earlier segment or
  // kernel left of it in shared memory: NaN is no maximum, so it moves no references, and nobody takes its output.
  const int live = min(s.rows * a.group - s.cg * kCE, kCE);
  const int n = s.cg * kCE + min(lane, live - 1), i = n / a.group, head = s.h * a.group + (n - i * a.group);
  const int64_t from = (int64_t)(s.row0 + i) * a.q_stride + (int64_t)head * kKvDim;
  const int start = a.seq_lens[s.b] - s.rows;      // position of row 0
  const int prefix = a.prefix_lens ? min(a.prefix_lens[s.b], s.len) : 0;
  const float slope = kMods && a.slopes ? a.slopes[head] * 1.4426950408889634f : 0.f;
  if (!ready()) return false;
  // then the values, 16 lanes a column: eight columns a step, the next eight on their way; a rolled loop, as code that a
  // CTA runs once or twice costs its way from L2
  const int part = lane & 15, half = lane >> 4;
  auto load = [&](int c) {
    const int64_t at = __shfl_sync(0xffffffffu, from, c & 31);
    return c < live ? *reinterpret_cast<const uint4*>(a.q + at + 8 * part) : make_uint4(0, 0, 0, 0);
  };
  uint4 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = load(2 * k + half);
  const int pos = start + i, limit = min(max(pos + 1, prefix), s.len);
  if (lane < live) {
    cm.limit[lane] = limit;
    cm.row[lane] = (float)i;
    cm.at[lane] = (s.row0 + i) * a.kv_heads * a.group + head;
    cm.slope[lane] = slope;
  } else if (lane < kCE) {
    cm.factor[lane] = __int_as_float(0x7FC00000);
  }
  int low = limit;                                 // (lanes without a column hold the last one's)
#pragma unroll 1
  for (int c0 = 0; c0 < live; c0 += 8) {
    uint4 y[4];
    uint32_t tops[4];                              // the largest |x| of each column as bf16 bits, side by side
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      y[k] = x[k];
      const uint32_t m = __vmaxu2(__vmaxu2(y[k].x & 0x7FFF7FFFu, y[k].y & 0x7FFF7FFFu), __vmaxu2(y[k].z & 0x7FFF7FFFu, y[k].w & 0x7FFF7FFFu));
      tops[k] = max(m & 0xFFFFu, m >> 16);
    }
    if (c0 + 8 < live) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = load(c0 + 8 + 2 * k + half);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) tops[k] = max(tops[k], __shfl_xor_sync(0xffffffffu, tops[k], o));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + 2 * k + half;
      const uint32_t w[4] = {y[k].x, y[k].y, y[k].z, y[k].w}, top = tops[k];
      const int E = pa_exponent(top);
      const __nv_bfloat162 up = pa_up(E);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pa_split<16>(w[e], up, hi[e], lo[e]);
      if (c < live) {
        const uint32_t at = (((part >> 1) ^ (c & 7)) << 4) + 8 * (part & 1);
        *reinterpret_cast<uint2*>(q_hi + c * kKvDim + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(q_hi + (kHalf + c) * kKvDim + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        if (part == 0) cm.factor[c] = pa_factor(top, E, a.scale_log2);
      }
    }
  }
  low = __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) {
    cm.min_limit = low;
    cm.start = start;
  }
  return true;
}

// Requests of many rows (paged_prompt.cu), and the join of both kernels' pieces (few: the first kernel's arguments, few_y
// groups of 8 columns); k_map: the K codes in boxes of a page.
cudaError_t launch_paged_prompt(const PagedAttnArgs& a, const PagedAttnArgs& few, int few_y, const CUtensorMap& k_map,
                                const uint8_t* v_codes, int ctas, cudaStream_t s);
cudaError_t launch_kv4_prompt(const PagedAttnArgs& a, const PagedAttnArgs& few, int few_y, const CUtensorMap& k_map, const uint8_t* v_codes,
                              int ctas, cudaStream_t s);
// The pieces of the few-row kernel's cut segments joined, where no request may have so many rows that the prompt kernel runs too
cudaError_t launch_paged_join(const PagedAttnArgs& a, int ctas, int columns, cudaStream_t s);
cudaError_t launch_prompt_join(const PagedAttnArgs& a, const PagedAttnArgs& few, int few_y, int ctas, cudaStream_t s);

// Where the workspace's parts lie, and which requests the kernel for few rows takes
inline void pa_layout(PagedAttnArgs& a, void* workspace, const PagedAttnPlan& plan, int ctas, int max_seq_len) {
  char* ws = static_cast<char*>(workspace);
  a.err = reinterpret_cast<uint32_t*>(ws);
  a.rec = reinterpret_cast<int32_t*>(ws + plan.rec_offset);
  a.part_o = reinterpret_cast<float*>(ws + plan.part_offset);
  a.part_ml = a.part_o + (size_t)2 * ctas * kPagedAttnColumns * kKvDim;
  // Requests of at most 1,024 keys are not cut: a CTA takes such a segment in less time than a second launch to join
  // its pieces would (8-bit cache, in replayed graphs, one request of 300 keys: 10.4 instead of 19.8 us; 4 prompts of 1,000 rows: 89
  // instead of 97; a single prompt of 1,000 rows and one K/V head, which leaves most SMs idle: 35.1 instead of 31.4).
  a.whole = max_seq_len <= 8 * kPaTok;
  a.lo_pairs = 0;
  a.hi_pairs = plan.prompt ? kPagedAttnDirect : INT32_MAX;
  // The prompt kernel's warps wait for each other with a bound of a second, and its writers for this kernel's end, so they
  // start early only where this kernel's CTAs cannot differ by as much: 2^23 tiles are 0.3 s of work for all of them.
  a.early = plan.prompt && (int64_t)a.num_requests * (((int64_t)max_seq_len + kPaTok - 1) / kPaTok) * a.kv_heads * 2 <= int64_t(1) << 23;
}

// The prompt kernel's requests and its parts of the workspace
inline PagedAttnArgs pa_prompt_args(const PagedAttnArgs& few, void* workspace, const PagedAttnPlan& plan, int ctas) {
  PagedAttnArgs a = few;
  char* ws = static_cast<char*>(workspace);
  a.lo_pairs = kPagedAttnDirect;
  a.hi_pairs = INT32_MAX;
  a.rec = reinterpret_cast<int32_t*>(ws + plan.prompt_rec_offset);
  a.part_o = reinterpret_cast<float*>(ws + plan.prompt_part_offset);
  a.part_ml = a.part_o + (size_t)2 * ctas * kPromptPairs * kKvDim;
  return a;
}

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
// Pieces and running sum are weighted means of V throughout: V's scales go up to 2^120 (4-bit cache: 2^125.4), and a sum over keys
// before its division by L would leave fp32's range.
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
