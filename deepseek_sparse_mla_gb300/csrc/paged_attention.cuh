// Shared by the two dense attention kernels: what a request brings, and the split of the units over CTAs.
#pragma once

#include <cuda.h>

#include "dsa_internal.cuh"

namespace dsa {

constexpr int kPaTok = 128;          // keys per tile

// Rows, first row and readable keys of request b.  rows is 0 where the call leaves the request alone: no rows, more
// than max_rows (reported), or a number of (row, head) pairs outside (lo, hi], which the other kernel takes.
struct PaShape {
  int rows, row0, len, tiles;        // tiles: of 128 keys, at least one
};

__device__ __forceinline__ PaShape pa_shape(const PagedAttnArgs& a, int b, uint32_t& bits) {
  PaShape s = {0, b, 0, 0};
  int n = 1;
  if (a.query_start_loc) {
    s.row0 = a.query_start_loc[b];
    const int64_t d = (int64_t)a.query_start_loc[b + 1] - s.row0;
    if (d <= 0 || s.row0 < 0 || s.row0 + d > a.num_rows) return s;
    if (d > a.max_rows) {
      bits |= DSA_DEVICE_BAD_LENGTH;
      return s;
    }
    n = (int)d;
  }
  const int64_t pairs = (int64_t)n * a.group;
  if (pairs <= a.lo_pairs || pairs > a.hi_pairs) return s;
  const int64_t room = (int64_t)a.table_stride << a.log2_page;
  int64_t len = max(a.seq_lens[b], 0);
  if (len > room) {
    bits |= DSA_DEVICE_BAD_PAGE;
    len = room;
  }
  s.rows = n;
  s.len = (int)len;
  s.tiles = max(1, (int)((len + kPaTok - 1) / kPaTok));
  return s;
}

// Requests of many rows (paged_prompt.cu); k_map: the K codes in boxes of a page.
cudaError_t launch_paged_prompt(const PagedAttnArgs& a, const CUtensorMap& k_map, const uint8_t* v_codes, int ctas,
                                cudaStream_t s);

// A capped score: cap * tanh(z / cap) = cap * (1 - 2 / (1 + 2^(in z))), in = 2 log2(e) / cap, all in log2 units.  Exact
// to about 2^-21 of the cap; past the range of 2^x the quotient is 0 or 2, and NaN stays.
__device__ __forceinline__ float capped(float z, float in, float cap) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * in));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return fmaf(-2.f * cap, r, cap);
}

// Units [start(c), start(c + 1)) belong to CTA c.
__device__ __forceinline__ int64_t pa_unit_start(int c, int64_t units, int ctas) { return units * c / ctas; }

__device__ __forceinline__ int pa_cta_of_unit(int64_t u, int64_t units, int ctas) {
  int c = (int)(u * ctas / units);
  while (c + 1 < ctas && pa_unit_start(c + 1, units, ctas) <= u) ++c;
  while (c > 0 && pa_unit_start(c, units, ctas) > u) --c;
  return c;
}

}  // namespace dsa
