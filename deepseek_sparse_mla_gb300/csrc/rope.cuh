// The position rotation that the appends apply on the way, and the queries that are rotated with them.
//
//   (a, b) -> (a c - b s, b c + a s)    c, s: cos and sin of the position's angle i, a and b dims (i, i + dim/2) or (2i, 2i + 1)
//
// Each product and the sum are rounded to fp32 apart (no fused multiply-add): a quantised value that lies near a border then
// falls on the same side wherever the same three operations are done.
//
// Eight neighbouring lanes hold a head, 16 dims each.  dim is a multiple of 32, so that a lane's dims all belong to
// the same half: the other values of pairs (i, i + dim/2) are in one other lane, as bf16, half a register each.
#pragma once

#include "dsa_internal.cuh"

namespace dsa {

constexpr int kRopeLaneDims = 16, kRopeLanes = kKvDim / kRopeLaneDims;   // dims a lane, lanes a head
constexpr int kRopeHeads = 16;                                           // query heads of a row that a warp takes: four steps of four

// cos and sin of a lane's dims at one position: 16 of each, or 8 for neighbouring pairs
struct RopeAngles {
  float4 c[4], s[4];
};

__device__ __forceinline__ void rope_load(const RopeArgs& r, int pos, int part, RopeAngles& a) {
  const int half = r.dim >> 1, d = kRopeLaneDims * part;
  if (d >= r.dim) return;
  const int i = r.interleaved ? d >> 1 : d < half ? d : d - half;
  const float4* p = reinterpret_cast<const float4*>(r.cos_sin + (int64_t)pos * r.dim + i);
  const float4* q = reinterpret_cast<const float4*>(r.cos_sin + (int64_t)pos * r.dim + half + i);
  const int n = r.interleaved ? 2 : 4;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < n) {
      a.c[k] = __ldg(p + k);
      a.s[k] = __ldg(q + k);
    }
  }
}

__device__ __forceinline__ float2 bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// 16 dims of a head (bf16, as loaded) rotated; every lane of the warp takes part, whether its dims are rotated or not
__device__ __forceinline__ void rope_turn(const RopeArgs& r, const RopeAngles& a, int part, const uint4 (&v)[2], float (&x)[16]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
  const float* c = reinterpret_cast<const float*>(a.c);
  const float* s = reinterpret_cast<const float*>(a.s);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 f = bf16x2(w[k]);
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
  const bool turned = kRopeLaneDims * part < r.dim;
  if (r.interleaved) {
    if (!turned) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float p = x[2 * k], q = x[2 * k + 1];
      x[2 * k] = __fsub_rn(__fmul_rn(p, c[k]), __fmul_rn(q, s[k]));
      x[2 * k + 1] = __fadd_rn(__fmul_rn(q, c[k]), __fmul_rn(p, s[k]));
    }
    return;
  }
  const int apart = r.dim / (2 * kRopeLaneDims);
  const bool low = part < apart;
  const int from = !turned ? part : low ? part + apart : part - apart;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 o = bf16x2(__shfl_sync(0xffffffffu, w[k], from, kRopeLanes));
    if (turned) {
      const float p = __fmul_rn(x[2 * k], c[2 * k]), q = __fmul_rn(x[2 * k + 1], c[2 * k + 1]);
      const float y = __fmul_rn(o.x, s[2 * k]), z = __fmul_rn(o.y, s[2 * k + 1]);
      x[2 * k] = low ? __fsub_rn(p, y) : __fadd_rn(p, y);
      x[2 * k + 1] = low ? __fsub_rn(q, z) : __fadd_rn(q, z);
    }
  }
}

// Request and position of row r.  False where the row belongs to no request, or to one whose offsets or length make no sense.
// Every lane of a warp asks for the same row; 32 probes a step.
__device__ __forceinline__ bool row_place(const int32_t* query_start_loc, const int32_t* seq_lens, int num_requests, int num_rows, int r,
                                          int& b, int& pos) {
  if (query_start_loc == nullptr) {
    b = r;
    pos = seq_lens[r] - 1;
    return pos >= 0;
  }
  const int lane = threadIdx.x & 31;
  int size = num_requests;
  b = 0;
  while (size > 1) {
    const int step = (size + 31) / 32, at = b + lane * step;
    const bool below = lane * step < size && query_start_loc[at] <= r;
    const int last = __popc(__ballot_sync(0xffffffffu, below)) - 1;      // (starts that do not ascend: checked below)
    if (last < 0) return false;
    b += last * step;
    size = min(step, size - last * step);
  }
  const int row0 = query_start_loc[b], end = query_start_loc[b + 1], len = seq_lens[b];
  if (row0 < 0 || r < row0 || r >= end || end > num_rows || len < end - row0) return false;
  pos = len - (end - row0) + (r - row0);
  return true;
}

// Query heads 16 job .. 16 job + 15 of row r, rotated and rounded to bf16.  Loads first: they do not wait for the position.
__device__ __forceinline__ void rope_queries(const RopeArgs& rope, const int32_t* query_start_loc, const int32_t* seq_lens,
                                             int num_requests, int num_rows, int r, int job) {
  const int lane = threadIdx.x & 31, part = lane & 7, sub = lane >> 3;
  uint4 v[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = kRopeHeads * job + 4 * i + sub;
    v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    if (h < rope.q_heads) {
      const uint4* p = reinterpret_cast<const uint4*>(rope.q + (int64_t)r * rope.q_stride + h * kKvDim) + 2 * part;
      v[i][0] = p[0];
      v[i][1] = p[1];
    }
  }
  int b, pos;
  if (!row_place(query_start_loc, seq_lens, num_requests, num_rows, r, b, pos) || pos >= rope.positions) return;
  RopeAngles a;
  rope_load(rope, pos, part, a);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = kRopeHeads * job + 4 * i + sub;
    float x[16];
    rope_turn(rope, a, part, v[i], x);
    if (h < rope.q_heads) {
      uint4 o[2];
      uint32_t* w = reinterpret_cast<uint32_t*>(o);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&y);
      }
      uint4* p = reinterpret_cast<uint4*>(rope.q_out + (int64_t)r * rope.q_out_stride + h * kKvDim) + 2 * part;
      p[0] = o[0];
      p[1] = o[1];
    }
  }
}

}  // namespace dsa
