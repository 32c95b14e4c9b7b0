// The position rotation that the appends apply on the way, and the queries that are rotated with them.
//
//   (a, b) -> (a c - b s, b c + a s)    c, s: cos and sin of the position's angle i, a and b dims (i, i + dim/2) or (2i, 2i + 1)
//
// Each product and the sum are rounded to fp32 apart (no fused multiply-add): a quantised value that lies near a border then
// falls on the same side wherever the same three operations are done.
//
// Keys: eight neighbouring lanes hold a head, 16 dims each in a row, as it is quantised.  dim is a multiple of 32, so that a lane's dims all belong to
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

// Request and position of row r, and the position of the request's first row: below 0 where it has more rows than tokens.  False
// where the row belongs to no request, or to one whose offsets make no sense.  Every lane of a warp asks for the same row; 32
// probes a step.
__device__ __forceinline__ bool row_place(const int32_t* query_start_loc, const int32_t* seq_lens, int num_requests, int num_rows, int r,
                                          int& b, int& pos, int& first) {
  if (query_start_loc == nullptr) {
    b = r;
    pos = first = max(seq_lens[r], 0) - 1;
    return true;
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
  if (row0 < 0 || r < row0 || r >= end || end > num_rows) return false;
  first = max(len, 0) - (end - row0);
  pos = first + (r - row0);
  return true;
}

// Query heads 16 job .. 16 job + 15 of row r, rotated and rounded to bf16.  (A row in front of its request's first token has no
// position: it may see a prefix, so its queries are copied as they are.)  Loads first: they do not wait for the position.  Nothing
// is quantised here, so a lane takes both halves of its pairs: eight dims and the eight that they turn with, and eight
// angles (with 16 dims in a row, 16 angles and the other halves from another lane, four prompts of 4,096 took 133 us instead of 100).
__device__ __forceinline__ void rope_queries(const RopeArgs& rope, const int32_t* query_start_loc, const int32_t* seq_lens,
                                             int num_requests, int num_rows, int r, int job) {
  const int lane = threadIdx.x & 31, part = lane & 7, sub = lane >> 3;
  const int half = rope.dim >> 1, parts = rope.dim / kRopeLaneDims;   // lanes with pairs to turn
  const bool turned = part < parts, apart = turned && !rope.interleaved;
  const int d0 = apart ? 8 * part : kRopeLaneDims * part, d1 = apart ? d0 + half : d0 + 8;
  const __nv_bfloat16* const from = rope.q + (int64_t)r * rope.q_stride + (kRopeHeads * job + sub) * kKvDim;
  const int heads = rope.q_heads - kRopeHeads * job - sub;            // from this lane's first on
  uint4 v[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    if (4 * i < heads) {
      v[i][0] = *reinterpret_cast<const uint4*>(from + 4 * i * kKvDim + d0);
      v[i][1] = *reinterpret_cast<const uint4*>(from + 4 * i * kKvDim + d1);
    }
  }
  int b, pos, first;
  if (!row_place(query_start_loc, seq_lens, num_requests, num_rows, r, b, pos, first) || pos >= rope.positions) return;
  const bool turns = turned && pos >= 0;
  float c[8], s[8];
  if (turns) {
    const float* const at = rope.cos_sin + (int64_t)pos * rope.dim + 8 * part;
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      *reinterpret_cast<float4*>(c + k) = __ldg(reinterpret_cast<const float4*>(at + k));
      *reinterpret_cast<float4*>(s + k) = __ldg(reinterpret_cast<const float4*>(at + half + k));
    }
  }
  __nv_bfloat16* const to = rope.q_out + (int64_t)r * rope.q_out_stride + (kRopeHeads * job + sub) * kKvDim;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (4 * i >= heads) break;
    uint4 o[2] = {v[i][0], v[i][1]};
    if (turns) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(v[i]);
      float x[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = bf16x2(w[k]);
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
      auto turn = [](float& p, float& q, float c, float s) {
        const float y = __fsub_rn(__fmul_rn(p, c), __fmul_rn(q, s));
        q = __fadd_rn(__fmul_rn(q, c), __fmul_rn(p, s));
        p = y;
      };
      if (rope.interleaved) {
#pragma unroll
        for (int k = 0; k < 8; ++k) turn(x[2 * k], x[2 * k + 1], c[k], s[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) turn(x[k], x[8 + k], c[k], s[k]);
      }
      uint32_t* u = reinterpret_cast<uint32_t*>(o);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        u[k] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
    *reinterpret_cast<uint4*>(to + 4 * i * kKvDim + d0) = o[0];
    *reinterpret_cast<uint4*>(to + 4 * i * kKvDim + d1) = o[1];
  }
}

}  // namespace dsa
