// Append to the dense layer's paged 4-bit K/V cache, with the position rotation of k (and of the step's queries) on the way.
//
//   K   per token, head and block of 32 dims: scale = 2^e, the smallest power of two with 6 * 2^e >= amax, -15 <= e <= 13
//   V   per token and head: scale = bf16(amax / 6), at least 2^-126
//   code = e2m1(x / scale), nearest-even, saturating; amax over the finite values; a NaN makes its block's (token's) scale NaN
// K's scales go to the tensor cores as they are (one exponent byte a block), so they are powers of two, and a block of 32
// keeps the few large dims of a rotated key from rounding the others away.  Their range is what e5m2 holds of code * scale
// exactly, the form in which the prompt kernel multiplies.  V's scale comes into the probabilities, one
// number a token whatever it is, so it wastes nothing of a code's range.
//
// What bounds it: the bytes (a query pair 4 read and 4 written, a cached value pair 4 read and 1 written) or, for a decode
// step, latency.  Tokens are independent, whatever page they fall into.  A warp takes 16 query heads or 8 K/V heads
// of one row: 8 lanes a head of 32 bytes each, all loads in flight before anything is looked up, and one set
// of cos and sin for all of its heads.
#include <cuda_fp4.h>

#include "rope.cuh"

namespace dsa {

namespace {
// One warp a CTA: warps share nothing, and their rows end at different times (four prompts of 4,096 with 64 query heads: 256 threads 160 us,
// 128 104, 64 100, 32 97).
constexpr int kThreads = 32, kWarps = kThreads / 32, kKvHeadsAWarp = 8;

// the largest finite |x| (its bits), and whether there is a NaN
__device__ __forceinline__ void largest(const float (&x)[16], uint32_t& top, bool& nan) {
  top = 0;
  nan = false;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint32_t b = __float_as_uint(x[k]) & 0x7FFFFFFFu;
    if (b < 0x7F800000u) top = max(top, b);
    nan |= b > 0x7F800000u;
  }
}

__device__ __forceinline__ uint32_t code2(float lo, float hi) {
  return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}

template <bool kRope>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4AppendArgs a, int q_jobs, int jobs) {
  const int lane = threadIdx.x & 31, part = lane & 7, sub = lane >> 3;
  pdl_wait();
  pdl_trigger();
  const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int r = unit / (uint32_t)jobs, job = unit - r * jobs;
  if (r >= a.num_rows) return;
  if (kRope && job < q_jobs) {
    rope_queries(a.rope, a.query_start_loc, a.seq_lens, a.num_requests, a.num_rows, r, job);
    return;
  }
  const int h0 = kKvHeadsAWarp * (job - q_jobs) + sub;
  uint4 k[2][2], v[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    k[i][0] = k[i][1] = v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    if (h0 + 4 * i < a.kv_heads) {
      const uint4* p = reinterpret_cast<const uint4*>(a.k + (int64_t)r * a.k_stride + (h0 + 4 * i) * kKvDim) + 2 * part;
      const uint4* q = reinterpret_cast<const uint4*>(a.v + (int64_t)r * a.v_stride + (h0 + 4 * i) * kKvDim) + 2 * part;
      k[i][0] = p[0];
      k[i][1] = p[1];
      v[i][0] = q[0];
      v[i][1] = q[1];
    }
  }
  int b, pos, first;
  if (!row_place(a.query_start_loc, a.seq_lens, a.num_requests, a.num_rows, r, b, pos, first) || first < 0) return;
  RopeAngles angles;
  if (kRope) {
    if (pos >= a.rope.positions) return;
    rope_load(a.rope, pos, part, angles);
  }
  const int lp = pos >> a.log2_page;
  if (lp >= a.table_stride) return;
  const int page = a.block_table[(int64_t)b * a.table_stride + lp];
  if (page < 0 || page >= a.num_pages) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int h = h0 + 4 * i;
    const bool there = h < a.kv_heads;
    const int64_t slot = (((int64_t)page * a.kv_heads + (there ? h : 0)) << a.log2_page) + (pos & ((1 << a.log2_page) - 1));
    float x[16];
    uint32_t top;
    bool nan;
    // ---- K
    if (kRope) {
      rope_turn(a.rope, angles, part, k[i], x);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float2 f = bf16x2(reinterpret_cast<const uint32_t*>(k[i])[q]);
        x[2 * q] = f.x;
        x[2 * q + 1] = f.y;
      }
    }
    largest(x, top, nan);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));        // a block is two lanes
    nan = nan | (__shfl_xor_sync(0xffffffffu, (int)nan, 1) != 0);
    // 6 = 1.5 * 2^2: amax = m * 2^E with m in [1, 2) wants 2^(E - 2), or 2^(E - 1) for m > 1.5
    int e = (int)(top >> 23) - 127 - 2 + ((top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    e = min(max(e, kKv4LowExp), kKv4HighExp);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < 8; ++q) c[q >> 2] |= code2(x[2 * q] * inv, x[2 * q + 1] * inv) << (8 * (q & 3));
    if (there) {
      reinterpret_cast<uint2*>(a.k_codes + slot * (kKvDim / 2))[part] = make_uint2(c[0], c[1]);
      if ((part & 1) == 0) a.k_scales[slot * kKv4Blocks + (part >> 1)] = nan ? 0xFFu : (uint8_t)(e + 127);
    }
    // ---- V
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float2 f = bf16x2(reinterpret_cast<const uint32_t*>(v[i])[q]);
      x[2 * q] = f.x;
      x[2 * q + 1] = f.y;
    }
    largest(x, top, nan);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      nan = nan | (__shfl_xor_sync(0xffffffffu, (int)nan, o) != 0);
    }
    const __nv_bfloat16 s = __float2bfloat16_rn(fmaxf(__fdiv_rn(__uint_as_float(top), 6.f), 0x1p-126f));
    const float sf = __bfloat162float(s);
    c[0] = c[1] = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) c[q >> 2] |= code2(__fdiv_rn(x[2 * q], sf), __fdiv_rn(x[2 * q + 1], sf)) << (8 * (q & 3));
    if (there) {
      reinterpret_cast<uint2*>(a.v_codes + slot * (kKvDim / 2))[part] = make_uint2(c[0], c[1]);
      if (part == 0) a.v_scales[slot] = nan ? __ushort_as_bfloat16(0x7FC0) : s;
    }
  }
}
}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t s) {
  const bool rope = a.rope.cos_sin != nullptr;
  const int q_jobs = (a.rope.q_heads + kRopeHeads - 1) / kRopeHeads, jobs = q_jobs + (a.kv_heads + kKvHeadsAWarp - 1) / kKvHeadsAWarp;
  const int64_t warps = (int64_t)a.num_rows * jobs;
  if (warps > INT32_MAX) return cudaErrorInvalidValue;           // the entry point refuses such a call
  const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps));
  const cudaError_t e = rope ? launch_pdl(kv4_append_kernel<true>, grid, dim3(kThreads), 0, s, a, q_jobs, jobs)
                             : launch_pdl(kv4_append_kernel<false>, grid, dim3(kThreads), 0, s, a, q_jobs, jobs);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dsa
