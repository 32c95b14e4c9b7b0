// Append to the dense layer's paged 8-bit K/V cache: one scale per block (= page) and head.
//
// For a page and head that the step writes, with the new tokens' largest finite |x| = amax:
//   want  = 2^ceil(log2(amax / 448))     (2^-126 where amax is 0: a later token then sets the scale)
//   scale = max(want, the page's scale)  if the page holds older tokens of the request, else want
//   code  = e4m3(x / scale), round to nearest even, saturating
// and where the scale grew, the older codes are re-coded: code' = e4m3(code * (old / scale)).
// A scale that is a power of two costs no precision (e4m3 keeps its 4 significant bits in every binade)
// and makes the division exact, and a re-coding exact too but for codes that become subnormal: a page
// filled a token at a time does not lose a little with every step, as it would with amax / 448.
//
// What bounds it: a prompt, the bytes (4 read and 2 written per cached value pair); a decode step, latency.
// One CTA owns one page of one head of K or of V, so nothing is shared and no atomics are needed: it
// holds the page's new values in registers between the maximum and the coding, and reads them once.  At
// most four 32-byte pieces a thread keep several CTAs on an SM (with eight, four prompts of 4,096 took 29.5 us instead of 20.8), and
// the values are asked for before the page's id and old scale, on which they do not depend.
//
// With a rotation of k on the way (rope.cuh) the same CTAs hold their values in fp32, rotated K is coded from fp32, and
// the step's queries are rotated by further CTAs of the same launch, in front.
#include "rope.cuh"

#include <type_traits>

namespace dsa {

namespace {
constexpr int kRowParts = kKvDim / 16;                                    // 16 values a thread

// 16 values of one token's head times `inv` (a power of two), as e4m3 codes
__device__ __forceinline__ uint4 code16(const uint4 (&v)[2], float inv) {
  uint4 out;
  uint32_t* w = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = reinterpret_cast<const uint32_t*>(&v[i >> 1])[2 * (i & 1)];
    const uint32_t hi = reinterpret_cast<const uint32_t*>(&v[i >> 1])[2 * (i & 1) + 1];
    float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&lo));
    float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi));
    a.x *= inv;
    a.y *= inv;
    b.x *= inv;
    b.y *= inv;
    w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
  }
  return out;
}

__device__ __forceinline__ uint4 code16(const float (&x)[16], float inv) {
  uint4 out;
  uint32_t* w = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3) << 16;
  return out;
}

// A scale's exponent: 448 = 1.75 * 2^8, so amax = m * 2^E with m in [1, 2) wants 2^(E - 8), or 2^(E - 7) for m > 1.75
__device__ __forceinline__ float wanted(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// e4m3(code * ratio) for the older codes of a page whose scale grew
template <int kThreads>
__device__ __forceinline__ void recode(uint4* codes, int pieces, float ratio) {
  for (int i = threadIdx.x; i < pieces; i += kThreads) {
    uint4 c = codes[i];
    uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t out = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[q] >> (16 * k)), __NV_E4M3);
        float2 x = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        x.x *= ratio;
        x.y *= ratio;
        out |= (uint32_t)__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3) << (16 * k);
      }
      w[q] = out;
    }
    codes[i] = c;
  }
}

// What the kernel with a rotation has besides.  (In the arguments of both, it would cost the other one 2 % of four prompts of 4,096.)
struct Rotation {
  RopeArgs rope;
  int q_ctas, q_jobs, units;
};
struct NoRotation {};

// kItems: pieces of a full page a thread.  kRope: one row of CTAs, the first q_ctas of which rotate queries; 24 warps on an SM, as far as
// registers go without spills (pages of 64 tokens, prompts of 1,633 rows: 16 warps 25.5 us, 24 23.1, 32 24.6).
template <int kThreads, int kItems, bool kRope>
__global__ void __launch_bounds__(kThreads, kRope && kItems < 4 ? 768 / kThreads : 1) kv8_append_kernel(const Kv8AppendArgs a, const std::conditional_t<kRope, Rotation, NoRotation> turn) {
  __shared__ uint32_t warp_max[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  int unit = blockIdx.x, h = blockIdx.y;
  bool is_v = blockIdx.z != 0;
  pdl_wait();
  pdl_trigger();
  if constexpr (kRope) {
    if (unit < turn.q_ctas) {
      const uint32_t w = (uint32_t)unit * (kThreads / 32) + (tid >> 5);
      const int r = w / (uint32_t)turn.q_jobs;
      if (r < a.num_rows) rope_queries(turn.rope, a.query_start_loc, a.seq_lens, a.num_requests, a.num_rows, r, w - r * turn.q_jobs);
      return;
    }
    unit -= turn.q_ctas;
    const int of_head = unit / turn.units;
    unit -= of_head * turn.units;
    h = of_head >> 1;
    is_v = of_head & 1;
  }
  // Which page: unit u belongs to the last request b with qsl[b] / P + 2 b <= u.  A request of n rows touches
  // at most n / P + 2 pages, which is no more than the units between its start and the next one's.  All
  // warps search alike, 32 probes a step.
  const int P = 1 << a.log2_page;
  const int u = unit;
  int b = 0, row0, n, j;
  if (a.query_start_loc == nullptr) {
    b = u >> 1;
    row0 = b;
    n = 1;
    j = u & 1;
  } else {
    int size = a.num_requests;
    while (size > 1) {
      const int step = (size + 31) / 32, at = b + lane * step;
      const bool below = lane * step < size && (a.query_start_loc[at] >> a.log2_page) + 2 * at <= u;
      const int last = __popc(__ballot_sync(0xffffffffu, below)) - 1;     // lane 0's probe always holds
      if (last < 0) return;                                               // starts that do not ascend
      b += last * step;
      size = min(step, size - last * step);
    }
    row0 = a.query_start_loc[b];
    n = a.query_start_loc[b + 1] - row0;
    j = u - ((row0 >> a.log2_page) + 2 * b);
    if (row0 < 0 || n <= 0 || row0 > a.num_rows - n) return;              // also rows past num_rows
  }
  if (b >= a.num_requests) return;
  const int start = a.seq_lens[b] - n;                                    // position of the first new token
  if (start < 0 || j < 0) return;
  const int lp = (start >> a.log2_page) + j;
  const int64_t page_pos = (int64_t)lp << a.log2_page;                    // position of the page's first token
  const int first = max((int)(start - page_pos), 0);                      // new tokens: offsets first .. last - 1
  int last = (int)min((int64_t)P, (int64_t)start + n - page_pos);
  if constexpr (kRope) last = (int)min((int64_t)last, turn.rope.positions - page_pos); // a token without a row of cos and sin is skipped
  if (first >= last || lp >= a.table_stride) return;
  const uint4* src = reinterpret_cast<const uint4*>(is_v ? a.v : a.k);
  const int64_t src_stride = (is_v ? a.v_stride : a.k_stride) / 8;        // in 16-byte chunks
  const int64_t row = row0 + (page_pos + first - start);                  // row of offset `first`
  uint4 v[kItems][2];
  const int items = (last - first) * kRowParts;
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const int i = tid + it * kThreads;
    v[it][0] = v[it][1] = make_uint4(0, 0, 0, 0);
    if (i < items) {
      const uint4* p = src + (row + i / kRowParts) * src_stride + h * (kKvDim / 8) + 2 * (i % kRowParts);
      v[it][0] = p[0];
      v[it][1] = p[1];
    }
  }
  const int page = a.block_table[(int64_t)b * a.table_stride + lp];
  if (page < 0 || page >= a.num_pages) return;
  const int64_t block = (int64_t)page * a.kv_heads + h;
  uint4* codes = reinterpret_cast<uint4*>((is_v ? a.v_codes : a.k_codes) + ((block << a.log2_page) * kKvDim));
  float* scale_at = (is_v ? a.v_scales : a.k_scales) + block;
  const float old_scale = first > 0 ? *scale_at : 0.f;

  float x[kRope ? kItems : 1][16];                                        // fp32, rotated
  uint32_t top = 0;                                                       // the bits of the largest finite |x|
  if constexpr (kRope) {
#pragma unroll
    for (int it = 0; it < kItems; ++it) {
      const int i = tid + it * kThreads, pos = (int)page_pos + first + i / kRowParts;
      if (!is_v) {
        RopeAngles angles;
        if (i < items && pos < turn.rope.positions) rope_load(turn.rope, pos, i % kRowParts, angles);
        rope_turn(turn.rope, angles, i % kRowParts, v[it], x[it]);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float2 f = bf16x2(reinterpret_cast<const uint32_t*>(v[it])[q]);
          x[it][2 * q] = f.x;
          x[it][2 * q + 1] = f.y;
        }
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const uint32_t w = __float_as_uint(x[it][q]) & 0x7FFFFFFFu;
        if (i < items && w < 0x7F800000u) top = max(top, w);
      }
    }
  } else {
#pragma unroll
    for (int it = 0; it < kItems; ++it)
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(&v[it][q])[e];
          const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
          if (lo < 0x7F80u) top = max(top, lo);
          if (hi < 0x7F80u) top = max(top, hi);
        }
    top <<= 16;
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) warp_max[tid >> 5] = top;
  __syncthreads();                                                        // the old scale has been read, too
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = max(top, warp_max[w]);
  const float want = wanted(top);
  const bool grown = first > 0 && !(old_scale >= want);
  const float scale = first > 0 && old_scale >= want ? old_scale : want;
  // an older scale need not be a power of two (a cache filled elsewhere): then the quotient is rounded
  const bool pow2 = (__float_as_uint(scale) & 0x7FFFFFu) == 0u;
  const float inv = pow2 ? __fdiv_rn(1.0f, scale) : 1.0f;
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const int i = tid + it * kThreads;
    if (i < items) {
      uint4 c;
      if (pow2) {
        if constexpr (kRope) c = code16(x[it], inv);
        else c = code16(v[it], inv);
      } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          w[q] = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float y;
            if constexpr (kRope) y = x[it][4 * q + k];
            else y = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(&v[it][0])[4 * q + k]);
            w[q] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(y, scale), __NV_SATFINITE, __NV_E4M3) << (8 * k);
          }
        }
      }
      codes[(first + i / kRowParts) * kRowParts + i % kRowParts] = c;
    }
  }
  if (grown) recode<kThreads>(codes, first * kRowParts, __fdiv_rn(old_scale, scale));
  if (tid == 0) *scale_at = scale;
}
}  // namespace

namespace {
template <int kThreads, int kItems>
cudaError_t launch_pages(const Kv8AppendArgs& a, const RopeArgs& rope, int64_t units, cudaStream_t s) {
  if (!rope.cos_sin)
    return launch_pdl(kv8_append_kernel<kThreads, kItems, false>, dim3((unsigned)units, a.kv_heads, 2), dim3(kThreads), 0, s, a, NoRotation{});
  const int q_jobs = max((rope.q_heads + kRopeHeads - 1) / kRopeHeads, 1), warps = kThreads / 32;
  const int64_t q_ctas = rope.q_heads ? ((int64_t)a.num_rows * q_jobs + warps - 1) / warps : 0, all = q_ctas + units * a.kv_heads * 2;
  if (all > INT32_MAX / 8) return cudaErrorInvalidValue;         // the entry point refuses such a call
  return launch_pdl(kv8_append_kernel<kThreads, kItems, true>, dim3((unsigned)all), dim3(kThreads), 0, s, a,
                    Rotation{rope, (int)q_ctas, q_jobs, (int)units});
}
}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, const RopeArgs& rope, cudaStream_t s) {
  const int64_t units = (a.query_start_loc ? (a.num_rows >> a.log2_page) : 0) + (int64_t)2 * a.num_requests;
  const cudaError_t e = a.log2_page == 4   ? launch_pages<128, 1>(a, rope, units, s)
                        : a.log2_page == 5 ? launch_pages<256, 1>(a, rope, units, s)
                        : a.log2_page == 6 ? launch_pages<256, 2>(a, rope, units, s)
                                           : launch_pages<256, 4>(a, rope, units, s);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dsa
