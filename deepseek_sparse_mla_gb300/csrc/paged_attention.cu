// Dense grouped-head attention over the paged 8-bit K/V cache, on tcgen05 tensor cores.
//
//   z_s = scale * q[r,h] . (k_code_s * ks)        [then the cap and the distance bias]
//   out[r,h] = sum_s softmax(z)_s * (v_code_s * vs),   lse[r,h] = ln sum_s exp(z_s)
// with one scale ks, vs per page and K/V head, and q bf16.
//
// The codes go to the tensor cores as they are (kind::f8f6f4), so nothing is expanded on chip, and the
// other operand is split into two e4m3 terms to keep its bits:
//   x = (hi + lo / 16) * 2^k,  hi = e4m3(x / 2^k),  lo = e4m3(16 (x / 2^k - hi)).
// e4m3 has 4 significant bits, so hi leaves a remainder of at most 2^-4 of x, which fits lo: bf16's 8 bits
// are kept exactly for values down to 2^-14 of the row's largest, and a probability keeps 8 bits or more
// (its remainder is rounded to 4 bits), with an absolute step of 2^-20 of the largest contribution.
// hi and lo are separate columns of the small operand and are added in fp32 after the products, which
// costs nothing: the large operand (128 keys, or 128 value dims) sets the time of these MMAs.
//
// A (row, head) pair of one request and K/V head is a column; up to 32 are taken together:
//   S^T [128 keys x columns]  = K [128 x 128] (K-major)   * Q^T          (M = 128, N = 2 x columns, K = 128)
//   O^T [128 dims x columns] += V^T (the same tile layout, MN-major) * P^T
// A thread of the softmax warpgroup holds one key's scores, so masks, scales and page lookups are per
// thread, and a column's maximum, where it is needed, is one warp-wide redux.
//
// The v scale would be lost in P's 8 bits if pages differ, so P' = p * vs is what is coded, against a
// running maximum of its own (of z + log2 vs), next to the softmax's maximum that the denominator uses.
// Both maxima move only when exceeded by 2^2, and the accumulator in TMEM is then rescaled.  A tile is first taken
// against the references as they are; only where a contribution exceeds them (one predicate over the
// warpgroup, on the barrier that P needs anyway) are the exact maxima found and the tile taken again.
//
// Work: (request, K/V head, column group, tile of 128 keys) units, laid out in that order and split into one
// contiguous range per CTA (persistent, one CTA per SM).  A segment (all tiles of one request, head and
// group) inside one CTA is written directly; one that is cut leaves fp32 pieces that a second kernel joins.
//
// Per CTA (12 warps): warp 0 looks pages up and issues TMA loads into a ring of 32 KB stages (K and V of
// a tile); warps 1 and 3 issue the products of the scores and of the outputs, each at its own pace (one warp
// doing both spent 1,500 cycles a tile on waits and issue: 788 us instead of 685 for 64 requests of
// 16K-128K tokens); warp 2 splits the coming segments' queries; warps 4-7 and 8-11 are two
// softmax warpgroups that take the even and the odd tiles.  A tile's softmax is one chain of waits (scores
// out of TMEM, maxima across the warps, probabilities into shared memory) about 2,000 cycles long, while at
// full HBM speed a tile arrives every 1,360 cycles; two chains side by side keep up.  They share nothing while they
// run: each has its own maxima, denominators and accumulator, joined in the segment's epilogue, which
// the warpgroups take in turn.
#include "paged_attention.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

#include <algorithm>
#include <type_traits>

namespace dsa {
using namespace sm100;

namespace pa {
constexpr int kTok = kPaTok;                    // keys per tile
constexpr int kTileBytes = kTok * kKvDim;       // 16 KB of codes
constexpr int kStageBytes = 2 * kTileBytes;     // K, then V
constexpr int kStages = 5;
constexpr int kColMax = kPagedAttnColumns;
constexpr int kQBytes = 2 * kColMax * kKvDim;   // hi and lo rows of 32 columns
constexpr int kPBytes = kTok * 2 * kColMax;
constexpr int kMaxPages = kTok / kKvMinPage;    // pages of a tile
constexpr int kThreads = 384;
constexpr int kScoreWarp = 1, kOutWarp = 3, kSoftWarp0 = 4;
constexpr uint32_t kRegsLow = 88, kRegsSoft = 208;   // 88 + 2 * 208 = 3 * 168, the launch's
constexpr int kQBufs = 3;                       // the scores run two tiles, so up to two segments, ahead of the outputs
constexpr uint32_t kTmemCols = 512;             // S^T of tile i at 64 (i % 4), O^T at 256 + 128 (segment % 2) + 64 warpgroup
constexpr uint32_t kColO = 256;
constexpr int kSBufs = 4;                       // two a warpgroup: one is kept until its tile is known to be done
constexpr float kSlackP = 4.f;                  // a reference may be exceeded by this factor
constexpr float kPOne = 64.f;                   // the code of a contribution at its reference: 2^2 above fits in 448
constexpr uint32_t kPolls = 1u << 18;           // of 3.8 us each or more: a second
// The query warp runs up to kQBufs segments ahead and then waits for a whole one to end: 57 ms for 2^22 tokens and 32
// columns, 15 s for 2^30.
constexpr uint32_t kSegPolls = 1u << 24;
constexpr int kFixedSmem = kStages * kStageBytes + kQBufs * kQBytes + 2 * kPBytes + 1024;
}  // namespace pa

// A run of tiles of one segment
struct PaSeg {
  int b, h, cg, tile, n;       // first tile and number of tiles of this piece
  int rows, row0, len, tiles;

  // Its t-th tile.  With a bias on distance the last keys come first: scores grow towards a row's own position, and the
  // references would move with every tile in rising order.  (Without one, beginning with the masked tiles costs
  // the verify case 1.5 %.)
  template <bool kFalling>
  __device__ __forceinline__ int tile_at(int t) const { return kFalling ? tile + n - 1 - t : tile + t; }
};

// The segment that unit u lies in, cut at u1.  end[b] = column groups * tiles of requests 0 .. b.
__device__ __forceinline__ PaSeg pa_segment(const PagedAttnArgs& a, const int32_t* end, int64_t u, int64_t u1) {
  int lo = 0, hi = a.num_requests - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)end[mid] * a.kv_heads > u) hi = mid;
    else lo = mid + 1;
  }
  PaSeg s;
  s.b = lo;
  const int first = lo ? end[lo - 1] : 0;
  uint32_t none = 0;
  const PaShape sh = pa_shape(a, lo, none);
  s.row0 = sh.row0;
  s.rows = sh.rows;
  s.len = sh.len;
  s.tiles = sh.tiles;
  const int64_t in = u - (int64_t)first * a.kv_heads;
  const int per_head = end[lo] - first;
  s.h = in < (int64_t(1) << 31) ? (int)((uint32_t)in / (uint32_t)per_head) : (int)(in / per_head);
  const int rest = (int)(in - (int64_t)s.h * per_head);
  s.cg = rest / sh.tiles;
  s.tile = rest - s.cg * sh.tiles;
  s.n = (int)min((int64_t)(sh.tiles - s.tile), u1 - u);
  return s;
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

// two e4m3 codes of (a, b), and of 16 times what they leave
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3);
  const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hr));
  lo = __nv_cvt_float2_to_fp8x2(make_float2(16.f * (a - back.x), 16.f * (b - back.y)), __NV_SATFINITE, __NV_E4M3);
}

// What the query warp leaves about a segment's columns
struct PaColumns {
  float factor[pa::kColMax];    // 2^k of the split query * softmax scale * log2 e
  int limit[pa::kColMax];       // keys below it are seen
  float row[pa::kColMax];       // of the request: its position is start + row
  float slope[pa::kColMax];     // * log2 e
  int at[pa::kColMax];          // row * query heads + head
  int min_limit;                // over the columns
  int start;                    // position of the request's first row
};

// kCE columns (8, 16 or 32); kModSet: score cap and distance bias compiled in
template <int kCE, PaMods kModSet>
__global__ void __launch_bounds__(pa::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                           const __grid_constant__ PagedAttnArgs a, int shared_keys) {
  using namespace pa;
  constexpr bool kMods = kModSet != kPaPlain;
  constexpr int kHalf = kCE < 16 ? 16 : kCE;          // columns of the hi half (and of the lo half)
  constexpr int kN = 2 * kHalf;                       // MMA N: 32 or 64
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;
  uint8_t* sQ = sKV + kStages * kStageBytes;
  uint8_t* sP = sQ + kQBufs * kQBytes;
  int32_t* end = reinterpret_cast<int32_t*>(sP + 2 * kPBytes);   // [requests]

  __shared__ uint64_t kv_full[kStages], kv_empty[kStages], s_full[kSBufs], s_empty[kSBufs], p_full[2];
  __shared__ uint64_t q_full[kQBufs], q_empty[kQBufs], stat_full[kQBufs], o_full[2], o_empty[2], mma_done;
  __shared__ float sks[kStages][kMaxPages], svs[kStages][kMaxPages];
  __shared__ uint32_t sbad[kStages];
  __shared__ __align__(16) PaColumns cols[kQBufs];
  __shared__ __align__(16) float refs[2][2][kCE];
  __shared__ float wmax[2][4][kCE], fin[2][2][kCE];
  __shared__ float stat[kQBufs][2][3][kCE];            // each warpgroup's m, mv and l of a segment
  __shared__ uint32_t stat_nan[kQBufs][2][kKvDim];
  __shared__ uint32_t nan_keys[2][4];
  __shared__ int32_t scan[kThreads / 32];
  __shared__ uint32_t tmem_base, bits_all;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&p_full[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 9);          // the last product that reads it, and eight softmax warps
      mbar_init(&stat_full[i], 8);
    }
    mbar_init(&mma_done, 2);
    bits_all = 0;
    fence_mbar_init();
    prefetch_tmap(&k_map);
    prefetch_tmap(&v_map);
  }
  if (warp == kScoreWarp) {
    tmem_alloc(&tmem_base, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  // The prompt kernel may start as SMs fall free (3 pieces of 700 rows over up to 9,000 tokens 380 instead of 400 us; the mixed
  // capped batch 95 instead of 93, both in replayed graphs).  A join may not: its CTAs coming early cost 32 requests at 8K
  // 2 us.
  if (a.early) pdl_trigger();
  if (tid == 0) reinterpret_cast<PaRecord*>(a.rec)[cta].tile = -1;   // no piece to join until it has been written
  // running sums of the requests' units: every thread a run of consecutive requests
  {
    uint32_t bits = 0;
    const int B = a.num_requests, per = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      const PaShape s = pa_shape(a, b, bits);
      sum += (s.rows * a.group + kCE - 1) / kCE * s.tiles;
      end[b] = sum;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < warp; ++w) before += scan[w];
    for (int b = b0; b < b1; ++b) end[b] += before;
    if (bits) atomicOr(&bits_all, bits);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int64_t units = (int64_t)end[a.num_requests - 1] * a.kv_heads;
  int64_t u0 = pa_unit_start(cta, units, ctas);
  const int64_t u1 = pa_unit_start(cta + 1, units, ctas);
  // segments are cut where the range ends, or (short requests) belong to the range they begin in as a whole
  const int64_t cut = a.whole ? units : u1;
  if (a.whole && u0 < u1) {
    const PaSeg s = pa_segment(a, end, u0, units);
    if (s.tile > 0) u0 += s.n;
  }
  uint32_t* const err = &bits_all;                    // this CTA's status bits, stored at the end

  if (warp < kSoftWarp0) {
  regs_dec<kRegsLow>();
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    const uint64_t policy = shared_keys ? l2_evict_normal() : l2_evict_first();
    const int lp = a.log2_page, ppt = kTok >> lp;
    const uint32_t page_bytes = (uint32_t)kKvDim << lp;
    int i = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok;) {
      const PaSeg s = pa_segment(a, end, u, cut);
      const int pages = (s.len + (1 << lp) - 1) >> lp;
      int batch = -1, page = -1;                       // 32 pages at a time, one a lane
      float ks = 0.f, vs = 0.f;
      for (int t = 0; t < s.n && ok; ++t, ++i) {
        const int p0 = s.template tile_at<kMods>(t) * ppt;
        if ((p0 >> 5) != batch) {
          batch = p0 >> 5;
          const int p = 32 * batch + lane;
          page = -1;
          ks = vs = 0.f;
          if (p < pages) {
            page = a.block_table[(int64_t)s.b * a.table_stride + p];
            if (page < 0 || page >= a.num_pages) {
              atomicOr(err, kErrBadPage);
              page = -1;
            }
          }
          if (page >= 0) {                             // (not waited for until the tile's loads are out)
            ks = a.k_scales[(int64_t)page * a.kv_heads + s.h];
            vs = a.v_scales[(int64_t)page * a.kv_heads + s.h];
          }
        }
        const int st = i % kStages, use = i / kStages;
        if (use > 0 && !mbar_wait_warp(&kv_empty[st], (use - 1) & 1, err, kErrMmaTimeout, kPolls)) {
          ok = false;
          break;
        }
        // this tile's pages sit in lanes o .. o + ppt - 1; lanes 0 .. ppt - 1 load K, 16 .. 16 + ppt - 1 V
        const int o = p0 & 31, mine = lane & 15;
        const int pg = __shfl_sync(0xffffffffu, page, (o + mine) & 31);
        const bool load = mine < ppt && pg >= 0;
        const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
        const uint32_t bad = __ballot_sync(0xffffffffu, mine < ppt && pg < 0) & 0xFFFFu;
        if (load)
          tma_load_2d_hint(sKV + st * kStageBytes + (lane >> 4) * kTileBytes + mine * page_bytes,
                           lane < 16 ? &k_map : &v_map, 0, (pg * a.kv_heads + s.h) << lp, &kv_full[st], policy);
        // the tile's arrival also stands for its scales
        const float k1 = __shfl_sync(0xffffffffu, ks, (o + mine) & 31), v1 = __shfl_sync(0xffffffffu, vs, (o + mine) & 31);
        if (lane < ppt) {
          sks[st][lane] = k1;
          svs[st][lane] = v1;
        }
        if (lane == 0) sbad[st] = bad;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&kv_full[st], loads * page_bytes);
      }
      u += s.n;
    }
    // nothing may still be landing in shared memory when the CTA exits
    for (int st = 0; st < kStages; ++st) {
      const int uses = (i - st + kStages - 1) / kStages;
      if (i > st) mbar_wait_warp(&kv_full[st], (uses - 1) & 1, err, kErrTmaTimeout, kPolls);
    }
  } else if (warp == kScoreWarp) {
    // ---------------------------------------------------------------- products of the scores
    // The warp walks together and one elected lane issues: addresses stay in uniform registers.  With
    // the walk itself inside a one-lane branch, issuing a tile's products took twice as long.
    const bool leader = elect_one();
    const uint32_t id_qk = idesc_e4m3(kTok, kN);
    const uint64_t d_k = smem_desc(smem_u32(sKV), 16, 1024, kSwizzle128B);
    const uint64_t d_q = smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
    int i = 0, seg = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok; ++seg) {
      const PaSeg s = pa_segment(a, end, u, cut);
      u += s.n;
      const int qb = seg % kQBufs;
      ok = mbar_wait_warp(&q_full[qb], (seg / kQBufs) & 1, err, kErrMmaTimeout, kPolls);
      for (int t = 0; t < s.n && ok; ++t, ++i) {
        const int st = i % kStages, sb = i % kSBufs;
        ok = mbar_spin_warp(&kv_full[st], (i / kStages) & 1, err, kErrTmaTimeout);
        if (ok && i >= kSBufs) ok = mbar_spin_warp(&s_empty[sb], (i / kSBufs - 1) & 1, err, kErrMmaTimeout);
        if (!ok) break;
        tc_fence_after();
        const uint64_t k = d_k + (uint64_t)((st * kStageBytes) >> 4), q = d_q + (uint64_t)((qb * kQBytes) >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kKvDim / 32; ++kk) mma_ss_f8(tmem + 64 * sb, k + 2 * kk, q + 2 * kk, id_qk, kk > 0);
          mma_commit(&s_full[sb]);
          if (t + 1 == s.n) mma_commit(&q_empty[qb]);
        }
        __syncwarp();
      }
    }
    // every MMA issued here has finished before TMEM is released
    if (leader) mma_commit(&mma_done);
    mbar_wait_warp(&mma_done, 0, err, kErrMmaTimeout, kPolls);
  } else if (warp == kOutWarp) {
    // ---------------------------------------------------------------- products of the outputs
    const bool leader = elect_one();
    const uint32_t id_pv = idesc_e4m3(kKvDim, kN) | (1u << 15) | (1u << 16);   // both operands MN-major
    constexpr SmemSwizzle kPSwizzle = kN == 64 ? kSwizzle64B : kSwizzle32B;
    const uint64_t d_v = smem_desc(smem_u32(sKV + kTileBytes), 16, 1024, kSwizzle128B);
    const uint64_t d_p = smem_desc(smem_u32(sP), 16, 8 * kN, kPSwizzle);
    int i = 0, seg = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok; ++seg) {
      const PaSeg s = pa_segment(a, end, u, cut);
      u += s.n;
      uint32_t fresh = 3;                              // accumulators of the segment without a product yet
      if (seg >= 2) ok = mbar_wait_warp(&o_empty[seg & 1], ((seg >> 1) - 1) & 1, err, kErrMmaTimeout, kPolls);
      for (int t = 0; t < s.n && ok; ++t, ++i) {
        const int st = i % kStages, pb = i & 1;
        ok = mbar_spin_warp(&p_full[pb], (i >> 1) & 1, err, kErrMmaTimeout);
        if (!ok) break;
        tc_fence_after();
        const uint64_t v = d_v + (uint64_t)((st * kStageBytes) >> 4), p = d_p + (uint64_t)((pb * kPBytes) >> 4);
        const bool first = (fresh >> pb) & 1u;
        fresh &= ~(1u << pb);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kTok / 32; ++kk)
            mma_ss_f8(tmem + kColO + 128 * (seg & 1) + 64 * pb, v + (uint64_t)((kk * 32 * kKvDim) >> 4),
                      p + (uint64_t)((kk * 32 * kN) >> 4), id_pv, !first || kk > 0);
          mma_commit(&kv_empty[st]);                   // K, V and this tile's probabilities have been read
          if (t + 1 == s.n) mma_commit(&o_full[seg & 1]);
        }
        __syncwarp();
      }
    }
    if (leader) mma_commit(&mma_done);
    mbar_wait_warp(&mma_done, 0, err, kErrMmaTimeout, kPolls);
  } else {
    // ---------------------------------------------------------------- queries
    int seg = 0;
    for (int64_t u = u0; u < u1; ++seg) {
      const PaSeg s = pa_segment(a, end, u, cut);
      u += s.n;
      const int buf = seg % kQBufs;
      // first what a lane knows of a column of its own.  A column without a pair scores NaN whatever an earlier segment or
      // kernel left of it in shared memory: NaN is no maximum, so it moves no references, and nobody takes its output.
      const int live = min(s.rows * a.group - s.cg * kCE, kCE);
      const int n = s.cg * kCE + min(lane, live - 1), i = n / a.group, head = s.h * a.group + (n - i * a.group);
      const int64_t from = (int64_t)(s.row0 + i) * a.q_stride + (int64_t)head * kKvDim;
      const int start = a.seq_lens[s.b] - s.rows;      // position of row 0
      const int prefix = a.prefix_lens ? min(a.prefix_lens[s.b], s.len) : 0;
      const float slope = kMods && a.slopes ? a.slopes[head] * 1.4426950408889634f : 0.f;
      if (seg >= kQBufs && !mbar_wait_warp(&q_empty[buf], (seg / kQBufs - 1) & 1, err, kErrMmaTimeout, kSegPolls)) break;
      uint8_t* q_hi = sQ + buf * kQBytes;
      PaColumns& cm = cols[buf];
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
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[buf]);
    }
  }
  } else {
    regs_inc<kRegsSoft>();
    // ---------------------------------------------------------------- softmax and outputs: one key a thread
    const int wg = (warp - kSoftWarp0) >> 2, bar = 1 + wg;
    const int quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    int i0 = 0, seg = 0;                               // i0: the CTA's tiles before this segment
    for (int64_t u = u0; u < u1; ++seg) {
      const PaSeg s = pa_segment(a, end, u, cut);
      u += s.n;
      const int qb = seg % kQBufs;
      if (!mbar_wait_warp(&q_full[qb], (seg / kQBufs) & 1, err, kErrMmaTimeout, kPolls)) break;
      const uint32_t acc = tmem + lanes + kColO + 128 * (seg & 1);
      const PaColumns& cm = cols[qb];
      const int min_limit = cm.min_limit;
      const int live = min(s.rows * a.group - s.cg * kCE, kCE);   // columns in use
      // the references of column `lane` (m: of z, mv: of z + log2 vs); every column's are in shared memory, as m and as
      // 2^(m - mv)
      float m_lane = -INFINITY, mv_lane = -INFINITY;
      float* const ref_m = refs[wg][0];
      float* const ref_e = refs[wg][1];
      float l[kCE];
#pragma unroll
      for (int c = 0; c < kCE; ++c) l[c] = 0.f;
      uint32_t poison = 0;                             // columns whose output at dim `row` is NaN
      bool ok = true, fresh = true;
      // One tile, with kNC columns in use (blocks of 8, 16 or 32).  Each form is a body of its own, chosen once a tile: with
      // guards and branches inside one body, the verify case (32 columns) took 394 us instead of 331.
      auto tile = [&](auto columns, auto with_masks, int i, int key0) {
        constexpr int kNC = decltype(columns)::value;
        constexpr bool kMasked = decltype(with_masks)::value;
        const int st = i % kStages, sb = i % kSBufs, j = key0 + row, pg = row >> a.log2_page;
        const float ks = sks[st][pg], vs = svs[st][pg], vs_one = vs * kPOne;
        const bool exists = !kMasked || (j < s.len && !((sbad[st] >> pg) & 1u));
        const float in = kMods && a.cap_log2 > 0.f ? 2.f * 1.4426950408889634f / a.cap_log2 : 0.f;
        // Distances are taken from the request's first row in integers: they, and the small row numbers, are exact in fp32
        // however far from 0 the positions are, up to 2^24 tokens away, and rounded like any fp32 value beyond.
        const float ahead = kMods ? (float)(j - cm.start) : 0.f;
        if (kMasked) {
          // A key's values meet a probability of 0 where it is not seen, and 0 * NaN is NaN: what lies behind
          // the request's tokens is zeroed here, and NaN codes of keys that only some columns see are taken out.
          uint4* vrow = reinterpret_cast<uint4*>(sKV + st * kStageBytes + kTileBytes + row * kKvDim);
          bool has_nan = false;
          if (!exists) {
#pragma unroll
            for (int q = 0; q < kKvDim / 16; ++q) vrow[q] = make_uint4(0, 0, 0, 0);
          } else if (j >= min_limit) {
            uint32_t hit = 0;
#pragma unroll 1
            for (int q = 0; q < kKvDim / 16; ++q) {
              const uint4 w = vrow[q];
              hit |= ((w.x & 0x7F7F7F7Fu) + 0x01010101u) | ((w.y & 0x7F7F7F7Fu) + 0x01010101u) |
                     ((w.z & 0x7F7F7F7Fu) + 0x01010101u) | ((w.w & 0x7F7F7F7Fu) + 0x01010101u);
            }
            has_nan = (hit & 0x80808080u) != 0;
          }
          if (group_or(bar, 128, has_nan)) {
            const uint32_t who = __ballot_sync(0xffffffffu, has_nan);
            if (lane == 0) nan_keys[wg][quarter] = who;
            group_sync(bar, 128);
            const uint8_t* vt = sKV + st * kStageBytes + kTileBytes;
            for (int w = 0; w < 4; ++w)
              for (uint32_t left = nan_keys[wg][w]; left; left &= left - 1) {
                const int k = 32 * w + __ffs(left) - 1;
                const uint8_t code = vt[k * kKvDim + ((((uint32_t)row >> 4) ^ (k & 7)) << 4) + (row & 15)];
                if ((code & 0x7Fu) == 0x7Fu)
                  for (int c = 0; c < kCE; ++c)
                    if (key0 + k < cm.limit[c]) poison |= 1u << c;
              }
            group_sync(bar, 128);
            if (has_nan) {
              uint32_t* words = reinterpret_cast<uint32_t*>(vrow);
              for (int q = 0; q < kKvDim / 4; ++q) {
                const uint32_t w = words[q], f = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;   // bit 7 of NaN bytes
                words[q] = w & ~((f >> 7) * 0xFFu);
              }
            }
          }
        }
        // the scores of c1 columns from what their products left
        auto finish = [&](auto& z, const uint32_t* hi, const uint32_t* lo, int c0, int c1) {
          // a loop each: a choice made inside one of them would leave the values no instructions to overlap with
#pragma unroll
          for (int c = 0; c < c1; ++c) z[c] = fmaf(__uint_as_float(lo[c]), 0.0625f, __uint_as_float(hi[c])) * (ks * cm.factor[c0 + c]);
          if (kMods && in != 0.f) {
#pragma unroll
            for (int c = 0; c < c1; ++c) z[c] = capped<kModSet>(z[c] * in, a.cap_log2);
          }
          if (kMods) {
#pragma unroll
            for (int c = 0; c < c1; ++c) z[c] = fmaf(-cm.slope[c0 + c], fabsf(cm.row[c0 + c] - ahead), z[c]);
          }
          if (kMasked) {
#pragma unroll
            for (int c = 0; c < c1; ++c)
              if (!exists || j >= cm.limit[c0 + c]) z[c] = -INFINITY;
          }
        };
        auto scores8 = [&](float (&z)[8], int c0) {
          uint32_t hi[8], lo[8];
          tmem_ld_cols8(tmem + lanes + 64 * sb + c0, hi);
          tmem_ld_cols8(tmem + lanes + 64 * sb + kHalf + c0, lo);
          tmem_wait_ld();
          finish(z, hi, lo, c0, 8);
        };
        auto scores = [&](float (&z)[kNC]) {
          constexpr int kC = kNC < 16 ? kNC : 16;      // columns at a time
#pragma unroll
          for (int c0 = 0; c0 < kNC; c0 += kC) {
            uint32_t hi[kC], lo[kC];
#pragma unroll
            for (int c = 0; c < kC; c += 8) {
              tmem_ld_cols8(tmem + lanes + 64 * sb + c0 + c, hi + c);
              tmem_ld_cols8(tmem + lanes + 64 * sb + kHalf + c0 + c, lo + c);
            }
            tmem_wait_ld();
            float y[kC];
            finish(y, hi, lo, c0, kC);
#pragma unroll
            for (int c = 0; c < kC; ++c) z[c0 + c] = y[c];
          }
        };
        // the exact maxima over the tile, where the references do not hold: they, and what was formed against them, move
        auto raise = [&]() {
          // log2 of the key's scale, -126 for one of 0: 2^(m - mv) and its product with a probability below 4 stay finite
          const float lv = fmaxf(__log2f(fabsf(vs)), -126.f);
          float mine = -INFINITY;
          // rolled: it runs for a segment's first tile, where a second copy of all columns' scores would have to come from L2
#pragma unroll 1
          for (int c0 = 0; c0 < kNC; c0 += 8) {
            float z[8];
            scores8(z, c0);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float r = warp_max_f32(z[c]);
              if (lane == c0 + c) mine = r;            // lane c of every warp ends up with column c's
            }
          }
          // A warp's 32 keys have one scale, but for pages of 16: there the maximum of z + lv may be another key's.  (A loop
          // of its own: inside the first one it took the verify case, whose pages are larger, 341 us instead of 334.)
          float mine_v = mine + lv;
          if (a.log2_page == 4) {
#pragma unroll 1
            for (int c0 = 0; c0 < kNC; c0 += 8) {
              float z[8];
              scores8(z, c0);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float r = warp_max_f32(z[c] + lv);
                if (lane == c0 + c) mine_v = r;
              }
            }
          }
          float* const wmax_v = reinterpret_cast<float*>(sP + wg * kPBytes);   // [4][kCE], before the tile's P is there
          if (lane < kCE) {
            wmax[wg][quarter][lane] = mine;
            wmax_v[quarter * kCE + lane] = mine_v;
          }
          group_sync(bar, 128);
          float m_new = m_lane, mv_new = mv_lane;
          if (lane < kCE) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              m_new = fmaxf(m_new, wmax[wg][w][lane]);
              mv_new = fmaxf(mv_new, wmax_v[w * kCE + lane]);
            }
          }
          const float al = m_lane == -INFINITY ? 0.f : ex2_approx(m_lane - m_new);
          const float ao = mv_lane == -INFINITY ? 0.f : ex2_approx(mv_lane - mv_new);
          m_lane = m_new;
          mv_lane = mv_new;
          if (quarter == 0 && lane < kCE) {
            ref_m[lane] = m_new == -INFINITY ? -1e30f : m_new;   // nothing seen yet: the first score that is exceeds it
            ref_e[lane] = mv_new == -INFINITY ? 1.f : ex2_approx(m_new - mv_new);
          }
          if (!fresh) {
#pragma unroll
            for (int c = 0; c < kNC; ++c) l[c] *= __shfl_sync(0xffffffffu, al, c);
            tc_fence_after();
            const uint32_t o = acc + 64 * wg;
#pragma unroll 1
            for (int c0 = 0; c0 < kNC; c0 += 8) {
              uint32_t r[16];
              tmem_ld_cols8(o + c0, r);
              tmem_ld_cols8(o + kHalf + c0, r + 8);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float f = __shfl_sync(0xffffffffu, ao, c0 + c);
                r[c] = __float_as_uint(__uint_as_float(r[c]) * f);
                r[8 + c] = __float_as_uint(__uint_as_float(r[8 + c]) * f);
              }
              tmem_st8(o + c0, r);
              tmem_st8(o + kHalf + c0, r + 8);
            }
            tmem_wait_st();
          }
          group_sync(bar, 128);
        };
        // the buffer is free, and the accumulator settled, once this warpgroup's previous product has completed
        if (i >= 2) {
          ok = mbar_wait_warp(&kv_empty[(i - 2) % kStages], ((i - 2) / kStages) & 1, err, kErrMmaTimeout, kPolls);
          if (!ok) return;
        }
        uint8_t* prow = sP + wg * kPBytes + row * kN;
        const int sw = kN == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
        float z[kNC];                                  // scores, then probabilities
        bool raised = fresh;
        if (fresh) raise();
        for (;;) {
          scores(z);
          // the probabilities, and their contributions in two e4m3 terms
          uint32_t hi[kHalf / 4], lo[kHalf / 4];
          float p_top = 0.f, x_top = 0.f;
#pragma unroll
          for (int c = 0; c < kHalf; c += 4) {
            hi[c / 4] = lo[c / 4] = 0;
            if (c >= kNC) continue;
            const float4 m4 = *reinterpret_cast<const float4*>(ref_m + c), e4 = *reinterpret_cast<const float4*>(ref_e + c);
            const float mm[4] = {m4.x, m4.y, m4.z, m4.w}, ee[4] = {e4.x, e4.y, e4.z, e4.w};
            float x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              z[c + q] = ex2_approx(z[c + q] - mm[q]);
              x[q] = (z[c + q] * ee[q]) * vs_one;     // in this order: 0 stays 0 whatever the scale of an unseen key
              p_top = fmaxf(p_top, z[c + q]);
              x_top = fmaxf(x_top, x[q]);
            }
            uint32_t h0, l0, h1, l1;
            split2(x[0], x[1], h0, l0);
            split2(x[2], x[3], h1, l1);
            hi[c / 4] = h0 | h1 << 16;
            lo[c / 4] = l0 | l1 << 16;
          }
#pragma unroll
          for (int q = 0; q < kHalf / 16; ++q) {
            *reinterpret_cast<uint4*>(prow + ((q ^ sw) << 4)) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
            *reinterpret_cast<uint4*>(prow + (((q + kHalf / 16) ^ sw) << 4)) =
                make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
          }
          fence_proxy_async_smem();
          tc_fence_before();
          if (!group_or(bar, 128, !raised && (p_top >= kSlackP || x_top > kSlackP * kPOne))) break;
          raised = true;                               // the same in all four warps
          raise();
        }
#pragma unroll
        for (int c = 0; c < kNC; ++c) l[c] += z[c];
        fresh = false;
        if (row == 0) mbar_arrive(&p_full[wg]);
        if (lane == 0) mbar_arrive(&s_empty[sb]);
      };
      for (int t = (i0 + wg) & 1; t < s.n && ok; t += 2) {
        const int i = i0 + t, key0 = s.template tile_at<kMods>(t) * kTok;
        ok = mbar_wait_warp(&kv_full[i % kStages], (i / kStages) & 1, err, kErrTmaTimeout, kPolls) &&
             mbar_wait_warp(&s_full[i % kSBufs], (i / kSBufs) & 1, err, kErrMmaTimeout, kPolls);
        if (!ok) break;
        tc_fence_after();
        using std::integral_constant;
        const bool masked = __any_sync(0xffffffffu, key0 + kTok > min_limit || sbad[i % kStages] != 0);
        if constexpr (kCE > 16) {
          if (live > 16) {
            if (masked) tile(integral_constant<int, 32>{}, std::true_type{}, i, key0);
            else tile(integral_constant<int, 32>{}, std::false_type{}, i, key0);
            continue;
          }
        }
        if constexpr (kCE > 8) {
          if (live > 8) {
            if (masked) tile(integral_constant<int, 16>{}, std::true_type{}, i, key0);
            else tile(integral_constant<int, 16>{}, std::false_type{}, i, key0);
            continue;
          }
        }
        if (masked) tile(integral_constant<int, 8>{}, std::true_type{}, i, key0);
        else tile(integral_constant<int, 8>{}, std::false_type{}, i, key0);
      }
      if (!ok) break;
      i0 += s.n;
      // ---- the segment's end: each warpgroup leaves its maxima and denominators, and one writes the outputs
#pragma unroll
      for (int c0 = 0; c0 < kCE; c0 += 8) {
        if (c0 >= live) continue;
#pragma unroll
        for (int c = c0; c < c0 + 8; ++c) {
          float v = l[c];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane == 0) wmax[wg][quarter][c] = v;
        }
      }
      group_sync(bar, 128);
      if (quarter == 0 && lane < live) {
        stat[qb][wg][0][lane] = m_lane;
        stat[qb][wg][1][lane] = mv_lane;
        stat[qb][wg][2][lane] = (wmax[wg][0][lane] + wmax[wg][1][lane]) + (wmax[wg][2][lane] + wmax[wg][3][lane]);
      }
      stat_nan[qb][wg][row] = poison;
      __syncwarp();
      if (lane == 0) mbar_arrive(&stat_full[qb]);
      if ((seg & 1) != wg) {
        if (lane == 0) mbar_arrive(&q_empty[qb]);
        group_sync(bar, 128);                      // the next segment's maxima go where these sums were read
        continue;
      }
      if (!mbar_wait_warp(&stat_full[qb], (seg / kQBufs) & 1, err, kErrMmaTimeout, kPolls)) break;
      const bool whole = s.n == s.tiles;
      const int pairs = s.rows * a.group;
      // of a CTA's two cut segments, the one that it goes on with and the one that it begins
      const int slot = s.tile > 0 ? 2 * cta : 2 * cta + 1;
      if (quarter == 0 && lane < live) {
        // out = sum_w f_w O_w: f_w = 2^(m_w - M) / (L 64 2^(m_w - mv_w)) = 2^(mv_w - M) / (64 L).  The factors stay apart, the
        // first one as two square roots: V's scales go from 2^-126 to 2^120, and O_w / (64 L) brings O_w to the size of V's codes first.
        const float ma = stat[qb][0][0][lane], mb = stat[qb][1][0][lane], la = stat[qb][0][2][lane], lb = stat[qb][1][2][lane];
        const bool has_a = la > 0.f || la != la, has_b = lb > 0.f || lb != lb;   // NaN counts as seen
        const float M = fmaxf(ma, mb);
        const float L = (has_a ? la * ex2_approx(ma - M) : 0.f) + (has_b ? lb * ex2_approx(mb - M) : 0.f);
        fin[wg][0][lane] = has_a ? ex2_approx(0.5f * (stat[qb][0][1][lane] - M)) : 0.f;
        fin[wg][1][lane] = has_b ? ex2_approx(0.5f * (stat[qb][1][1][lane] - M)) : 0.f;
        stat[qb][0][2][lane] = 1.f / L / kPOne;          // (la has been read)
        if (whole) {
          if (a.lse) a.lse[cm.at[lane]] = has_a || has_b ? (M + __log2f(L)) * 0.69314718055994530942f : -INFINITY;
        } else {
          float* ml = a.part_ml + ((int64_t)slot * kColMax + lane) * 2;
          ml[0] = M;
          ml[1] = L;
        }
      }
      if (row == 0 && u - s.n == u0)                     // for the join: this CTA's first piece
        reinterpret_cast<PaRecord*>(a.rec)[cta] = {units, s.tile, s.tiles, s.row0, pairs, s.cg * kCE, s.h};
      poison = stat_nan[qb][0][row] | stat_nan[qb][1][row];
      group_sync(bar, 128);
      if (!mbar_wait_warp(&o_full[seg & 1], (seg >> 1) & 1, err, kErrMmaTimeout, kPolls)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < live; c0 += 8) {
        uint32_t r[32];
        tmem_ld_cols8(acc + c0, r);
        tmem_ld_cols8(acc + kHalf + c0, r + 8);
        tmem_ld_cols8(acc + 64 + c0, r + 16);
        tmem_ld_cols8(acc + 64 + kHalf + c0, r + 24);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c0 + c >= live) break;
          const float fa = fin[wg][0][c0 + c], fb = fin[wg][1][c0 + c], over = stat[qb][0][2][c0 + c];
          // an accumulator without a seen key holds nothing of this column (or was never written)
          float v = 0.f;
          if (fa != 0.f) v = fmaf(__uint_as_float(r[8 + c]), 0.0625f, __uint_as_float(r[c])) * over * fa * fa;
          if (fb != 0.f) v = fmaf(fmaf(__uint_as_float(r[24 + c]), 0.0625f, __uint_as_float(r[16 + c])) * over * fb, fb, v);
          if ((poison >> (c0 + c)) & 1u) v = __int_as_float(0x7FC00000);
          if (whole) {
            a.out[(int64_t)cm.at[c0 + c] * kKvDim + row] = __float2bfloat16_rn(v);
          } else {
            a.part_o[((int64_t)slot * kColMax + c0 + c) * kKvDim + row] = v;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&o_empty[seg & 1]);
        mbar_arrive(&q_empty[qb]);
      }
    }
    group_leave(bar, 128);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0) {
    a.err[kStatusCtaWords + cta] = bits_all;
    if (cta == 0) {
      a.err[0] = 0;
      a.err[1] = (uint32_t)ctas;
    }
  }
}

// Joins the pieces of segments that were cut, where no request may have so many rows that the other kernel runs too
__global__ void __launch_bounds__(256) paged_attention_join_kernel(const __grid_constant__ PagedAttnArgs a, int ctas) {
  pdl_wait();
  pdl_trigger();
  pa_join(a, ctas, blockIdx.x + 1, blockIdx.y);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
PagedAttnPlan plan_paged_attention(int max_query_len, int group) {
  PagedAttnPlan p;
  const int ctas = device_sm_count();
  p.prompt = (int64_t)max_query_len * group > kPagedAttnDirect;
  p.rec_offset = kWorkspaceHeader + ((size_t)ctas * sizeof(uint32_t) + 255) / 256 * 256;
  // each kernel's records and pieces: one launch joins both kernels'
  const size_t recs = ((size_t)ctas * sizeof(PaRecord) + 255) / 256 * 256, few = (size_t)2 * ctas * kPagedAttnColumns * (kKvDim + 2);
  const size_t many = p.prompt ? (size_t)2 * ctas * kPromptPairs * (kKvDim + 2) : 0;
  p.prompt_rec_offset = p.rec_offset + recs;
  p.part_offset = p.prompt_rec_offset + (p.prompt ? recs : 0);
  p.prompt_part_offset = p.part_offset + few * sizeof(float);
  p.workspace_bytes = p.prompt_part_offset + many * sizeof(float);
  return p;
}

namespace {
template <int kCE>
cudaError_t launch_columns(const PagedAttnArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map, int ctas, bool join,
                           cudaStream_t s) {
  const size_t smem = pa::kFixedSmem + (size_t)a.num_requests * sizeof(int32_t);
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = once_per_device(ready, [] {
    const int most = pa::kFixedSmem + DSA_MAX_REQUESTS * (int)sizeof(int32_t);
    cudaError_t r = cudaFuncSetAttribute(paged_attention_kernel<kCE, kPaPlain>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(paged_attention_kernel<kCE, kPaCapBias>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(paged_attention_kernel<kCE, kPaLargeCap>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return r;
  });
  if (e != cudaSuccess) return e;
  const int shared_keys = std::min<int64_t>((int64_t)a.max_rows * a.group, a.hi_pairs) > kCE ? 1 : 0;   // column groups share keys
  const PaMods mods = pa_mods(a);
  auto kernel = mods == kPaPlain     ? paged_attention_kernel<kCE, kPaPlain>
                : mods == kPaCapBias ? paged_attention_kernel<kCE, kPaCapBias>
                                     : paged_attention_kernel<kCE, kPaLargeCap>;
  e = launch_pdl(kernel, dim3(ctas), dim3(pa::kThreads), smem, s, k_map, v_map, a, shared_keys);
  count_launches(1);
  if (e != cudaSuccess) return e;
  if (ctas > 1 && !a.whole && join) {
    e = launch_pdl(paged_attention_join_kernel, dim3(ctas - 1, kCE / 8), dim3(256), 0, s, a, ctas);
    count_launches(1);
  }
  return e;
}
}  // namespace

cudaError_t launch_paged_attention(PagedAttnArgs a, const uint8_t* k_codes, const uint8_t* v_codes, int max_seq_len, void* workspace,
                                   const PagedAttnPlan& plan, cudaStream_t s) {
  char* ws = static_cast<char*>(workspace);
  const int ctas = device_sm_count();
  a.err = reinterpret_cast<uint32_t*>(ws);
  a.rec = reinterpret_cast<int32_t*>(ws + plan.rec_offset);
  a.part_o = reinterpret_cast<float*>(ws + plan.part_offset);
  // Requests of at most 1,024 keys are not cut: a CTA takes such a segment in less time than a second launch to join
  // its pieces would (in replayed graphs, one request of 300 keys: 10.4 instead of 19.8 us; 4 prompts of 1,000 rows: 89 instead
  // of 97; a single prompt of 1,000 rows and one K/V head, which leaves most SMs idle: 35.1 instead of 31.4).
  a.whole = max_seq_len <= 8 * kPaTok;
  a.lo_pairs = 0;
  a.hi_pairs = plan.prompt ? kPagedAttnDirect : INT32_MAX;
  // The prompt kernel's warps wait for each other with a bound of a second, and its writers for this kernel's end, so they
  // start early only where this kernel's CTAs cannot differ by as much: 2^23 tiles are 0.3 s of work for all of them.
  a.early = plan.prompt && (int64_t)a.num_requests * (((int64_t)max_seq_len + kPaTok - 1) / kPaTok) * a.kv_heads * 2 <= int64_t(1) << 23;
  a.part_ml = a.part_o + (size_t)2 * ctas * kPagedAttnColumns * kKvDim;
  const uint64_t rows = (uint64_t)a.num_pages * a.kv_heads << a.log2_page;
  CUtensorMap k_map, v_map;
  if (!encode_2d(&k_map, k_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kKvDim, rows, kKvDim, kKvDim, 1u << a.log2_page) ||
      !encode_2d(&v_map, v_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kKvDim, rows, kKvDim, kKvDim, 1u << a.log2_page))
    return cudaErrorInvalidValue;
  const int64_t pairs = (int64_t)a.max_rows * a.group;
  cudaError_t e = pairs <= 8    ? launch_columns<8>(a, k_map, v_map, ctas, !plan.prompt, s)
                  : pairs <= 16 ? launch_columns<16>(a, k_map, v_map, ctas, !plan.prompt, s)
                                : launch_columns<32>(a, k_map, v_map, ctas, !plan.prompt, s);
  if (e == cudaSuccess && plan.prompt) {
    PagedAttnArgs many = a;
    many.lo_pairs = kPagedAttnDirect;
    many.hi_pairs = INT32_MAX;
    many.rec = reinterpret_cast<int32_t*>(ws + plan.prompt_rec_offset);
    many.part_o = reinterpret_cast<float*>(ws + plan.prompt_part_offset);
    many.part_ml = many.part_o + (size_t)2 * ctas * kPromptPairs * kKvDim;
    e = launch_paged_prompt(many, a, kPagedAttnColumns / 8, k_map, v_codes, ctas, s);   // more than 64 pairs: 32 columns above
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dsa
