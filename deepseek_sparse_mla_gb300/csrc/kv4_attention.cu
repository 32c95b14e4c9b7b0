// Dense grouped-head attention over the paged 4-bit K/V cache, on tcgen05 tensor cores: the kernel for few rows a request, and the
// launches.  (Requests of many rows: kv4_prompt.cu.)
//
//   z_s = scale * q[r,h] . (k_code_s * 2^e_s)     [then the cap and the distance bias]
//   out[r,h] = sum_s softmax(z)_s * (v_code_s * vs_s),   lse[r,h] = ln sum_s exp(z_s)
// with e2m1 codes, an exponent e for each 32 dims of a key and one scale vs a token for V.
//
// Nothing is widened on chip.  TMA writes 16 codes into the first half of each 16-byte unit, the form in which the tensor
// cores take 4-bit operands beside 8-bit ones:
//   S^T [128 keys x columns]  = K [128 x 128] (K-major, its block scales from TMEM) * Q^T     kind::mxf8f6f4
//   O^T [128 dims x columns] += V^T (the same layout, MN-major) * P^T                         kind::f8f6f4
// The small operands are two e4m3 terms, hi and lo with hi + lo / 16 (see paged_attention.cu): columns of their own; Q's lo
// terms have a block scale of 2^-4.  With 32 columns TMEM has no room for both of S's, and Q's terms are two products into
// the same columns.  V's scale is in what P codes, p * vs, against a running maximum of z + log2 vs of its own.
// A product with 128 rows takes 40 cycles a 32-deep step whatever its columns (48 with 64), as the 128 rows are read at 128
// bytes a cycle: 320 cycles a tile of 128 keys here.  4-bit codes are finite whatever the bits are, so what lies behind a
// request's tokens needs a probability of 0 and no more.
//
// Bound by HBM: 134 bytes a key and head, 17 KB a tile, which arrive every 740 cycles.  What stands against that is latency and
// instructions, not products: a CTA's loops run side by side, each with its own wait, and the ring's stages hold half
// as many bytes as they take.  So: loads, orders, products and softmax are warps of their own with short loops; rings of K
// and V apart, as K is done with early; one warp finds segments for all; references and factors of 8 columns stay in
// registers; probabilities are formed in pairs (f32x2, then f16x2 for the two terms).
//
// Work, pieces and their join as in paged_attention.cu.  Per CTA (16 warps): 0 and 4 load K, 2 and 6 V; 5 orders K's scales; 1 issues
// the products of the scores, 3 of the outputs; 7 finds the segments and splits their queries; 8-11 and 12-15 are the softmax,
// two warpgroups that take the tiles in turn, one key a thread.
#include "paged_attention.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

#include <algorithm>
#include <type_traits>

namespace dsa {
using namespace sm100;

namespace p4 {
constexpr int kTok = kPaTok;                    // keys per tile
constexpr int kTileBytes = kTok * kKvDim;       // of K or V in shared memory: 16-byte units, half used
constexpr int kKScales = kTok * kKv4Blocks, kVScales = kTok * 2;   // bytes of a tile's scales
constexpr int kLoadKWarp = 0, kScoreWarp = 1, kLoadVWarp = 2, kOutWarp = 3, kOrderWarp = 5, kQueryWarp = 7, kSoftWarp0 = 8;   // loaders: 0 and 4, 2 and 6
constexpr int kQBufs = 3, kSegBufs = 4, kOBufs = 2;   // segments with queries, with a description and with accumulators
// Three softmax warpgroups instead of two: 480 us instead of 476 for 64 requests of 16K-128K, and with 32 columns (where TMEM then holds one
// segment's accumulators) 291 instead of 301 for the verify rows at 240K but 92 instead of 90 for the mixed capped batch.
constexpr int kWgs = 2, kThreads = 256 + 128 * kWgs;
constexpr uint32_t kRegsLow = 80, kRegsSoft = 176;   // 2 * 80 + 2 * 176 = 4 * 128: the launch's
constexpr uint32_t kTmemCols = 512, kColScales = 192, kColQScales = 216, kColO = 256;
constexpr float kSlackP = 4.f;                  // a reference may be exceeded by this factor
constexpr float kPOne = 64.f;                   // the code of a contribution at its reference: 2^2 above fits in 448
// kPOne's factors: 2^4 comes in with a column's references and the rest with a key's scale, so that scales below 2^126 (more than the
// append writes) stay finite.  References are formed with scales of at least 2^-121: 2^(m - mv + 4) times a probability below 4 stays finite, too.
constexpr int kColumnLog2 = 4, kLowScaleLog2 = -121;
constexpr float kKeyPOne = kPOne / (1 << kColumnLog2);
static_assert(kColumnLog2 - kLowScaleLog2 + 2 < 128, "fp32's range");
constexpr uint32_t kPolls = 1u << 18;           // of 3.8 us each or more: a second
constexpr uint32_t kSegPolls = 1u << 24;        // for the end of a whole segment: a minute
// Polls are rolled: the bodies of many roles share the instruction caches.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t code, uint32_t polls = kPolls) {
  return mbar_wait_warp<1>(bar, parity, err, code, polls);
}

template <int kCE>
struct Form {
  static constexpr int kHalf = kCE < 16 ? 16 : kCE, kN = 2 * kHalf;   // columns of the hi terms, and of both
  static constexpr bool kApart = kCE <= 16;           // Q's two terms have columns of their own
  static constexpr int kColsS = kApart ? kN : kHalf;  // TMEM columns of a tile's scores
  // Rings: K's tiles and their scores, V's tiles and their probabilities.  One barrier says that a product has been computed,
  // which frees what it read and hands over what it wrote.
  static constexpr int kKStages = kCE <= 16 ? 5 : 4, kVStages = kCE <= 16 ? 6 : 5;
  static constexpr int kQBytes = kN * kKvDim, kPBytes = kTok * kN;
  static constexpr int kSmem = (kKStages + kVStages) * kTileBytes + kQBufs * kQBytes + kVStages * kPBytes + kKStages * kKScales + kVStages * kVScales + 1024;
  static_assert(kKStages * kColsS <= (int)kColScales && kColScales + 4 * kKStages <= kColQScales && kColO + kOBufs * kWgs * kN <= kTmemCols, "TMEM columns");
};

// A run of tiles of one segment, as the segment warp leaves it for the others
struct __align__(16) Seg {
  int n, tile, tiles, b;           // its tiles and the first of them (n = 0: no further segment); the segment's tiles; the request
  int h, cg, rows, row0;
  int len, pad[3];
  // The last keys first where a bias on distance would move the references with every tile (see paged_attention.cu)
  template <bool kFalling>
  __device__ __forceinline__ int tile_at(int t) const { return kFalling ? tile + n - 1 - t : tile + t; }
};

// A place in a ring of kN stages and the parity of its turn
template <int kN>
struct Ring {
  int st = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void next() {
    if (++st == kN) {
      st = 0;
      turn ^= 1;
    }
  }
};

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
}  // namespace p4

// kCE columns (8, 16 or 32); kModSet: score cap and distance bias compiled in
template <int kCE, PaMods kModSet>
__global__ void __launch_bounds__(p4::kThreads, 1)
    kv4_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                         const __grid_constant__ PagedAttnArgs a, int shared_keys) {
  using namespace p4;
  using F = Form<kCE>;
  constexpr bool kMods = kModSet != kPaPlain;
  constexpr int kHalf = F::kHalf, kN = F::kN, kKStages = F::kKStages, kVStages = F::kVStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sK = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sV = sK + kKStages * kTileBytes;
  uint8_t* const sQ = sV + kVStages * kTileBytes;
  uint8_t* const sP = sQ + kQBufs * F::kQBytes;
  uint8_t* const sScaleK = sP + kVStages * F::kPBytes;
  uint8_t* const sScaleV = sScaleK + kKStages * kKScales;

  __shared__ uint64_t k_full[kKStages], sf_full[kKStages], s_full[kKStages], s_empty[kKStages];
  __shared__ uint64_t v_full[kVStages], p_full[kVStages], pv_done[kVStages];
  __shared__ uint64_t q_full[kQBufs], q_empty[kQBufs], stat_full[kQBufs], o_full[kOBufs], o_empty[kOBufs], mma_done;
  __shared__ uint64_t seg_full[kSegBufs], seg_empty[kSegBufs];
  __shared__ Seg segs[kSegBufs];
  __shared__ uint32_t sbad[kVStages];                  // pages of a tile that are not there
  __shared__ __align__(16) PaColumns cols[kQBufs];
  __shared__ __align__(16) float refs[kWgs][2][kCE];
  __shared__ float wmax[kWgs][4][kCE], fin[kWgs][kWgs][kCE];
  __shared__ float stat[kQBufs][kWgs][3][kCE];            // each warpgroup's m, mv and l of a segment
  __shared__ int32_t scan[kThreads / 32], total;
  __shared__ uint32_t tmem_base, bits_all;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&sf_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&p_full[i], 1);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < kOBufs; ++i) {
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1 + 4 * kWgs);            // the last product that reads it, and the softmax warps
      mbar_init(&stat_full[i], 4 * kWgs);
    }
    for (int i = 0; i < kSegBufs; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 7 + 4 * kWgs);                   // every warp that reads it
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
  if (a.early) pdl_trigger();                          // for the prompt kernel, not for a join (see paged_attention.cu)
  if (tid == 0) reinterpret_cast<PaRecord*>(a.rec)[cta].tile = -1;   // no piece to join until it has been written
  // the requests' units
  {
    uint32_t bits = 0;
    int sum = 0;
    for (int b = tid; b < a.num_requests; b += kThreads) {
      const PaShape s = pa_shape(a, b, bits);
      sum += (s.rows * a.group + kCE - 1) / kCE * s.tiles;
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) scan[warp] = sum;
    if (bits) atomicOr(&bits_all, bits);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) {
    int sum = 0;
    for (int w = 0; w < kThreads / 32; ++w) sum += scan[w];
    total = sum;
  }
  const uint32_t tmem = tmem_base;
  // the queries' block scales: 1 for the hi terms, 2^-4 for the lo ones, which are rows of their own (a lane each) or have byte 1
  if (warp < 4) {
    const uint32_t word = !F::kApart ? 0x7B7Fu : lane < kHalf ? 0x7Fu : 0x7Bu;
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tmem + kColQScales + ((uint32_t)(32 * warp) << 16)),
                 "r"(word)
                 : "memory");
    tmem_wait_st();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int64_t units = (int64_t)total * a.kv_heads;
  uint32_t* const err = &bits_all;                     // this CTA's status bits, stored at the end

  if (warp < kSoftWarp0) {
    regs_dec<kRegsLow>();
    const int lp = a.log2_page, ppt = kTok >> lp;
    // one segment after the other: its place in the ring, and a copy of what it is
    int seg = -1;
    auto next_segment = [&](Seg& s) {
      ++seg;
      if (!wait_warp(&seg_full[seg % kSegBufs], (seg / kSegBufs) & 1, err, kErrMmaTimeout)) return false;
      s = segs[seg % kSegBufs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[seg % kSegBufs]);
      return s.n > 0;
    };
    // 32 pages of a segment from page 32 * batch on, one a lane: their ids (as they are in the table; -1 behind the request's
    // tokens), asked for well before they are used, and then their first rows (-1: not there).
    auto pages_of = [&](const Seg& s, int batch) {
      const int p = 32 * batch + lane;
      return p >= 0 && p < (s.len + (1 << lp) - 1) >> lp ? a.block_table[(int64_t)s.b * a.table_stride + p] : -1;
    };
    auto rows_of = [&](const Seg& s, int batch, int page, bool report) {
      if (page >= 0 && page < a.num_pages) return (page * a.kv_heads + s.h) << lp;
      if (report && 32 * batch + lane < (s.len + (1 << lp) - 1) >> lp) atomicOr(err, kErrBadPage);
      return -1;
    };
    const uint64_t policy = shared_keys ? l2_evict_normal() : l2_evict_first();
    // Every other tile of K or V, codes (lanes 0 .. ppt - 1, a page each) and scales (lanes 8 ..).  4-bit codes count 64 bytes a row
    // on the barrier.  Getting one tile's copies out takes a warp some 900 cycles of one thing after the other, so two warps
    // take turns.
    auto load = [&](auto of_v) {
      constexpr bool kV = decltype(of_v)::value;
      constexpr int kRing = kV ? kVStages : kKStages, kScale = kV ? 2 : kKv4Blocks, kWay = kMods ? -1 : 1;   // scale bytes of a token
      uint64_t* const full = kV ? v_full : k_full;
      uint64_t* const empty = kV ? pv_done : s_full;
      const uint8_t* const scales = kV ? reinterpret_cast<const uint8_t*>(a.v_scales4) : a.k_scales4;
      const int mine = lane & 7;
      const bool codes = lane < 8, used = mine < ppt && lane < 16;
      uint8_t* const dst = codes ? (kV ? sV : sK) + mine * (kKvDim << lp) : (kV ? sScaleV : sScaleK) + mine * (kScale << lp);
      int i = warp >> 2, i0 = 0, st = i;               // the tile to load (its place in the ring, and the ring's turn), and the CTA's before the segment
      uint32_t turn = 0;
      bool ok = true;
      for (Seg s; ok && next_segment(s); i0 += s.n) {
        if (i - i0 >= s.n) continue;
        int batch = (s.template tile_at<kMods>(i - i0) * ppt) >> 5, row32 = rows_of(s, batch, pages_of(s, batch), kV), ahead = pages_of(s, batch + kWay);
        for (; i - i0 < s.n; i += 2) {
          const int p0 = s.template tile_at<kMods>(i - i0) * ppt;
          if ((p0 >> 5) != batch) {
            batch += kWay;
            row32 = rows_of(s, batch, ahead, kV);
            ahead = pages_of(s, batch + kWay);
          }
          if (i >= kRing) ok = wait_warp(&empty[st], turn ^ 1, err, kErrMmaTimeout);
          if (!ok) break;
          const int row = __shfl_sync(0xffffffffu, row32, (p0 + mine) & 31);
          const uint32_t bad = __ballot_sync(0xffffffffu, codes && used && row < 0);
          if (lane == 0) {
            if (kV) sbad[st] = bad;
            mbar_arrive_expect_tx(&full[st], (uint32_t)(ppt - __popc(bad)) * ((uint32_t)(kKvDim / 2 + kScale) << lp));
          }
          __syncwarp();
          if (used && row >= 0) {
            if (codes) tma_load_2d_hint(dst + st * kTileBytes, kV ? &v_map : &k_map, 0, row, &full[st], policy);
            else bulk_load_hint(dst + st * (kTok * kScale), scales + (int64_t)row * kScale, kScale << lp, &full[st], policy);
          }
          st += 2;
          if (st >= kRing) {
            st -= kRing;
            turn ^= 1;
          }
        }
      }
      // nothing may still be landing in shared memory when the CTA exits: this warp's among the last kRing tiles (the stages of
      // earlier ones have been filled again since).  Where the wait for tile i's place ran out, those before tile i, and what that
      // place holds, whichever warp's it is.  (Tiles before that one have been used, and so have landed.)
      const int end = ok ? i0 : i;
      if (!ok) wait_warp(&full[st], turn ^ 1, err, kErrTmaTimeout);
      for (i -= 2; i >= 0 && i >= end - kRing; i -= 2) {
        st -= 2;
        if (st < 0) {
          st += kRing;
          turn ^= 1;
        }
        wait_warp(&full[st], turn, err, kErrTmaTimeout);
      }
    };
    if ((warp & 3) == kLoadKWarp) {
      load(std::false_type{});
    } else if ((warp & 3) == kLoadVWarp) {
      load(std::true_type{});
    } else if (warp == kOrderWarp) {
      // ---------------------------------------------------------------- K's scales as tcgen05.cp takes them
      // Those of keys l, l + 32, l + 64 and l + 96 go into the l-th 16 bytes.
      // The arrival on sf_full also says that the place of the tile's scores is free, so that the product's issuer waits once.
      Ring<kKStages> r;
      bool ok = true, first = true;
      for (Seg s; ok && next_segment(s);)
        for (int t = 0; t < s.n; ++t) {
          ok = wait_warp(&k_full[r.st], r.turn, err, kErrTmaTimeout);
          if (!ok) break;
          uint32_t* const raw = reinterpret_cast<uint32_t*>(sScaleK + r.st * kKScales);
          uint32_t w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = raw[32 * c + lane];
          __syncwarp();
          reinterpret_cast<uint4*>(raw)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
          fence_proxy_async_smem();
          ok = first || wait_warp(&s_empty[r.st], r.turn ^ 1, err, kErrMmaTimeout);
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sf_full[r.st]);
          r.next();
          if (r.st == 0) first = false;
        }
    } else if (warp == kScoreWarp) {
      // ---------------------------------------------------------------- products of the scores
      // The warp walks together and one elected lane issues: addresses stay in uniform registers.
      const bool leader = elect_one();
      const uint32_t id_qk = idesc_mx(kTok, F::kApart ? kN : kHalf, kFmtE2m1, kFmtE4m3);
      const uint64_t d_k = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B), d_q = smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
      const uint64_t d_sf = smem_desc(smem_u32(sScaleK), 16, 128, kSwizzleNone);
      Ring<kKStages> r;
      bool ok = true;
      for (Seg s; ok && next_segment(s);) {
        const int qb = seg % kQBufs;
        ok = wait_warp(&q_full[qb], (seg / kQBufs) & 1, err, kErrMmaTimeout);
        const uint64_t q = d_q + (uint64_t)((qb * F::kQBytes) >> 4);
        for (int t = 0; t < s.n && ok; ++t) {
          ok = wait_warp(&sf_full[r.st], r.turn, err, kErrTmaTimeout);
          if (!ok) break;
          tc_fence_after();
          const uint64_t k = d_k + (uint64_t)((r.st * kTileBytes) >> 4);
          if (leader) {
            const uint32_t sf = tmem + kColScales + 4 * r.st, to = tmem + F::kColsS * r.st;
            tmem_cp_scales(sf, d_sf + (uint64_t)((r.st * kKScales) >> 4));
#pragma unroll
            for (int kk = 0; kk < (F::kApart ? 1 : 2) * kKvDim / 32; ++kk) {   // (in the same columns: hi, then lo)
              const uint32_t block = kk & 3, term = kk >> 2;
              mma_ss_mx(to, k + 2 * block, q + 2 * block + (uint64_t)((term * kHalf * kKvDim) >> 4), id_qk | block << 29 | term << 4, sf,
                        tmem + kColQScales, kk > 0);
            }
            mma_commit(&s_full[r.st]);
            if (t + 1 == s.n) mma_commit(&q_empty[qb]);
          }
          __syncwarp();
          r.next();
        }
      }
      // every MMA issued here has finished before TMEM is released
      if (leader) mma_commit(&mma_done);
      wait_warp(&mma_done, 0, err, kErrMmaTimeout);
    } else if (warp == kOutWarp) {
      // ---------------------------------------------------------------- products of the outputs
      const bool leader = elect_one();
      const uint32_t id_pv = idesc_e4m3(kKvDim, kN) | (1u << 15) | (1u << 16) | (kFmtE2m1 << 7);   // both operands MN-major
      const uint64_t d_v = smem_desc(smem_u32(sV), 16, 1024, kSwizzle128B);
      const uint64_t d_p = smem_desc(smem_u32(sP), 16, 8 * kN, kN == 64 ? kSwizzle64B : kSwizzle32B);
      Ring<kVStages> r;
      uint32_t wg = 0;                                 // whose tile it is
      bool ok = true;
      for (Seg s; ok && next_segment(s);) {
        uint32_t fresh = (1u << kWgs) - 1;                            // accumulators of the segment without a product yet
        if (seg >= kOBufs) ok = wait_warp(&o_empty[seg % kOBufs], (seg / kOBufs - 1) & 1, err, kErrMmaTimeout);
        for (int t = 0; t < s.n; ++t) {
          ok = ok && wait_warp(&p_full[r.st], r.turn, err, kErrMmaTimeout);
          if (!ok) break;
          tc_fence_after();
          const uint64_t v = d_v + (uint64_t)((r.st * kTileBytes) >> 4), p = d_p + (uint64_t)((r.st * F::kPBytes) >> 4);
          const uint32_t to = tmem + kColO + kWgs * kN * (seg % kOBufs) + kN * wg;
          const bool add = !((fresh >> wg) & 1u);
          fresh &= ~(1u << wg);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kTok / 32; ++kk)
              mma_ss_f8(to, v + (uint64_t)((kk * 32 * kKvDim) >> 4), p + (uint64_t)((kk * 32 * kN) >> 4), id_pv, add || kk > 0);
            mma_commit(&pv_done[r.st]);
            if (t + 1 == s.n) mma_commit(&o_full[seg % kOBufs]);
          }
          __syncwarp();
          r.next();
          if (++wg == kWgs) wg = 0;
        }
      }
      if (leader) mma_commit(&mma_done);
      wait_warp(&mma_done, 0, err, kErrMmaTimeout);
    } else if (warp == kQueryWarp) {
      // ---------------------------------------------------------------- segments (and an end mark), and their queries
      int64_t u = pa_unit_start(cta, units, ctas);
      const int64_t u1 = pa_unit_start(cta + 1, units, ctas);
      // segments are cut where the range ends, or (short requests) belong to the range they begin in as a whole
      const int64_t cut = a.whole ? units : u1;
      int b = 0;                                       // units of the requests before b, without heads
      int64_t before = 0;
      bool ok = true;
      for (Seg s;;) {
        s = {};
        while (u < u1 && s.n == 0) {
          // the request that holds u: 32 at a time
          for (;;) {
            uint32_t none = 0;
            int count = 0;
            if (b + lane < a.num_requests) {
              const PaShape sh = pa_shape(a, b + lane, none);
              count = (sh.rows * a.group + kCE - 1) / kCE * sh.tiles;
            }
            int incl = count;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int v = __shfl_up_sync(0xffffffffu, incl, o);
              if (lane >= o) incl += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, (before + incl) * a.kv_heads > u);
            if (hit) {
              const int l = __ffs(hit) - 1;
              b += l;
              before += __shfl_sync(0xffffffffu, incl - count, l);
              break;
            }
            b += 32;
            before += __shfl_sync(0xffffffffu, incl, 31);
          }
          uint32_t none = 0;
          const PaShape sh = pa_shape(a, b, none);
          const int per_head = (sh.rows * a.group + kCE - 1) / kCE * sh.tiles;
          const int64_t in = u - before * a.kv_heads;
          s.h = in < (int64_t(1) << 31) ? (int)((uint32_t)in / (uint32_t)per_head) : (int)(in / per_head);
          const int rest = (int)(in - (int64_t)s.h * per_head);
          s.cg = rest / sh.tiles;
          s.tile = rest - s.cg * sh.tiles;
          s.n = (int)min((int64_t)(sh.tiles - s.tile), cut - u);
          u += s.n;
          if (a.whole && s.tile > 0) s.n = 0;          // the range before has it
          s.tiles = sh.tiles;
          s.b = b;
          s.rows = sh.rows;
          s.row0 = sh.row0;
          s.len = sh.len;
        }
        ++seg;
        if (seg >= kSegBufs) ok = wait_warp(&seg_empty[seg % kSegBufs], (seg / kSegBufs - 1) & 1, err, kErrMmaTimeout, kSegPolls);
        if (!ok) break;
        if (lane == 0) {
          segs[seg % kSegBufs] = s;
          mbar_arrive(&seg_full[seg % kSegBufs]);
        }
        __syncwarp();
        if (s.n == 0) break;
        const int buf = seg % kQBufs;
        if (!pa_query_columns<kCE, kHalf, kMods>(a, s, sQ + buf * F::kQBytes, cols[buf], [&] {
              return seg < kQBufs || wait_warp(&q_empty[buf], (seg / kQBufs - 1) & 1, err, kErrMmaTimeout, kSegPolls);
            }))
          break;
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
    const int sw = kN == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
    constexpr bool kHold = kCE == 8;                   // references and factors stay in registers
    float* const ref_m = refs[wg][0];                  // as -m
    float* const ref_e = refs[wg][1];                  // 2^(m - mv + 4)
    int i0 = 0, i = wg;                                // the CTA's tiles before this segment; this warpgroup's next one
    int kst = wg, vst = wg;                            // its places in the rings (longer than kWgs), and their turns
    uint32_t k_turn = 0, v_turn = 0;
    for (int seg = 0;; ++seg) {
      const int sb_ = seg % kSegBufs, qb = seg % kQBufs;
      if (!wait_warp(&seg_full[sb_], (seg / kSegBufs) & 1, err, kErrMmaTimeout)) break;
      const Seg s = segs[sb_];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[sb_]);
      if (s.n == 0) break;
      if (!wait_warp(&q_full[qb], (seg / kQBufs) & 1, err, kErrMmaTimeout)) break;
      const uint32_t acc = tmem + lanes + kColO + kWgs * kN * (seg % kOBufs);
      const PaColumns& cm = cols[qb];
      const int min_limit = cm.min_limit;
      const int live = min(s.rows * a.group - s.cg * kCE, kCE);   // columns in use
      // the references of column `lane` (m: of z, mv: of z + log2 vs)
      float m_lane = -INFINITY, mv_lane = -INFINITY;
      uint64_t l2[kCE / 2], hold_f[kHold ? 4 : 1], hold_m[kHold ? 4 : 1], hold_e[kHold ? 4 : 1];
#pragma unroll
      for (int c = 0; c < kCE / 2; ++c) l2[c] = 0;
      if (kHold) {
#pragma unroll
        for (int c = 0; c < 4; ++c) hold_f[c] = pack2(cm.factor[2 * c], cm.factor[2 * c + 1]);
      }
      bool ok = true, fresh = true;
      // One tile, with kNC columns in use (8, 16 or 32): a body of its own each, chosen once a tile
      auto tile = [&](auto columns, auto with_masks, int key0) {
        constexpr int kNC = decltype(columns)::value;
        constexpr bool kMasked = decltype(with_masks)::value;
        const int j = key0 + row;
        const bool exists = !kMasked || (j < s.len && !((sbad[vst] >> (row >> a.log2_page)) & 1u));
        const float vs = exists ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(sScaleV + vst * kVScales)[row]) : 0.f;
        const uint32_t from = tmem + lanes + F::kColsS * kst;
        const float in = kMods && a.cap_log2 > 0.f ? 2.f * 1.4426950408889634f / a.cap_log2 : 0.f;
        // distances in integers from the request's first row, exact up to 2^24 (see paged_attention.cu)
        const float ahead = kMods ? (float)(j - cm.start) : 0.f;
        // products as they are, in pairs: all columns at once, one wait
        auto products = [&](auto& z, int c0) {
          constexpr int kC = sizeof(z) / 4;
          uint32_t hi[kC], lo[F::kApart ? kC : 1];
#pragma unroll
          for (int c = 0; c < kC; c += 8) {
            tmem_ld_cols8(from + c0 + c, hi + c);
            if (F::kApart) tmem_ld_cols8(from + kHalf + c0 + c, lo + c);
          }
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < kC / 2; ++c) {
            z[c] = pack2(__uint_as_float(hi[2 * c]), __uint_as_float(hi[2 * c + 1]));
            if (F::kApart) z[c] = add2(z[c], pack2(__uint_as_float(lo[2 * c]), __uint_as_float(lo[2 * c + 1])));
          }
        };
        // four columns of a shared array
        auto four = [&](const float* x, uint64_t (&r)[2]) {
          const float4 v = *reinterpret_cast<const float4*>(x);
          r[0] = pack2(v.x, v.y);
          r[1] = pack2(v.z, v.w);
        };
        // .. and 8 of them as scores
        auto scores = [&](float (&z)[8], const uint64_t* y, int c0) {
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            uint64_t f[2];
            if (kHold) {
              f[0] = hold_f[c];
              f[1] = hold_f[c + 1];
            } else {
              four(cm.factor + c0 + 2 * c, f);
            }
            const float2 v = unpack2(mul2(y[c], f[0])), w = unpack2(mul2(y[c + 1], f[1]));
            z[2 * c] = v.x;
            z[2 * c + 1] = v.y;
            z[2 * c + 2] = w.x;
            z[2 * c + 3] = w.y;
          }
          if (kMods && in != 0.f) {
#pragma unroll
            for (int c = 0; c < 8; ++c) z[c] = capped<kModSet>(z[c] * in, a.cap_log2);
          }
          if (kMods) {
#pragma unroll
            for (int c = 0; c < 8; ++c) z[c] = fmaf(-cm.slope[c0 + c], fabsf(cm.row[c0 + c] - ahead), z[c]);
          }
        };
        auto seen = [&](int c) { return exists && j < cm.limit[c]; };
        // the exact maxima over the tile, where the references do not hold: they, and what was formed against them, move
        auto raise = [&]() {
          const float lv = fmaxf(__log2f(fabsf(vs)), (float)kLowScaleLog2);   // log2 of the key's scale, which may be 0
          float mine = -INFINITY, mine_v = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < kNC; c0 += 8) {
            uint64_t y[4];
            float z[8];
            products(y, c0);
            scores(z, y, c0);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if (kMasked && !seen(c0 + c)) z[c] = -INFINITY;
              const float r = warp_max_f32(z[c]), rv = warp_max_f32(z[c] + lv);
              if (lane == c0 + c) {                    // lane c of every warp ends up with column c's
                mine = r;
                mine_v = rv;
              }
            }
          }
          float* const wmax_v = reinterpret_cast<float*>(sP + vst * F::kPBytes);   // [4][kCE], before the tile's P is there
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
            ref_m[lane] = m_new == -INFINITY ? 1e30f : -m_new;   // nothing seen yet: the first score that is exceeds it
            ref_e[lane] = mv_new == -INFINITY ? 1.f : ex2_approx(m_new - mv_new + (float)kColumnLog2);
          }
          if (!fresh) {
            // the accumulator is settled when the tile before has been added
            const bool back = vst < kWgs;
            ok = wait_warp(&pv_done[back ? vst + kVStages - kWgs : vst - kWgs], back ? v_turn ^ 1 : v_turn, err, kErrMmaTimeout) && ok;
#pragma unroll
            for (int c = 0; c < kNC / 2; ++c)
              l2[c] = mul2(l2[c], pack2(__shfl_sync(0xffffffffu, al, 2 * c), __shfl_sync(0xffffffffu, al, 2 * c + 1)));
            tc_fence_after();
            const uint32_t o = acc + kN * wg;
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
          if (kHold) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              hold_m[c] = *reinterpret_cast<const uint64_t*>(ref_m + 2 * c);
              hold_e[c] = *reinterpret_cast<const uint64_t*>(ref_e + 2 * c);
            }
          }
        };
        // (P's place is free: V's tile was loaded once the product that read both before had been computed)
        uint8_t* const prow = sP + vst * F::kPBytes + row * kN;
        const uint64_t vs2 = pack2(vs * kKeyPOne, vs * kKeyPOne);
        uint64_t p[kNC / 2];
        bool raised = fresh;
        if (fresh) raise();
        for (;;) {
          // the probabilities, and their contributions in two e4m3 terms
          uint64_t all[kNC / 2];
          uint32_t raw[kNC > 16 ? 16 : 1];
          if constexpr (kNC > 16) {
            uint64_t y16[8];
            products(y16, 0);
#pragma unroll
            for (int c = 0; c < 8; ++c) all[c] = y16[c];
            tmem_ld_cols8(from + 16, raw);
            tmem_ld_cols8(from + 24, raw + 8);
          } else {
            products(all, 0);
          }
          uint32_t hi[kHalf / 4], lo[kHalf / 4];
          float p_top = 0.f;                           // (a NaN is no maximum: a column without a pair asks for nothing)
          __half2 x_top = __float2half2_rn(0.f);
#pragma unroll
          for (int c0 = 0; c0 < kHalf; c0 += 8) {
            hi[c0 / 4] = hi[c0 / 4 + 1] = lo[c0 / 4] = lo[c0 / 4 + 1] = 0;
            if (c0 >= kNC) continue;
            if constexpr (kNC > 16) {
              if (c0 == 16) {
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c) all[8 + c] = pack2(__uint_as_float(raw[2 * c]), __uint_as_float(raw[2 * c + 1]));
              }
            }
            uint64_t* const y = all + c0 / 2;
            uint64_t mm[4], ee[4];
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
              uint64_t m2[2] = {}, e2[2] = {}, f2[2] = {};
              if (!kHold) {
                four(ref_m + c0 + 2 * c, m2);
                four(ref_e + c0 + 2 * c, e2);
                if (!kMods) four(cm.factor + c0 + 2 * c, f2);
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                mm[c + k] = kHold ? hold_m[c + k] : m2[k];
                ee[c + k] = kHold ? hold_e[c + k] : e2[k];
                if (!kMods) y[c + k] = fma2(y[c + k], kHold ? hold_f[c + k] : f2[k], mm[c + k]);
              }
            }
            if (kMods) {
              float z[8];
              scores(z, y, c0);
#pragma unroll
              for (int c = 0; c < 4; ++c) y[c] = add2(pack2(z[2 * c], z[2 * c + 1]), mm[c]);
            }
            uint32_t h8[4], l8[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float2 d = unpack2(y[c]);
              float2 e = make_float2(ex2_approx(d.x), ex2_approx(d.y));
              if (kMasked) {
                if (!seen(c0 + 2 * c)) e.x = 0.f;
                if (!seen(c0 + 2 * c + 1)) e.y = 0.f;
              }
              p[(c0 >> 1) + c] = pack2(e.x, e.y);
              p_top = max3(p_top, e.x, e.y);
              // in this order: 0 stays 0 whatever the scale of an unseen key ..
              float2 x = unpack2(mul2(mul2(p[(c0 >> 1) + c], ee[c]), vs2));
              if (kMasked) {                           // .. and of one that some columns do not see even NaN
                if (!seen(c0 + 2 * c)) x.x = 0.f;
                if (!seen(c0 + 2 * c + 1)) x.y = 0.f;
              }
              // in fp16: 11 bits of a contribution, of which the two terms keep 8
              const __half2 h = __floats2half2_rn(x.x, x.y);
              x_top = __hmax2(x_top, __habs2(h));
              h8[c] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
              const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h8[c], __NV_E4M3);
              const __half2 rest = __hmul2(__hsub2(h, __half2(back)), __float2half2_rn(16.f));
              l8[c] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E4M3);
            }
            hi[c0 / 4] = h8[0] | h8[1] << 16;
            hi[c0 / 4 + 1] = h8[2] | h8[3] << 16;
            lo[c0 / 4] = l8[0] | l8[1] << 16;
            lo[c0 / 4 + 1] = l8[2] | l8[3] << 16;
          }
#pragma unroll
          for (int q = 0; q < kHalf / 16; ++q) {
            *reinterpret_cast<uint4*>(prow + ((q ^ sw) << 4)) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
            *reinterpret_cast<uint4*>(prow + (((q + kHalf / 16) ^ sw) << 4)) =
                make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
          }
          fence_proxy_async_smem();
          tc_fence_before();
          const float x_most = fmaxf(__low2float(x_top), __high2float(x_top));
          if (!group_or(bar, 128, !raised && (p_top >= kSlackP || x_most > kSlackP * kPOne))) break;
          raised = true;                               // the same in all four warps
          raise();
        }
#pragma unroll
        for (int c = 0; c < kNC / 2; ++c) l2[c] = add2(l2[c], p[c]);
        fresh = false;
        if (row == 0) mbar_arrive(&p_full[vst]);
        if (lane == 0) mbar_arrive(&s_empty[kst]);
      };
      for (; ok && i - i0 < s.n; i += kWgs) {
        const int key0 = s.template tile_at<kMods>(i - i0) * kTok;
        ok = wait_warp(&v_full[vst], v_turn, err, kErrTmaTimeout) && wait_warp(&s_full[kst], k_turn, err, kErrMmaTimeout);
        if (!ok) break;
        tc_fence_after();
        using std::integral_constant;
        const bool masked = __any_sync(0xffffffffu, key0 + kTok > min_limit || sbad[vst] != 0);
        auto with_columns = [&](auto columns) {
          if (masked) tile(columns, std::true_type{}, key0);
          else tile(columns, std::false_type{}, key0);
        };
        if constexpr (kCE == 32) {
          if (live > 16) with_columns(integral_constant<int, 32>{});
          else if (live > 8) with_columns(integral_constant<int, 16>{});
          else with_columns(integral_constant<int, 8>{});
        } else if constexpr (kCE == 16) {
          if (live > 8) with_columns(integral_constant<int, 16>{});
          else with_columns(integral_constant<int, 8>{});
        } else {
          with_columns(integral_constant<int, 8>{});
        }
        kst += kWgs;
        if (kst >= kKStages) {
          kst -= kKStages;
          k_turn ^= 1;
        }
        vst += kWgs;
        if (vst >= kVStages) {
          vst -= kVStages;
          v_turn ^= 1;
        }
      }
      if (!ok) break;
      i0 += s.n;
      // ---- the segment's end: each warpgroup leaves its maxima and denominators, and one writes the outputs
#pragma unroll
      for (int c0 = 0; c0 < kCE; c0 += 8) {
        if (c0 >= live) continue;
#pragma unroll
        for (int c = c0; c < c0 + 8; c += 2) {
          float2 v = unpack2(l2[c >> 1]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
          }
          if (lane == 0) {
            wmax[wg][quarter][c] = v.x;
            wmax[wg][quarter][c + 1] = v.y;
          }
        }
      }
      group_sync(bar, 128);
      if (quarter == 0 && lane < live) {
        stat[qb][wg][0][lane] = m_lane;
        stat[qb][wg][1][lane] = mv_lane;
        stat[qb][wg][2][lane] = (wmax[wg][0][lane] + wmax[wg][1][lane]) + (wmax[wg][2][lane] + wmax[wg][3][lane]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&stat_full[qb]);
      if ((seg & 1) != wg) {                           // (the first two write outputs in turn)
        if (lane == 0) mbar_arrive(&q_empty[qb]);
        group_sync(bar, 128);                          // the next segment's maxima go where these sums were read
        continue;
      }
      if (!wait_warp(&stat_full[qb], (seg / kQBufs) & 1, err, kErrMmaTimeout)) break;
      const bool whole = s.n == s.tiles;
      const int pairs = s.rows * a.group;
      // of a CTA's two cut segments, the one that it goes on with and the one that it begins
      const int slot = s.tile > 0 ? 2 * cta : 2 * cta + 1;
      if (quarter == 0 && lane < live) {
        // out = sum_w f_w O_w, f_w = 2^(mv_w - M) / (64 L), in an order that keeps V's extreme scales finite (see paged_attention.cu)
        float M = -INFINITY, L = 0.f;
        bool any = false;
#pragma unroll
        for (int w = 0; w < kWgs; ++w) M = fmaxf(M, stat[qb][w][0][lane]);
#pragma unroll
        for (int w = 0; w < kWgs; ++w) {
          const float lw = stat[qb][w][2][lane];
          const bool has = lw > 0.f || lw != lw;           // NaN counts as seen
          if (has) L += lw * ex2_approx(stat[qb][w][0][lane] - M);
          fin[wg][w][lane] = has ? ex2_approx(0.5f * (stat[qb][w][1][lane] - M)) : 0.f;
          any |= has;
        }
        stat[qb][0][2][lane] = 1.f / L / kPOne;        // (it has been read)
        if (whole) {
          if (a.lse) a.lse[cm.at[lane]] = any ? (M + __log2f(L)) * 0.69314718055994530942f : -INFINITY;
        } else {
          float* ml = a.part_ml + ((int64_t)slot * kPagedAttnColumns + lane) * 2;
          ml[0] = M;
          ml[1] = L;
        }
      }
      if (row == 0 && seg == 0)                        // for the join: this CTA's first piece
        reinterpret_cast<PaRecord*>(a.rec)[cta] = {units, s.tile, s.tiles, s.row0, pairs, s.cg * kCE, s.h};
      group_sync(bar, 128);
      if (!wait_warp(&o_full[seg % kOBufs], (seg / kOBufs) & 1, err, kErrMmaTimeout)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < live; c0 += 8) {
        uint32_t r[16 * kWgs];
#pragma unroll
        for (int w = 0; w < kWgs; ++w) {
          tmem_ld_cols8(acc + kN * w + c0, r + 16 * w);
          tmem_ld_cols8(acc + kN * w + kHalf + c0, r + 16 * w + 8);
        }
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c0 + c >= live) break;
          const float over = stat[qb][0][2][c0 + c];
          // an accumulator without a seen key holds nothing of this column (or was never written)
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kWgs; ++w) {
            const float f = fin[wg][w][c0 + c];
            if (f != 0.f) v = fmaf(fmaf(__uint_as_float(r[16 * w + 8 + c]), 0.0625f, __uint_as_float(r[16 * w + c])) * over * f, f, v);
          }
          if (whole) a.out[(int64_t)cm.at[c0 + c] * kKvDim + row] = __float2bfloat16_rn(v);
          else a.part_o[((int64_t)slot * kPagedAttnColumns + c0 + c) * kKvDim + row] = v;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&o_empty[seg % kOBufs]);
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

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {
template <int kCE>
cudaError_t launch_columns4(const PagedAttnArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map, int ctas, bool join, cudaStream_t s) {
  constexpr int smem = p4::Form<kCE>::kSmem;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = once_per_device(ready, [] {
    cudaError_t r = cudaFuncSetAttribute(kv4_attention_kernel<kCE, kPaPlain>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(kv4_attention_kernel<kCE, kPaCapBias>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(kv4_attention_kernel<kCE, kPaLargeCap>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return r;
  });
  if (e != cudaSuccess) return e;
  const int shared_keys = std::min<int64_t>((int64_t)a.max_rows * a.group, a.hi_pairs) > kCE ? 1 : 0;   // column groups share keys
  const PaMods mods = pa_mods(a);
  auto kernel = mods == kPaPlain     ? kv4_attention_kernel<kCE, kPaPlain>
                : mods == kPaCapBias ? kv4_attention_kernel<kCE, kPaCapBias>
                                     : kv4_attention_kernel<kCE, kPaLargeCap>;
  e = launch_pdl(kernel, dim3(ctas), dim3(p4::kThreads), smem, s, k_map, v_map, a, shared_keys);
  count_launches(1);
  if (e == cudaSuccess && ctas > 1 && !a.whole && join) e = launch_paged_join(a, ctas, kCE, s);
  return e;
}
}  // namespace

cudaError_t launch_kv4_attention(PagedAttnArgs a, const uint8_t* k_codes, const uint8_t* v_codes, int max_seq_len, void* workspace,
                                 const PagedAttnPlan& plan, cudaStream_t s) {
  const int ctas = device_sm_count();
  pa_layout(a, workspace, plan, ctas, max_seq_len);
  a.k_codes4 = k_codes;
  const uint64_t rows = (uint64_t)a.num_pages * a.kv_heads << a.log2_page;
  CUtensorMap k_map, v_map;
  if (!encode_2d(&k_map, k_codes, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 1, kKvDim, rows, kKvDim / 2, kKvDim, 1u << a.log2_page) ||
      !encode_2d(&v_map, v_codes, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 1, kKvDim, rows, kKvDim / 2, kKvDim, 1u << a.log2_page))
    return cudaErrorInvalidValue;
  const int64_t pairs = (int64_t)a.max_rows * a.group;
  cudaError_t e = pairs <= 8    ? launch_columns4<8>(a, k_map, v_map, ctas, !plan.prompt, s)
                  : pairs <= 16 ? launch_columns4<16>(a, k_map, v_map, ctas, !plan.prompt, s)
                                : launch_columns4<32>(a, k_map, v_map, ctas, !plan.prompt, s);
  if (e == cudaSuccess && plan.prompt)
    e = launch_kv4_prompt(pa_prompt_args(a, workspace, plan, ctas), a, kPagedAttnColumns / 8, k_map, v_codes, ctas, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dsa
