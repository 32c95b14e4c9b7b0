// Dense attention over the paged 8-bit K/V cache for requests of many rows (prompt pieces), on tcgen05 tensor
// cores.  Definition as in paged_attention.cu:
//   z_s = scale * q[r,h] . (k_code_s * ks),  out = softmax(z) (v_code * vs),  lse = ln sum exp(z)
//
// Here the products bound the call (4 * 128 flop per visible pair and head), so the tiles are square and the
// codes are widened once per tile for 256 (row, head) pairs:
//   S [128 pairs x 128 keys]  = Q [128 x 128] K^T     Q and K in fp16 from shared memory
//   O [128 pairs x 128 dims] += P [128 x 128] V       P in fp16 from TMEM, V in fp16 from shared memory
// fp16 holds e4m3 codes exactly, and bf16 queries too once a row is scaled by a power of two that brings its
// largest value below 2^15 (8 bits down to 2^-31 of it).  ks stays out of K: it multiplies the scores of its
// page, one fp32 factor per 16 keys.  vs goes into V relative to the largest of the request's pages, exactly
// for the powers of two that the append writes.  P carries 2^8 times the probability (11 bits of it, and
// an absolute step of 2^-33 of the row's largest), so that V's and P's ranges together fit fp16.
// e4m3 products with a two-term Q would take the same time (fp8 runs twice as fast) but keep only 2^-18
// of a row's largest value, as both terms would have to share one accumulator.
//
// Work: (request, 256 pairs, K/V head, tile of 128 keys) units split into one contiguous range per CTA
// (persistent, one CTA per SM), as in paged_attention.cu; a segment that is cut leaves fp32 pieces for a join.
// Segments count the tiles their last row sees, so causal rows are balanced over the CTAs.
//
// Per CTA (20 warps): warps 0-3 and 4-7 are the softmax of the two 128-pair halves, one pair a thread (no
// cross-lane work at all), which alternate with each other on the tensor cores; warps 8-15 load codes, widen
// them and write the K and V tiles; warp 16 issues the products; warps 17-19 load the next segment's queries.
// TMEM (all 512 columns): S of half q at 128 q, with P over its first 64 columns; O of half q at 256 + 128 q.
#include "paged_attention.cuh"
#include "sm100.cuh"

#include <cuda_fp16.h>

namespace dsa {
using namespace sm100;

namespace pp {
constexpr int kTok = kPaTok;
constexpr int kHalfPairs = 128;
constexpr int kTileBytes = kTok * kKvDim * 2;        // 32 KB of fp16: two 64-wide column chunks of 128-byte rows
constexpr int kChunkBytes = kTok * 128;
constexpr int kThreads = 640;
constexpr int kConvWarp0 = 8, kMmaWarp = 16, kQueryWarp0 = 17;
constexpr uint32_t kRegsSoft = 112, kRegsConv = 96, kRegsRest = 64;   // 2 * 112 + 2 * 96 + 64 = 480 = 5 * 96, the launch's
constexpr uint32_t kTmemCols = 512, kColO = 256;
constexpr float kSlack = 6.f;                        // log2 by which a row's maximum may be exceeded
constexpr float kPLog2 = 8.f;                        // P = 2^8 p
constexpr uint32_t kPolls = 1u << 22;
constexpr int kRuns = 512;                           // runs of (request, pairs) entries that are summed
constexpr int kMetaBufs = 4;
constexpr int kFixedSmem = 6 * kTileBytes + 1024;    // two halves of Q, two K tiles, two V tiles
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

__device__ __forceinline__ PpEntry pp_entry(const PagedAttnArgs& a, int b, int qt) {
  PpEntry e;
  uint32_t none = 0;
  e.b = b;
  e.qt = qt;
  e.shape = pa_shape(a, b, none);
  e.start = a.seq_lens[b] - e.shape.rows;
  e.prefix = a.prefix_lens ? min(a.prefix_lens[b], e.shape.len) : 0;
  const int last = min(e.shape.rows - 1, ((qt + 1) * kPromptPairs - 1) / a.group);
  e.tiles = max(1, (pp_limit(e, last) + pp::kTok - 1) / pp::kTok);
  return e;
}

// A run of tiles of one segment (entry and K/V head)
struct PpSeg {
  PpEntry e;
  int h, tile, n;
};

// Where a role stands: the entry and how many units before it
struct PpCursor {
  int b, qt;
  int64_t before;                  // units of the entries before this one
};

// The segment that unit u lies in, cut at u1; the cursor moves up to its entry.
__device__ __forceinline__ PpSeg pp_segment(const PagedAttnArgs& a, PpCursor& c, int64_t u, int64_t u1) {
  PpSeg s;
  for (;;) {
    uint32_t none = 0;
    const PaShape sh = pa_shape(a, c.b, none);
    if (c.qt >= pp_entries(a, sh)) {
      ++c.b;
      c.qt = 0;
      continue;
    }
    s.e = pp_entry(a, c.b, c.qt);
    const int64_t units = (int64_t)s.e.tiles * a.kv_heads;
    if (u < c.before + units) break;
    c.before += units;
    ++c.qt;
  }
  const int in = (int)(u - c.before);
  s.h = in / s.e.tiles;
  s.tile = in - s.h * s.e.tiles;
  s.n = (int)min((int64_t)(s.e.tiles - s.tile), u1 - u);
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

// eight columns, as tmem_st16
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// A softmax thread's row: its reference m (log2 units), its sum l of P, and what masks and biases need.
struct PpRow {
  float m, l, cf, slope;
  int limit, pos;
};

// A row's reference moves from m to m + something: what was summed and stored against the old one shrinks by al.
// done: 16-key groups of this tile whose P is in TMEM already.
__device__ __forceinline__ void pp_shrink(uint32_t tS, uint32_t tO, int done, bool has_o, float al) {
  const __half2 h = __float2half2_rn(al);
#pragma unroll 1
  for (int g = 0; g < done; ++g) {
    uint32_t p[8];
    tmem_ld8(tS + 8 * g, p);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = mul2(p[k], h);
    tmem_st8(tS + 8 * g, p);
  }
  if (has_o) {
#pragma unroll 1
    for (int c = 0; c < kKvDim; c += 8) {
      uint32_t o[8];
      tmem_ld8(tO + c, o);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
      tmem_st8(tO + c, o);
    }
  }
  tmem_wait_st();
}

// One tile of a row, in one pass over its scores: 16 keys at a time the scores come out of TMEM, their largest
// is held against the reference (which moves only when exceeded by 2^kSlack, seldom after the first
// keys), and P goes back over scores that have been read.  Holding all 128 scores for an exact maximum
// first took 176 registers, and reading them twice 15 % more time.
template <bool kMods, bool kMasked>
__device__ __forceinline__ void pp_tile(PpRow& w, const PagedAttnArgs& a, uint32_t tS, uint32_t tO, int key0, uint32_t bad,
                                        const float* ks, bool has_o) {
  const float in = kMods && a.cap_log2 > 0.f ? 2.f * 1.4426950408889634f / a.cap_log2 : 0.f;
  uint64_t sum = 0;
  uint32_t r[2][16];
  float shift = pp::kPLog2 - (w.m == -INFINITY ? 0.f : w.m);
  tmem_ld16(tS, r[0]);
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    tmem_wait_ld();
    if (g < 7) tmem_ld16(tS + 16 * (g + 1), r[(g + 1) & 1]);
    uint32_t* x = r[g & 1];
    float kc = ks[g] * w.cf;
    if (kMods) {
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        float z = __uint_as_float(x[c]) * kc;
        if (in != 0.f) {
          const float y = z * in;
          z = a.cap_log2 * (1.f - __fdividef(2.f, 1.f + ex2_approx(y > 64.f ? 64.f : y)));   // NaN stays
        }
        x[c] = __float_as_uint(z - w.slope * (float)abs(w.pos - (key0 + 16 * g + c)));
      }
      kc = 1.f;
    }
    if (kMasked) {
      // a masked score is -inf whatever the factor (which may be 0): they are scaled first
      const int left = ((bad >> g) & 1u) ? 0 : w.limit - key0 - 16 * g;   // keys of the group that are seen
#pragma unroll
      for (int c = 0; c < 16; ++c) x[c] = c < left ? __float_as_uint(__uint_as_float(x[c]) * kc) : 0xFF800000u;
      kc = 1.f;
    }
    float top = __uint_as_float(x[0]);
#pragma unroll
    for (int c = 1; c < 16; ++c) top = fmaxf(top, __uint_as_float(x[c]));
    top *= kc;
    const bool grow = top > w.m + pp::kSlack || (w.m == -INFINITY && top > w.m);
    if (__any_sync(0xffffffffu, grow)) {
      const float m_new = grow ? top : w.m;
      const float al = m_new == w.m ? 1.f : w.m == -INFINITY ? 0.f : ex2_approx(w.m - m_new);
      pp_shrink(tS, tO, g, has_o, al);
      w.l *= al;
      sum = fma2(sum, pack2(al, al), 0);
      w.m = m_new;
      shift = pp::kPLog2 - (m_new == -INFINITY ? 0.f : m_new);
    }
    const uint64_t kc2 = pack2(kc, kc), shift2 = pack2(shift, shift);
    uint32_t p[8];
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      float y0, y1;
      unpack2(fma2(pack2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), kc2, shift2), y0, y1);
      y0 = ex2_approx(y0);
      y1 = ex2_approx(y1);
      sum = add2(sum, pack2(y0, y1));
      const __half2 h = __floats2half2_rn(y0, y1);
      p[c >> 1] = *reinterpret_cast<const uint32_t*>(&h);
    }
    // columns 8 g .. 8 g + 7 hold scores that have been read
    tmem_st8(tS + 8 * g, p);
  }
  float s0, s1;
  unpack2(sum, s0, s1);
  w.l += s0 + s1;
  tmem_wait_st();
}

template <bool kMods>
__global__ void __launch_bounds__(pp::kThreads, 1)
    paged_prompt_kernel(const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ v_codes,
                        const __grid_constant__ PagedAttnArgs a) {
  using namespace pp;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * kTileBytes;
  uint8_t* sV = sK + 2 * kTileBytes;
  int32_t* entry_end = reinterpret_cast<int32_t*>(sV + 2 * kTileBytes);   // [requests] entries of requests 0 .. b

  __shared__ uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], o_empty[2];
  __shared__ uint64_t q_full, q_empty, mma_done;
  __shared__ __align__(16) float sks[kMetaBufs][8];   // K scale of each 16 keys of a tile
  __shared__ uint32_t sbad[kMetaBufs];                // 16-key groups without a valid page
  __shared__ float factor[2][kPromptPairs];
  __shared__ int nan_key[kMetaBufs][kKvDim];          // first key with a NaN code that only some rows see, by dim
  __shared__ int32_t run_units[kRuns];                // units (without heads) of the runs before
  __shared__ int32_t scan[kThreads / 32];
  __shared__ float vmax_part[4], v_ref[kMetaBufs];    // V's reference of a segment
  __shared__ int seg_tiles[kMetaBufs];
  __shared__ uint32_t tmem_base, bits_all;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 2);                        // the products, and their issuer
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 2);
      mbar_init(&o_empty[i], 4);
    }
    mbar_init(&q_full, 3);
    mbar_init(&q_empty, 1);
    mbar_init(&mma_done, 1);
    bits_all = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_base, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  const int B = a.num_requests;
  // block-wide inclusive sum of one value a thread
  auto block_sum = [&](int v) {
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += scan[w];
    return before + incl;
  };
  {
    uint32_t bits = 0;
    const int per = (B + kThreads - 1) / kThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      sum += pp_entries(a, pa_shape(a, b, bits));
      entry_end[b] = sum;
    }
    const int before = block_sum(sum) - sum;
    for (int b = b0; b < b1; ++b) entry_end[b] += before;
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
        while (c.qt >= pp_entries(a, pa_shape(a, c.b, none))) {
          ++c.b;
          c.qt = 0;
        }
        sum += pp_entry(a, c.b, c.qt).tiles;
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
  // every role starts at the run that holds u0
  PpCursor cur = {0, 0, 0};
  if (u0 < u1) {
    int lo = 0, hi = kRuns - 1;                       // the last run whose units begin at or before u0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)run_units[mid] * a.kv_heads <= u0) lo = mid;
      else hi = mid - 1;
    }
    cur.before = (int64_t)run_units[lo] * a.kv_heads;
    find(min(lo * run, entries - 1), cur);
  }

  if (warp < kConvWarp0) {
    regs_inc<kRegsSoft>();
    // ---------------------------------------------------------------- softmax and outputs: one pair a thread
    const int q = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t tS = tmem + lanes + 128 * q, tO = tmem + lanes + kColO + 128 * q;
    int i = 0, seg = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok; ++seg) {
      const PpSeg s = pp_segment(a, cur, u, u1);
      const int64_t u_first = u;
      u += s.n;
      const int pairs = s.e.shape.rows * a.group;
      const int n = s.e.qt * kPromptPairs + kHalfPairs * q + row;     // this thread's pair
      const int r = min(n, pairs - 1) / a.group, head = s.h * a.group + (min(n, pairs - 1) - r * a.group);
      const int limit = pp_limit(s.e, r), pos = s.e.start + r;
      // keys below it are seen by every pair of this half
      const int min_limit = pp_limit(s.e, min(s.e.qt * kPromptPairs + kHalfPairs * q, pairs - 1) / a.group);
      const float slope = kMods && a.slopes ? a.slopes[head] * 1.4426950408889634f : 0.f;
      PpRow w = {-INFINITY, 0.f, 0.f, slope, limit, pos};
      for (int t = 0; t < s.n; ++t, ++i) {
        const int key0 = (s.tile + t) * kTok;
        // The scores' arrival also stands for the tile's scales and the queries' factors: their own barriers may be
        // a phase further by the time this warpgroup looks.
        ok = mbar_wait(&s_full[q], i & 1, err, kErrMmaTimeout, kPolls);
        if (!ok) break;
        tc_fence_after();
        if (t == 0) w.cf = factor[seg & 1][kHalfPairs * q + row];
        const float* ks = sks[i % kMetaBufs];
        const uint32_t bad = sbad[i % kMetaBufs];
        if (key0 + kTok > min_limit || bad) pp_tile<kMods, true>(w, a, tS, tO, key0, bad, ks, t > 0);
        else pp_tile<kMods, false>(w, a, tS, tO, key0, bad, ks, t > 0);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[q]);
      }
      if (!ok) break;
      // ---- the segment's end
      const bool whole = s.n == s.e.tiles;
      const int slot = u_first == u0 ? 2 * cta : 2 * cta + 1;
      ok = mbar_wait(&o_full[q], seg & 1, err, kErrMmaTimeout, kPolls);
      if (!ok) break;
      tc_fence_after();
      const float m = w.m, l = w.l;
      const bool any = l > 0.f || l != l;
      const int64_t at = (int64_t)(s.e.shape.row0 + r) * a.kv_heads * a.group + head;
      const float vref = v_ref[seg % kMetaBufs];
      const float f = !any ? 0.f : whole ? vref / l : vref;
      const int* nk = nan_key[seg % kMetaBufs];
#pragma unroll 1
      for (int c = 0; c < kKvDim; c += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c, o);
        tmem_wait_ld();
        if (n < pairs) {
          float x[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            x[k] = any ? __uint_as_float(o[k]) * f : 0.f;
            if (nk[c + k] < limit) x[k] = __int_as_float(0x7FC00000);
          }
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + at * kKvDim + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint4 w;
              uint32_t* ww = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
              for (int k2 = 0; k2 < 4; ++k2) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[8 * k + 2 * k2], x[8 * k + 2 * k2 + 1]);
                ww[k2] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              dst[k] = w;
            }
          } else {
            // [slot][dim / 4][pair] float4: a warp's stores are contiguous
            float4* dst = reinterpret_cast<float4*>(a.part_o) + ((int64_t)slot * (kKvDim / 4) + c / 4) * kPromptPairs + kHalfPairs * q + row;
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[k * kPromptPairs] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          }
        }
      }
      if (n < pairs) {
        if (!whole) {
          reinterpret_cast<float2*>(a.part_ml)[(int64_t)slot * kPromptPairs + kHalfPairs * q + row] = make_float2(m, l);
        } else if (a.lse) {
          a.lse[at] = any ? (m - kPLog2 + __log2f(l)) * 0.69314718055994530942f : -INFINITY;
        }
      }
      if (tid == 0 && u_first == u0) {                 // for the join: this CTA's first piece
        int32_t* rec = a.rec + 8 * cta;
        rec[0] = s.e.b;
        rec[1] = s.h;
        rec[2] = s.e.qt;
        rec[3] = s.tile;
        rec[4] = s.e.tiles;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[q]);
    }
  } else if (warp < kMmaWarp) {
    regs_dec<kRegsConv>();
    // ---------------------------------------------------------------- K and V tiles: codes to fp16
    // Four warps for K and four for V: eight lanes a row of 16-byte pieces, 16 rows a pass, so that a pass is one
    // 16-key group and lies in one page.  A tile's loads go out right after the last tile's fence, which
    // waits for the loads in flight too: one warp doing both K and V with its loads ahead took 7,000 cycles
    // a tile, most of them in fences, against the 2,000 of the products.
    const bool is_v = warp >= kConvWarp0 + 4;
    const int cw = (warp - kConvWarp0) & 3, part = lane & 7, sub = 4 * cw + (lane >> 3), lp = a.log2_page;
    const int unit = 2 * (part & 3), swap = part >> 2;
    uint64_t* const full = is_v ? v_full : k_full;
    uint64_t* const empty = is_v ? v_empty : k_empty;
    const float* const scales = is_v ? a.v_scales : a.k_scales;
    uint8_t* const tiles = (is_v ? sV : sK) + (part >> 2) * kChunkBytes;
    int i = 0, seg = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok; ++seg) {
      const PpSeg s = pp_segment(a, cur, u, u1);
      u += s.n;
      const int len = s.e.shape.len, pages = (len + (1 << lp) - 1) >> lp;
      const int32_t* table = a.block_table + (int64_t)s.e.b * a.table_stride;
      // this lane's 16 bytes of row 0 of page 0; a page further is page_step bytes on
      const uint8_t* const base = (is_v ? v_codes : k_codes) + ((int64_t)s.h << lp) * kKvDim + 16 * part;
      const int64_t page_step = ((int64_t)a.kv_heads << lp) * kKvDim;
      constexpr int kNoPage = INT32_MIN;               // past the request's pages
      auto id_of = [&](int key) {
        const int p = key >> lp;
        return p < pages ? table[p] : kNoPage;
      };
      auto checked = [&](int id) {
        if (id >= 0 && id < a.num_pages) return id;
        if (id != kNoPage) atomicOr(err, kErrBadPage);
        return -1;
      };
      // V's reference: the power of two at or below the piece's largest scale
      float vinv = 1.f;
      if (is_v) {
        float top = 0.f;
        const int p0 = (s.tile * kTok) >> lp, p1 = min(pages, ((s.tile + s.n) * kTok) >> lp);
#pragma unroll 4
        for (int p = p0 + 32 * cw + lane; p < p1; p += 128) {
          const int id = table[p];
          if (id >= 0 && id < a.num_pages) top = fmaxf(top, fabsf(scales[(int64_t)id * a.kv_heads + s.h]));
        }
        top = warp_max_f32(top);
        if (lane == 0) vmax_part[cw] = top;
        nan_key[seg % kMetaBufs][32 * cw + lane] = INT32_MAX;
        named_bar_sync(1, 128);
        top = fmaxf(fmaxf(vmax_part[0], vmax_part[1]), fmaxf(vmax_part[2], vmax_part[3]));
        const uint32_t top_bits = __float_as_uint(top) & 0x7F800000u;
        const float vref = top_bits && top_bits < 0x7F800000u ? __uint_as_float(top_bits) : 1.f;
        if (cw == 0 && lane == 0) v_ref[seg % kMetaBufs] = vref;
        vinv = 1.f / vref;
        named_bar_sync(1, 128);
      }
      const int min_limit = pp_limit(s.e, min(s.e.qt * kPromptPairs, s.e.shape.rows * a.group - 1) / a.group);

      uint4 x[8];
      float scale = 0.f;
      // lane g (and g + 8, ..): the page of 16-key group g, of this tile and (not checked yet) of the next one
      int id = checked(id_of(s.tile * kTok + 16 * part)), id2 = id_of((s.tile + 1) * kTok + 16 * part);
      auto load = [&](int key0) {
        scale = id >= 0 ? scales[(int64_t)id * a.kv_heads + s.h] : 0.f;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const int page = __shfl_sync(0xffffffffu, id, g), key = key0 + 16 * g + sub;
          x[g] = make_uint4(0, 0, 0, 0);
          if (page >= 0 && key < len)
            x[g] = __ldg(reinterpret_cast<const uint4*>(base + page * page_step + (key & ((1 << lp) - 1)) * kKvDim));
        }
      };
      load(s.tile * kTok);
      for (int t = 0; t < s.n; ++t, ++i) {
        const int key0 = (s.tile + t) * kTok, buf = i & 1;
        if (i >= 2) ok = mbar_wait(&empty[buf], ((i >> 1) - 1) & 1, err, kErrMmaTimeout, kPolls);
        if (!ok) break;
        // a NaN code of a key that only some rows see: out of the tile, and noted for the rows that see it
        if (is_v && key0 + kTok > min_limit) {
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&x[g]);
            uint32_t any = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) any |= ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            if (any) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t f = ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                for (int k = 0; k < 4; ++k)
                  if ((f >> (8 * k + 7)) & 1u) atomicMin(&nan_key[seg % kMetaBufs][16 * part + 4 * e + k], key0 + 16 * g + sub);
                w[e] &= ~((f >> 7) * 0xFFu);
              }
            }
          }
        }
        uint8_t* tile = tiles + buf * kTileBytes;
        const float ratio = scale * vinv;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const int r = 16 * g + sub;
          uint4 lo = widen8(x[g].x, x[g].y), hi = widen8(x[g].z, x[g].w);
          if (is_v) {
            const __half2 f = __float2half2_rn(__shfl_sync(0xffffffffu, ratio, g));
            lo = make_uint4(mul2(lo.x, f), mul2(lo.y, f), mul2(lo.z, f), mul2(lo.w, f));
            hi = make_uint4(mul2(hi.x, f), mul2(hi.y, f), mul2(hi.z, f), mul2(hi.w, f));
          }
          // lanes of the two column chunks start with different units, so that eight lanes fill all banks
          *reinterpret_cast<uint4*>(tile + r * 128 + (((unit + swap) ^ (r & 7)) << 4)) = swap ? hi : lo;
          *reinterpret_cast<uint4*>(tile + r * 128 + (((unit + 1 - swap) ^ (r & 7)) << 4)) = swap ? lo : hi;
        }
        if (!is_v && cw == 0) {
          if (lane < 8) sks[i % kMetaBufs][lane] = scale;
          const uint32_t bad = __ballot_sync(0xffffffffu, lane < 8 && id < 0);
          if (lane == 0) sbad[i % kMetaBufs] = bad;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[buf]);
        if (t + 1 < s.n) {
          id = checked(id2);
          id2 = id_of(key0 + 2 * kTok + 16 * part);
          load(key0 + kTok);
        }
      }
    }
  } else {
    regs_dec<kRegsRest>();
    if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- products
      // Order: .. O0(i) S0(i+1) O1(i) S1(i+1) ..: while one half's softmax runs, the tensor cores work for the other.
      // S0(i+1) overwrites P0(i), which O0(i) has read (products issue and complete in order).
      const bool leader = elect_one();
      const uint32_t id_s = idesc_f16(128, kTok, false, false, false, false);
      const uint32_t id_o = idesc_f16(128, kKvDim, false, false, false, true);
      const uint64_t d_q = smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
      const uint64_t d_k = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
      const uint64_t d_v = smem_desc(smem_u32(sV), kChunkBytes, 1024, kSwizzle128B);
      const int n_tiles = (int)(u1 - u0);
      int s_left = 0, o_left = 0, s_seg = -1, o_seg = -1;
      bool ok = true, o_first = false;
      for (int i = -1; i < n_tiles && ok; ++i) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (i >= 0) {
            if (q == 0) {
              if (o_left == 0) {
                ++o_seg;
                o_left = seg_tiles[o_seg % kMetaBufs];
                o_first = true;
              }
              --o_left;
              ok = ok && mbar_spin(&v_full[i & 1], (i >> 1) & 1, err, kErrMmaTimeout);
            }
            if (o_first && o_seg > 0) ok = ok && mbar_spin(&o_empty[q], (o_seg - 1) & 1, err, kErrMmaTimeout);
            ok = ok && mbar_spin(&p_full[q], i & 1, err, kErrMmaTimeout);
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = d_v + (uint64_t)(((i & 1) * kTileBytes) >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kTok / 16; ++kk)
                mma_ts(tmem + kColO + 128 * q, tmem + 128 * q + 8 * kk, v + (uint64_t)((kk * 16 * 128) >> 4), id_o, !o_first || kk > 0);
              if (q == 1) mma_commit(&v_empty[i & 1]);
              if (o_left == 0) {
                mma_commit(&o_full[q]);
                mbar_arrive(&o_full[q]);
              }
            }
            __syncwarp();
            if (q == 1) o_first = false;
          }
          if (i + 1 < n_tiles) {
            const int j = i + 1;
            if (q == 0) {
              if (s_left == 0) {
                ++s_seg;
                ok = ok && mbar_wait(&q_full, s_seg & 1, err, kErrMmaTimeout, kPolls);
                s_left = seg_tiles[s_seg % kMetaBufs];
              }
              --s_left;
              ok = ok && mbar_spin(&k_full[j & 1], (j >> 1) & 1, err, kErrMmaTimeout);
            }
            if (!ok) break;
            tc_fence_after();
            const uint64_t qd = d_q + (uint64_t)((q * kTileBytes) >> 4), k = d_k + (uint64_t)(((j & 1) * kTileBytes) >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kKvDim / 16; ++kk) {
                const uint64_t off = (uint64_t)(((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4);
                mma_ss(tmem + 128 * q, qd + off, k + off, id_s, kk > 0);
              }
              mma_commit(&s_full[q]);
              mbar_arrive(&s_full[q]);
              if (q == 1) {
                mma_commit(&k_empty[j & 1]);
                if (s_left == 0) mma_commit(&q_empty);
              }
            }
            __syncwarp();
          }
        }
      }
      if (leader) mma_commit(&mma_done);
      mbar_wait(&mma_done, 0, err, kErrMmaTimeout, kPolls);
    } else {
      // ---------------------------------------------------------------- queries: 16 lanes a row
      const int slot = 2 * (warp - kQueryWarp0) + (lane >> 4), part = lane & 15;
      int seg = 0;
      for (int64_t u = u0; u < u1; ++seg) {
        const PpSeg s = pp_segment(a, cur, u, u1);
        u += s.n;
        if (seg > 0 && !mbar_wait(&q_empty, (seg - 1) & 1, err, kErrMmaTimeout, kPolls)) break;
        const int pairs = s.e.shape.rows * a.group;
        if (warp == kQueryWarp0 && lane == 0) seg_tiles[seg % kMetaBufs] = s.n;
#pragma unroll 1
        for (int r0 = 0; r0 < kPromptPairs; r0 += 24) {
          uint4 x[4];
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int r = r0 + 6 * it + slot, n = s.e.qt * kPromptPairs + r;
            x[it] = make_uint4(0, 0, 0, 0);
            if (r < kPromptPairs && n < pairs) {
              const int i = n / a.group, g = n - i * a.group;
              x[it] = *reinterpret_cast<const uint4*>(a.q + (int64_t)(s.e.shape.row0 + i) * a.q_stride + (s.h * a.group + g) * kKvDim + 8 * part);
            }
          }
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int r = r0 + 6 * it + slot;
            uint32_t* w = reinterpret_cast<uint32_t*>(&x[it]);
            uint32_t top = 0;                          // largest finite |x|, as bf16 bits
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t p = w[e] & 0x7FFFu, y = (w[e] >> 16) & 0x7FFFu;
              if (p < 0x7F80u) top = max(top, p);
              if (y < 0x7F80u) top = max(top, y);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            // the largest goes to [2^14, 2^15): x * 2^(14 - E), E its exponent (held at -100: smaller rows score 0)
            const int E = max((int)(top >> 7) - 127, -100);
            const float up = __uint_as_float((uint32_t)(14 - E + 127) << 23);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // an infinity becomes NaN, as its product with a key's zeros or mixed signs is
              const uint32_t wl = w[e] << 16, wh = w[e] & 0xFFFF0000u;
              const float xl = (wl & 0x7F800000u) == 0x7F800000u ? __int_as_float(0x7FC00000) : __uint_as_float(wl) * up;
              const float xh = (wh & 0x7F800000u) == 0x7F800000u ? __int_as_float(0x7FC00000) : __uint_as_float(wh) * up;
              const __half2 h = __floats2half2_rn(xl, xh);
              w[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            if (r < kPromptPairs) {
              const int rr = r & (kHalfPairs - 1);
              *reinterpret_cast<uint4*>(sQ + (r >> 7) * kTileBytes + (part >> 3) * kChunkBytes + rr * 128 + (((part & 7) ^ (rr & 7)) << 4)) = x[it];
              if (part == 0) factor[seg & 1][r] = __uint_as_float((uint32_t)(E - 14 + 127) << 23) * a.scale_log2;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0) {
    a.err[kStatusCtaWords + cta] |= bits_all;          // beside what the first kernel reported
    if (cta == 0) *reinterpret_cast<int64_t*>(a.err + 4) = units;
  }
}

// Joins the pieces of the segments that CTA boundaries cut, as paged_attention_join_kernel: a thread a pair, 16 dims
// of it per blockIdx.y.
__global__ void __launch_bounds__(kPromptPairs) paged_prompt_join_kernel(const __grid_constant__ PagedAttnArgs a, int ctas) {
  pdl_wait();
  pdl_trigger();
  const int64_t units = *reinterpret_cast<const int64_t*>(a.err + 4);
  const int c = blockIdx.x + 1;
  const int64_t u = pa_unit_start(c, units, ctas);
  if (u == pa_unit_start(c + 1, units, ctas)) return;     // a range without units
  const int32_t* rec = a.rec + 8 * c;
  const int b = __ldcg(rec), h = __ldcg(rec + 1), qt = __ldcg(rec + 2), tile = __ldcg(rec + 3), tiles = __ldcg(rec + 4);
  if (tile == 0) return;                                   // the range begins with a segment
  const int64_t seg = u - tile;
  const int first = pa_cta_of_unit(u - 1, units, ctas);
  if (pa_unit_start(first, units, ctas) > seg) return;     // an earlier boundary cuts it, too
  uint32_t none = 0;
  const PaShape s = pa_shape(a, b, none);
  const int n = qt * kPromptPairs + threadIdx.x;
  if (n >= s.rows * a.group) return;
  const int last = pa_cta_of_unit(seg + tiles - 1, units, ctas);
  const int first_slot = pa_unit_start(first, units, ctas) == seg ? 2 * first : 2 * first + 1;
  float M = -INFINITY, L = 0.f;
  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int p = first; p <= last; ++p) {
    if (pa_unit_start(p, units, ctas) == pa_unit_start(p + 1, units, ctas)) continue;
    const int64_t slot = p == first ? first_slot : 2 * p;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot * kPromptPairs + threadIdx.x);
    if (ml.y == 0.f) continue;                             // a piece that sees nothing (NaN counts as seen)
    float4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (slot * (kKvDim / 4) + 4 * blockIdx.y + k) * kPromptPairs + threadIdx.x);
    const float Mn = fmaxf(M, ml.x);
    const float sc = M == -INFINITY ? 0.f : exp2f(M - Mn), w = exp2f(ml.x - Mn);
    L = L * sc + w * ml.y;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      acc[4 * k] = fmaf(w, x[k].x, acc[4 * k] * sc);
      acc[4 * k + 1] = fmaf(w, x[k].y, acc[4 * k + 1] * sc);
      acc[4 * k + 2] = fmaf(w, x[k].z, acc[4 * k + 2] * sc);
      acc[4 * k + 3] = fmaf(w, x[k].w, acc[4 * k + 3] * sc);
    }
    M = Mn;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int i = n / a.group;
  const int64_t at = (int64_t)(s.row0 + i) * a.kv_heads * a.group + h * a.group + (n - i * a.group);
  uint4 v[2];
  __nv_bfloat162* xo = reinterpret_cast<__nv_bfloat162*>(v);
#pragma unroll
  for (int e = 0; e < 8; ++e) xo[e] = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  uint4* dst = reinterpret_cast<uint4*>(a.out + at * kKvDim) + 2 * blockIdx.y;
  dst[0] = v[0];
  dst[1] = v[1];
  if (a.lse && blockIdx.y == 0) a.lse[at] = L == 0.f ? -INFINITY : (M - pp::kPLog2 + log2f(L)) * 0.69314718055994530942f;
}

cudaError_t launch_paged_prompt(const PagedAttnArgs& a, const uint8_t* k_codes, const uint8_t* v_codes, int ctas,
                                cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = once_per_device(ready, [] {
    const int most = pp::kFixedSmem + DSA_MAX_REQUESTS * (int)sizeof(int32_t);
    cudaError_t r = cudaFuncSetAttribute(paged_prompt_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(paged_prompt_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return r;
  });
  if (e != cudaSuccess) return e;
  const size_t smem = pp::kFixedSmem + (size_t)a.num_requests * sizeof(int32_t);
  e = launch_pdl(a.cap_log2 > 0.f || a.slopes ? paged_prompt_kernel<true> : paged_prompt_kernel<false>, dim3(ctas),
                 dim3(pp::kThreads), smem, s, k_codes, v_codes, a);
  count_launches(1);
  if (e != cudaSuccess) return e;
  if (ctas > 1) {
    e = launch_pdl(paged_prompt_join_kernel, dim3(ctas - 1, kKvDim / 16), dim3(kPromptPairs), 0, s, a, ctas);
    count_launches(1);
  }
  return e;
}

}  // namespace dsa
