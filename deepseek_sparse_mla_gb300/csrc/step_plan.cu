// Block tables and slot maps of one step, built on the device from the requests' lengths.
//
// Request b holds L_b tokens and brings n_b new ones; pages hold P tokens.
//   need_b = ceil((L_b + n_b) / P) - ceil(L_b / P)          new pages
//   off_b  = need_0 + .. + need_{b-1}                       their places on the stack of free pages
//   new page i of request b = free[count - 1 - off_b - i]
//   row r of request b at position p = L_b + i              slot = table[b][p / P] * P + p % P
// The requests admitted are the longest prefix whose rows fit into num_rows and whose pages the stack
// holds; the others keep their length and get no rows.  Both running sums grow with b, so the prefix is
// where the two limits still hold, and no request depends on another's outcome.
//
// What bounds it: latency (a few KB of lengths in, 12 bytes a row out), so it is one launch.  The sums
// over the requests are one block scan that every CTA repeats for itself (8 bytes a request out of L2);
// the rows and the new table entries are shared out over the CTAs of one cluster, each of which finds a row's
// request by binary search in shared memory.  One cluster rather than a grid: seq_lens_out may be
// seq_lens and free_count_out may be free_count, so every CTA must have read them before any writes,
// which a cluster barrier orders inside the launch.
#include "dsa_internal.cuh"
#include "sm100.cuh"

namespace dsa {

namespace {
constexpr int kPlanThreads = 1024;
constexpr int kPlanClusterMax = 16;      // more than 8 where the device says that such a cluster fits

// Inclusive sums of (x, y) over the block's threads; every thread passes its own values.
__device__ __forceinline__ void block_scan2(int64_t& x, int64_t& y, int64_t (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    part[warp][0] = x;
    part[warp][1] = y;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t a = part[lane][0], b = part[lane][1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, a, o), v = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) {
        a += u;
        b += v;
      }
    }
    part[lane][0] = a;
    part[lane][1] = b;
  }
  __syncthreads();
  if (warp > 0) {
    x += part[warp - 1][0];
    y += part[warp - 1][1];
  }
}

// The first b with ends[b] > r (ends ascends; the caller knows there is one).
__device__ __forceinline__ int request_of(const int32_t* ends, int n, int r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > r) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The same from a b whose predecessors are known to end at or before r: neighbouring rows are mostly few requests on,
// so the range is doubled until it holds the answer.
__device__ __forceinline__ int request_from(const int32_t* ends, int n, int b, int r) {
  int lo = b, step = 1;
  while (lo + step - 1 < n - 1 && ends[lo + step - 1] <= r) {
    lo += step;
    step *= 2;
  }
  int hi = min(lo + step - 1, n - 1);
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > r) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) step_plan_kernel(const StepPlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  const int B = a.num_requests;
  int32_t* old_len = plan_smem;           // [B] tokens held
  int32_t* row_end = plan_smem + B;       // [B] admitted rows of requests 0 .. b
  int32_t* page_end = plan_smem + 2 * B;  // [B] admitted new pages of requests 0 .. b
  __shared__ int64_t part[32][2];
  __shared__ uint32_t total_rows, total_pages;         // at most num_rows, and the count of free pages
  __shared__ uint32_t bits;
  const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x;
  if (tid == 0) {
    total_rows = total_pages = 0;
    bits = 0;
  }
  pdl_wait();
  pdl_trigger();
  const int P = 1 << a.log2_page;
  const int64_t count = min(max(*a.free_count, 0), a.free_capacity);
  // each request's new rows and pages: none where its lengths do not make sense or its table row is too short
  uint32_t my_bits = 0;
  constexpr int kEach = kPlanMaxRequests / kPlanThreads;
  int tokens[kEach], brings[kEach];                     // every load in flight before the first is used
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int b = tid + k * kPlanThreads;
    tokens[k] = b < B ? a.seq_lens[b] : 0;
    brings[k] = b < B ? a.new_lens[b] : 0;
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int b = tid + k * kPlanThreads;
    if (b >= B) break;
    const int64_t L = tokens[k];
    int64_t n = brings[k], need = 0;
    const int64_t pages = (L + n + P - 1) >> a.log2_page;
    if (L < 0 || n < 0 || L + n > INT32_MAX || (n > 0 && pages > a.table_stride)) {
      my_bits |= DSA_DEVICE_BAD_LENGTH;
      n = 0;
    } else {
      need = pages - ((L + P - 1) >> a.log2_page);
    }
    old_len[b] = (int32_t)L;
    row_end[b] = (int32_t)n;
    page_end[b] = (int32_t)need;
  }
  __syncthreads();
  // every thread sums a run of consecutive requests, then the runs are scanned
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int64_t rows = 0, pages = 0;
  for (int b = b0; b < b1; ++b) {
    rows += row_end[b];
    pages += page_end[b];
  }
  int64_t row_first = rows, page_first = pages;
  block_scan2(row_first, page_first, part);
  row_first -= rows;
  page_first -= pages;
  int64_t row_sum = row_first, page_sum = page_first, row_top = 0, page_top = 0;
  for (int b = b0; b < b1; ++b) {
    row_sum += row_end[b];
    page_sum += page_end[b];
    if (row_sum <= a.num_rows && page_sum <= count) {
      row_top = row_sum;
      page_top = page_sum;
    } else if (row_end[b] > 0) {
      my_bits |= row_sum > a.num_rows ? DSA_DEVICE_ROWS_FULL : DSA_DEVICE_POOL_EMPTY;
    }
  }
  // one atomic a warp: 1,024 of 64 bits took 8,900 cycles
  const uint32_t warp_rows = __reduce_max_sync(0xffffffffu, (uint32_t)row_top), warp_pages = __reduce_max_sync(0xffffffffu, (uint32_t)page_top);
  my_bits = __reduce_or_sync(0xffffffffu, my_bits);
  if ((tid & 31) == 0) {
    atomicMax(&total_rows, warp_rows);
    atomicMax(&total_pages, warp_pages);
    if (my_bits) atomicOr(&bits, my_bits);
  }
  __syncthreads();
  const int64_t R = total_rows, N = total_pages;
  // beyond the last admitted request the sums stay at their totals (they only grow from there)
  row_sum = row_first;
  page_sum = page_first;
  for (int b = b0; b < b1; ++b) {
    row_sum += row_end[b];
    page_sum += page_end[b];
    row_end[b] = (int32_t)min(row_sum, R);
    page_end[b] = (int32_t)min(page_sum, N);
  }
  __syncthreads();
  // from here on memory that may be an input's is written
  if (ctas > 1) sm100::cluster_sync();
  if (rank == 0) {
    for (int b = tid; b < B; b += kPlanThreads) {
      const int first = b ? row_end[b - 1] : 0;
      a.seq_lens_out[b] = old_len[b] + (row_end[b] - first);
      a.query_start_loc[b + 1] = row_end[b];
    }
    if (tid == 0) {
      a.query_start_loc[0] = 0;
      *a.free_count_out = (int32_t)(count - N);
      if (a.status) {
        a.status[0] = bits;
        a.status[1] = 0;
      }
    }
  }
  const int stride = ctas * kPlanThreads;
  for (int64_t k = rank * kPlanThreads + tid; k < N; k += stride) {
    const int b = request_of(page_end, B, (int)k);
    const int first = b ? page_end[b - 1] : 0;
    const int held = (int)(((int64_t)old_len[b] + P - 1) >> a.log2_page);
    a.block_table[(int64_t)b * a.table_stride + held + ((int)k - first)] = a.free_pages[count - 1 - k];
  }
  // Each warp takes a run of consecutive rows, 128 at a time (four a lane, their page ids in flight together): the
  // requests of the first and the last bound the others', which are searched for side by side.
  const int warps = ctas * (kPlanThreads / 32), lane = tid & 31;
  const int64_t run = ((a.num_rows + warps - 1) / warps + 31) / 32 * 32;
  const int64_t run0 = run * (rank * (kPlanThreads / 32) + (tid >> 5)), run1 = min((int64_t)a.num_rows, run0 + run);
  int low = run0 < R ? request_of(row_end, B, (int)run0) : 0;
  for (int64_t r0 = run0; r0 < run1; r0 += 128) {
    int page[4], pos[4], of[4], high[4];
    const int64_t end = min(min(r0 + 128, run1), R);   // the rows that requests have
    const int top = end > r0 ? request_from(row_end, B, low, (int)end - 1) : low;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      of[k] = low;
      high[k] = top;
    }
    for (int w = top - low; w > 0; w >>= 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int mid = (of[k] + high[k]) >> 1;
        if (row_end[mid] > r0 + 32 * k + lane) high[k] = mid;
        else of[k] = min(mid + 1, top);
      }
    }
    low = top;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t r = r0 + 32 * k + lane;
      page[k] = -1;
      pos[k] = -1;
      if (r < end) {
        const int b = of[k];
        const int first = b ? row_end[b - 1] : 0, page_first_b = b ? page_end[b - 1] : 0;
        pos[k] = old_len[b] + ((int)r - first);
        const int held = (int)(((int64_t)old_len[b] + P - 1) >> a.log2_page), lp = pos[k] >> a.log2_page;
        // a page that this call hands out is read from the stack: another thread writes its table entry
        page[k] = lp < held ? a.block_table[(int64_t)b * a.table_stride + lp]
                            : a.free_pages[count - 1 - (page_first_b + (lp - held))];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t r = r0 + 32 * k + lane;
      if (r < run1) {
        a.slot_mapping[r] = page[k] < 0 ? -1 : ((int64_t)page[k] << a.log2_page) + (pos[k] & (P - 1));
        if (a.positions) a.positions[r] = pos[k];
      }
    }
  }
}

// Returns the pages of finished requests to the stack of free pages, in request order.  A warp counts a
// request's valid page ids (it reads the table row anyway), one scan places them, and the warp then
// compacts the ids with ballots.  One CTA: a step finishes a few requests, and free_count is read and
// written in place.
__global__ void __launch_bounds__(kPlanThreads) pages_release_kernel(const PagesReleaseArgs a) {
  extern __shared__ int32_t plan_smem[];
  int32_t* end = plan_smem;               // [B] pages of finished requests 0 .. b
  __shared__ int64_t part[32][2];
  __shared__ uint32_t bits;
  const int B = a.num_requests, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) bits = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  auto held = [&](int b) {
    if (a.finished[b] == 0) return 0;
    const int64_t pages = ((int64_t)max(a.seq_lens[b], 0) + (1 << a.log2_page) - 1) >> a.log2_page;
    return (int)min(pages, (int64_t)a.table_stride);
  };
  auto valid = [&](int b, int n, int i) {
    const int page = i < n ? a.block_table[(int64_t)b * a.table_stride + i] : -1;
    return page >= 0 && page < a.num_pages ? page : -1;
  };
  for (int b = warp; b < B; b += kPlanThreads / 32) {
    const int n = held(b);
    int sum = 0;
    for (int i = 0; i < n; i += 32) sum += __popc(__ballot_sync(0xffffffffu, valid(b, n, i + lane) >= 0));
    if (lane == 0) {
      end[b] = sum;
      if (sum < n) atomicOr(&bits, (uint32_t)DSA_DEVICE_BAD_PAGE);
    }
  }
  __syncthreads();
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int64_t sum = 0, zero = 0;
  for (int b = b0; b < b1; ++b) sum += end[b];
  const int64_t mine = sum;
  block_scan2(sum, zero, part);
  sum -= mine;
  const int64_t count = min(max(*a.free_count, 0), a.free_capacity), room = a.free_capacity - count;
  for (int b = b0; b < b1; ++b) {
    sum += end[b];
    end[b] = (int32_t)min(sum, (int64_t)INT32_MAX);
  }
  __syncthreads();
  // every thread has read the count and the lengths' uses below are per request: written from here on
  for (int b = warp; b < B; b += kPlanThreads / 32) {
    const int first = b ? end[b - 1] : 0;
    // a stack too full for a request's pages keeps the request as it is (a page released twice does that)
    if (end[b] > room) {
      if (lane == 0 && end[b] > first) atomicOr(&bits, (uint32_t)DSA_DEVICE_POOL_FULL);
      continue;
    }
    const int n = held(b);
    int at = first;
    for (int i = 0; i < n; i += 32) {
      const int page = valid(b, n, i + lane);
      const uint32_t ok = __ballot_sync(0xffffffffu, page >= 0);
      if (page >= 0) a.free_pages[count + at + __popc(ok & ((1u << lane) - 1u))] = page;
      if (i + lane < n) a.block_table[(int64_t)b * a.table_stride + i + lane] = -1;
      at += __popc(ok);
    }
    __syncwarp();
    if (lane == 0 && a.finished[b] != 0) a.seq_lens[b] = 0;
  }
  __syncthreads();
  if (tid == 0) {
    // the released prefix: the largest end that fits
    int lo = 0, hi = B;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (end[mid] <= room) lo = mid + 1;
      else hi = mid;
    }
    *a.free_count = (int32_t)(count + (lo ? end[lo - 1] : 0));
    if (a.status) {
      a.status[0] = bits;
      a.status[1] = 0;
    }
  }
}

void plan_cluster(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* at, int ctas, int requests) {
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = (size_t)3 * requests * sizeof(int32_t);
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
}

std::atomic<uint64_t> g_plan_ready{0}, g_plan_wide{0};   // by device: set up, and found to hold the widest cluster
cudaError_t plan_set_up(int& widest) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
  e = once_per_device(g_plan_ready, [bit] {
    cudaError_t r = cudaFuncSetAttribute(step_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         3 * kPlanMaxRequests * (int)sizeof(int32_t));
    if (r == cudaSuccess) r = cudaFuncSetAttribute(step_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (r != cudaSuccess) return r;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    plan_cluster(cfg, at, kPlanClusterMax, kPlanMaxRequests);
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, step_plan_kernel, &cfg) == cudaSuccess && clusters > 0)
      g_plan_wide.fetch_or(bit, std::memory_order_acq_rel);
    else
      (void)cudaGetLastError();
    return cudaSuccess;
  });
  widest = g_plan_wide.load(std::memory_order_acquire) & bit ? kPlanClusterMax : 8;
  return e;
}
}  // namespace

cudaError_t launch_step_plan(const StepPlanArgs& a, cudaStream_t s) {
  int widest = 8;
  cudaError_t e = plan_set_up(widest);
  if (e != cudaSuccess) return e;
  // One CTA a few thousand rows keep busy; more rows are shared out, as the searches of a row's request are bound by
  // shared memory (69,632 rows of 4,096 requests: 12.4 us with 16 CTAs, 15.1 with 8).
  int ctas = 1;
  while (ctas < widest && (int64_t)ctas * 4 * kPlanThreads < a.num_rows) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  plan_cluster(cfg, at, ctas, a.num_requests);
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = s;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, step_plan_kernel, a);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_pages_release(const PagesReleaseArgs& a, cudaStream_t s) {
  cudaError_t e = launch_pdl(pages_release_kernel, dim3(1), dim3(kPlanThreads),
                             (size_t)a.num_requests * sizeof(int32_t), s, a);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dsa
