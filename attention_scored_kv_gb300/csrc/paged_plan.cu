// Block tables, slot maps and lengths of the paged cache, from the requests' lengths.
//
// What it computes: for request r with c cached and q new tokens, blocks
// ceil(c/16) .. ceil((c+q)/16) - 1 take pages from the free stack (the j-th page taken
// overall is free[count - 1 - j]); rows are packed at the exclusive sums of q; row i of r
// is position c + i with slot page * 16 + position % 16.
//
// How: everything follows from two prefix sums over the requests (rows and pages), which
// are a few hundred integers, so every CTA computes them for itself, 512 requests at a
// time, and then fills its share of the tables and rows: no CTA waits for another's
// result.  The one hazard is an output that is also an input (kv_len over ctx_len, the
// count in place): those calls run as one cluster of 8 CTAs whose barrier separates the
// last read from the first write; calls with outputs of their own use as many CTAs as
// the rows feed.  Rows go four to a thread (one binary search in shared memory and one
// 16-byte store each); a page's table entry is a thread's.  Bound by launch latency for a
// decode step (16 requests: 7 us a call), by the two searches and the table's loads for
// large batches (64 prompts, 1.2 M rows, 75 k pages: 10 us, 10 MB; in place, on 8 CTAs, eight times that).
#include "paged.cuh"

namespace kvs {
namespace {

constexpr int kThreads = 512;
constexpr int kChunk = kThreads;         // requests of one round
constexpr int kAliasCtas = 8;            // a portable cluster

struct Item {
  long long rows, pages;
};

__device__ __forceinline__ Item add(Item a, Item b) { return {a.rows + b.rows, a.pages + b.pages}; }

// Inclusive prefix sums over the block's threads.
__device__ Item block_scan(Item x, Item* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x.rows, o), b = __shfl_up_sync(0xffffffffu, x.pages, o);
    if (lane >= o) { x.rows += a; x.pages += b; }
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    Item w = lane < kThreads / 32 ? warp_sums[lane] : Item{0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, w.rows, o), b = __shfl_up_sync(0xffffffffu, w.pages, o);
      if (lane >= o) { w.rows += a; w.pages += b; }
    }
    if (lane < kThreads / 32) warp_sums[lane] = w;
  }
  __syncthreads();
  return warp ? add(x, warp_sums[warp - 1]) : x;
}

__device__ __forceinline__ void cluster_arrive() { __syncwarp(); asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { __syncwarp(); asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

struct Args {
  PagedDev d;
  int n, stride, free_capacity, capacity;
  const int32_t* ctx; const int32_t* add;          // ctx may be null (all 0)
  int32_t* table;
  const int32_t* free_pages; const int32_t* count_in; int32_t* count_out;
  int32_t* row_start; int32_t* kv_len; int32_t* slots; int32_t* positions; int32_t* denied;
};

// TAKE: pages are taken (kvs_paged_plan); else tables are read only (kvs_paged_slot_map).
template <bool TAKE>
__global__ void __launch_bounds__(kThreads) plan_kernel(const Args a) {
  __shared__ Item warp_sums[kThreads / 32];
  __shared__ int s_start[kChunk + 1];      // first row of the request
  __shared__ int s_ctx[kChunk];            // its cached tokens; negative: denied
  __shared__ int s_page[kChunk + 1];       // pages taken before it
  const int tid = threadIdx.x, G = gridDim.x, cta = blockIdx.x;
  const long long most = (long long)a.stride * kBlock;
  const int count = TAKE ? max(0, min(*a.count_in, a.free_capacity)) : 0;
  Item carry{0, 0};
  int err = 0, denied = 0;
  long long taken = 0;
  for (int r0 = 0; r0 < a.n; r0 += kChunk) {
    const int m = min(kChunk, a.n - r0), r = r0 + tid;
    int c = 0, q = 0;
    if (tid < m) {
      c = a.ctx ? a.ctx[r] : 0;
      q = a.add[r];
      if (c < 0 || q < 0) err |= kErrState;
      c = max(c, 0);
      q = max(q, 0);
    }
    if (TAKE) cluster_arrive();              // this CTA has read the chunk's lengths and the count
    const bool fits = (long long)c + q <= most;
    const int held = (c + kBlock - 1) / kBlock;
    const int need = TAKE && fits ? (c + q + kBlock - 1) / kBlock - held : 0;
    const Item incl = add(carry, block_scan(Item{q, need}, warp_sums));
    const bool grant = !TAKE || (fits && (need == 0 || incl.pages <= count));
    if (tid < m) {
      s_start[tid] = (int)min(incl.rows - q, (long long)INT32_MAX);
      s_ctx[tid] = grant ? c : -1 - c;
      s_page[tid] = (int)min(incl.pages - need, (long long)INT32_MAX);
      if (!grant) ++denied;
      if (grant && need) taken = max(taken, incl.pages);
      if (!TAKE && !fits && q > 0) err |= kErrCapacity;
    }
    if (tid == m - 1) {
      s_start[m] = (int)min(incl.rows, (long long)INT32_MAX);
      s_page[m] = (int)min(incl.pages, (long long)INT32_MAX);
    }
    carry = add(carry, warp_sums[kThreads / 32 - 1]);
    __syncthreads();
    if (TAKE) cluster_wait();
    if (cta == 0 && tid < m) {
      a.row_start[r] = s_start[tid];
      if (r == a.n - 1) a.row_start[a.n] = s_start[m];
      if (TAKE) a.kv_len[r] = grant ? c + q : c;
    }
    if (TAKE) {
      // Table entries, a thread to a page.  Pages that are wanted past the stack's are of denied requests; together
      // they may pass 32 bits.
      const int pages = min(s_page[m], count);
      for (long long j0 = (long long)s_page[0] + cta * kThreads + tid; j0 < pages; j0 += (long long)G * kThreads) {
        const int j = (int)j0;
        int i = 0, top = m - 1;
        while (i < top) {
          const int mid = (i + top + 1) >> 1;
          if (s_page[mid] <= j) i = mid; else top = mid - 1;
        }
        const int ci = s_ctx[i];
        if (ci < 0) continue;                // denied
        a.table[(size_t)(r0 + i) * a.stride + (ci + kBlock - 1) / kBlock + (j - s_page[i])] = a.free_pages[count - 1 - j];
      }
    }
    // rows, four to a thread
    const int lo = s_start[0], hi = min(s_start[m], a.capacity);
    for (int t0 = lo < hi ? (lo & ~3) + 4 * (cta * kThreads + tid) : hi; t0 < hi; t0 += 4 * G * kThreads) {
      int i = 0, top = m - 1;                // the last request that starts at or before the first row
      const int key = max(t0, lo);
      while (i < top) {
        const int mid = (i + top + 1) >> 1;
        if (s_start[mid] <= key) i = mid; else top = mid - 1;
      }
      int slot[4], pos[4], block = -1, page = -1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + u;
        slot[u] = -1;
        pos[u] = 0;
        if (t < lo || t >= hi) continue;
        while (s_start[i + 1] <= t) { ++i; block = -1; }
        const int ci = s_ctx[i];
        const bool ok = ci >= 0;
        const long long p = (long long)(ok ? ci : -1 - ci) + (t - s_start[i]);
        pos[u] = (int)min(p, (long long)INT32_MAX);
        if (!ok || p >= most) continue;
        if ((int)(p >> 4) != block) {
          block = (int)(p >> 4);
          const int h = (ci + kBlock - 1) / kBlock;
          page = (TAKE && block >= h) ? a.free_pages[count - 1 - (s_page[i] + block - h)]
                                      : a.table[(size_t)(r0 + i) * a.stride + block];
          if (page < 0 || page >= a.d.num_pages) { err |= kErrState; page = -1; }
        }
        if (page >= 0) slot[u] = page * kBlock + (int)(p & 15);
      }
      if (t0 >= lo && t0 + 4 <= hi && !(reinterpret_cast<uintptr_t>(a.slots) & 15)) {
        *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (t0 + u >= lo && t0 + u < hi) a.slots[t0 + u] = slot[u];
      }
      if (a.positions) {
        if (t0 >= lo && t0 + 4 <= hi && !(reinterpret_cast<uintptr_t>(a.positions) & 15)) {
          *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (t0 + u >= lo && t0 + u < hi) a.positions[t0 + u] = pos[u];
        }
      }
    }
    __syncthreads();                         // before the next round overwrites the shared arrays
  }
  // rows past the last
  const int end = (int)min(carry.rows, (long long)a.capacity);
  for (int t = end + cta * kThreads + tid; t < a.capacity; t += G * kThreads) {
    a.slots[t] = -1;
    if (a.positions) a.positions[t] = 0;
  }
  if (carry.rows > a.capacity) err |= kErrCapacity;
  if (cta == 0) {
    if (denied) err |= kErrCapacity;
    if (TAKE) {
      __shared__ int s_denied;
      __shared__ unsigned long long s_taken;
      if (tid == 0) { s_denied = 0; s_taken = 0; }
      __syncthreads();
      if (denied) atomicAdd(&s_denied, denied);
      if (taken) atomicMax(&s_taken, (unsigned long long)taken);
      __syncthreads();
      if (tid == 0) {
        *a.count_out = count - (int)s_taken;
        if (a.denied) *a.denied = s_denied;
      }
    }
  }
  if (err) paged_error(a.d, err);
}

// One CTA walks the pages from the last to the first, so that a page's place on the stack is the number of
// those after it that are pages: what is not one is left out without knowing the total first.  A thread has four
// pages in a row, whose table entries are loaded together.  Bound by the latency of a round of 2048 pages (search,
// load, scan: 2 us): 64 contexts of 68866 pages 81 us, 16 of 44 pages 7 us.
constexpr int kReleaseChunk = 256;       // requests of one round: their pages are counted in 32 bits
static_assert((long long)kReleaseChunk * kMaxTableStride <= 1ll << 30, "pages of a round");
__global__ void __launch_bounds__(kThreads) release_kernel(const PagedDev d, int n, const int32_t* kv_len,
                                                           int32_t* table, int stride, int32_t* free_pages,
                                                           int free_capacity, int32_t* free_count) {
  __shared__ Item warp_sums[kThreads / 32];
  __shared__ int s_first[kReleaseChunk + 1];
  const int tid = threadIdx.x;
  long long count = max(0, min(*free_count, free_capacity));
  int err = 0;
  for (int r0 = (n - 1) / kReleaseChunk * kReleaseChunk; r0 >= 0; r0 -= kReleaseChunk) {
    const int m = min(kReleaseChunk, n - r0);
    const int mine = tid < m ? (int)min((max((long long)kv_len[r0 + tid], 0ll) + kBlock - 1) / kBlock, (long long)stride) : 0;
    const Item incl = block_scan(Item{0, mine}, warp_sums);
    if (tid < m) s_first[tid] = (int)(incl.pages - mine);
    const int here = (int)warp_sums[kThreads / 32 - 1].pages;
    if (tid == 0) s_first[m] = here;
    __syncthreads();
    for (int top = here; top > 0; top -= 4 * kThreads) {       // pages [top - 2048, top), the last four first
      int page[4], good = 0;
      const int j0 = top - 1 - 4 * tid;
      int i = 0, last = m - 1;
      while (i < last) {
        const int mid = (i + last + 1) >> 1;
        if (s_first[mid] <= max(j0, 0)) i = mid; else last = mid - 1;
      }
      int32_t* entry[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 - u;
        while (j >= 0 && j < s_first[i]) --i;
        entry[u] = j >= 0 ? table + (size_t)(r0 + i) * stride + (j - s_first[i]) : nullptr;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) page[u] = entry[u] ? *entry[u] : -1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!entry[u]) continue;
        *entry[u] = -1;
        if (page[u] >= 0 && page[u] < d.num_pages) {
          ++good;
        } else {
          page[u] = -1;
          err |= kErrState;
        }
      }
      long long at = count + block_scan(Item{0, good}, warp_sums).pages - good;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (page[u] < 0) continue;
        if (at < free_capacity) free_pages[at] = page[u];
        else err |= kErrCapacity;
        ++at;
      }
      count += warp_sums[kThreads / 32 - 1].pages;
      __syncthreads();
    }
  }
  if (tid == 0) *free_count = (int)min(count, (long long)free_capacity);
  if (err) paged_error(d, err);
}

template <bool TAKE>
cudaError_t launch(const Args& a, int grid, bool cluster, cudaStream_t st) {
  if (!cluster || grid == 1) {
    plan_kernel<TAKE><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = grid;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel<TAKE>, a);
}

// CTAs that `capacity` rows feed: two rounds of four rows a thread each, at most four CTAs to an SM.
int grid_for(int capacity, int sms) {
  const int want = (int)cdiv64(capacity, 2 * 4 * kThreads);
  return want < 1 ? 1 : (want < 4 * sms ? want : 4 * sms);
}

}  // namespace

cudaError_t launch_paged_plan(const PagedDev& d, int n, const int32_t* ctx, const int32_t* add, int32_t* table,
                              int stride, const int32_t* free_pages, int free_capacity, const int32_t* count_in,
                              int32_t* count_out, int32_t* row_start, int32_t* kv_len, int32_t* slots,
                              int32_t* positions, int capacity, int32_t* denied, int sms, cudaStream_t st) {
  const Args a{d, n, stride, free_capacity, capacity, ctx, add, table, free_pages, count_in, count_out,
               row_start, kv_len, slots, positions, denied};
  const bool alias = kv_len == ctx || count_out == count_in;
  int grid = grid_for(capacity, sms);
  if (alias && grid > kAliasCtas) grid = kAliasCtas;
  return launch<true>(a, grid, alias, st);
}

cudaError_t launch_paged_slot_map(const PagedDev& d, int n, const int32_t* first, const int32_t* len,
                                  const int32_t* table, int stride, int32_t* row_start, int32_t* slots,
                                  int32_t* positions, int capacity, int sms, cudaStream_t st) {
  const Args a{d, n, stride, 0, capacity, first, len, const_cast<int32_t*>(table), nullptr, nullptr, nullptr,
               row_start, nullptr, slots, positions, nullptr};
  return launch<false>(a, grid_for(capacity, sms), false, st);
}

cudaError_t launch_paged_release(const PagedDev& d, int n, const int32_t* kv_len, int32_t* table, int stride,
                                 int32_t* free_pages, int free_capacity, int32_t* free_count, cudaStream_t st) {
  release_kernel<<<1, kThreads, 0, st>>>(d, n, kv_len, table, stride, free_pages, free_capacity, free_count);
  return cudaGetLastError();
}

}  // namespace kvs
