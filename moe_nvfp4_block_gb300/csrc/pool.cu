// pool.cu -- pages of a paged cache handed out to growing sequences and taken
// back, on the device.
//
// With grow_b the pages that sequence b lacks and end_b their running sum, the
// call's k-th page is the stack's k-th from its top and belongs to the first b
// with k < end_b.  A sequence is granted its pages if end_b does not pass the
// stack, so the granted ones are those of the first sequences that need any,
// and the k below the last granted end_b have no gaps.  A release runs the same
// sums over the pages given back, to the same places.
//
// What bounds it: three dependent reads (the sequences' ints, the stack or the
// table, their stores) and the launch.  Every CTA forms the sums of all
// sequences itself (at most 1024: 1 us) rather than wait for another's, then
// takes its share of the call's pages and rows, a search of the sums each.  The
// counts that the sums are formed from change only when every CTA has read
// them: the last one to say so writes them.
// Measured: 64 sequences, 160 rows handed out and taken back (two calls) 8.6 us;
// 1000 sequences, 264,000 rows 11.9.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kPoolThreads = 256;
constexpr int kPoolEach = kPagedMaxSeqs / kPoolThreads;  // sequences of a thread
constexpr long long kIntMax = 0x7fffffff;

// Exclusive sums of v over the CTA's threads; total: of all.
__device__ __forceinline__ long long scan_cta(long long v, long long* s_warp, long long& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();  // the last use of s_warp is over
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  long long base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPoolThreads / 32; ++w) {
    if (w < warp) base += s_warp[w];
    total += s_warp[w];
  }
  return base + inc - v;
}

// The first b < n with k < end[b] (n if there is none); end does not decrease.
__device__ __forceinline__ int first_above(const int* end, int n, int k) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] <= k) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void record(int* err, int e) { atomicCAS(err, 0, e); }

// True in every thread of one CTA: the last to call it.  (Its reads so far are
// done before it says so.)
__device__ __forceinline__ bool last_cta(unsigned* ticket) {
  __shared__ bool s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    s_last = true;
    if (gridDim.x > 1) {
      __threadfence();
      s_last = atomicAdd(ticket, 1u) == gridDim.x - 1;
      if (s_last) *ticket = 0;  // ready for the next call
    }
  }
  __syncthreads();
  return s_last;
}

}  // namespace

__global__ void __launch_bounds__(kPoolThreads) k_paged_reserve(const __grid_constant__ PoolArgs a) {
  __shared__ long long s_warp[kPoolThreads / 32];
  __shared__ int s_row[kPagedMaxSeqs + 1];  // first row of each sequence
  __shared__ int s_end[kPagedMaxSeqs];      // running sums of the pages wanted
  __shared__ int s_len[kPagedMaxSeqs], s_held[kPagedMaxSeqs];
  __shared__ bool s_ok[kPagedMaxSeqs];
  __shared__ int s_pages;  // of the granted sequences
  const int n = a.n_seqs, tid = threadIdx.x;
  const bool first = blockIdx.x == 0;
  pdl_wait();
  pdl_launch_dependents();
  int err = 0;
  int n_free = *a.n_free;
  if (n_free < 0 || n_free > a.n_pages) {
    err = MOE_ERR_INVALID_ARG;
    n_free = 0;
  }
  long long grow[kPoolEach], rows[kPoolEach], sum_g = 0, sum_r = 0;
  bool can[kPoolEach];
#pragma unroll
  for (int i = 0; i < kPoolEach; ++i) {
    const int b = tid * kPoolEach + i;
    grow[i] = rows[i] = 0;
    can[i] = false;
    if (b >= n) continue;
    const int len = a.kv_len[b], r = a.rows[b], held = a.held[b];
    s_len[b] = len;
    s_held[b] = held;
    if (len < 0 || r < 0 || held < 0 || held > a.max_pages) {
      err = MOE_ERR_INVALID_ARG;
      continue;
    }
    rows[i] = r;
    const long long need = ((long long)len + r + (1 << a.lps) - 1) >> a.lps;
    can[i] = need <= a.max_pages;
    if (can[i]) grow[i] = need > held ? need - held : 0;
    else if (!err) err = MOE_ERR_CAPACITY;
    sum_g += grow[i];
    sum_r += rows[i];
  }
  if (tid == 0) s_pages = 0;
  long long total_r, total_g;
  long long at_r = scan_cta(sum_r, s_warp, total_r);
  long long at_g = scan_cta(sum_g, s_warp, total_g);
#pragma unroll
  for (int i = 0; i < kPoolEach; ++i) {
    const int b = tid * kPoolEach + i;
    if (b >= n) break;
    s_row[b] = (int)min(at_r, kIntMax);
    at_r += rows[i];
    at_g += grow[i];
    s_end[b] = (int)min(at_g, kIntMax);
    const bool ok = can[i] && (grow[i] == 0 || at_g <= n_free);
    if (can[i] && !ok && !err) err = MOE_ERR_CAPACITY;
    if (ok && grow[i] > 0) atomicMax(&s_pages, (int)at_g);
    s_ok[b] = ok;
  }
  if (tid == 0) s_row[n] = (int)min(total_r, kIntMax);
  if (tid == 0 && a.n_rows > 0 && total_r > a.n_rows && !err) err = MOE_ERR_CAPACITY;
  if (first && err) record(a.err, err);
  const bool last = last_cta(a.ticket);  // (and a barrier)
  const int pages = s_pages;

  if (last) {
    for (int b = tid; b < n; b += kPoolThreads) {
      const int g = s_end[b] - (b ? s_end[b - 1] : 0);
      if (s_ok[b] && g > 0) a.held[b] = s_held[b] + g;
    }
    if (tid == 0 && pages > 0) *a.n_free = n_free - pages;
  }
  if (first) {
    for (int b = tid; b <= n; b += kPoolThreads) a.row_start[b] = s_row[b];
    if (a.granted)
      for (int b = tid; b < n; b += kPoolThreads) a.granted[b] = s_ok[b];
  }
  const int step = gridDim.x * kPoolThreads, t0 = blockIdx.x * kPoolThreads + tid;
  for (long long k = t0; k < pages; k += step) {
    const int b = first_above(s_end, n, (int)k);
    const int page = a.free_pages[n_free - 1 - (int)k];
    if (page < 0 || page >= a.n_pages) record(a.err, MOE_ERR_INVALID_ARG);
    const int g = (int)k - (b ? s_end[b - 1] : 0);
    a.table[(size_t)b * a.max_pages + s_held[b] + g] = page;
  }
  // four rows a thread: one search, their pages in flight together
  const bool whole = ((reinterpret_cast<uintptr_t>(a.slot) | reinterpret_cast<uintptr_t>(a.pos)) & 15u) == 0;
  for (long long t4 = 4LL * t0; t4 < a.n_rows; t4 += 4LL * step) {
    int b = first_above(s_row + 1, n, (int)t4), pos[4], page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = (int)min(t4 + k, (long long)a.n_rows - 1);
      while (b < n && s_row[b + 1] <= t) ++b;  // the sequence of row t: the last one that starts at or before it
      pos[k] = page[k] = -1;
      if (b == n) continue;
      pos[k] = (int)min((long long)s_len[b] + (t - s_row[b]), kIntMax);
      if (!s_ok[b]) continue;
      const int j = pos[k] >> a.lps, fresh = j - s_held[b];
      page[k] = fresh < 0 ? a.table[(size_t)b * a.max_pages + j] : a.free_pages[n_free - 1 - (fresh + (b ? s_end[b - 1] : 0))];
    }
    int slot[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      slot[k] = page[k] >= 0 && page[k] < a.n_pages ? (page[k] << a.lps) + (pos[k] & ((1 << a.lps) - 1)) : -1;
    if (whole && t4 + 4 <= a.n_rows) {
      if (a.slot) *reinterpret_cast<int4*>(a.slot + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.pos) *reinterpret_cast<int4*>(a.pos + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (t4 + k >= a.n_rows) continue;
        if (a.slot) a.slot[t4 + k] = slot[k];
        if (a.pos) a.pos[t4 + k] = pos[k];
      }
    }
  }
}

__global__ void __launch_bounds__(kPoolThreads) k_paged_release(const __grid_constant__ PoolArgs a) {
  __shared__ long long s_warp[kPoolThreads / 32];
  __shared__ int s_end[kPagedMaxSeqs];  // running sums of the pages given back
  __shared__ int s_kept[kPagedMaxSeqs];
  __shared__ bool s_ok[kPagedMaxSeqs];
  __shared__ int s_pages;
  const int n = a.n_seqs, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  int err = 0;
  const int n_free = *a.n_free;
  const bool stack = n_free >= 0 && n_free <= a.n_pages;
  if (!stack) err = MOE_ERR_INVALID_ARG;
  long long back[kPoolEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kPoolEach; ++i) {
    const int b = tid * kPoolEach + i;
    back[i] = 0;
    if (b >= n) continue;
    const int held = a.held[b], keep = max(a.keep[b], 0);
    if (held < 0 || held > a.max_pages) {
      err = MOE_ERR_INVALID_ARG;
      continue;
    }
    const int kept = max((int)(((long long)keep + (1 << a.lps) - 1) >> a.lps), a.shared ? a.shared[b] : 0);
    s_kept[b] = kept;
    back[i] = held > kept ? held - kept : 0;
    sum += back[i];
  }
  if (tid == 0) s_pages = 0;
  long long total;
  long long at = scan_cta(sum, s_warp, total);
#pragma unroll
  for (int i = 0; i < kPoolEach; ++i) {
    const int b = tid * kPoolEach + i;
    if (b >= n) break;
    at += back[i];
    s_end[b] = (int)min(at, kIntMax);
    const bool ok = back[i] > 0 && stack && n_free + at <= a.n_pages;
    if (back[i] > 0 && !ok) err = MOE_ERR_INVALID_ARG;
    if (ok) atomicMax(&s_pages, (int)at);
    s_ok[b] = ok;
  }
  if (blockIdx.x == 0 && err) record(a.err, err);
  const bool last = last_cta(a.ticket);
  const int pages = s_pages;
  if (last) {
    for (int b = tid; b < n; b += kPoolThreads)
      if (s_ok[b]) a.held[b] = s_kept[b];
    if (tid == 0 && pages > 0) *a.n_free = n_free + pages;
  }
  const int step = gridDim.x * kPoolThreads;
  for (long long k = blockIdx.x * kPoolThreads + tid; k < pages; k += step) {
    const int b = first_above(s_end, n, (int)k);
    int32_t* entry = a.table + (size_t)b * a.max_pages + s_kept[b] + ((int)k - (b ? s_end[b - 1] : 0));
    const int page = *entry;
    if (page < 0 || page >= a.n_pages) record(a.err, MOE_ERR_INVALID_ARG);
    a.free_pages[n_free + pages - 1 - (int)k] = page;
    *entry = -1;
  }
}

namespace {

template <auto KERN>
cudaError_t launch_pool(const PoolArgs& a, long long work, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // one CTA up to 2048 entries; more: 1024 a CTA, at most two an SM
  const long long want = work <= 2048 ? 1 : (work + 1023) / 1024;
  cfg.gridDim = dim3((unsigned)(want < 2 * num_sms() ? want : 2 * num_sms()));
  cfg.blockDim = dim3(kPoolThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = prepare_kernel<KERN>(0);
  return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, KERN, a) : e;
}

}  // namespace

// How many pages change hands is on the device.  Where the call asks for its
// rows' slots, a row in 16 at most asks for one.  Else, and at a release, a
// sequence is taken to have 32 (700 sequences that take 60,000 pages without
// slots and give them back: 173 us with the reserve on one CTA, 23 so; 1024 of a
// page each 10.4 and 8.8; 64 are one CTA either way, 6.4).  More a sequence only
// take longer: 5 of 3750 pages each 64 us.
cudaError_t launch_paged_reserve(const PoolArgs& a, cudaStream_t s) {
  const long long pages = 32LL * a.n_seqs;
  return launch_pool<k_paged_reserve>(a, a.n_rows > 0 ? a.n_rows : pages < a.n_pages ? pages : a.n_pages, s);
}
cudaError_t launch_paged_release(const PoolArgs& a, cudaStream_t s) {
  return launch_pool<k_paged_release>(a, 32LL * a.n_seqs, s);
}

}  // namespace moe
