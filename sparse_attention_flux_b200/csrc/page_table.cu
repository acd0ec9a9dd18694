// page_table.cu -- block tables, slot map and positions of a paged cache, built
// on the GPU from the request lengths before and after a step.
//
// With np(x) = ceil(x / page) and, for a ring, cap = sink + window pages (else
// infinity), request b takes need_b = min(np(new), cap) - min(np(old), cap)
// pages from the free list; an exclusive scan of need gives each request its
// place in the list, a scan of new - old each token its request.  Logical page
// j lives in the physical page of comp(j) = j below cap, else
// sink + (j - sink) mod window, which either is fresh (comp >= the pages held
// before) or stands in the table already.
#include "q4.h"

namespace flux {

namespace {

constexpr int kThreads = 1024;

__device__ __forceinline__ int pages_of(int len, int page) {
  return len > 0 ? (len - 1) / page + 1 : 0;
}

__global__ void __launch_bounds__(kThreads) page_table_kernel(const PageTableLaunch a) {
  extern __shared__ int32_t smem[];
  int32_t* cu = smem;                 // [B + 1] tokens before each request
  int32_t* pg = smem + a.B + 1;       // [B + 1] fresh pages before each request
  __shared__ unsigned long long wsum_t[32], wsum_p[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = a.window_pages > 0 ? a.sink_pages + a.window_pages : 0x7fffffff;
  unsigned long long carry_t = 0, carry_p = 0;
  bool bad = false;
  for (int base = 0; base < a.B; base += kThreads) {
    const int b = base + tid;
    unsigned long long t = 0, p = 0;
    if (b < a.B) {
      const int o = a.old_lens[b], n = a.new_lens[b];
      if (o < 0 || n < o || pages_of(n, a.page_size) > a.max_pages) {
        bad = true;
      } else {
        t = n - o;
        p = min(pages_of(n, a.page_size), cap) - min(pages_of(o, a.page_size), cap);
      }
    }
    const unsigned long long t0 = t, p0 = p;
    for (int s = 1; s < 32; s <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, t, s);
      const unsigned long long y = __shfl_up_sync(0xffffffffu, p, s);
      if (lane >= s) { t += x; p += y; }
    }
    if (lane == 31) { wsum_t[warp] = t; wsum_p[warp] = p; }
    __syncthreads();
    unsigned long long bt = carry_t, bp = carry_p;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) { bt += wsum_t[w]; bp += wsum_p[w]; }
      carry_t += wsum_t[w];
      carry_p += wsum_p[w];
    }
    if (b < a.B) {
      cu[b] = static_cast<int>(bt + t - t0);
      pg[b] = static_cast<int>(bp + p - p0);
    }
    __syncthreads();
  }
  bad = __syncthreads_or(bad);
  const int cursor = *a.cursor;
  const bool fits = carry_t <= static_cast<unsigned long long>(a.n_slots) && cursor >= 0 &&
                    cursor <= a.n_free &&
                    carry_p <= static_cast<unsigned long long>(a.n_free - cursor);
  const bool ok = !bad && fits;
  const int total = ok ? static_cast<int>(carry_t) : 0;
  if (tid == 0) {
    if (bad) raise_error(a.err, DEV_ERR_SEQLEN);
    else if (!fits) raise_error(a.err, DEV_ERR_CAPACITY);
    cu[a.B] = total;
  }
  __syncthreads();
  auto page_of = [&](int b, int j, int held) {
    const int c = j < cap ? j : a.sink_pages + (j - a.sink_pages) % a.window_pages;
    const int id = c >= held ? a.free_pages[cursor + pg[b] + c - held]
                             : a.page_table[static_cast<size_t>(b) * a.max_pages + c];
    if (id < 0) raise_error(a.err, DEV_ERR_PAGE);
    return id;
  };
  for (int i = tid; i < a.n_slots; i += kThreads) {
    int64_t slot = -1;
    int pos = 0;
    if (i < total) {
      int lo = 0, hi = a.B - 1;                  // the last b with cu[b] <= i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= i) lo = mid; else hi = mid - 1;
      }
      const int o = a.old_lens[lo];
      pos = o + i - cu[lo];
      const int j = pos / a.page_size;
      const int last = pages_of(a.new_lens[lo], a.page_size);
      if (j < a.sink_pages || a.window_pages == 0 || j >= last - a.window_pages) {
        const int id = page_of(lo, j, min(pages_of(o, a.page_size), cap));
        if (id >= 0) slot = static_cast<int64_t>(id) * a.page_size + pos % a.page_size;
      }
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  if (ok) {
    for (int b = warp; b < a.B; b += kThreads / 32) {
      const int j0 = pages_of(a.old_lens[b], a.page_size), j1 = pages_of(a.new_lens[b], a.page_size);
      for (int j = j0 + lane; j < j1; j += 32)
        a.page_table[static_cast<size_t>(b) * a.max_pages + j] = page_of(b, j, min(j0, cap));
    }
  }
  if (a.cu_new)
    for (int b = tid; b <= a.B; b += kThreads) a.cu_new[b] = ok ? cu[b] : 0;
  if (tid == 0) *a.cursor_out = ok ? cursor + static_cast<int>(carry_p) : cursor;
}

}  // namespace

cudaError_t launch_page_table(const PageTableLaunch& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const int smem = 2 * (p.B + 1) * static_cast<int>(sizeof(int32_t));
  cudaError_t e = cudaFuncSetAttribute(page_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       2 * (kPageTableMaxB + 1) * static_cast<int>(sizeof(int32_t)));
  if (e != cudaSuccess) return e;
  page_table_kernel<<<1, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace flux
