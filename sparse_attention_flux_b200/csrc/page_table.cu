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
//
// One launch.  Every CTA makes both scans for itself (they read 8 bytes a
// request, which costs less than a second kernel or a wait between CTAs) and
// then writes its share of the tokens and of the requests' new pages.  The
// cursor may be updated in place, so the CTA that takes the last ticket, when
// all have read it, writes it.  Bound: the latency of its few dependent loads
// and barriers for a decode step, the 12 bytes a token for long prompts.
#include "q4.h"

namespace flux {

namespace {

__device__ __forceinline__ int pages_of(int len, int page) {
  return len > 0 ? (len - 1) / page + 1 : 0;
}

template <int T>
__global__ void __launch_bounds__(T) page_table_kernel(const PageTableLaunch a) {
  extern __shared__ int32_t smem[];
  int32_t* cu = smem;                 // [B + 1] tokens before each request
  int32_t* pg = smem + a.B + 1;       // [B + 1] fresh pages before each request
  __shared__ unsigned long long wsum_t[2][T / 32], wsum_p[2][T / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = a.window_pages > 0 ? a.sink_pages + a.window_pages : 0x7fffffff;
  griddep_launch_dependents();
  griddep_wait();
  __shared__ int sm_cursor;           // one read per CTA, over before the first barrier
  if (tid == 0) sm_cursor = *a.cursor;
  unsigned long long carry_t = 0, carry_p = 0;
  bool bad = false;
  for (int base = 0, turn = 0; base < a.B; base += T, turn ^= 1) {
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
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, t, s);
      const unsigned long long y = __shfl_up_sync(0xffffffffu, p, s);
      if (lane >= s) { t += x; p += y; }
    }
    if (lane == 31) { wsum_t[turn][warp] = t; wsum_p[turn][warp] = p; }
    __syncthreads();
    unsigned long long bt = carry_t, bp = carry_p;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
      if (w < warp) { bt += wsum_t[turn][w]; bp += wsum_p[turn][w]; }
      carry_t += wsum_t[turn][w];
      carry_p += wsum_p[turn][w];
    }
    if (b < a.B) {
      cu[b] = static_cast<int>(bt + t - t0);
      pg[b] = static_cast<int>(bp + p - p0);
    }
  }
  bad = __syncthreads_or(bad);
  const int cursor = sm_cursor;
  const bool fits = carry_t <= static_cast<unsigned long long>(a.n_slots) && cursor >= 0 &&
                    cursor <= a.n_free &&
                    carry_p <= static_cast<unsigned long long>(a.n_free - cursor);
  const bool ok = !bad && fits;
  const int total = ok ? static_cast<int>(carry_t) : 0;
  if (tid == 0) {
    if (blockIdx.x == 0) {
      if (bad) raise_error(a.err, DEV_ERR_SEQLEN);
      else if (!fits) raise_error(a.err, DEV_ERR_CAPACITY);
    }
    // Every CTA has its cursor: the last to say so may write it.
    bool last = true;
    if (gridDim.x > 1) {
      __threadfence();
      last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
      if (last) *a.ticket = 0;
    }
    if (last) *a.cursor_out = ok ? cursor + static_cast<int>(carry_p) : cursor;
  }
  auto page_of = [&](int b, int j, int held) {
    const int c = j < cap ? j : a.sink_pages + (j - a.sink_pages) % a.window_pages;
    const int id = c >= held ? a.free_pages[cursor + pg[b] + c - held]
                             : a.page_table[static_cast<size_t>(b) * a.max_pages + c];
    if (id < 0) raise_error(a.err, DEV_ERR_PAGE);
    return id;
  };
  const int stride = gridDim.x * T;
  for (int i = blockIdx.x * T + tid; i < a.n_slots; i += stride) {
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
    if (i > 0x7fffffff - stride) break;
  }
  if (ok) {
    for (int b = blockIdx.x * (T / 32) + warp; b < a.B; b += gridDim.x * (T / 32)) {
      const int j0 = pages_of(a.old_lens[b], a.page_size), j1 = pages_of(a.new_lens[b], a.page_size);
      for (int j = j0 + lane; j < j1; j += 32)
        a.page_table[static_cast<size_t>(b) * a.max_pages + j] = page_of(b, j, min(j0, cap));
    }
  }
  if (a.cu_new && blockIdx.x == 0)
    for (int b = tid; b <= a.B; b += T) a.cu_new[b] = !ok ? 0 : b < a.B ? cu[b] : total;
}

template <int T>
cudaError_t launch_t(const PageTableLaunch& p, int num_sms, cudaStream_t stream) {
  constexpr int max_smem = 2 * (kPageTableMaxB + 1) * static_cast<int>(sizeof(int32_t));
  const int smem = 2 * (p.B + 1) * static_cast<int>(sizeof(int32_t));
  if (smem > 40 << 10) {      // with the static arrays past 48 KB
    const cudaError_t e =
        cudaFuncSetAttribute(page_table_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
    if (e != cudaSuccess) return e;
  }
  // A token a thread, or a warp per eight requests, in one wave.  (Four tokens a
  // thread on a CTA per SM: 10.3 us for 48 prompts of 170k tokens against 7.7.)
  const long long want = (static_cast<long long>(p.n_slots) + T - 1) / T;
  const long long rows = (static_cast<long long>(p.B) + T / 4 - 1) / (T / 4);
  const long long ctas = want > rows ? want : rows, wave = static_cast<long long>(2048 / T) * num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < wave ? ctas : wave));
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_table_kernel<T>, p);
}

}  // namespace

// Few requests: 256 threads (their barriers cost less); many: 1024, a scan step per 1024.
cudaError_t launch_page_table(const PageTableLaunch& p, int num_sms, cudaStream_t stream) {
  return p.B <= 1024 ? launch_t<256>(p, num_sms, stream) : launch_t<1024>(p, num_sms, stream);
}

}  // namespace flux
