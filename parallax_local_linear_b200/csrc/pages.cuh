// Page plan: page tables, slot map and positions of a serving step, built from
// the requests' lengths (the definition is at parallax_page_plan in
// parallax.h).
//
// Two exclusive prefix sums over the requests fix everything: of the new rows
// (which rows belong to whom) and of the new pages (which free pages go to
// whom).  Every CTA forms both for itself in shared memory, so that no CTA
// waits for another and one launch does the whole plan: 8 bytes a request
// from L2, and two block-wide scans.  The rows are then cut evenly over the
// grid, and a row finds its request by a binary search in shared memory.  A
// row's page is an old table entry or a free page found from the prefix sum,
// never a table entry that this launch writes, so rows and table entries are
// written in any order.  Latency bounds it: 128 requests of one row take 3.5 us,
// 1024 requests of 300 000 rows (3.6 MB) 7 us, device time.
#pragma once

#include "ptx.cuh"

namespace plx {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxBatch = 8192;
constexpr int kPage = 64;

struct PagePlanArgs {
  const int32_t* cached;
  const int32_t* fresh;            // new tokens of each request
  int32_t* table;                  // [B, max_pages]
  const int32_t* free_pages;
  const int32_t* free_head;        // or null
  int32_t* seq_lens;
  int32_t* cu;
  int64_t* slots;
  int32_t* positions;
  int32_t* used;
  int B, rows, num_pages, max_pages, num_free;
};

// Request b's first row is cu[b]; `off[b]` free pages go to the requests
// before it; have[b] is its number of cached tokens, or -1 if it failed.
__host__ __device__ constexpr int plan_smem_bytes(int B) { return (3 * B + 1) * 4; }

// Sum over the block's earlier threads of (x, y), and the block's totals.
__device__ __forceinline__ void block_scan2(long long& x, long long& y, long long& tx, long long& ty) {
  __shared__ long long part[2][kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ux = __shfl_up_sync(0xffffffffu, ix, o), uy = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) {
      ix += ux;
      iy += uy;
    }
  }
  if (lane == 31) {
    part[0][warp] = ix;
    part[1][warp] = iy;
  }
  __syncthreads();
  long long bx = 0, by = 0;
  tx = ty = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w == warp) {
      bx = tx;
      by = ty;
    }
    tx += part[0][w];
    ty += part[1][w];
  }
  x = bx + ix - x;
  y = by + iy - y;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  int32_t* cu = plan_smem;          // [B + 1]
  int32_t* off = cu + a.B + 1;      // [B]
  int32_t* have = off + a.B;        // [B]
  __shared__ int s_used;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool first = blockIdx.x == 0;   // the CTA that reports a request's faults
  if (tid == 0) s_used = 0;

  int head = a.free_head ? __ldg(a.free_head) : 0;
  if (head < 0 || head > a.num_free) {
    if (first && tid == 0) report_error(16 /* PLX_DEVERR_NO_PAGES */);
    head = a.num_free;
  }
  const long long avail = a.num_free - head;

  // A thread takes a run of requests; rows and pages in 64 bits, since
  // lengths that break the rules may add up to anything.
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long nrow = 0, npage = 0;
  for (int b = b0; b < b1; ++b) {
    const long long c = __ldg(a.cached + b), n = __ldg(a.fresh + b);
    nrow += n > 0 ? n : 0;
    if (c >= 0 && n >= 0 && c + n <= (long long)a.max_pages * kPage) npage += (c + n + kPage - 1) / kPage - (c + kPage - 1) / kPage;
  }
  long long trow, tpage;
  block_scan2(nrow, npage, trow, tpage);
  for (int b = b0; b < b1; ++b) {
    const long long c = __ldg(a.cached + b), n = __ldg(a.fresh + b);
    const long long end = nrow + (n > 0 ? n : 0);
    const bool valid = c >= 0 && n >= 0 && c + n <= (long long)a.max_pages * kPage;
    const long long need = valid ? (c + n + kPage - 1) / kPage - (c + kPage - 1) / kPage : 0;
    // Once rows or pages run out, they do for every later request that needs
    // any, so the pages handed out are a prefix of the sum.
    const bool fits = n <= 0 || end <= a.rows, granted = need == 0 || npage + need <= avail;
    const bool ok = valid && fits && granted;
    cu[b] = (int)min(nrow, (long long)a.rows);
    off[b] = (int)min(npage, (long long)INT32_MAX);
    have[b] = ok ? (int)c : -1;
    if (first) {
      if (!valid || !fits) report_error(4 /* PLX_DEVERR_BAD_LENGTH */);
      else if (!granted) report_error(16 /* PLX_DEVERR_NO_PAGES */);
      a.seq_lens[b] = ok ? (int)(c + n) : 0;
      a.cu[b] = cu[b];
      if (need > 0 && ok) atomicMax(&s_used, (int)(npage + need));
    }
    nrow = end;
    npage += need;
  }
  if (tid == 0) cu[a.B] = (int)min(trow, (long long)a.rows);
  __syncthreads();
  if (first && tid == 0) {
    a.cu[a.B] = cu[a.B];
    *a.used = s_used;
  }

  // New table entries: a warp per request.
  const int lane = tid & 31, nwarps = gridDim.x * (kPlanThreads / 32);
  for (int b = blockIdx.x * (kPlanThreads / 32) + (tid >> 5); b < a.B; b += nwarps) {
    const int c = have[b];
    if (c < 0) continue;
    const int n = cu[b + 1] - cu[b];
    const int p0 = (c + kPage - 1) / kPage, p1 = (int)(((long long)c + n + kPage - 1) / kPage);
    for (int i = p0 + lane; i < p1; i += 32) {
      int page = __ldg(a.free_pages + head + off[b] + (i - p0));
      if (page < 0 || page >= a.num_pages) {
        report_error(1 /* PLX_DEVERR_BAD_PAGE */);
        page = -1;
      }
      a.table[(size_t)b * a.max_pages + i] = page;
    }
  }

  // Rows.
  const int live = cu[a.B];
  for (long long r = (long long)blockIdx.x * kPlanThreads + tid; r < a.rows; r += (long long)gridDim.x * kPlanThreads) {
    int pos = -1;
    long long slot = -1;
    if (r < live) {
      int lo = 0, hi = a.B - 1;   // last request with cu[b] <= r
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= r) lo = mid; else hi = mid - 1;
      }
      const int c = have[lo];
      if (c >= 0) {
        pos = c + (int)r - cu[lo];
        const int p0 = (c + kPage - 1) / kPage, i = pos / kPage;
        const int page = i < p0 ? a.table[(size_t)lo * a.max_pages + i]
                                : __ldg(a.free_pages + head + off[lo] + (i - p0));
        if (page < 0 || page >= a.num_pages)
          report_error(1 /* PLX_DEVERR_BAD_PAGE */);
        else
          slot = (long long)page * kPage + pos % kPage;
      }
    }
    a.slots[r] = slot;
    a.positions[r] = pos;
  }
}

}  // namespace plx
