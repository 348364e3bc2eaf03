// Page tables and slot maps built on the GPU from request lengths, and the
// return of pages (include/sd_kv8.h: sd_pages_extend, sd_pages_release).
//
// Both are a prefix sum over the batch followed by an independent fill, and
// their bytes are few (4 per new token and 8 per new page), so a call is
// bound by its latency: one launch, in which every CTA repeats the prefix
// sums of the at most 256 sequences (one load round and a block scan) instead
// of waiting for another kernel's, then writes its share of the page entries
// and of the slot map.  The inputs are never written, so no CTA sees another's
// half-done state; outputs are separate arrays.
//
// The free list is a stack: entry e (in batch order) of the pages that a call
// takes is free_list[count - 1 - e], so page p of a sequence can be computed
// by whoever needs it, without the page table having been written.
#include "common.cuh"
#include "kernels.h"

namespace sdv {
namespace {

constexpr int kPagesThreads = 256;   // one thread per sequence in the prefix sums (SD_MAX_BATCH)
constexpr int kPathThreads = 1024;   // with accepted paths: one CTA, which must have seen every path first
static_assert(kPagesThreads >= kMaxBatch, "one thread per sequence");

// Inclusive sums of two 64-bit values over the block's first 256 threads
// (eight warps); every thread of the block calls it.
__device__ __forceinline__ void scan2(long long& a, long long& b) {
  __shared__ long long wa[8], wb[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long ua = __shfl_up_sync(0xffffffffu, a, d), ub = __shfl_up_sync(0xffffffffu, b, d);
    if (lane >= d) { a += ua; b += ub; }
  }
  if (lane == 31 && warp < 8) { wa[warp] = a; wb[warp] = b; }
  __syncthreads();
  if (warp < 8)
    for (int w = 0; w < warp; ++w) { a += wa[w]; b += wb[w]; }
}

// Sequence of element e: the last b with start[b] <= e (starts never fall; start[0] = 0).
__device__ __forceinline__ int find_seq(const int* start, int batch, int e) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= e) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Page j of sequence b after the call, without the page table having been written.
__device__ __forceinline__ int page_of(const PagesParams& p, const int* held, const int* first_new, int count, int b, int j) {
  return j < held[b] ? p.page_table[(size_t)b * p.max_pages + j] : p.free_list[count - 1 - (first_new[b] + j - held[b])];
}

template <bool PATH>
__global__ void __launch_bounds__(PATH ? kPathThreads : kPagesThreads)
pages_extend_kernel(const PagesParams p, const BatchDesc bd) {
  __shared__ int s_row[kMaxBatch + 1], s_page[kMaxBatch + 1];   // first row / first new page of each sequence
  __shared__ int s_ctx[kMaxBatch], s_held[kMaxBatch];
  __shared__ int s_bad;
  const int t = threadIdx.x, B = p.batch;
  const int count = *p.free_count;
  int ctx = 0, add = 0, held = 0;
  if (t < B) { ctx = p.ctx_lens[t]; add = p.add_lens[t]; held = p.held[t]; }
  if (t == 0) s_bad = 0;
  __syncthreads();
  int bad = 0;
  const long long most = (long long)p.max_pages * kPage;
  if (t < B && (ctx < 0 || add < 0 || (long long)ctx + add > most || held < 0 || held > p.max_pages ||
                (long long)held * kPage < ctx)) {
    bad |= SD_DEV_BAD_CTX;
    ctx = add = held = 0;
  }
  if (PATH && t < B && (add > p.max_path || add > bd.q_indptr[t + 1] - bd.q_indptr[t])) {
    bad |= SD_DEV_BAD_ACCEPT;
    add = 0;
  }
  const int need = max(held, (int)(((long long)ctx + add + kPage - 1) / kPage));
  long long rows = add, pages = need - held;
  scan2(rows, pages);
  // the totals decide before they are cut to 32 bits
  if (t == B - 1) {
    if (rows > p.max_rows) bad |= SD_DEV_BAD_SLOT;
    if (count < 0 || count > p.num_pool_pages || pages > count) bad |= SD_DEV_NO_PAGES;
  }
  if (t < B) {
    if (t == 0) s_row[0] = s_page[0] = 0;
    s_row[t + 1] = (int)min(rows, (long long)INT_MAX);
    s_page[t + 1] = (int)min(pages, (long long)INT_MAX);
    s_ctx[t] = ctx;
    s_held[t] = held;
  }
  if (PATH) {
    // every accepted node of the batch, before anything is written
    __syncthreads();
    const int n = min(s_row[B], p.max_rows);
    for (int r = t; r < n; r += blockDim.x) {
      const int b = find_seq(s_row, B, r);
      const int i = r - s_row[b], node = p.path[(size_t)b * p.max_path + i];
      if (node < 0 || node >= bd.q_indptr[b + 1] - bd.q_indptr[b]) bad |= SD_DEV_BAD_ACCEPT;
    }
  }
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  const bool ok = s_bad == 0;
  if (blockIdx.x == 0) {
    if (t == 0) {
      if (!ok) report(p.dev_status, s_bad);
      *p.new_free_count = ok ? count - s_page[B] : count;
    }
    if (t < B) {
      p.new_held[t] = ok ? need : p.held[t];
      if (p.new_ctx_lens != nullptr) p.new_ctx_lens[t] = ok ? ctx + add : p.ctx_lens[t];
    }
    if (p.row_indptr != nullptr)
      for (int b = t; b <= B; b += blockDim.x) p.row_indptr[b] = ok ? s_row[b] : 0;
  }
  const int step = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + t;
  if (ok) {
    const int n_new = s_page[B];
    for (int e = first; e < n_new; e += step) {
      const int b = find_seq(s_page, B, e);
      p.page_table[(size_t)b * p.max_pages + s_held[b] + (e - s_page[b])] = p.free_list[count - 1 - e];
    }
  }
  // The slot map: a warp takes 512 consecutive rows at a time, a lane four quads of rows (one 16-byte store each, lanes
  // side by side) whose page lookups are all in flight together; behind the last row: -1.  The warp searches its first
  // row's sequence once, lanes walk on from there.
  const int n_rows = ok ? s_row[B] : 0;
  bool bad_page = false;
  constexpr int U = 4;
  const int lane = t & 31;
  for (long long w0 = (long long)(first - lane) * (4 * U); w0 < p.max_rows; w0 += (long long)step * (4 * U)) {
    int b0 = w0 < n_rows ? find_seq(s_row, B, (int)w0) : 0;
    int seq[U], pos[U], page[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = w0 + 128 * u + 4 * lane;
      seq[u] = -1;
      if (r < n_rows) {
        while ((int)r >= s_row[b0 + 1]) ++b0;      // ends: r < s_row[B]
        seq[u] = b0;
        pos[u] = s_ctx[b0] + (int)r - s_row[b0];
        page[u] = page_of(p, s_held, s_page, count, b0, pos[u] / kPage);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r0 = w0 + 128 * u + 4 * lane;
      int slot[4], src[4];
      int b = seq[u], j = b >= 0 ? pos[u] / kPage : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const long long r = r0 + k;
        slot[k] = src[k] = -1;
        if (r < n_rows) {
          int at = b;
          while ((int)r >= s_row[at + 1]) ++at;
          const int i = (int)r - s_row[at], x = s_ctx[at] + i;
          if (at != b || x / kPage != j) {         // the quad ends a page or a sequence
            b = at;
            j = x / kPage;
            page[u] = page_of(p, s_held, s_page, count, b, j);
          }
          const bool in = page[u] >= 0 && page[u] < p.num_pool_pages;
          bad_page |= !in;
          slot[k] = in ? page[u] * kPage + x % kPage : -1;
          src[k] = PATH ? bd.q_indptr[at] + p.path[(size_t)at * p.max_path + i] : (int)r;
        }
      }
      if (r0 + 4 <= p.max_rows && p.vec) {
        *reinterpret_cast<int4*>(p.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        if (p.rows != nullptr) *reinterpret_cast<int4*>(p.rows + r0) = make_int4(src[0], src[1], src[2], src[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r0 + k < p.max_rows) {
            p.slots[r0 + k] = slot[k];
            if (p.rows != nullptr) p.rows[r0 + k] = src[k];
          }
      }
    }
  }
  if (bad_page) report(p.dev_status, SD_DEV_BAD_PAGE);
}

__global__ void __launch_bounds__(kPagesThreads) pages_release_kernel(const PagesParams p) {
  __shared__ int s_page[kMaxBatch + 1], s_keep[kMaxBatch];
  __shared__ int s_bad;
  const int t = threadIdx.x, B = p.batch;
  const int count = *p.free_count;
  int keep_len = 0, held = 0, bad = 0;
  if (t < B) { keep_len = p.ctx_lens[t]; held = p.held[t]; }
  if (t == 0) s_bad = 0;
  __syncthreads();
  const int held_in = held;
  if (keep_len < 0 || held < 0 || held > p.max_pages) { bad |= SD_DEV_BAD_CTX; keep_len = held = 0; }
  const int keep = min(held, (int)(((long long)keep_len + kPage - 1) / kPage));
  long long pages = held - keep, unused = 0;
  scan2(pages, unused);
  if (t == B - 1 && (count < 0 || count + pages > p.num_pool_pages)) bad |= SD_DEV_BAD_PAGE;
  if (t < B) {
    if (t == 0) s_page[0] = 0;
    s_page[t + 1] = (int)min(pages, (long long)INT_MAX);
    s_keep[t] = keep;
  }
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  const bool ok = s_bad == 0;
  if (blockIdx.x == 0) {
    if (t == 0) {
      if (!ok) report(p.dev_status, s_bad);
      *p.new_free_count = ok ? count + s_page[B] : count;
    }
    if (t < B) p.new_held[t] = ok ? keep : held_in;
  }
  if (!ok) return;
  const int n = s_page[B];
  bool bad_page = false;
  for (int e = blockIdx.x * blockDim.x + t; e < n; e += gridDim.x * blockDim.x) {
    const int b = find_seq(s_page, B, e);
    const int page = p.page_table[(size_t)b * p.max_pages + s_keep[b] + (e - s_page[b])];
    bad_page |= page < 0 || page >= p.num_pool_pages;
    p.free_list_out[count + e] = page;
  }
  if (bad_page) report(p.dev_status, SD_DEV_BAD_PAGE);
}

int blocks_for(long long elements, int per_block) {
  const long long n = (elements + per_block - 1) / per_block;
  return (int)(n < 1 ? 1 : n > 8 * kSMs ? 8 * kSMs : n);   // one wave at most
}

}  // namespace

cudaError_t launch_pages_extend(const PagesParams& p, const BatchDesc& bd, cudaStream_t st) {
  if (p.path != nullptr)
    pages_extend_kernel<true><<<1, kPathThreads, 0, st>>>(p, bd);
  else
    pages_extend_kernel<false><<<blocks_for(p.max_rows, 16 * kPagesThreads), kPagesThreads, 0, st>>>(p, bd);
  return cudaGetLastError();
}

cudaError_t launch_pages_release(const PagesParams& p, cudaStream_t st) {
  pages_release_kernel<<<blocks_for((long long)p.batch * p.max_pages, 2 * kPagesThreads), kPagesThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace sdv
