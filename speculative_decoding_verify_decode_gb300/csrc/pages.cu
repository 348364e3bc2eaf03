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
__global__ void __launch_bounds__(PATH ? kPathThreads : kPagesThreads, PATH ? 1 : 6)
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
  const unsigned n_rows = ok ? (unsigned)s_row[B] : 0u, max_rows = (unsigned)p.max_rows;
  bool bad_page = false;
  constexpr unsigned U = 4;
  const unsigned lane = t & 31;
  auto slot_of = [&](int page, unsigned pos) {
    const bool in = (unsigned)page < (unsigned)p.num_pool_pages;
    bad_page |= !in;
    return in ? page * kPage + (int)(pos % kPage) : -1;
  };
  // first * 16 rows is below 2^31 for every warp with work; the step keeps within 2^32 of it
  for (unsigned w0 = ((unsigned)first - lane) * (4 * U); w0 < max_rows; w0 += (unsigned)step * (4 * U)) {
    const int b0 = w0 < n_rows ? find_seq(s_row, B, (int)w0) : 0;
    int seq[U], page[U], page2[U];
    unsigned pos[U];
#pragma unroll
    for (unsigned u = 0; u < U; ++u) {
      const unsigned r = w0 + 128 * u + 4 * lane;
      seq[u] = -1;
      pos[u] = 0;
      page[u] = page2[u] = -1;
      if (r < n_rows) {
        const int b = (int)r < s_row[b0 + 1] ? b0 : find_seq(s_row, B, (int)r);
        seq[u] = b;
        pos[u] = (unsigned)(s_ctx[b] + (int)r - s_row[b]);
        page[u] = page_of(p, s_held, s_page, count, b, (int)(pos[u] / kPage));
        // the page that the quad's last row lands on, if it is another and the sequence's
        if (pos[u] % kPage > kPage - 4 && (int)r + 3 < s_row[b + 1])
          page2[u] = page_of(p, s_held, s_page, count, b, (int)(pos[u] / kPage) + 1);
      }
    }
#pragma unroll
    for (unsigned u = 0; u < U; ++u) {
      const unsigned r0 = w0 + 128 * u + 4 * lane;
      if (r0 >= max_rows) break;
      int slot[4] = {-1, -1, -1, -1}, src[4] = {-1, -1, -1, -1};
      const int b = seq[u];
      if (b >= 0 && (int)r0 + 3 < s_row[b + 1]) {      // four rows of one sequence, on one page or two
#pragma unroll
        for (unsigned k = 0; k < 4; ++k) {
          slot[k] = slot_of(pos[u] % kPage + k < kPage ? page[u] : page2[u], pos[u] + k);
          src[k] = PATH ? bd.q_indptr[b] + p.path[(size_t)b * p.max_path + ((int)(r0 + k) - s_row[b])] : (int)(r0 + k);
        }
      } else if (b >= 0) {                             // a sequence, or all rows, end in the quad
        int at = b;
#pragma unroll 1
        for (unsigned k = 0; k < 4 && r0 + k < n_rows; ++k) {
          const int r = (int)(r0 + k);
          while (r >= s_row[at + 1]) ++at;             // ends: r < s_row[B]
          const unsigned x = (unsigned)(s_ctx[at] + r - s_row[at]);
          const int s = slot_of(page_of(p, s_held, s_page, count, at, (int)(x / kPage)), x);
          const int from = PATH ? bd.q_indptr[at] + p.path[(size_t)at * p.max_path + (r - s_row[at])] : r;
#pragma unroll
          for (unsigned e = 0; e < 4; ++e) {
            slot[e] = e == k ? s : slot[e];
            src[e] = e == k ? from : src[e];
          }
        }
      }
      if (max_rows - r0 >= 4 && p.vec) {
        *reinterpret_cast<int4*>(p.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        if (p.rows != nullptr) *reinterpret_cast<int4*>(p.rows + r0) = make_int4(src[0], src[1], src[2], src[3]);
      } else {
#pragma unroll
        for (unsigned k = 0; k < 4; ++k)
          if (k < max_rows - r0) {
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
  return (int)(n < 1 ? 1 : n > 6 * kSMs ? 6 * kSMs : n);   // one wave at most
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
