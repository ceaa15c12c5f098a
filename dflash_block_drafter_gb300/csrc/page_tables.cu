// Page tables and slot maps of requests whose lengths only the device knows
// (dflash_page_tables in include/dflash.h).
//
// Per request: need = ceil((length + new_rows) / page); it takes need - held
// pages from the ring of free pages or gives held - need back.  Which page is
// whose, and where a request's rows lie, are prefix sums over the requests.
// The work is a few bytes per request and per row, so launches are what it
// costs: one launch does it all.  Every CTA forms the prefix sums of all
// requests in its own shared memory (at most kMaxRequests of them), then the
// rows (four neighbours a thread, for one search and one store), taken pages
// and given pages are shared out over all CTAs, each item finding its request
// by binary search.  The CTAs form one cluster, whose barrier orders their
// last read of held / ring_state before the first CTA updates them, so that
// both may be updated in place.
// Measured (cold caches): 16 requests with 8 rows each 7 to 9 us, 2000 requests with
// 194,000 rows 18 us (8 CTAs with a row a thread: 41).
#include "common.cuh"
#include "internal.h"
#include "kernels.h"

namespace dflash {
namespace {

constexpr int kMaxRequests = 4096;
constexpr int kThreads = 1024;
constexpr int kCluster = 16;  // CTAs at most

struct PageArgs {
  const int32_t* lengths;
  const int32_t* new_rows;
  int n_seq, page_shift, n_pages;
  const int32_t* held_in;
  int32_t* held_out;
  int32_t* table;
  int table_stride;
  int32_t* ring;
  const int32_t* ring_in;
  int32_t* ring_out;
  int32_t* row_offsets;
  int32_t* slots;
  int32_t* positions;
  int row_cap;
  int32_t* status;
};

__device__ __forceinline__ int saturate(long long v) { return v > 0x7fffffffll ? 0x7fffffff : static_cast<int>(v); }

// What a request asks for.
struct Request {
  bool valid, fits;  // in play; its pages fit the table's width
  int held, need, rows;
};
__device__ __forceinline__ Request request(const PageArgs& a, int s) {
  Request q;
  const int len = a.lengths[s], rows = a.new_rows[s];
  q.valid = len >= 0 && rows >= 0;
  q.held = min(max(a.held_in[s], 0), a.table_stride);
  const long long total = static_cast<long long>(len) + rows;
  const long long need = q.valid ? (total + (1 << a.page_shift) - 1) >> a.page_shift : 0;
  q.fits = q.valid && need <= a.table_stride;
  q.need = q.fits ? static_cast<int>(need) : q.held;
  q.rows = q.valid ? rows : 0;
  return q;
}

// First s with end[s] > x (end ascending, x < end[n - 1]).
__device__ __forceinline__ int upper(const int* end, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_tables_kernel(const PageArgs a) {
  // [5][n_seq]: rows, pages taken, pages given, up to and with a request; its
  // length; its pages held before (their complement where it has no place in
  // the table)
  extern __shared__ int ends[];
  __shared__ long long part[3][33];
  __shared__ int s_taken;
  int* row_end = ends;
  int* take_end = ends + a.n_seq;
  int* give_end = ends + 2 * a.n_seq;
  int* s_len = ends + 3 * a.n_seq;
  int* s_held = ends + 4 * a.n_seq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x;  // one cluster: the grid is the cluster
  const int head = a.ring_in[0], free_pages = min(max(a.ring_in[1], 0), a.n_pages);
  const int ring0 = head >= 0 && head < a.n_pages ? head : 0;
  if (tid == 0) {
    s_taken = 0;
    if (rank == 0 && (ring0 != head || free_pages != a.ring_in[1])) set_status(a.status, DFLASH_DEV_CAPACITY);
  }
  long long carry[3] = {0, 0, 0};
  for (int s0 = 0; s0 < a.n_seq; s0 += kThreads) {
    const int s = s0 + tid;
    long long v[3] = {0, 0, 0};
    if (s < a.n_seq) {
      const Request q = request(a, s);
      v[0] = q.rows;
      v[1] = max(q.need - q.held, 0);
      v[2] = max(q.held - q.need, 0);
      s_len[s] = a.lengths[s];
      s_held[s] = q.fits ? q.held : ~q.held;
      if (rank == 0 && ((q.valid && !q.fits) || q.held != a.held_in[s])) set_status(a.status, DFLASH_DEV_CAPACITY);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const long long u = __shfl_up_sync(0xffffffffu, v[j], o);
        if (lane >= o) v[j] += u;
      }
    if (lane == 31)
      for (int j = 0; j < 3; ++j) part[j][warp] = v[j];
    __syncthreads();
    if (warp < 3) {  // warp j: prefix sums of the warps' totals of quantity j
      long long x = part[warp][lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
      }
      __syncwarp();
      part[warp][lane + 1] = x;
      if (lane == 0) part[warp][0] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      if (s < a.n_seq) ends[j * a.n_seq + s] = saturate(carry[j] + part[j][warp] + v[j]);
      carry[j] += part[j][32];
    }
    __syncthreads();
  }
  // requests whose pages are all there get them: those up to the first that
  // asks for more than is left, and those that ask for none
  for (int s = tid; s < a.n_seq; s += kThreads)
    if (take_end[s] <= free_pages) atomicMax(&s_taken, take_end[s]);
  __syncthreads();
  const int taken = s_taken;
  const int rows = saturate(carry[0]);
  const int given_all = saturate(carry[2]);
  const int given = min(given_all, a.n_pages - free_pages);  // more: a page was both free and held
  if (rank == 0 && tid == 0 && (rows > a.row_cap || given < given_all || carry[1] > free_pages))
    set_status(a.status, DFLASH_DEV_CAPACITY);
  const int t0 = rank * kThreads + tid, step = gridDim.x * kThreads;
  bool bad = false;
  // pages taken: ring -> table
  for (int i = t0; i < taken; i += step) {
    const int s = upper(take_end, a.n_seq, i);
    const int first = s ? take_end[s - 1] : 0;
    int at = ring0 + i;
    if (at >= a.n_pages) at -= a.n_pages;
    a.table[static_cast<size_t>(s) * a.table_stride + s_held[s] + (i - first)] = a.ring[at];
  }
  // pages given back: table -> ring's tail
  for (int i = t0; i < given; i += step) {
    const int s = upper(give_end, a.n_seq, i);
    const int first = s ? give_end[s - 1] : 0;
    const int need = s_held[s] - (give_end[s] - first);
    const int page = a.table[static_cast<size_t>(s) * a.table_stride + need + (i - first)];
    long long at = static_cast<long long>(ring0) + free_pages + i;
    at -= at >= a.n_pages ? a.n_pages : 0;
    at -= at >= a.n_pages ? a.n_pages : 0;
    a.ring[at] = page;
    bad |= page < 0 || page >= a.n_pages;
  }
  // slots and positions of the rows
  const bool wide = (reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) % 16 == 0;
  for (long long r0 = 4ll * t0; r0 < a.row_cap; r0 += 4ll * step) {
    int slot[4], pos[4];
    int s = r0 < rows ? upper(row_end, a.n_seq, static_cast<int>(r0)) : 0;
    int seen_s = -1, seen_p = -1, page = -1;  // the page looked up last
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long r = r0 + j;
      slot[j] = pos[j] = -1;
      if (r >= rows || r >= a.row_cap) continue;
      while (row_end[s] <= r) ++s;
      const int before = s ? row_end[s - 1] : 0, held = s_held[s];
      const int take0 = s ? take_end[s - 1] : 0, take1 = take_end[s];
      pos[j] = saturate(s_len[s] + (r - before));
      if (held < 0 || (take1 > take0 && take1 > free_pages)) continue;
      const int p = pos[j] >> a.page_shift;
      if (s != seen_s || p != seen_p) {
        if (p < held) {
          page = a.table[static_cast<size_t>(s) * a.table_stride + p];
        } else {
          int at = ring0 + take0 + (p - held);
          if (at >= a.n_pages) at -= a.n_pages;
          page = a.ring[at];
        }
        seen_s = s;
        seen_p = p;
      }
      if (page >= 0 && page < a.n_pages) slot[j] = (page << a.page_shift) + (pos[j] & ((1 << a.page_shift) - 1));
      else bad = true;
    }
    if (wide && r0 + 4 <= a.row_cap) {
      *reinterpret_cast<int4*>(a.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.positions) *reinterpret_cast<int4*>(a.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int j = 0; j < 4 && r0 + j < a.row_cap; ++j) {
        a.slots[r0 + j] = slot[j];
        if (a.positions) a.positions[r0 + j] = pos[j];
      }
    }
  }
  if (bad) set_status(a.status, DFLASH_DEV_CAPACITY);
  // every CTA has read what the first now updates
  if (gridDim.x > 1) {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (rank != 0) return;
  for (int s = tid; s < a.n_seq; s += kThreads) {
    const int take0 = s ? take_end[s - 1] : 0, take1 = take_end[s], give0 = s ? give_end[s - 1] : 0;
    const int held = s_held[s];
    a.held_out[s] = held < 0 ? ~held : take1 == take0 ? held - (give_end[s] - give0) : take1 <= free_pages ? held + take1 - take0 : held;
    a.row_offsets[s + 1] = row_end[s];
  }
  if (tid == 0) {
    a.row_offsets[0] = 0;
    int h = ring0 + taken;
    if (h >= a.n_pages) h -= a.n_pages;
    a.ring_out[0] = h;
    a.ring_out[1] = free_pages - taken + given;
  }
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_page_tables(const int32_t* lengths, const int32_t* new_rows, int32_t n_seq, int32_t page_size,
                                  int32_t n_pages, const int32_t* held_in, int32_t* held_out, int32_t* table,
                                  int32_t table_stride, int32_t* ring, const int32_t* ring_in, int32_t* ring_out,
                                  int32_t* row_offsets, int32_t* slots, int32_t* positions, int32_t row_cap,
                                  int32_t* dev_status, dflash_stream_t stream) {
  if (!lengths || !new_rows || !held_in || !held_out || !table || !ring || !ring_in || !ring_out || !row_offsets)
    return DFLASH_ERR_INVALID_ARG;
  if (n_seq < 1 || table_stride < 1 || n_pages < 1 || row_cap < 0 || (row_cap > 0 && !slots))
    return DFLASH_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return DFLASH_ERR_UNSUPPORTED;
  // (n_seq * table_stride: the sums of pages taken and given back stay within 31 bits)
  if (n_seq > kMaxRequests || static_cast<long long>(n_pages) * page_size > 0x7fffffffll ||
      static_cast<long long>(n_seq) * table_stride >= 0x7fffffffll)
    return DFLASH_ERR_CAPACITY;
  PageArgs a{lengths, new_rows, n_seq, 0, n_pages, held_in, held_out, table, table_stride, ring, ring_in, ring_out,
             row_offsets, slots, positions, row_cap, dev_status};
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  cudaLaunchConfig_t cfg = {};
  // a CTA for every 4096 rows: one for a decoding step, the largest cluster for prompts
  int ctas = 1;
  while (ctas < kCluster && row_cap > 4 * kThreads * ctas) ctas *= 2;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 5 * sizeof(int) * n_seq;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  cudaError_t e = cudaSuccess;
  if (cfg.dynamicSmemBytes > 40 * 1024)
    e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             5 * static_cast<int>(sizeof(int)) * kMaxRequests);
  if (e == cudaSuccess && ctas > 8)  // beyond the portable size
    e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return cuda_status(e, "page tables");
  return cuda_status(cudaLaunchKernelEx(&cfg, page_tables_kernel, a), "page tables");
}
