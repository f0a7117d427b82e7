// Bookkeeping of a paged KV cache on the device: copying, growing, forking, freeing and
// compacting pages.
//
// The state is the caller's: ref[n_pages] (how many lists hold each page; 0: free) and the page
// lists (page_indptr, page_indices) of the paged decode. Free pages are always taken lowest
// number first, in the order of the requests, so the result does not depend on timing; counts
// of holders are changed by integer atomics alone. The searches are one CTA's scan of the counts (4 bytes
// a page: 131 KB for 32768 pages), bound by latency and the launch, not by bytes; the copies are bound
// by HBM.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace sta {
namespace {

constexpr int kThreads = 256;
constexpr int kScanThreads = 1024;
constexpr int kMaxBufs = 256;        // cache buffers of one launch
constexpr int kSlice = 16384;        // bytes of a page that a CTA copies at a time
// CTAs of a copy: 3 an SM, whose slices in flight fill the memory system (a pool of 8 buffers compacted,
// 409 MB read and as much written: 142.5 us; with 2 an SM 157, with 4 146, with 6 148.6)
constexpr int kCopyCtas = 152 * 3;

struct PageBufs {
  uint8_t* p[kMaxBufs];
};

struct Lists {
  int32_t* ref;
  const int32_t* indptr;
  int32_t* indices;
  const int32_t* kv_indptr;
  int n_pages, n_req, page_size;
  int* err;
};

__device__ __forceinline__ int pages_of(int64_t tokens, int page) {
  return tokens > 0 ? (int)((tokens + page - 1) / page) : 0;
}
__device__ __forceinline__ int64_t tokens_of(const int32_t* kv_indptr, int r) {
  return (int64_t)__ldg(kv_indptr + r + 1) - __ldg(kv_indptr + r);
}

// Exclusive prefix of v over the block (1024 threads) and its total.
__device__ __forceinline__ int block_scan(int v, int& total, int* s_warp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();  // s_warp free
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  const int w = s_warp[lane];  // 32 warps
  int wi = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) wi += x;
  }
  total = __shfl_sync(0xffffffffu, wi, 31);
  const int before = __shfl_sync(0xffffffffu, wi - w, warp);
  return before + incl - v;
}

// Copies page src[i] onto page dst[i] of every buffer (a negative number: no copy). With page_map,
// first the entries that the requests hold take their pages' new numbers, `runs` warps a request.
__global__ void __launch_bounds__(kThreads) pages_copy_kernel(const __grid_constant__ PageBufs bufs, int n_bufs,
                                                              int64_t page_bytes, int n_pages, const int32_t* src,
                                                              const int32_t* dst, int n, const int32_t* n_dev,
                                                              const Lists L, const int32_t* page_map, int runs, int* err) {
  if (page_map) {
    const int lane = threadIdx.x & 31, warps = gridDim.x * (kThreads / 32);
    for (int64_t w = (blockIdx.x * kThreads + threadIdx.x) >> 5; w < (int64_t)L.n_req * runs; w += warps) {
      const int r = (int)(w / runs), b = __ldg(L.indptr + r);
      const int held = min(pages_of(tokens_of(L.kv_indptr, r), L.page_size), __ldg(L.indptr + r + 1) - b);
      for (int k = (int)(w % runs) * 32 + lane; k < held; k += 32 * runs) {
        const int page = L.indices[b + k];
        if (page < 0) continue;  // no page: there was none left when the request grew
        if (page >= n_pages) record_error(err, 0x601);
        else L.indices[b + k] = __ldg(page_map + page);
      }
    }
  }
  const int slices = (int)((page_bytes + kSlice - 1) / kSlice);
  const int64_t pairs = n_dev ? min(n, __ldg(n_dev)) : n;
  const int64_t items = pairs * n_bufs * slices;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t pair = it / ((int64_t)n_bufs * slices);
    const int rest = (int)(it - pair * n_bufs * slices), b = rest / slices, sl = rest - b * slices;
    const int s = src[pair], d = dst[pair];
    if (s < 0 || d < 0 || s == d) continue;
    if (s >= n_pages || d >= n_pages) {
      if (threadIdx.x == 0) record_error(err, 0x601);
      continue;
    }
    const int64_t off = (int64_t)sl * kSlice;
    const uint4* from = reinterpret_cast<const uint4*>(bufs.p[b] + s * page_bytes + off);
    uint4* to = reinterpret_cast<uint4*>(bufs.p[b] + d * page_bytes + off);
    const int nv = (int)(min((int64_t)kSlice, page_bytes - off) >> 4);
    uint4 v[kSlice / 16 / kThreads];
#pragma unroll
    for (int u = 0; u < kSlice / 16 / kThreads; ++u)
      if (threadIdx.x + u * kThreads < nv) v[u] = __ldg(from + threadIdx.x + u * kThreads);
#pragma unroll
    for (int u = 0; u < kSlice / 16 / kThreads; ++u)
      if (threadIdx.x + u * kThreads < nv) to[threadIdx.x + u * kThreads] = v[u];
  }
}

// Bit e: page p + e (of 16) is there and its count is 0 (free) or, with `live`, above 0. Counts are read
// 16 bytes at a time where they are aligned and 16 are left (32768 pages searched and 256 requests grown
// and freed: 17.5 us, 21.2 one by one), else one by one.
__device__ __forceinline__ uint32_t page_bits(const Lists& L, int p, bool live) {
  uint32_t bits = 0;
  if (p + 16 <= L.n_pages && !((uintptr_t)L.ref & 15)) {
    int4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const int4*>(L.ref + p + 4 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) bits |= (uint32_t)(live ? x[e] > 0 : x[e] == 0) << (4 * i + e);
    }
  } else {
    for (int e = 0; e < 16 && p + e < L.n_pages; ++e) bits |= (uint32_t)(live ? L.ref[p + e] > 0 : L.ref[p + e] == 0) << e;
  }
  return bits;
}

// The lowest free pages, ascending, into taken[0 .. want): returns how many there are. 16 pages a
// thread and step.
__device__ int take_free(const Lists& L, int want, int32_t* taken, int* s_warp) {
  int found = 0;
  for (int64_t p0 = 0; p0 < L.n_pages && found < want; p0 += 16 * kScanThreads) {
    const int p = (int)min(p0 + 16 * (int)threadIdx.x, (int64_t)L.n_pages);
    uint32_t bits = page_bits(L, p, false);
    int total;
    int k = found + block_scan(__popc(bits), total, s_warp);
    for (; bits && k < want; bits &= bits - 1, ++k) taken[k] = p + __ffs(bits) - 1;
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

// Entries that request r gains when it grows from old to now tokens (0 when its list is too short).
__device__ __forceinline__ int grow_want(const Lists& L, const int32_t* now, int r, int& first) {
  first = pages_of(tokens_of(L.kv_indptr, r), L.page_size);
  const int n = pages_of(tokens_of(now, r), L.page_size);
  if (n <= first) return 0;
  if (n > __ldg(L.indptr + r + 1) - __ldg(L.indptr + r)) {
    record_error(L.err, 0x604);
    return 0;
  }
  return n - first;
}

// One block. The requests' wants are added up, the pages taken, then the lists filled, 1024 requests at
// a time: the block runs over all their new entries, each looked up among the requests, so that one long
// prompt is no longer than many short ones. (8 requests of 940 to 1900 pages leave and grow again: 21.6 us
// for both calls, 91 with a thread a request and a warp a freed list; 256 requests, 32 leaving: 17.5, 21.6
// before.)
__global__ void __launch_bounds__(kScanThreads) pages_grow_kernel(const Lists L, const int32_t* now, int32_t* taken,
                                                                  int32_t* status) {
  __shared__ int s_warp[32];
  __shared__ int s_from[kScanThreads];  // a request's first new entry among the round's
  __shared__ int s_at[kScanThreads];    // and its place in the lists
  // a batch of no more than 1024 needs the wants only once
  const bool once = L.n_req <= kScanThreads;
  int want = 0, n = 0, k0 = 0, first = 0;
  for (int r0 = 0; r0 < L.n_req; r0 += kScanThreads) {
    const int r = r0 + threadIdx.x;
    int total;
    n = r < L.n_req ? grow_want(L, now, r, first) : 0;
    k0 = block_scan(n, total, s_warp);
    want += total;
  }
  const int got = take_free(L, want, taken, s_warp);
  int base = 0;
  for (int r0 = 0; r0 < L.n_req; r0 += kScanThreads) {
    const int r = r0 + threadIdx.x;
    int total = want;
    if (!once) {
      n = r < L.n_req ? grow_want(L, now, r, first) : 0;
      k0 = block_scan(n, total, s_warp);
    }
    s_from[threadIdx.x] = k0;
    s_at[threadIdx.x] = n > 0 ? __ldg(L.indptr + r) + first : 0;
    __syncthreads();
    for (int j = threadIdx.x; j < total; j += kScanThreads) {
      int q = 0;  // the last request of the round whose entries begin at or before j: one that gains some
#pragma unroll
      for (int step = kScanThreads / 2; step > 0; step >>= 1)
        if (s_from[q + step] <= j) q += step;
      const int k = base + j, page = k < got ? taken[k] : -1;
      L.indices[s_at[q] + (j - s_from[q])] = page;
      if (page >= 0) L.ref[page] = 1;
    }
    base += total;
    __syncthreads();
  }
  if (threadIdx.x == 0 && status) {
    status[0] = got;
    status[1] = want - got;
  }
}

// Fork i: the pages it shares and whether it needs a page of its own for a last, partly filled one.
__device__ __forceinline__ bool fork_of(const Lists& L, const int32_t* parent, const int32_t* child, int i, int& p,
                                        int& c, int& whole, int& part) {
  p = __ldg(parent + i);
  c = __ldg(child + i);
  if (p < 0 || p >= L.n_req || c < 0 || c >= L.n_req || p == c) {
    record_error(L.err, 0x602);
    return false;
  }
  if (tokens_of(L.kv_indptr, c) > 0) {  // the child holds pages of its own
    record_error(L.err, 0x605);
    return false;
  }
  const int64_t len = max((int64_t)0, tokens_of(L.kv_indptr, p));
  whole = (int)(len / L.page_size);
  part = len % L.page_size != 0;
  if (whole + part > __ldg(L.indptr + p + 1) - __ldg(L.indptr + p) ||
      whole + part > __ldg(L.indptr + c + 1) - __ldg(L.indptr + c)) {
    record_error(L.err, 0x604);
    return false;
  }
  return true;
}

// Block 0 takes the pages that partly filled last pages need and writes the copies to make;
// the other blocks share the whole pages, `runs` warps per fork. (A page is free or not before the
// call: sharing raises counts that are above zero already, so the two do not meet.) Of two
// forks onto one child the first counts.
__global__ void __launch_bounds__(kScanThreads) pages_fork_kernel(const Lists L, const int32_t* parent,
                                                                  const int32_t* child, int n, int32_t* taken,
                                                                  int32_t* src, int32_t* dst, int32_t* owner,
                                                                  int runs, int32_t* status) {
  __shared__ int s_warp[32];
  int p, c, whole, part;
  if (blockIdx.x > 0) {
    const int lane = threadIdx.x & 31;
    for (int64_t w = ((int)blockIdx.x - 1) * 32 + (int)(threadIdx.x >> 5); w < (int64_t)n * runs; w += ((int)gridDim.x - 1) * 32) {
      const int i = (int)(w / runs);
      if (!fork_of(L, parent, child, i, p, c, whole, part)) continue;
      bool again = false;
      for (int j = lane; j < i; j += 32) again |= __ldg(child + j) == c;
      if (__any_sync(0xffffffffu, again)) continue;
      for (int k = (int)(w % runs) * 32 + lane; k < whole; k += 32 * runs) {
        int page = L.indices[__ldg(L.indptr + p) + k];
        if (page < 0 || page >= L.n_pages) {
          record_error(L.err, 0x601);
          page = -1;
        } else {
          atomicAdd(L.ref + page, 1);
        }
        L.indices[__ldg(L.indptr + c) + k] = page;
      }
    }
    return;
  }
  for (int r = threadIdx.x; r < L.n_req; r += kScanThreads) owner[r] = INT32_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kScanThreads) {
    c = __ldg(child + i);
    if (c >= 0 && c < L.n_req) atomicMin(owner + c, i);
  }
  __syncthreads();
  // the page that fork i needs for a last, partly filled one (old: the parent's; without it there is
  // nothing to copy, so the child's entry holds no page either and none is taken)
  int old = -1;
  auto own_page = [&](int i) -> int {
    if (i >= n || !fork_of(L, parent, child, i, p, c, whole, part)) return 0;
    if (*(volatile int32_t*)(owner + c) != i) {
      record_error(L.err, 0x605);
      return 0;
    }
    if (!part) return 0;
    old = L.indices[__ldg(L.indptr + p) + whole];
    if (old >= 0 && old < L.n_pages) return 1;
    record_error(L.err, 0x601);
    L.indices[__ldg(L.indptr + c) + whole] = -1;
    return 0;
  };
  // then what the first look found is still there for the second (4 forks: 15.5 us, 17.5 looking twice)
  const bool once = n <= kScanThreads;
  int want = 0, w = 0, k = 0;
  for (int i0 = 0; i0 < n; i0 += kScanThreads) {
    int total;
    w = own_page(i0 + threadIdx.x);
    k = block_scan(w, total, s_warp);
    want += total;
  }
  const int got = take_free(L, want, taken, s_warp);
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += kScanThreads) {
    const int i = i0 + threadIdx.x;
    if (!once) {
      int total;
      w = own_page(i);
      k = base + block_scan(w, total, s_warp);
      base += total;
    }
    if (i >= n) continue;
    src[i] = dst[i] = -1;
    if (!w) continue;
    const int page = k < got ? taken[k] : -1;
    L.indices[__ldg(L.indptr + c) + whole] = page;
    if (page < 0) continue;
    L.ref[page] = 1;
    src[i] = old;
    dst[i] = page;
  }
  if (threadIdx.x == 0 && status) {
    status[0] = got;
    status[1] = want - got;
  }
}

// `runs` warps per listed request: its held entries become -1, their pages lose a holder. The entry
// is taken by an exchange, so a request listed twice is freed once; one that is reported is put back.
__global__ void __launch_bounds__(kThreads) pages_free_kernel(const Lists L, const int32_t* reqs, int n,
                                                              int runs) {
  const int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int i = (int)(w / runs), lane = threadIdx.x & 31;
  if (i >= n) return;
  const int r = __ldg(reqs + i);
  if (r < 0 || r >= L.n_req) {
    record_error(L.err, 0x602);
    return;
  }
  const int b = __ldg(L.indptr + r), held = min(pages_of(tokens_of(L.kv_indptr, r), L.page_size), __ldg(L.indptr + r + 1) - b);
  for (int k = (int)(w % runs) * 32 + lane; k < held; k += 32 * runs) {
    const int page = atomicExch(L.indices + b + k, -1);
    if (page < 0) continue;
    if (page >= L.n_pages) {
      atomicExch(L.indices + b + k, page);
      record_error(L.err, 0x601);
      continue;
    }
    if (atomicSub(L.ref + page, 1) <= 0) {  // the page was free already: its count stays 0
      atomicAdd(L.ref + page, 1);
      atomicExch(L.indices + b + k, page);
      record_error(L.err, 0x603);
    }
  }
}

// One block: counts the live pages, pairs the live ones numbered at or past that count with the
// free ones below it (both ascending), writes every page's new number and moves the counts.
__global__ void __launch_bounds__(kScanThreads) pages_plan_compact_kernel(const Lists L, int32_t* page_map, int32_t* src,
                                                                          int32_t* dst, int32_t* n_moves,
                                                                          int32_t* status) {
  __shared__ int s_warp[32];
  __shared__ uint32_t s_live[kScanThreads];  // a thread's 16 pages, for the coalesced writes of the map
  int used = 0;
  for (int64_t p0 = 16 * threadIdx.x; p0 < L.n_pages; p0 += 16 * kScanThreads) used += __popc(page_bits(L, (int)p0, true));
  int all;
  block_scan(used, all, s_warp);
  used = all;
  int holes = 0, movers = 0;
  for (int64_t r0 = 0; r0 < L.n_pages; r0 += 16 * kScanThreads) {
    const int p = (int)min(r0 + 16 * (int)threadIdx.x, (int64_t)L.n_pages);
    const uint32_t in = p + 16 <= L.n_pages ? 0xffffu : (1u << (L.n_pages - p)) - 1u;
    const uint32_t live = page_bits(L, p, true);
    const uint32_t low = used >= p + 16 ? 0xffffu : (used <= p ? 0u : (1u << (used - p)) - 1u);  // below `used`
    uint32_t hole = in & low & ~live, mover = live & ~low;
    // both counts in one scan: at most 16384 of each a round
    int total;
    const int k = block_scan(__popc(hole) | (__popc(mover) << 16), total, s_warp);
    int32_t *h = dst + holes + (k & 0xffff), *m = src + movers + (k >> 16);
    for (; hole; hole &= hole - 1) *h++ = p + __ffs(hole) - 1;
    for (; mover; mover &= mover - 1) *m++ = p + __ffs(mover) - 1;
    holes += total & 0xffff;
    movers += total >> 16;
    s_live[threadIdx.x] = live;
    __syncthreads();  // (the next round's scan separates these reads from its writes)
    const int here = (int)min((int64_t)16 * kScanThreads, L.n_pages - r0);
    for (int i = threadIdx.x; i < here; i += kScanThreads) {
      const int page = (int)r0 + i;
      page_map[page] = (s_live[i >> 4] >> (i & 15)) & 1 ? page : -1;
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < movers; k += kScanThreads) {
    page_map[src[k]] = dst[k];
    L.ref[dst[k]] = L.ref[src[k]];
    L.ref[src[k]] = 0;
  }
  if (threadIdx.x == 0) {
    *n_moves = movers;
    if (status) {
      status[0] = used;
      status[1] = movers;
    }
  }
}

bool aligned4(std::initializer_list<const void*> ps) {
  uintptr_t x = 0;
  for (const void* p : ps) x |= (uintptr_t)p;
  return (x & 3) == 0;
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

sta_status check_bufs(void* const* bufs, int n_bufs, size_t page_bytes) {
  if (n_bufs < 0 || (n_bufs > 0 && (!bufs || page_bytes == 0))) return STA_ERR_INVALID_ARG;
  if (n_bufs > 0 && (page_bytes & 15)) return STA_ERR_UNSUPPORTED;
  for (int b = 0; b < n_bufs; ++b) {
    if (!bufs[b]) return STA_ERR_INVALID_ARG;
    if ((uintptr_t)bufs[b] & 15) return STA_ERR_UNSUPPORTED;
  }
  return STA_OK;
}

// Warps that share a list when there are n lists: with one, a list of 1000 entries is a chain of 32
// dependent rounds. (4 forks of lists of about 1400: 17.5 us, 29.8 with one warp each. Many short lists
// lose nothing: 120 forks 37 us both ways.)
int runs_of(int n) { return std::min(std::max(152 * 32 / std::max(n, 1), 1), 32); }

// n: pairs at most (the grid is sized by it), n_dev: their number on the device, or null.
sta_status launch_copy(void* const* bufs, int n_bufs, size_t page_bytes, int n_pages, const int32_t* src,
                       const int32_t* dst, int n, const int32_t* n_dev, const Lists& L, const int32_t* page_map, int* err,
                       cudaStream_t st) {
  const int64_t slices = cdiv((int64_t)page_bytes, kSlice);
  const int runs = runs_of(L.n_req);
  const unsigned remap = page_map ? (unsigned)std::min<int64_t>(cdiv((int64_t)L.n_req * runs, kThreads / 32), kCopyCtas) : 0;
  for (int b0 = 0; b0 == 0 || b0 < n_bufs; b0 += kMaxBufs) {
    PageBufs pb;
    const int nb = std::min(kMaxBufs, n_bufs - b0);
    for (int b = 0; b < nb; ++b) pb.p[b] = static_cast<uint8_t*>(bufs[b0 + b]);
    const int64_t items = (int64_t)n * nb * slices;
    const unsigned grid = std::max((unsigned)std::min<int64_t>(items, kCopyCtas), b0 == 0 ? remap : 0u);
    if (grid == 0) continue;
    pages_copy_kernel<<<grid, kThreads, 0, st>>>(pb, nb, (int64_t)page_bytes, n_pages, src, dst, n, n_dev, L,
                                                 b0 == 0 ? page_map : nullptr, runs, err);
    STA_LAUNCH_CHECK();
  }
  return STA_OK;
}

sta_status check_lists(const int32_t* ref, int n_pages, const int32_t* indptr, const int32_t* indices,
                       const int32_t* kv_indptr, int n_req, int page_size, int* err, Lists& L) {
  if (n_pages < 1 || n_pages > (1 << 30) || n_req < 1 || page_size < 1) return STA_ERR_INVALID_ARG;
  L = Lists{const_cast<int32_t*>(ref), indptr, const_cast<int32_t*>(indices), kv_indptr, n_pages, n_req, page_size, err};
  return STA_OK;
}

// The workspace protocol: *bytes set and *query true when there is none.
sta_status check_workspace(void* workspace, size_t* bytes, size_t need, bool& query) {
  if (!bytes) return STA_ERR_INVALID_ARG;
  query = workspace == nullptr;
  if (query) {
    *bytes = need;
    return STA_OK;
  }
  if (*bytes < need) return STA_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255) return STA_ERR_UNSUPPORTED;
  return STA_OK;
}

}  // namespace
}  // namespace sta

using namespace sta;

extern "C" sta_status sta_pages_copy(void* const* bufs_host, int n_bufs, size_t page_bytes, int n_pages,
                                     const int32_t* src_dev, const int32_t* dst_dev, int n, sta_stream stream) {
  sta_status st = check_bufs(bufs_host, n_bufs, page_bytes);
  if (st != STA_OK) return st;
  if (n < 0 || n_pages < 1) return STA_ERR_INVALID_ARG;
  if (n == 0 || n_bufs == 0) return STA_OK;
  if (!src_dev || !dst_dev) return STA_ERR_INVALID_ARG;
  if (!aligned4({src_dev, dst_dev})) return STA_ERR_UNSUPPORTED;
  return launch_copy(bufs_host, n_bufs, page_bytes, n_pages, src_dev, dst_dev, n, nullptr, Lists{}, nullptr,
                     device_error_word(), (cudaStream_t)stream);
}

extern "C" sta_status sta_pages_grow(int32_t* ref_dev, int n_pages, const int32_t* page_indptr_dev,
                                     int32_t* page_indices_dev, const int32_t* kv_indptr_dev,
                                     const int32_t* new_kv_indptr_dev, int n_req, int page_size, int32_t* status_dev,
                                     void* workspace, size_t* workspace_bytes, sta_stream stream) {
  Lists L;
  sta_status st = check_lists(ref_dev, n_pages, page_indptr_dev, page_indices_dev, kv_indptr_dev, n_req, page_size, nullptr, L);
  if (st != STA_OK) return st;
  bool query;
  st = check_workspace(workspace, workspace_bytes, al256((size_t)n_pages * 4), query);
  if (st != STA_OK || query) return st;
  if (!ref_dev || !page_indptr_dev || !page_indices_dev || !kv_indptr_dev || !new_kv_indptr_dev) return STA_ERR_INVALID_ARG;
  if (!aligned4({ref_dev, page_indptr_dev, page_indices_dev, kv_indptr_dev, new_kv_indptr_dev, status_dev})) return STA_ERR_UNSUPPORTED;
  L.err = device_error_word();
  pages_grow_kernel<<<1, kScanThreads, 0, (cudaStream_t)stream>>>(L, new_kv_indptr_dev, static_cast<int32_t*>(workspace), status_dev);
  STA_LAUNCH_CHECK();
  return STA_OK;
}

extern "C" sta_status sta_pages_fork(void* const* bufs_host, int n_bufs, size_t page_bytes, int32_t* ref_dev, int n_pages,
                                     const int32_t* page_indptr_dev, int32_t* page_indices_dev,
                                     const int32_t* kv_indptr_dev, int n_req, int page_size, const int32_t* parent_dev,
                                     const int32_t* child_dev, int n_forks, int32_t* status_dev, void* workspace,
                                     size_t* workspace_bytes, sta_stream stream) {
  Lists L;
  sta_status st = check_bufs(bufs_host, n_bufs, page_bytes);
  if (st != STA_OK) return st;
  st = check_lists(ref_dev, n_pages, page_indptr_dev, page_indices_dev, kv_indptr_dev, n_req, page_size, nullptr, L);
  if (st != STA_OK) return st;
  if (n_forks < 0 || n_forks > n_req) return STA_ERR_INVALID_ARG;
  const size_t part = al256((size_t)std::max(n_forks, 1) * 4);
  bool query;
  st = check_workspace(workspace, workspace_bytes, 3 * part + al256((size_t)n_req * 4), query);
  if (st != STA_OK || query) return st;
  if (!ref_dev || !page_indptr_dev || !page_indices_dev || !kv_indptr_dev || (n_forks > 0 && (!parent_dev || !child_dev)))
    return STA_ERR_INVALID_ARG;
  if (!aligned4({ref_dev, page_indptr_dev, page_indices_dev, kv_indptr_dev, parent_dev, child_dev, status_dev})) return STA_ERR_UNSUPPORTED;
  L.err = device_error_word();
  cudaStream_t s = (cudaStream_t)stream;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* taken = reinterpret_cast<int32_t*>(ws);
  int32_t* src = reinterpret_cast<int32_t*>(ws + part);
  int32_t* dst = reinterpret_cast<int32_t*>(ws + 2 * part);
  const int runs = runs_of(n_forks);
  pages_fork_kernel<<<1 + (unsigned)std::min<int64_t>(cdiv((int64_t)n_forks * runs, 32), 151), kScanThreads, 0, s>>>(
      L, parent_dev, child_dev, n_forks, taken, src, dst, reinterpret_cast<int32_t*>(ws + 3 * part), runs, status_dev);
  STA_LAUNCH_CHECK();
  return launch_copy(bufs_host, n_bufs, page_bytes, n_pages, src, dst, n_forks, nullptr, L, nullptr, L.err, s);
}

extern "C" sta_status sta_pages_free(int32_t* ref_dev, int n_pages, const int32_t* page_indptr_dev,
                                     int32_t* page_indices_dev, const int32_t* kv_indptr_dev, int n_req, int page_size,
                                     const int32_t* reqs_dev, int n, sta_stream stream) {
  Lists L;
  const sta_status st = check_lists(ref_dev, n_pages, page_indptr_dev, page_indices_dev, kv_indptr_dev, n_req, page_size, nullptr, L);
  if (st != STA_OK) return st;
  if (n < 0) return STA_ERR_INVALID_ARG;
  if (n == 0) return STA_OK;
  if (!ref_dev || !page_indptr_dev || !page_indices_dev || !kv_indptr_dev || !reqs_dev) return STA_ERR_INVALID_ARG;
  if (!aligned4({ref_dev, page_indptr_dev, page_indices_dev, kv_indptr_dev, reqs_dev})) return STA_ERR_UNSUPPORTED;
  L.err = device_error_word();
  const int runs = runs_of(n);
  pages_free_kernel<<<(unsigned)cdiv((int64_t)n * runs, kThreads / 32), kThreads, 0, (cudaStream_t)stream>>>(L, reqs_dev, n, runs);
  STA_LAUNCH_CHECK();
  return STA_OK;
}

extern "C" sta_status sta_pages_compact(void* const* bufs_host, int n_bufs, size_t page_bytes, int32_t* ref_dev,
                                        int n_pages, const int32_t* page_indptr_dev, int32_t* page_indices_dev,
                                        const int32_t* kv_indptr_dev, int n_req, int page_size, int32_t* page_map_dev,
                                        int32_t* status_dev, void* workspace, size_t* workspace_bytes,
                                        sta_stream stream) {
  Lists L;
  sta_status st = check_bufs(bufs_host, n_bufs, page_bytes);
  if (st != STA_OK) return st;
  st = check_lists(ref_dev, n_pages, page_indptr_dev, page_indices_dev, kv_indptr_dev, n_req, page_size, nullptr, L);
  if (st != STA_OK) return st;
  const size_t most = (size_t)n_pages / 2 + 1;  // at most half of the pages can move
  const size_t part = al256(most * 4);
  bool query;
  st = check_workspace(workspace, workspace_bytes, 2 * part + 256, query);
  if (st != STA_OK || query) return st;
  if (!ref_dev || !page_indptr_dev || !page_indices_dev || !kv_indptr_dev || !page_map_dev) return STA_ERR_INVALID_ARG;
  if (!aligned4({ref_dev, page_indptr_dev, page_indices_dev, kv_indptr_dev, page_map_dev, status_dev})) return STA_ERR_UNSUPPORTED;
  L.err = device_error_word();
  cudaStream_t s = (cudaStream_t)stream;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* src = reinterpret_cast<int32_t*>(ws);
  int32_t* dst = reinterpret_cast<int32_t*>(ws + part);
  int32_t* n_moves = reinterpret_cast<int32_t*>(ws + 2 * part);
  pages_plan_compact_kernel<<<1, kScanThreads, 0, s>>>(L, page_map_dev, src, dst, n_moves, status_dev);
  STA_LAUNCH_CHECK();
  return launch_copy(bufs_host, n_bufs, page_bytes, n_pages, src, dst, (int)most, n_moves, L, page_map_dev, L.err, s);
}
