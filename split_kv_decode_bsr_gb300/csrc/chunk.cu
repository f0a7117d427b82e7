// Attention of chunks of new tokens over a paged KV cache, for sm_103a.
//
// Rows. The G = Hq / Hkv query heads that share a KV head, of 128 / G consecutive new tokens, are
// the 128 rows of a query tile (row = token * G + head of the group; a last few rows are unused
// when G does not divide 128). K and V of a KV head are then read once for the whole group, and a
// causal tile spans few positions. A CTA works on one item: two neighbouring query tiles of one
// (request, KV head), in two slots that share every K / V tile (128 keys) in shared memory; when
// a request has one tile left, both slots take that tile and every other key tile each, and the
// two results are merged at the end (a single token's long cache is then two interleaved
// streams). The key tiles of an item are those that some of its tokens see: [0, n_global) and the
// window, as two ranges of tile numbers. Items of few rows over a long cache are further cut into
// chunks of their tile list, whose normalised fp32 partials a second kernel merges by
// log-sum-exp.
//
// Roles (12 warps, one CTA an SM): warps 0..3 and 4..7 the softmax of slots 0 and 1 (a thread a
// row), warp 8 issues the MMAs, warps 9 and 10 load V and K, warp 11 finds items and loads Q.
// S = Q K^T (M 128, N 128) and O += P V (P bf16 over the first half of S in tensor memory) run as
// tcgen05.mma; a slot's order on the tensor core is PV(j), QK(j + 1), and one slot's MMAs run
// under the other's softmax. S and O of both slots fill the 512 TMEM columns. The softmax is the
// online one with a lazy maximum: O is rescaled only when a row's maximum grows by more than 2^8.
//
// Pages. A page of P tokens is copied by TMA in boxes of gcd(P, 128) tokens when that is a
// multiple of 8 (whole swizzle atoms). For other P of 40 or more, runs of 32 and of 8 tokens that a
// page holds whole go by TMA, and the groups of 8 that a page's end cuts by 16-byte copies
// (cp.async) to the same swizzled places; smaller pages by such copies alone. (64 single tokens over
// pages of 33: 353 us by copies, 368 by runs; of 60: 351 and 327; of 100: 384 and 329. An 8192-token
// prompt over pages of 33: 433 and 437, of 60: 443 and 341, of 100: 433 and 323, by runs of 8 alone
// 413.) Rows of V behind the sequence are set to zero, since what a page holds there may be NaN; rows
// of K there only reach masked scores.
//
// What bounds it (32 query and 8 KV heads of 128; here and below, unless it says otherwise, times of a
// CUDA graph replayed from a cold L2, some 4 to 5 us of events and graph launch included). An 8192-token
// prompt: 306 to 316 us, 1.74 to 1.79 PFLOP/s where cuBLAS reaches 1.90 in a burst (back to back, at the
// lower clocks of a card at its power limit, 333 to 354 us, 1.55 to 1.65 PFLOP/s; cuBLAS 1.68); the tensor cores,
// with the softmax just below them. 64 single tokens over 522,892 cached ones: 333 to 339 us, 6.3 to 6.4
// TB/s where a copy reaches 6.77 (back to back 319 to 326 us, 6.6 to 6.7 TB/s); HBM. Chunks with a window of 256 keys:
// 58.5 us for 700 items of some 4 tiles; each item's fixed part (the wait for its Q, the first product and
// softmax, its result) is a third of that. Heads of 64: a prompt takes 272 to 318 us for half the products,
// bound by the instructions of the softmax, which are as many as for heads of 128, and the latency between
// them.
//
// Shared prefixes (SHARED). A group's requests have their first pages in common: its prefix is an item list of its own, whose
// rows are those of all the group's new tokens one after the other (64 single tokens of 4 heads a KV head fill two query
// tiles) and which nothing masks; a request's other keys are a list with positions counted from the prefix's end; a
// second kernel joins a row's partials of both by log-sum-exp. O = sum_i e^(L_i - M) O_i / sum_i e^(L_i - M), M = max L_i:
// exact but for the roundings, whatever the cuts. Own parts of few rows go to CTAs that do nothing else (few_rows, below).
// Graph of calls back to back: 64 single tokens behind 8192 shared ones, 20523 of their own, pages of 16: 37 us (each request
// alone 222; 17.5 are the cache once at copy speed): 5 or so until the first tiles are there, 20 for 85 CTAs' runs of 17 tiles of
// 16 keys and, beside them, 64 items of 8 key tiles of the prefix, and the merge. 120 forks of 32768 tokens: 83 (1380 alone; 58.6 the cache, 0.40
// GB of DRAM reads counted). Questions of up to 1024 tokens behind a document of 12000: 576 (612; 439 at cuBLAS' rate), 77 % of the tensor
// pipe in the attention's 522, and 35 of the merge, which reads 136 MB of partials. With heads of 32 / 8, 128 elements each.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <numeric>
#include <vector>

#include "internal.h"
#include "ptx.cuh"
#include "shares.h"

namespace sta {
namespace {

constexpr int kBM = 128;  // rows of a query tile
constexpr int kBN = 128;  // keys of a tile
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kVWarp = 9, kKWarp = 10, kQWarp = 11;
constexpr int kRunPage = 40;  // tokens of a page, no multiple of 8, from which its runs are copied by TMA
constexpr int kAhead = 4;  // K tiles of an item that are still to load when the next item is taken
constexpr float kRescaleThreshold = 8.0f;  // log2 units

struct ChunkArgs {
  __nv_bfloat16* o;  // [N, Hq, d]
  float* lse;        // [N, Hq] or null
  const __nv_bfloat16* q;
  int64_t q_stride;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  const int32_t* q_indptr;
  const int32_t* kv_indptr;
  float* part_o;     // [partial rows, d]
  float* part_lse;   // [partial rows]
  int N, Hq, Hkv, d, G, TQ;  // TQ tokens a query tile
  int page_size, n_pages;
  uint32_t page_mul;      // division of a position by page_size: high word of the product with this,
  int page_shift;         // shifted right (by -1: page_size is 1)
  int box;                // tokens of a TMA box, or 0: cp.async
  int row_box;            // and of one of few_rows: 16 or 8; 0: there are none
  float scale_log2;
  int causal;
  int64_t win_lo, win_hi, n_global;
  int* err;
};

// What the host planned: the requests with new tokens, longest key lists first. Rank k has the items
// base[k] .. base[k+1]-1: ((pair of query tiles, from the last down) * Hkv + KV head) * ns + chunk.
//
// With shared prefixes a rank is a request of its own (skip 0), what a request has behind its group's prefix
// of `skip` tokens (pre: the prefix's rank), or that prefix itself (pre -2), whose rows are those of all the group's
// requests req .. end - 1 and whose pages are those of request `lead`. The first ranks, those of few rows, have no
// items: base counts their tiles of 16 keys, kStart more for each, in one row, of which each CTA of few rows takes an equal
// run. A rank's numbers lie side by side there: each part of a parameter that a kernel first reads by an index
// costs it a round trip to memory.
template <int CAP, bool SHARED>
struct Plan {
  int n;                // ranks
  int32_t base[CAP + 1];
  int32_t rows[CAP];    // merged rows up to and with the rank's (those of requests that are cut)
  int32_t part[CAP];    // first partial row
  int32_t qn[CAP];      // new tokens of the request on the host
  uint16_t req[CAP];    // request, from the launch's first
  uint16_t ns[CAP];     // chunks
};
constexpr int kStart = 2;  // what the start and the end of a piece of few rows cost, in tiles
struct Rank {
  int32_t part, qn, skip;
  uint16_t req, ns, end, lead;
  int16_t pre;  // -1: neither
  uint16_t pad;
};
template <int CAP>
struct Plan<CAP, true> {
  int n;
  int n_rows, row_ctas, ctas;  // ranks of few rows, CTAs that do them (the grid's first), the other CTAs
  int runs, run;               // CTAs of few rows for each group of KV heads, length of their runs
  int32_t base[CAP + 1];
  int32_t rows[CAP];
  Rank rank[CAP];
};
template <int CAP>
__device__ __forceinline__ Rank rank_of(const Plan<CAP, false>& P, int i) {
  return Rank{P.part[i], P.qn[i], 0, P.req[i], P.ns[i], 0, 0, -1, 0};
}
template <int CAP>
__device__ __forceinline__ Rank rank_of(const Plan<CAP, true>& P, int i) {
  return P.rank[i];
}

struct Item {
  int end;         // no more items
  int r, hk, c, ns, rank;
  int q0;          // first row of the request in q
  int n;           // new tokens computed
  int t0;          // first token of slot 0 (slot 1: t0 + TQ when dual)
  int dual;
  int len;         // tokens of the sequence
  int pos0;        // position of the request's token 0
  int gt, wl;      // tile list: [0, gt), then wl, wl + 1, ...
  int j0, j1;      // this chunk's part of it
  int j1a;         // slot 0's end in dual items (its last tokens come earlier)
  int pb, pe;      // the request's page list
  __device__ int tile(int j) const { return j < gt ? j : wl + (j - gt); }
  __device__ int count(int slot) const {
    return dual ? (slot == 1 ? j1 - j0 : j1a - j0) : (j1 - j0 + 1 - slot) / 2;
  }
};

// An item out of shared memory, by a whole warp: a word a lane, then broadcasts, which tell the
// compiler that the fields are the same in every lane (the MMA operands that follow from them then
// stay in uniform registers).
__device__ __forceinline__ Item read_item(const Item* s) {
  static_assert(sizeof(Item) == 19 * 4, "one word a lane");
  const int lane = threadIdx.x & 31, v = lane < 19 ? reinterpret_cast<const int*>(s)[lane] : 0;
  auto f = [&](int i) { return __shfl_sync(0xffffffffu, v, i); };
  return Item{f(0), f(1), f(2), f(3), f(4), f(5), f(6), f(7), f(8), f(9), f(10), f(11), f(12), f(13), f(14), f(15), f(16), f(17), f(18)};
}

// Ranges of keys that tokens at positions p0 .. p1 see among them.
struct Seen {
  int g1;      // last key seen as a global one, or -1
  int lo, hi;  // first and last key of the window, hi < lo: none
};
template <class A>
__host__ __device__ inline Seen seen(const A& a, int64_t p0, int64_t p1, int64_t len) {
  const int64_t jmax = a.causal && p1 < len - 1 ? p1 : len - 1;
  int64_t g = a.n_global - 1 < jmax ? a.n_global - 1 : jmax, lo = p0 + a.win_lo, hi = p1 + a.win_hi;
  if (lo < 0) lo = 0;
  if (hi > jmax) hi = jmax;
  Seen s;
  s.g1 = (int)(g < -1 ? -1 : g);
  s.lo = (int)(lo > INT32_MAX ? INT32_MAX : lo);
  s.hi = (int)(hi < -1 ? -1 : hi);
  return s;
}
__host__ __device__ inline int tile_list(const Seen& s, int& gt, int& wl) {
  gt = s.g1 >= 0 ? s.g1 / kBN + 1 : 0;
  wl = s.lo / kBN > gt ? s.lo / kBN : gt;
  const int wh = s.hi >= s.lo ? s.hi / kBN : -1;
  return gt + (wh >= wl ? wh - wl + 1 : 0);
}

// A word of the lists and lengths. As a constant (__ldg) only where the launch does not start before the one before it has
// ended, which may have written it.
template <bool SHARED>
__device__ __forceinline__ int32_t list_word(const int32_t* p) {
  if constexpr (SHARED) return *p;
  else return __ldg(p);
}

template <int CAP, bool SHARED>
__device__ __forceinline__ bool get_item(const ChunkArgs& A, const Plan<CAP, SHARED>& P, int req0, int item, Item& it) {
  int lo = 0, hi = P.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (P.base[mid] <= item) lo = mid;
    else hi = mid;
  }
  it.end = 0;
  it.rank = lo;
  const Rank k = rank_of(P, lo);
  it.ns = k.ns;
  const int x = item - P.base[lo], per_u = A.Hkv * it.ns, units = (P.base[lo + 1] - P.base[lo]) / per_u;
  const int u = units - 1 - x / per_u, y = x - (x / per_u) * per_u;
  it.hk = y / it.ns;
  it.c = y - it.hk * it.ns;
  it.r = req0 + k.req;
  int kr = it.r, q_end = it.r + 1;  // whose keys, whose last row
  if constexpr (SHARED) {
    q_end = req0 + k.end;
    if (k.pre == -2) kr = req0 + k.lead;
  }
  const int q0 = list_word<SHARED>(A.q_indptr + it.r), q1 = list_word<SHARED>(A.q_indptr + q_end);
  int64_t len = (int64_t)list_word<SHARED>(A.kv_indptr + kr + 1) - list_word<SHARED>(A.kv_indptr + kr);
  it.pb = list_word<SHARED>(A.page_indptr + kr);  // (with the lengths, not later by the loaders: a 2048-token prompt 36 us, 39)
  it.pe = list_word<SHARED>(A.page_indptr + kr + 1);
  int n = q1 - q0;
  int64_t pos0 = len - n;
  if constexpr (SHARED) {
    const int skip = k.skip, pre = k.pre;
    if (pre >= 0 && n > 0 && pos0 < skip) record_error(A.err, 0x608);  // new tokens that are not behind the prefix
    if (pre == -2) {  // every row is behind all of its keys
      len = skip;
      pos0 = skip;
    } else if (pre >= 0) {  // keys and positions counted from the prefix's end
      pos0 -= skip;
      len = len > skip ? len - skip : 0;
      it.pb += skip / A.page_size;
    }
  }
  if (n > k.qn) {
    record_error(A.err, 0x606);
    n = k.qn;
  }
  if (q0 < 0 || n < 0 || q0 > A.N - n || len < 0 || len > INT32_MAX - 2 * kBN) {
    record_error(A.err, 0x111);
    return false;
  }
  it.q0 = q0;
  it.n = n;
  it.t0 = 2 * u * A.TQ;
  if (it.t0 >= n) return false;
  it.dual = it.t0 + A.TQ < n;
  it.len = (int)len;
  it.pos0 = (int)pos0;
  const int te = min(n, it.t0 + (it.dual ? 2 : 1) * A.TQ);
  const Seen s = seen(A, it.pos0 + it.t0, it.pos0 + te - 1, len);
  const int nt = tile_list(s, it.gt, it.wl);
  const int each = nt / it.ns, over = nt - each * it.ns;
  it.j0 = it.c * each + it.c * over / it.ns;  // c nt / ns
  it.j1 = (it.c + 1) * each + (it.c + 1) * over / it.ns;
  it.j1a = it.j1;
  if (it.dual) {  // tiles past what slot 0's tokens see
    const Seen a = seen(A, it.pos0 + it.t0, it.pos0 + it.t0 + A.TQ - 1, len);
    const int last = max(a.g1, a.hi >= a.lo ? a.hi : -1);
    const int lt = last >= 0 ? last / kBN : -1;  // last tile of slot 0
    const int na = lt < 0 ? 0 : (lt < it.gt ? lt + 1 : it.gt + max(0, lt - it.wl + 1));
    it.j1a = max(it.j0, min(it.j1, na));
  }
  if constexpr (SHARED) {
    if (k.pre != -1) it.ns = 2;  // a partial result, whether it is cut or not
  }
  return true;
}

// A position in the ring of K and V stages, and the parity of its use.
template <int ST>
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ Ring next(int n) const {  // n <= ST
    Ring r;
    const bool wrap = s + n >= ST;
    r.s = wrap ? s + n - ST : s + n;
    r.parity = wrap ? parity ^ 1u : parity;
    return r;
  }
};

// Behind the tiles in shared memory.
template <int ST>
struct Shared {
  uint4 clc;  // answer to a request for another CTA's item
  // full[s] / empty[s]: a K or V tile is in stage s / may be overwritten. s_full[x]: S of slot x is in
  // TMEM (and every earlier MMA is done); p_half[x], p_full[x]: the P of its first 64 keys, of all of
  // them is (4 warps each); o_full[x]: the item's last PV of slot x is done; o_free[x]: its O has been
  // read (4 warps); x_full: slot 1's row maxima and sums of a single tile are in row; item_full /
  // item_empty: item holds an item / has been read by the softmax, MMA, K and V warps; want: the
  // item's last K tiles are being loaded.
  uint64_t full[ST], empty[ST], s_full[2], p_half[2], p_full[2], o_full[2], o_free[2], q_full, q_empty, x_full, tail,
      drain, clc_full, want, item_full[2], item_empty[2];
  Item item[2];
  uint32_t tmem;
  float2 row[kBM];           // slot 1's row maxima (base 2) and sums, for the merge of a single tile
};

template <int D>
struct Cfg {
  static constexpr int KH = D / 64;            // 128-byte column blocks of a row
  static constexpr int TILE = kBN * D * 2;     // a Q, K or V tile
  static constexpr int STAGES = D == 128 ? 5 : 10;
  static constexpr int OFF_Q = 0;              // two tiles
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_S = OFF_KV + STAGES * TILE;  // Shared
  static constexpr int SMEM = OFF_S + (int)sizeof(Shared<STAGES>);
  static_assert(SMEM <= 227 * 1024, "one CTA an SM");
  static constexpr uint32_t IDESC_QK = umma_idesc_bf16(kBM, kBN, 0, 0);
  static constexpr uint32_t IDESC_PV = umma_idesc_bf16(kBM, D, 0, 1);
  static constexpr int S_COL = 0;              // slot s: + 128 s; P over its first 64 columns
  static constexpr int O_COL = 256;            // slot s: + 128 s
};

// 8 consecutive TMEM columns of this thread's lane, accessed and waited for in one statement.
__device__ __forceinline__ void tmem_ld8_sync(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8_sync(uint32_t taddr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// 128 consecutive TMEM columns of this thread's lane, loaded and waited for in one statement.
#define STA_R(i) "=r"(r[i])
#define STA_R8(i) STA_R(i), STA_R(i + 1), STA_R(i + 2), STA_R(i + 3), STA_R(i + 4), STA_R(i + 5), STA_R(i + 6), STA_R(i + 7)
#define STA_R32X(i) STA_R8(i), STA_R8(i + 8), STA_R8(i + 16), STA_R8(i + 24)
__device__ __forceinline__ void tmem_ld128_sync(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, "
      "%37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, "
      "%59, %60, %61, %62, %63, %64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, %80, "
      "%81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, %96, %97, %98, %99, %100, %101, "
      "%102, %103, %104, %105, %106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, %117, %118, %119, "
      "%120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : STA_R32X(0), STA_R32X(32), STA_R32X(64), STA_R32X(96)
      : "r"(taddr)
      : "memory");
}
#undef STA_R32X
#undef STA_R8
#undef STA_R

// 16 bytes, or 16 zero bytes where `some` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
// One arrival of this thread on `bar` once all its cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// True in one lane of the (whole, converged) warp. Unlike lane == 0 it tells the compiler that a
// single thread runs what follows, so that the operands of its MMAs stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Asks for one CTA of this grid that has not started yet, to do its work here: the answer (16 bytes)
// arrives on `bar`.
__device__ __forceinline__ void clc_request(void* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// blockIdx.x of the CTA that was taken over, or -1: none is left (no further request may be made).
__device__ __forceinline__ int clc_answer(const void* answer) {
  uint32_t got, x = 0;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\tld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
      : "=&r"(got), "=&r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return got ? (int)x : -1;
}

// mbar_wait by all lanes of a converged warp, which vote on each try and on the time: one outcome
// for all of them. (Each by its own tries and its own reading of the timer, some could go on and others
// leave when the phase completes as the time runs out, and the votes, shuffles and .aligned instructions
// that follow would wait for lanes that never come. A vote on the outcome of mbar_wait would do too, but
// a try that has to leave its loop first costs more: an 8192-token prompt 310 us,
// 308 as here, 306 with lanes on their own; back to back 333 both ways.)
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, int* err, int err_code) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait_suspend(bar, parity, kSuspendHintNs))) return true;
    if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs)) {
      record_error(err, err_code);
      return false;
    }
  }
}

// 32 bytes to one place, a whole sector at once (both halves of it where p is not 32-byte aligned).
__device__ __forceinline__ void store32(void* p, const uint32_t* r) {
  if (((uintptr_t)p & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// Bits of keys k0 .. k0 + 31 that lie in [lo, hi].
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int k0) {
  const int a = lo - k0, b = hi - k0;
  if (a > 31 || b < 0 || b < a) return 0u;
  return (a <= 0 ? ~0u : ~0u << a) & (b >= 31 ? ~0u : (2u << b) - 1u);
}

// Few rows: the (at most 16) rows of a request's new tokens for each KV head, over a piece of its keys, on mma.sync. Beside
// a shared prefix, whose rows fill the tensor cores' tiles, what a request has of its own is a short list for each KV head:
// an item of it would take a CTA's 128-row tiles for 4 rows or so, and some 6 us between its lookups, its loads, its
// one product and its result. Here a CTA takes a piece for up to 8 KV heads at once: two warps copy K and V of 16 tokens by
// TMA, 16-KB boxes of all the heads (a warp that looked up and copied for its own head alone spent more issue slots on that
// than on the products), and 8 warps compute, one a head, or several a head that take tiles in turn where there are
// fewer heads. The first CTAs of the grid do nothing else, beside those of the prefix. (64 single tokens behind 8192 shared ones
// 37 us, all in items 44; 120 forks 83 and 124; a single KV head's short lists 33 and 28: RowTimes::few and the estimates choose.)
template <int D>
struct RowCfg {
  static constexpr int KEYS = 16;              // of a tile
  static constexpr int KH = D / 64;            // 128-byte column blocks of a row
  static constexpr int HEAD = KEYS * 128;      // a head's part of such a block
  static constexpr int BYTES = kRowRing;
  static constexpr int WARPS = 8, PIECES = 4;
  static constexpr bool turns_divide_stages() {
    for (int heads = 1; heads <= 8; ++heads)
      if (row_stages(D, heads) % row_turns(heads)) return false;
    return true;
  }
  static_assert(turns_divide_stages(), "see row_first");
};

// Partials beside shared prefixes: those of chunk c of a rank are [D / 8][rows][8], rows by KV head, token and head of the
// group, so that the threads of a warp, a row each, write whole lines (a row's 512 bytes by one thread took an item of two
// query tiles 2 us longer).
struct SharedPart {
  int64_t first;  // row of the chunk's first
  int rows, row;
  __device__ __forceinline__ SharedPart(const Rank& k, int Hq, int G, int c, int hk, int t, int g)
      : first(k.part + (int64_t)c * k.qn * Hq), rows(k.qn * Hq), row((hk * k.qn + t) * G + g) {}
  __device__ __forceinline__ int64_t lse() const { return first + row; }
  __device__ __forceinline__ int64_t values(int D, int eighth) const { return first * D + ((int64_t)eighth * rows + row) * 8; }
};

// K and V in boxes of ChunkArgs::row_box tokens.
template <bool SHARED>
struct RowMaps {};
template <>
struct RowMaps<true> {
  CUtensorMap k, v;
};

// The launches with shared prefixes may start while the one before them ends. grid_wait(): it has ended, and what it wrote is
// there. grid_go(): the next one may start (when all CTAs have come here). The first kernel touches no memory of the
// call before its wait, and lets the merge start after it, since that looks its rows up before its own: what wrote the lists and
// lengths has ended before the merge begins. The merge lets the next launch start at once, beside the first kernel's last
// CTAs; that launch waits for the merge's end, which comes after theirs.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A piece: the rank's rows of KV heads h0 .. , chunk c of its 16-key tiles (j0 .. j1 - 1).
struct Piece {
  int rank, h0, c;      // rank -1: none
  int q0, n, pos0, len; // first row in q, new tokens, position of the first one, keys
  int pb, pe;           // page list
  int j0, j1;
};
struct RowShared {  // behind the ring
  uint64_t full[16], empty[16], piece_full[4], piece_empty[4];
  Piece piece[4];
};

template <int D, int CAP>
__device__ __forceinline__ void few_rows(const ChunkArgs& A, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                         const Plan<CAP, true>& P, int req0, uint8_t* smem) {
  using C = RowCfg<D>;
  static_assert(C::BYTES + (int)sizeof(RowShared) <= Cfg<D>::SMEM, "beside the other CTAs' shared memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  RowShared& sh = *reinterpret_cast<RowShared*>(smem + C::BYTES);
  const int HB = row_heads(A.Hkv), turns = row_turns(A.Hkv), half = HB * C::KH * C::HEAD;  // K's or V's part of a stage
  const int ST = row_stages(D, HB);
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&sh.full[s], 2);
      mbar_init(&sh.empty[s], HB);
    }
    for (int i = 0; i < C::PIECES; ++i) {
      mbar_init(&sh.piece_full[i], 1);
      mbar_init(&sh.piece_empty[i], HB * turns);
    }
    fence_mbar_init();
  }
  __syncthreads();
  grid_wait();
  grid_go();
  const int P0 = A.page_size;
  auto page_no = [&](int tok) -> int { return A.page_shift < 0 ? tok : (int)(__umulhi((uint32_t)tok, A.page_mul) >> A.page_shift); };

  if (warp >= C::WARPS) {
    // ------------------------------------------------------------ K and the pieces, V
    const int me = warp - C::WARPS, is_v = me;
    if (me > 1) return;
    // This CTA's run, over as many ranks as it touches: a piece of each.
    const int group = blockIdx.x / P.runs, x0 = (blockIdx.x - group * P.runs) * P.run, x1 = min(x0 + P.run, P.base[P.n_rows]);
    int lo = 0, hi = P.n_rows;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (P.base[mid] <= x0) lo = mid;
      else hi = mid;
    }
    int from = P.base[lo], a = 0, b = 0, tiles = 1;  // the next piece: where its rank begins, its tiles of all there were on the host
    // The next piece's rank, heads and chunk; a lane loads one of the six numbers that it goes by.
    auto take = [&](Piece& p) -> int {
      p.rank = -1;
      if (lo >= P.n_rows || from >= x1) return 0;
      const Rank k = rank_of(P, lo);
      const int to = P.base[lo + 1];
      p.rank = lo;
      p.h0 = group * HB;
      p.c = from < x0 ? x0 / P.run - from / P.run : 0;
      tiles = to - from - kStart;
      a = max(max(x0, from) - from - kStart, 0);
      b = max(min(x1, to) - from - kStart, 0);
      ++lo;
      from = to;
      const int32_t* in = lane < 2 ? A.q_indptr : (lane < 4 ? A.kv_indptr : A.page_indptr);
      return lane < 6 ? list_word<true>(in + req0 + k.req + (lane & 1)) : 0;
    };
    auto settle = [&](Piece& p, int loaded) {
      const int q0 = __shfl_sync(0xffffffffu, loaded, 0), q1 = __shfl_sync(0xffffffffu, loaded, 1);
      int64_t len = (int64_t)__shfl_sync(0xffffffffu, loaded, 3) - __shfl_sync(0xffffffffu, loaded, 2);
      p.pb = __shfl_sync(0xffffffffu, loaded, 4);
      p.pe = __shfl_sync(0xffffffffu, loaded, 5);
      p.n = p.j0 = p.j1 = 0;
      if (p.rank < 0) return;
      const Rank k = rank_of(P, p.rank);
      int n = q1 - q0;
      int64_t pos0 = len - n;
      if (n > k.qn) {
        record_error(A.err, 0x606);
        n = k.qn;
      }
      if (q0 < 0 || n < 0 || q0 > A.N - n || len < 0 || len > INT32_MAX - 2 * kBN) {
        record_error(A.err, 0x111);
        return;
      }
      if (k.pre >= 0) {  // keys and positions counted from the prefix's end
        if (n > 0 && pos0 < k.skip) record_error(A.err, 0x608);  // new tokens that are not behind the prefix
        pos0 -= k.skip;
        len = len > k.skip ? len - k.skip : 0;
        p.pb += page_no(k.skip);
      }
      p.q0 = q0;
      p.n = n;
      p.pos0 = (int)pos0;
      p.len = (int)len;
      if (n == 0) return;
      const int nt = (p.len + C::KEYS - 1) / C::KEYS;
      p.j0 = nt == tiles ? a : (int)((int64_t)a * nt / tiles);  // (other lengths than the host's: the same parts of them)
      p.j1 = nt == tiles ? b : (int)((int64_t)b * nt / tiles);
    };
    bool ok = true;
    uint32_t T = 0;  // tiles of earlier pieces
    Piece next;
    int loaded = take(next);
    for (uint32_t k = 0; ok; ++k) {
      Piece p = next;
      settle(p, loaded);
      if (me == 0) {
        if (k >= C::PIECES) ok = mbar_wait_warp(&sh.piece_empty[k % C::PIECES], ((k / C::PIECES) & 1u) ^ 1u, A.err, 0x635);
        if (!ok) break;
        if (lane == 0) {
          sh.piece[k % C::PIECES] = p;
          mbar_arrive(&sh.piece_full[k % C::PIECES]);
        }
      }
      if (p.rank < 0) break;
      loaded = take(next);
      // A lane holds one entry of the page list, and one of the 32 after them; -1 behind the list.
      auto entry = [&](int e) -> int {
        const int o = p.pb + e;
        return o >= 0 && o < p.pe && (int64_t)e * P0 < p.len && A.page_indices ? list_word<true>(A.page_indices + o) : -1;
      };
      int window = page_no(p.j0 * C::KEYS), pages = -1, later = -1;
      if (p.j0 < p.j1) {
        pages = entry(window + lane);
        later = entry(window + 32 + lane);
      }
      for (int j = p.j0; j < p.j1; ++j, ++T) {
        const int tok0 = j * C::KEYS, in = min(C::KEYS, p.len - tok0);
        if (page_no(tok0) >= window + 32) {
          window += 32;
          pages = later;
          later = entry(window + 32 + lane);
        }
        const int tok = tok0 + (lane & 15) * A.row_box;  // the first of the tile's box, or of the two of 8
        const bool some = (lane & 15) * A.row_box < in;
        const int no = page_no(some ? tok : tok0);
        const int near = __shfl_sync(0xffffffffu, pages, no - window), far = __shfl_sync(0xffffffffu, later, no - window - 32);
        int page = no < window + 32 ? near : far, row = -1;
        if (some) {
          if (page < 0 || page >= A.n_pages) {
            record_error(A.err, 0x110);
            page = 0;
          }
          row = page * P0 + tok - no * P0;
        }
        const int s = T % ST;
        if (T >= (uint32_t)ST && !(ok = mbar_wait_warp(&sh.empty[s], ((T / ST) & 1u) ^ 1u, A.err, 0x636))) break;
        uint8_t* to = smem + s * 2 * half + is_v * half;
        const int nb = A.row_box == C::KEYS ? 1 : (in + 7) >> 3;
        const int row1 = __shfl_sync(0xffffffffu, row, 1);
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.full[s], (uint32_t)(nb * A.row_box * HB * 128 * C::KH));
#pragma unroll
          for (int kh = 0; kh < C::KH; ++kh) {
            // [KH][box][HB][tokens of a box] rows of 128 bytes
            tma_load_3d(to + kh * (HB * C::HEAD), is_v ? &tm_v : &tm_k, kh * 64, row, p.h0, &sh.full[s]);
            if (nb > 1) tma_load_3d(to + kh * (HB * C::HEAD) + HB * 1024, is_v ? &tm_v : &tm_k, kh * 64, row1, p.h0, &sh.full[s]);
          }
        }
        __syncwarp();
      }
    }
    // shared memory is not released under a copy
    for (uint32_t t = T > (uint32_t)ST ? T - ST : 0; t < T; ++t)
      if (!mbar_wait_warp(&sh.full[t % ST], (t / ST) & 1u, A.err, 0x637)) break;
    return;
  }

  // -------------------------------------------------------------- products and softmax of a head, by turns
  constexpr int NB = C::KEYS / 8;
  const float c = A.scale_log2;
  const int head = warp % HB, turn = warp / HB;
  if (turn >= turns) return;
  // this lane's rows of a piece, lane / 4 and that + 8: their tokens and heads of the group
  const int r0 = lane >> 2, r1 = r0 + 8, t0 = r0 / A.G, t1 = r1 / A.G, g0 = r0 - t0 * A.G, g1 = r1 - t1 * A.G;
  const int mi = lane >> 3, mr = lane & 7;
  // a head's rows 0 .. 7 and 8 .. 15 of a tile: in one box, or in two
  const int at_head = A.row_box == 8 ? head * 1024 : head * C::HEAD, to_second = A.row_box == 8 ? HB * 1024 : 1024;
  bool ok = true;
  uint32_t T = 0;
  for (uint32_t k = 0; ok; ++k) {
    if (!(ok = mbar_wait_warp(&sh.piece_full[k % C::PIECES], (k / C::PIECES) & 1u, A.err, 0x638))) break;
    const Piece p = sh.piece[k % C::PIECES];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.piece_empty[k % C::PIECES]);
    if (p.rank < 0) break;
    const int hk = p.h0 + head;
    const bool mine = hk < A.Hkv, live0 = mine && t0 < p.n, live1 = mine && t1 < p.n;  // (rows past the last: zeros)
    uint32_t qa[D / 16][4];
    {  // (q may be what the merge before this launch wrote while it ran already: not by way of the cache for what is constant)
      auto q_row = [&](int t, int g) { return A.q + (int64_t)(p.q0 + t) * A.q_stride + ((int64_t)hk * A.G + g) * D; };
      const __nv_bfloat16 *a0 = q_row(t0, g0), *a1 = q_row(t1, g1);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int e = i * 16 + (lane & 3) * 2;
        qa[i][0] = live0 ? *reinterpret_cast<const uint32_t*>(a0 + e) : 0u;
        qa[i][1] = live1 ? *reinterpret_cast<const uint32_t*>(a1 + e) : 0u;
        qa[i][2] = live0 ? *reinterpret_cast<const uint32_t*>(a0 + e + 8) : 0u;
        qa[i][3] = live1 ? *reinterpret_cast<const uint32_t*>(a1 + e + 8) : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    const int nt = p.j1 - p.j0;
    for (int i = row_first(T, turn, turns); i < nt; i += turns) {
      const int j = p.j0 + i, tail = p.len - j * C::KEYS, st = (T + i) % ST;  // tail: keys of this tile
      if (!(ok = mbar_wait_warp(&sh.full[st], ((T + i) / ST) & 1u, A.err, 0x639))) break;
      const uint8_t* kt = smem + st * 2 * half + at_head;
      float s[NB][4], s2[NB][4];  // (two short chains of products rather than one long)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[b][e] = s2[b][e] = 0.f;
      {
        const uint32_t base = smem_u32(kt) + (mi >> 1) * to_second + mr * 128;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          uint32_t f[4];
          ldsm_x4(base + (x >> 2) * (HB * C::HEAD) + ((((2 * x + (mi & 1)) & 7) ^ mr) << 4), f);
          mma_bf16_16816(x & 1 ? s2[0] : s[0], qa[x], f[0], f[1]);
          mma_bf16_16816(x & 1 ? s2[1] : s[1], qa[x], f[2], f[3]);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[b][e] += s2[b][e];
      if (j * C::KEYS + C::KEYS - 1 > p.pos0) {  // keys that some row does not see
        const int k0 = j * C::KEYS + (lane & 3) * 2, see0 = p.pos0 + t0 - k0, see1 = p.pos0 + t1 - k0;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (b * 8 + (e & 1) > (e < 2 ? see0 : see1) || b * 8 + (e & 1) + (lane & 3) * 2 >= tail) s[b][e] = -INFINITY;
      }
      float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])), x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
      }
      x0 *= c;
      x1 *= c;
      float a0 = 1.f, a1 = 1.f;
      if (x0 > m0 + kRescaleThreshold) {
        if (m0 != -INFINITY) a0 = ex2(m0 - x0);
        m0 = x0;
      }
      if (x1 > m1 + kRescaleThreshold) {
        if (m1 != -INFINITY) a1 = ex2(m1 - x1);
        m1 = x1;
      }
      if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a0;
          o[i][2] *= a1;
          o[i][3] *= a1;
        }
      }
      const float n0 = m0 == -INFINITY ? 0.f : -m0, n1 = m1 == -INFINITY ? 0.f : -m1;
      uint32_t pa[4];  // P in bf16 for the product, off by 2^-8 at most; the sums take the fp32 values
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float w0 = ex2(fmaf(s[b][0], c, n0)), w1 = ex2(fmaf(s[b][1], c, n0));
        const float w2 = ex2(fmaf(s[b][2], c, n1)), w3 = ex2(fmaf(s[b][3], c, n1));
        l0 += w0 + w1;
        l1 += w2 + w3;
        pa[b * 2] = pack_bf16x2(w0, w1);
        pa[b * 2 + 1] = pack_bf16x2(w2, w3);
      }
      uint8_t* vt = smem + st * 2 * half + half + at_head;
      if (tail < C::KEYS) {  // rows behind the sequence: what a page holds there may be NaN
        for (int z = tail * 8 + lane; z < C::KEYS * 8; z += 32)
#pragma unroll
          for (int kh = 0; kh < C::KH; ++kh)
            *reinterpret_cast<uint4*>(vt + kh * (HB * C::HEAD) + (z >= 64 ? to_second + (z - 64) * 16 : z * 16)) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
      }
      {
        const uint32_t base = smem_u32(vt) + (mi & 1) * to_second + mr * 128;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          uint32_t f[4];
          ldsm_x4_t(base + (x >> 2) * (HB * C::HEAD) + ((((2 * x + (mi >> 1)) & 7) ^ mr) << 4), f);
          mma_bf16_16816(o[2 * x], pa, f[0], f[1]);
          mma_bf16_16816(o[2 * x + 1], pa, f[2], f[3]);
        }
      }
      __syncwarp();  // the tile has been read by all lanes
      if (lane == 0) mbar_arrive(&sh.empty[st]);
    }
    T += nt;
    if (!ok) break;
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    const Rank rk = rank_of(P, p.rank);
    auto result = [&](bool live, int t, int g, float m, float l, int e) {
      if (!live) return;
      const float inv = l != 0.f ? 1.f / l : 0.f;  // a NaN among the scores stays one
      const float lse = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      const int h = hk * A.G + g;
      if (rk.ns > 1 || rk.pre != -1) {
        const SharedPart to(rk, A.Hq, A.G, p.c * turns + turn, hk, t, g);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(A.part_o + to.values(D, i) + (lane & 3) * 2) = make_float2(o[i][e] * inv, o[i][e + 1] * inv);
        if ((lane & 3) == 0) A.part_lse[to.lse()] = lse == lse ? lse : INFINITY;  // the merge makes a NaN of it again
      } else {
        const int64_t to = (int64_t)(p.q0 + t) * A.Hq + h;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<uint32_t*>(A.o + to * D + i * 8 + (lane & 3) * 2) = pack_bf16x2(o[i][e] * inv, o[i][e + 1] * inv);
        if ((lane & 3) == 0 && A.lse) A.lse[to] = lse;
      }
    };
    result(live0, t0, g0, m0, l0, 0);
    result(live1, t1, g1, m1, l1, 2);
  }
}

template <int D, int CAP, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k4,
                 const __grid_constant__ CUtensorMap tm_v4, const __grid_constant__ RowMaps<SHARED> R,
                 const __grid_constant__ ChunkArgs A, const __grid_constant__ Plan<CAP, SHARED> P, int req0) {
  using C = Cfg<D>;
  constexpr int ST = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<ST>& sh = *reinterpret_cast<Shared<ST>*>(smem + C::OFF_S);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(smem) & 1023) {  // swizzle atoms start on 1024-byte boundaries
    record_error(A.err, 0x607);
    return;
  }
  if constexpr (SHARED) {
    if ((int)blockIdx.x < P.row_ctas) {
      few_rows<D, CAP>(A, R.k, R.v, P, req0, smem);
      return;
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&sh.full[s], A.box > 0 ? 1 : (A.page_size >= kRunPage ? 33 : 32));  // TMA bytes, the copying lanes
      mbar_init(&sh.empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh.s_full[x], 1);
      mbar_init(&sh.p_half[x], 4);
      mbar_init(&sh.p_full[x], 4);
      mbar_init(&sh.o_full[x], 1);
      mbar_init(&sh.o_free[x], 4);
      mbar_init(&sh.item_full[x], 1);
      mbar_init(&sh.item_empty[x], kMmaWarp + 3);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.x_full, 4);
    mbar_init(&sh.tail, 1);
    mbar_init(&sh.drain, 1);
    mbar_init(&sh.clc_full, 1);
    mbar_init(&sh.want, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if constexpr (SHARED) {
    grid_wait();
    grid_go();
  }

  // Every role runs over the same items: item k is in sh.item[k & 1]. A wait that runs out ends the
  // role's loop, and then, by their own waits, the others'.
  if (warp == kQWarp) {
    // ------------------------------------------------------------ items and Q
    // The CTA starts with its own item and takes over those of CTAs that have not started yet, in
    // the grid's order (heaviest first): the next one when the last K tiles of this one are being
    // loaded. (Taken as early as there is room for them, items lie waiting in CTAs that are busy with
    // long ones while others run out of work: 366 us against 333 for 64 single tokens, 52 against 40 for a
    // 2048-token prompt.)
    if (lane == 0) {
      bool ok = true;
      int item = blockIdx.x, k = 0, nq = 0;
      if constexpr (SHARED) item += P.base[P.n_rows] - P.row_ctas;
      Item it;
      for (int n = 0; ok && item >= 0;) {
        if (get_item(A, P, req0, item, it)) {
          if (k >= 2) ok = mbar_wait(&sh.item_empty[k & 1], ((k >> 1) & 1u) ^ 1u, A.err, 0x62b);
          if (ok) {
            sh.item[k & 1] = it;
            mbar_arrive(&sh.item_full[k & 1]);
            ++k;
          }
          if (ok && it.j1 > it.j0) {
            if (nq > 0) ok = mbar_wait(&sh.q_empty, (nq - 1) & 1u, A.err, 0x620);
            if (ok) {
              const uint32_t bytes = (uint32_t)(A.G * A.TQ * 128 * C::KH);
              mbar_arrive_expect_tx(&sh.q_full, bytes * (it.dual ? 2 : 1));
              for (int x = 0; x <= it.dual; ++x)
#pragma unroll
                for (int kh = 0; kh < C::KH; ++kh)
                  tma_load_3d(smem + C::OFF_Q + x * C::TILE + kh * (kBM * 128), &tm_q, kh * 64, it.hk * A.G,
                              it.q0 + it.t0 + x * A.TQ, &sh.q_full);
              ++nq;
            }
          }
          ok = ok && mbar_wait(&sh.want, (k - 1) & 1u, A.err, 0x632);
        }
        if (!ok) break;
        if constexpr (SHARED) {
          if (P.row_ctas > 0) {  // CTAs of few rows may not be taken over: the others go round by themselves
            item += P.ctas;
            if (item >= P.base[P.n]) break;
            continue;
          }
        }
        clc_request(&sh.clc, &sh.clc_full);
        item = mbar_wait(&sh.clc_full, n & 1u, A.err, 0x62c) ? clc_answer(&sh.clc) : -1;
        fence_proxy_async_smem();  // the answer has been read before the next one is written
        ++n;
      }
      if (ok && k >= 2) ok = mbar_wait(&sh.item_empty[k & 1], ((k >> 1) & 1u) ^ 1u, A.err, 0x62b);
      if (ok) {
        sh.item[k & 1].end = 1;
        mbar_arrive(&sh.item_full[k & 1]);
      }
      if (nq > 0) mbar_wait(&sh.q_full, (nq - 1) & 1u, A.err, 0x620);  // shared memory is not released under a copy
    }
  } else if (warp == kKWarp || warp == kVWarp) {
    // ------------------------------------------------------------ K or V: ring stages 2i and 2i + 1
    const bool is_v = warp == kVWarp;
    const int P0 = A.page_size;
    int pb = 0, pe = 0;
    auto page_no = [&](int tok) -> int {  // tok / P0
      return A.page_shift < 0 ? tok : (int)(__umulhi((uint32_t)tok, A.page_mul) >> A.page_shift);
    };
    auto page_at = [&](int tok) -> int {  // list entry of a token, unchecked; -1 behind the list
      const int o = pb + page_no(tok);
      return o >= 0 && o < pe && A.page_indices ? list_word<SHARED>(A.page_indices + o) : -1;
    };
    auto row_at = [&](int page, int tok) -> int {  // cache row; a page outside the cache reads page 0
      if (page < 0 || page >= A.n_pages) {
        record_error(A.err, 0x110);
        page = 0;
      }
      return page * P0 + tok - page_no(tok) * P0;
    };
    bool ok = true;
    int T = 0, n_tail = 0;  // tiles of earlier items; tail tiles so far
    for (int k = 0; ok; ++k) {
      if (!mbar_wait_warp(&sh.item_full[k & 1], (k >> 1) & 1u, A.err, 0x62d)) break;
      const Item it = read_item(&sh.item[k & 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_empty[k & 1]);
      if (it.end) break;
      const int nj = it.j1 - it.j0;
      const int ask = is_v ? -1 : max(nj - kAhead, 0);  // the tile at which the next item is asked for
      int i = 0;
      if (ask == 0 && lane == 0) mbar_arrive(&sh.want);
      pb = it.pb;
      pe = it.pe;
      if (A.box > 0) {
        // a lane per TMA box (column block kh of box b); the next tile's page numbers are fetched
        // while this tile's stage is waited for
        const int b = lane / C::KH, kh = lane % C::KH, off = b * A.box;
        const int boxes = kBN / A.box, box_shift = __ffs(A.box) - 1;  // (a power of 2)
        // With a shared prefix, whose tiles come from memory rather than from L2, page numbers one tile ahead are a round
        // trip to memory for each tile: there a lane holds one page number of the next 32 / boxes tiles, and the 32 after
        // them are on their way (2.5 us a tile over pages of 16 otherwise, 1.5 so).
        const int in_window = 32 / boxes;
        auto window = [&](int i0) -> int {
          const int t = i0 + lane / boxes;
          return t < nj ? page_at(it.tile(it.j0 + t) * kBN + (lane & (boxes - 1)) * A.box) : -1;
        };
        int pg = -1, later = -1;
        if constexpr (SHARED) {
          pg = window(0);
          later = window(in_window);
        } else {
          pg = nj > 0 && b < boxes ? page_at(it.tile(it.j0) * kBN + off) : -1;
        }
        for (; i < nj; ++i) {
          const int y = 2 * (T + i) + is_v, s = y % ST, tok0 = it.tile(it.j0 + i) * kBN;
          int page = pg;
          if constexpr (SHARED) {
            const int at = i & (in_window - 1);
            if (i > 0 && at == 0) {
              pg = later;
              later = window(i + in_window);
            }
            page = __shfl_sync(0xffffffffu, pg, at * boxes + min(b, boxes - 1));
          } else {
            if (i + 1 < nj && b < boxes) pg = page_at(it.tile(it.j0 + i + 1) * kBN + off);
          }
          const int in = min(boxes, (it.len - tok0 + A.box - 1) >> box_shift);  // boxes with tokens
          const bool tail_v = is_v && tok0 + kBN > it.len;                 // rows behind the sequence
          if (i > 0 && i == ask && lane == 0) mbar_arrive(&sh.want);
          // every lane waits, for one that waits alone leaves the warp diverged (349 us against 338 for 64 single
          // tokens; over pages of one token, below, 625 against 439)
          ok = mbar_wait_warp(&sh.empty[s], ((y / ST) & 1u) ^ 1u, A.err, 0x621);
          if (!ok) break;
          uint8_t* dst = smem + C::OFF_KV + s * C::TILE;
          uint64_t* bar = tail_v ? &sh.tail : &sh.full[s];
          if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(in * A.box * 128 * C::KH));
          __syncwarp();
          if (b < in)
            tma_load_3d(dst + kh * (kBN * 128) + off * 128, is_v ? &tm_v : &tm_k, kh * 64, it.hk, row_at(page, tok0 + off), bar);
          if (tail_v) {  // (the last tile of a list at most)
            if (!(ok = mbar_wait_warp(&sh.tail, n_tail & 1u, A.err, 0x622))) {
              mbar_wait_warp(&sh.tail, n_tail & 1u, A.err, 0x622);  // shared memory is not released under a copy
              break;
            }
            ++n_tail;
            for (int z = (it.len - tok0) * 8 + lane; z < kBN * 8; z += 32)
#pragma unroll
              for (int k = 0; k < C::KH; ++k) *reinterpret_cast<uint4*>(dst + k * (kBN * 128) + z * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.full[s]);
          }
        }
      } else if (P0 >= kRunPage) {
        // Groups of 8 tokens: lane b (of 16) looks up the cache row of group b's first token, lane 16 + b
        // that of its last. Rows that follow one another go by TMA, a lane per column block; groups that
        // a page's end cuts (once at most) or the sequence's end go row by row in
        // 16-byte copies of all lanes.
        constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes a row, rows an instruction
        const int ch = lane % LPR, hi = lane / LPR, b = lane & 15, far = lane >> 4;
        const __nv_bfloat16* src = (is_v ? A.v : A.k) + (int64_t)it.hk * D + ch * 8;
        const int64_t row_elems = (int64_t)A.Hkv * D;
        auto token = [&](int t0) { return min(t0 + 8 * b + 7 * far, it.len - 1); };  // this lane's of the tile at t0
        int pg = nj > 0 ? page_at(token(it.tile(it.j0) * kBN)) : -1;
        for (; i < nj; ++i) {
          const int y = 2 * (T + i) + is_v, s = y % ST, tok0 = it.tile(it.j0 + i) * kBN, page = pg;
          if (i + 1 < nj) pg = page_at(token(it.tile(it.j0 + i + 1) * kBN));
          const bool live = tok0 + 8 * b < it.len;
          const int row = live ? row_at(page, token(tok0)) : -1;
          const int first = __shfl_sync(0xffffffffu, row, b), last = __shfl_sync(0xffffffffu, row, b + 16);
          const bool whole = tok0 + 8 * b + 7 < it.len && last == first + 7;
          // four groups in one run of rows (a page ends once among them at most) in one box
          const int first4 = __shfl_sync(0xffffffffu, row, b & 12), last4 = __shfl_sync(0xffffffffu, row, (b | 3) + 16);
          const bool whole4 = tok0 + 8 * (b | 3) + 7 < it.len && last4 == first4 + 31;
          const uint32_t boxes = __ballot_sync(0xffffffffu, whole) & 0xffffu;
          const uint32_t rest = __ballot_sync(0xffffffffu, !whole && (is_v || live)) & 0xffffu;
          if (i > 0 && i == ask && lane == 0) mbar_arrive(&sh.want);
          ok = mbar_wait_warp(&sh.empty[s], ((y / ST) & 1u) ^ 1u, A.err, 0x621);
          if (!ok) break;
          uint8_t* tile = smem + C::OFF_KV + s * C::TILE;
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], (uint32_t)(__popc(boxes) * 1024 * C::KH));
          __syncwarp();
          if (whole && far < C::KH && (!whole4 || (b & 3) == 0))
            tma_load_3d(tile + far * (kBN * 128) + b * 1024, whole4 ? (is_v ? &tm_v4 : &tm_k4) : (is_v ? &tm_v : &tm_k),
                        far * 64, it.hk, first, &sh.full[s]);
          const uint32_t dst = smem_u32(tile) + (ch >> 3) * (kBN * 128);
          for (uint32_t left = rest; left; left &= left - 1) {
            const int g = __ffs(left) - 1, t0 = tok0 + 8 * g, in = min(it.len - t0, 8);  // tokens of the group
            const int f = __shfl_sync(0xffffffffu, row, g), e = __shfl_sync(0xffffffffu, row, g + 16);
            const int here = P0 - (t0 - page_no(t0) * P0);  // of which in the first one's page
#pragma unroll
            for (int r0 = 0; r0 < 8; r0 += RPI) {
              const int r = r0 + hi, m = 8 * g + r, at = r < here ? f + r : e - (in - 1 - r);
              cp_async16(dst + m * 128 + (((ch & 7) ^ (m & 7)) << 4), src + (r < in ? at : 0) * row_elems, r < in);
            }
          }
          cp_async_arrive(&sh.full[s]);
        }
      } else {
        // Small pages: 16-byte copies alone. Lane l looks up the rows of tokens l, l + 32, .. of the tile,
        // which the copies take from it by shuffles.
        constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes a row, rows an instruction
        const int ch = lane % LPR;
        const __nv_bfloat16* src = (is_v ? A.v : A.k) + (int64_t)it.hk * D + ch * 8;
        const int64_t row_elems = (int64_t)A.Hkv * D;
        int pg[kBN / 32];
#pragma unroll
        for (int g = 0; g < kBN / 32; ++g) {
          const int tok = nj > 0 ? it.tile(it.j0) * kBN + 32 * g + lane : it.len;
          pg[g] = tok < it.len ? page_at(tok) : -1;
        }
        for (; i < nj; ++i) {
          const int y = 2 * (T + i) + is_v, s = y % ST, tok0 = it.tile(it.j0 + i) * kBN;
          int row[kBN / 32];
#pragma unroll
          for (int g = 0; g < kBN / 32; ++g) {
            const int tok = tok0 + 32 * g + lane;
            row[g] = tok < it.len ? row_at(pg[g], tok) : -1;
            const int next = i + 1 < nj ? it.tile(it.j0 + i + 1) * kBN + 32 * g + lane : it.len;
            pg[g] = next < it.len ? page_at(next) : -1;
          }
          if (i > 0 && i == ask && lane == 0) mbar_arrive(&sh.want);
          ok = mbar_wait_warp(&sh.empty[s], ((y / ST) & 1u) ^ 1u, A.err, 0x621);
          if (!ok) break;
          const uint32_t dst = smem_u32(smem + C::OFF_KV + s * C::TILE) + (ch >> 3) * (kBN * 128);
#pragma unroll
          for (int g = 0; g < kBN / 32; ++g) {
            int at[32 / RPI];
#pragma unroll
            for (int r = 0; r < 32 / RPI; ++r) at[r] = __shfl_sync(0xffffffffu, row[g], r * RPI + lane / LPR);
#pragma unroll
            for (int r = 0; r < 32 / RPI; ++r) {
              const int m = 32 * g + r * RPI + lane / LPR;  // rows behind the sequence: zeros
              cp_async16(dst + m * 128 + (((ch & 7) ^ (m & 7)) << 4), src + max(at[r], 0) * row_elems, at[r] >= 0);
            }
          }
          cp_async_arrive(&sh.full[s]);
        }
      }
      T += i;
    }
    if (lane == 0)  // shared memory is not released under a copy
      for (int i = max(0, T - (ST + 1) / 2); i < T; ++i) {
        const int y = 2 * i + is_v;
        if (y + ST >= 2 * T) mbar_wait(&sh.full[y % ST], (y / ST) & 1u, A.err, 0x623);
      }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // One thread issues both slots' products in turn, PV(j) and QK(j + 1) of slot 0, then of slot 1, so
    // that each slot's softmax has the time of the other's products. (An issuing thread for each slot
    // let the two fall into step, both in the softmax at once and then both on the tensor core: 542 us
    // against 470 us for an 8192-token prompt, before the elected lane issued.)
    const uint64_t q0 = umma_sdesc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
    const uint64_t k0 = umma_sdesc_sw128(smem_u32(smem + C::OFF_KV), 16, 1024);
    const uint64_t v0 = umma_sdesc_sw128(smem_u32(smem + C::OFF_KV), kBN * 128, 1024);
    bool ok = true;
    Ring<ST> ring;                           // the next item's first K
    int nq = 0;                              // Q loads of earlier items
    int np0 = 0, np1 = 0, nf0 = 0, nf1 = 0;  // tiles, and items with tiles, of each slot so far
    const bool by_lanes = A.box == 0;
    for (int k = 0; ok; ++k) {
      if (!mbar_wait_warp(&sh.item_full[k & 1], (k >> 1) & 1u, A.err, 0x62d)) break;
      const Item it = read_item(&sh.item[k & 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_empty[k & 1]);
      if (it.end) break;
      const bool dual = it.dual;
      const int nj = it.j1 - it.j0, na = it.j1a - it.j0;
      if (elect_one() && nj > 0) {
        // a wait that has run out fails the later ones at once; the products then issued read
        // nothing but shared and tensor memory, and their results are not used
        auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
          if (!mbar_try_wait(bar, parity)) ok = ok && mbar_wait(bar, parity, A.err, code);
        };
        auto wait_full = [&](const Ring<ST>& r) {
          wait(&sh.full[r.s], r.parity, 0x625);
          if (by_lanes) fence_proxy_async_smem();  // cp.async wrote through the generic proxy
        };
        auto qk = [&](int x, const Ring<ST>& r) {
          const uint64_t a = q0 + (uint64_t)((dual && x ? C::TILE : 0) >> 4), b = k0 + (uint64_t)((r.s * C::TILE) >> 4);
          const uint32_t tS = tmem + C::S_COL + x * 128;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int off = (kk >> 2) * (kBN * 128) + (kk & 3) * 32;
            umma_bf16(tS, a + (uint64_t)(off >> 4), b + (uint64_t)(off >> 4), C::IDESC_QK, kk > 0 ? 1u : 0u);
          }
          umma_commit(&sh.s_full[x]);
        };
        auto pv = [&](int x, const Ring<ST>& r, uint32_t parity, bool first) {
          const uint64_t b = v0 + (uint64_t)((r.s * C::TILE) >> 4);
          const uint32_t tS = tmem + C::S_COL + x * 128, tO = tmem + C::O_COL + x * 128;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            wait(half ? &sh.p_full[x] : &sh.p_half[x], parity, 0x626);
            tc_fence_after();
#pragma unroll
            for (int kk = half * (kBN / 32); kk < (half + 1) * (kBN / 32); ++kk)
              umma_bf16_ts(tO, tS + kk * 8, b + (uint64_t)((kk * 2048) >> 4), C::IDESC_PV, (kk > 0 || !first) ? 1u : 0u);
          }
        };
        wait(&sh.q_full, nq & 1u, 0x624);
        Ring<ST> r = ring;  // the current tile's K; its V is the next entry
        if (dual) {
          wait_full(r);
          if (na > 0) qk(0, r);
          qk(1, r);
          umma_commit(&sh.empty[r.s]);
          if (nj == 1) umma_commit(&sh.q_empty);
          if (nf0 > 0 && na > 0) wait(&sh.o_free[0], (nf0 - 1) & 1u, 0x62e);
          if (nf1 > 0) wait(&sh.o_free[1], (nf1 - 1) & 1u, 0x62e);
          uint32_t par0 = np0 & 1u, par1 = np1 & 1u;
          for (int n = 0; ok && n < nj; ++n) {
            const Ring<ST> v = r.next(1);
            r = r.next(2);
            wait_full(v);
            if (n < na) {
              pv(0, v, par0, n == 0);
              if (n + 1 < na) {
                wait_full(r);
                qk(0, r);
              } else {
                umma_commit(&sh.o_full[0]);
              }
            }
            pv(1, v, par1, n == 0);
            umma_commit(&sh.empty[v.s]);
            if (n + 1 < nj) {
              if (n + 1 >= na) wait_full(r);
              qk(1, r);
              umma_commit(&sh.empty[r.s]);
              if (n + 2 == nj) umma_commit(&sh.q_empty);
            } else {
              umma_commit(&sh.o_full[1]);
            }
            par0 ^= 1u;
            par1 ^= 1u;
          }
        } else {
          for (int x = 0; x < 2 && x < nj; ++x) {
            const Ring<ST> e = x ? r.next(2) : r;
            wait_full(e);
            qk(x, e);
            umma_commit(&sh.empty[e.s]);
            if (x + 1 == nj) umma_commit(&sh.q_empty);
          }
          if (nf0 > 0) wait(&sh.o_free[0], (nf0 - 1) & 1u, 0x62e);
          if (nf1 > 0 && nj > 1) wait(&sh.o_free[1], (nf1 - 1) & 1u, 0x62e);
          for (int e = 0; ok && e < nj; ++e) {
            const int x = e & 1;
            const Ring<ST> v = r.next(1), f = r.next(4);
            r = r.next(2);
            wait_full(v);
            pv(x, v, ((x ? np1 : np0) + (e >> 1)) & 1u, e < 2);
            umma_commit(&sh.empty[v.s]);
            if (e + 2 < nj) {
              wait_full(f);
              qk(x, f);
              umma_commit(&sh.empty[f.s]);
              if (e + 3 == nj) umma_commit(&sh.q_empty);
            } else {
              umma_commit(&sh.o_full[x]);
            }
          }
        }
        if (!ok) {  // TMEM is not freed under an MMA
          umma_commit(&sh.drain);
          mbar_wait(&sh.drain, 0, A.err, 0x628);
        }
      }
      ok = !__any_sync(0xffffffffu, !ok);
      {
        const int y = ring.s + 2 * nj, turns = y / ST;
        ring.s = y - turns * ST;
        ring.parity ^= turns & 1u;
      }
      nq += nj > 0;
      np0 += it.count(0);
      np1 += it.count(1);
      nf0 += it.count(0) > 0;
      nf1 += it.count(1) > 0;
    }
  } else {
    // ------------------------------------------------------------ softmax of one slot, a thread a row
    const int x = warp >> 2, qd = warp & 3, m = qd * 32 + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(qd * 32) << 16);
    const uint32_t tS = t_lane + C::S_COL + x * 128, tO = t_lane + C::O_COL + x * 128;
    const float c = A.scale_log2;
    // an arrival of the whole warp
    auto arrive = [&](uint64_t* bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    uint32_t ns = 0, no = 0, nx = 0;  // tiles, results and merges of this slot so far
    const int tt = m / A.G;
    // this row's part of item k, if there is one
    struct Part {
      int cnt, dual, t, some;
      bool live;
      Seen sn;
    };
    auto look = [&](int k, Part& p) {
      const Item& it = sh.item[k & 1];
      p.some = mbar_wait_warp(&sh.item_full[k & 1], (k >> 1) & 1u, A.err, 0x62d) && !it.end;
      if (!p.some) return;
      p.cnt = it.count(x);
      p.dual = it.dual;
      p.t = it.t0 + (p.dual ? x * A.TQ : 0) + tt;
      p.live = tt < A.TQ && p.t < it.n;
      p.sn = seen(A, it.pos0 + p.t, it.pos0 + p.t, it.len);
    };
    Part part;
    look(0, part);
    for (int k = 0; ok && part.some; ++k) {
      const Item& it = sh.item[k & 1];  // given back at the end: few registers are left beside S
      const int cnt = part.cnt, dual = part.dual, t = part.t;
      const bool live = part.live, warp_live = __any_sync(0xffffffffu, live);
      const Seen sn = part.sn;
      float m_ref = -INFINITY, l = 0.f;
      for (int n = 0; ok && n < cnt; ++n) {
        const int k0 = it.tile(it.j0 + (dual ? n : 2 * n + x)) * kBN;
        if (!(ok = mbar_wait_warp(&sh.s_full[x], ns++ & 1u, A.err, 0x629))) break;
        tc_fence_after();
        if (warp_live) {
          float s[128];
          tmem_ld128_sync(tS, s);
          const bool all = (k0 >= sn.lo && k0 + kBN - 1 <= sn.hi) || k0 + kBN - 1 <= sn.g1 || !live;
          if (!__all_sync(0xffffffffu, all)) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t bits = range_bits(sn.lo, sn.hi, k0 + 32 * w) | range_bits(0, sn.g1, k0 + 32 * w);
#pragma unroll
              for (int e = 0; e < 32; ++e) s[32 * w + e] = (bits & (1u << e)) ? s[32 * w + e] : -INFINITY;
            }
          }
          float m8[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            m8[y] = fmax3(s[y], s[y + 8], s[y + 16]);
#pragma unroll
            for (int z = 24; z < 120; z += 16) m8[y] = fmax3(m8[y], s[y + z], s[y + z + 8]);
            m8[y] = fmaxf(m8[y], s[y + 120]);
          }
          const float mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * c;
          float alpha = 1.f;
          bool need = false;
          if (mx > m_ref + kRescaleThreshold) {
            if (m_ref != -INFINITY) {
              alpha = ex2(m_ref - mx);
              need = true;
            }
            m_ref = mx;
          }
          if (__any_sync(0xffffffffu, need)) {  // (S of this tile is there: the earlier PV is done)
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 8) {  // rare, and S is in registers
              float o[8];
              tmem_ld8_sync(tO + c0, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= alpha;
              tmem_st8_sync(tO + c0, o);
            }
          }
          const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
          const uint64_t c2 = f32x2_pack(c, c), nm2 = f32x2_pack(neg_m, neg_m);
          uint64_t l2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float a0, a1;
              f32x2_unpack(f32x2_fma(f32x2_pack(s[64 * half + 2 * e], s[64 * half + 2 * e + 1]), c2, nm2), a0, a1);
              const float p0 = ex2(a0), p1 = ex2(a1);
              l2[e & 3] = f32x2_add(l2[e & 3], f32x2_pack(p0, p1));
              pk[e] = pack_bf16x2(p0, p1);  // bf16 for the MMA, off by 2^-8 at most; the sum takes the fp32 values
            }
            tmem_st32_sync(tS + 32 * half, pk);
            arrive(half ? &sh.p_full[x] : &sh.p_half[x]);
          }
          float lp[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) f32x2_unpack(l2[y], lp[2 * y], lp[2 * y + 1]);
          l = l * alpha + (((lp[0] + lp[1]) + (lp[2] + lp[3])) + ((lp[4] + lp[5]) + (lp[6] + lp[7])));
        } else if (lane == 0) {
          mbar_arrive(&sh.p_half[x]);
          mbar_arrive(&sh.p_full[x]);
        }
      }
      look(k + 1, part);  // under the last PV (eight 1024-token prompts: 74.9 us, 76.9 when looked up afterwards)
      // ---- result
      if (ok && cnt > 0) ok = mbar_wait_warp(&sh.o_full[x], no++ & 1u, A.err, 0x62a);
      tc_fence_after();
      float w0 = 1.f, w1 = 0.f;  // weights of this slot's O and, for a single tile, of slot 1's
      const bool other = !dual && x == 0 && it.count(1) > 0;
      if (!dual && x == 1 && cnt > 0) {  // (slot 0 gives O, and with it row, back)
        sh.row[m] = make_float2(m_ref, l);
        arrive(&sh.x_full);
      }
      if (other) {
        if (ok) ok = mbar_wait_warp(&sh.x_full, nx++ & 1u, A.err, 0x62f);
        tc_fence_after();
        const float2 ml = sh.row[m];
        const float M = fmaxf(m_ref, ml.x);
        if (M != -INFINITY) {
          w0 = exp2f(m_ref - M);
          w1 = exp2f(ml.x - M);
          l = l * w0 + ml.y * w1;
          m_ref = M;
        } else {
          l += ml.y;  // 0, or NaN where the query is one: maxima pass over NaN
        }
      }
      if (warp_live && (dual || x == 0)) {
        const float inv = l != 0.f ? 1.f / l : 0.f;  // a NaN among the scores stays one
        const float row_lse = l != 0.f ? (m_ref + log2f(l)) * kLn2 : -INFINITY;
        w0 *= inv;
        w1 *= inv;
        const int h = it.hk * A.G + (m - tt * A.G);
        const int64_t row = (int64_t)(it.q0 + t) * A.Hq + h;
        int64_t prow = 0, step = 8;  // the row's LSE; elements between eighths of its values
        float* pvalues = nullptr;
        if (it.ns > 1) {
          const Rank rk = rank_of(P, it.rank);
          if constexpr (SHARED) {
            const SharedPart to(rk, A.Hq, A.G, it.c, it.hk, t, m - tt * A.G);
            prow = to.lse();
            pvalues = A.part_o + to.values(D, 0);
            step = (int64_t)to.rows * 8;
          } else {
            prow = rk.part + ((int64_t)it.c * rk.qn + t) * A.Hq + h;
            pvalues = A.part_o + prow * D;
          }
        }
        // (Short code: a CTA comes here once an item and has to fetch it. With the loops unrolled, windowed
        // chunks took 62.6 us against 59, an 8192-token prompt 318 against 315. Four lanes that exchanged
        // pieces of their rows by shuffles, to store whole 128-byte lines, lost 4 us to the exchange.)
        if (it.ns == 1 && !other && cnt > 0) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            tmem_ld32_sync(tO + c0, o);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(o[2 * e] * w0, o[2 * e + 1] * w0);
            if (live) {
              store32(A.o + row * D + c0, w);
              store32(A.o + row * D + c0 + 16, w + 8);
            }
          }
        } else {
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
          if (cnt > 0) {
            tmem_ld32_sync(tO + c0, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= w0;
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
          if (other) {
            float o1[32];
            tmem_ld32_sync(tO + 128 + c0, o1);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(o1[e], w1, o[e]);
          }
          if (live) {
            if (it.ns > 1) {
#pragma unroll
              for (int e = 0; e < 32; e += 8)
                store32(pvalues + (c0 + e) / 8 * step, reinterpret_cast<const uint32_t*>(o) + e);
            } else {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
              store32(A.o + row * D + c0, w);
              store32(A.o + row * D + c0 + 16, w + 8);
            }
          }
        }
        }
        if (live) {
          if (it.ns > 1) A.part_lse[prow] = row_lse == row_lse ? row_lse : INFINITY;  // the merge makes a NaN of it again
          else if (A.lse) A.lse[row] = row_lse;
        }
      }
      // what has been read of O may be overwritten by the slot's next item
      if ((dual || x == 0) && cnt > 0) arrive(&sh.o_free[x]);
      if (other) arrive(&sh.o_free[1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_empty[k & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// One warp per (new token, query head) of the requests that were cut. It reads ns fp32 partials of d + 1
// a row, which stay in L2 (one 30,000-token sequence, 32 rows in 19 pieces: 44 us with the attention, of
// which 18 are the cache at copy speed).
template <int D, int CAP>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const __grid_constant__ ChunkArgs A,
                                                          const __grid_constant__ Plan<CAP, false> P, int req0, int n_rows) {
  constexpr int E = D / 32;
  const int64_t mr = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (mr >= n_rows) return;
  int lo = 0, hi = P.n - 1;  // the first rank whose rows end behind this one
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (P.rows[mid] > mr) hi = mid;
    else lo = mid + 1;
  }
  const int y = (int)mr - (lo > 0 ? P.rows[lo - 1] : 0), r = req0 + P.req[lo], t = y / A.Hq;
  const int q0 = __ldg(A.q_indptr + r), n = __ldg(A.q_indptr + r + 1) - q0;
  if (q0 < 0 || t >= n || q0 > A.N - min(n, P.qn[lo])) return;
  const int64_t pr = (int64_t)P.part[lo] + y;
  const size_t stride = (size_t)P.qn[lo] * A.Hq;
  float out[E];
  const float L = merge_row<E>(A.part_o + pr * D, stride * D, A.part_lse + pr, stride, P.ns[lo], lane, out);
  const int64_t row = (int64_t)(q0 + t) * A.Hq + y % A.Hq;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(A.o + row * D + lane * E + e) = pack_bf16x2(out[e], out[e + 1]);
  if (A.lse && lane == 0) A.lse[row] = L;
}

// Four merged rows a warp: a rank's own partials, and before them its prefix's. Lane (eighth x of 4, row y of 4, half z):
// 16 bytes of its row's eighths x, x + 4, .., so that four rows side by side are whole lines. It starts as the first
// kernel's CTAs end, finds its rows, then waits for the last of them.
// U partials of a row are on their way at once: 4, or 2 with twice the warps, for more rows than the SMs take at once otherwise
// that have three partials or fewer on average (132224 rows of two 35 us, 49 by four; calls of 16384 rows of more 67 us, 64
// by four, of 2048 rows 45.7 and 37.3).
template <int D, int CAP, int U>
__global__ void __launch_bounds__(128, U == 2 ? 8 : 1) chunk_merge_shared_kernel(const __grid_constant__ ChunkArgs A,
                                                                                 const __grid_constant__ Plan<CAP, true> P, int req0,
                                                                                 int n_rows) {
  constexpr int NV = D / 32;  // 16-byte parts of a lane
  const int lane = threadIdx.x & 31, z = lane & 1, sub = (lane >> 3) * 2 + z;  // sub: of the 8 lanes of a row
  grid_go();
  const int64_t mr = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * 4 + ((lane >> 1) & 3);
  bool some = mr < n_rows;
  int lo = 0, hi = P.n - 1;  // the first rank whose rows end behind this one
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (P.rows[mid] > mr) hi = mid;
    else lo = mid + 1;
  }
  const Rank k = rank_of(P, lo);
  const int y = some ? (int)mr - (lo > 0 ? P.rows[lo - 1] : 0) : 0, r = req0 + k.req;
  const int g = y % A.G, ht = y / A.G, hk = ht / k.qn, t = ht - hk * k.qn;
  const int q0 = list_word<true>(A.q_indptr + r), n = list_word<true>(A.q_indptr + r + 1) - q0;
  some = some && q0 >= 0 && t < n && q0 <= A.N - min(n, k.qn);
  SharedPart own(k, A.Hq, A.G, 0, hk, t, g), pre = own;
  int na = 0;  // the prefix's partials
  if (k.pre >= 0) {
    const Rank kp = rank_of(P, k.pre);
    const int64_t tg = (int64_t)q0 + t - list_word<true>(A.q_indptr + req0 + kp.req);  // its token of the group's
    some = some && tg >= 0 && tg < kp.qn;
    if (some) pre = SharedPart(kp, A.Hq, A.G, 0, hk, (int)tg, g);
    na = kp.ns;
    if (some && y == 0 && sub == 0) {  // the request's list holds the pages that were read for it
      const int e = k.skip / A.page_size - 1, lead = req0 + k.lead;
      const int a = list_word<true>(A.page_indptr + r) + e, b = list_word<true>(A.page_indptr + lead) + e;
      if (a < 0 || a >= list_word<true>(A.page_indptr + r + 1) || b < 0 || b >= list_word<true>(A.page_indptr + lead + 1) ||
          list_word<true>(A.page_indices + a) != list_word<true>(A.page_indices + b))
        record_error(A.err, 0x609);
    }
  }
  grid_wait();  // the partials: written while this kernel ran, so not by way of the cache for what is constant
  const int s = some ? na + k.ns : 0;
  int most = s;
#pragma unroll
  for (int d = 2; d <= 4; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
  auto lse_at = [&](int i) {
    return i < s ? A.part_lse[i < na ? pre.lse() + (int64_t)i * pre.rows : own.lse() + (int64_t)(i - na) * own.rows] : -INFINITY;
  };
  auto value = [&](int i, int v) {
    const SharedPart& p = i < na ? pre : own;
    const int64_t c = (int64_t)(i < na ? i : i - na) * p.rows;  // rows of the chunks before
    return *reinterpret_cast<const float4*>(A.part_o + p.values(D, (lane >> 3) + 4 * v) + c * D + z * 4);
  };
  float4 x[U][NV];
  float w[U];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[u] = lse_at(i0 + u);
      if (i0 + u < s)
#pragma unroll
        for (int v = 0; v < NV; ++v) x[u][v] = value(i0 + u, v);
    }
  };
  load(0);  // (before the maximum is known)
  float M = -INFINITY;
  for (int i = sub; i < most; i += 8) M = fmaxf(M, lse_at(i));
#pragma unroll
  for (int d : {1, 8, 16}) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float4 out[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) out[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int i0 = 0; i0 < most; i0 += U) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < s && M != -INFINITY) {
        const float e = exp2f((w[u] - M) * kLog2e);
        sum += e;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          out[v].x = fmaf(e, x[u][v].x, out[v].x);
          out[v].y = fmaf(e, x[u][v].y, out[v].y);
          out[v].z = fmaf(e, x[u][v].z, out[v].z);
          out[v].w = fmaf(e, x[u][v].w, out[v].w);
        }
      }
  }
  if (!some) return;
  const float inv = M != -INFINITY ? 1.f / sum : 0.f;
  const int64_t row = (int64_t)(q0 + t) * A.Hq + hk * A.G + g;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    *reinterpret_cast<uint2*>(A.o + row * D + ((lane >> 3) + 4 * v) * 8 + z * 4) =
        make_uint2(pack_bf16x2(out[v].x * inv, out[v].y * inv), pack_bf16x2(out[v].z * inv, out[v].w * inv));
  if (A.lse && sub == 0) A.lse[row] = M != -INFINITY ? M + logf(sum) : -INFINITY;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
               : nullptr;
  }();
  return fn;
}

// [rows, heads, d] bf16 as a 3-D tensor (d, heads, rows), `stride` elements between rows; box (64, bh, br).
bool make_map(CUtensorMap* m, const void* base, int d, int heads, int64_t rows, int64_t stride, int bh, int br) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)br}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cache's [rows, heads, d] as (d, rows, heads), boxes of 64 x br x the heads of a CTA of few rows.
bool make_row_map(CUtensorMap* m, const void* base, int d, int heads, int64_t rows, int br) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {(cuuint64_t)heads * d * 2, (cuuint64_t)d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)br, (cuuint32_t)row_heads(heads)}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Requests from r0 on as one launch: its ranks, and how much scratch they need.
struct Group {
  int r0 = 0;
  int64_t items = 0, rows = 0, parts = 0;  // items; merged rows; partial rows
  struct Rank {
    int req, qn, ns;
    int64_t base, row1, part;
    int skip, pre, end, lead;  // with shared prefixes
  };
  bool shared = false;  // some prefix is computed once for its group
  int n_rows = 0, row_ctas = 0, ctas = 0, runs = 0, run = 0;
  std::vector<Rank> ranks;
};

// Ranks of a launch: the plan travels in the launch's parameters, 1.2 KB of them for up to 64 requests,
// 18 KB for more (copied at each launch: 58 us of host time a call of 64 requests, 88 with the large one).
constexpr int kSmallPlan = 64, kLargePlan = 1024;
constexpr int kSmallShared = 96, kLargeShared = 768;  // (64 requests and their prefixes)

// Requests that share their first tokens, on the host: requests indptr[i] .. indptr[i + 1] - 1 the first prefix[i].
struct Prefixes {
  int n = 0;
  const int32_t* indptr = nullptr;
  const int32_t* prefix = nullptr;
};

// What the host plans with: a request, what it has behind its group's prefix, or a prefix.
struct Req {
  int req, n, units, first, last, ns;  // new tokens, pairs of query tiles, key tiles of the first and last pair
  int skip, pre, end, lead;            // as in Plan; pre: number of the prefix among reqs, -1 none, -2 itself one
  int few;                             // few rows: their own keys, else 0
};
constexpr int kMaxAuto = 256;    // chunks that the plan cuts a list into at most
constexpr double kItem = 2.0;    // an item's prologue and epilogue, in key tiles
constexpr double kMerge = 4.0;   // the merge launch

constexpr double kPieceUs = 0.25;  // merge: a partial of a row (it reads four at a time)
// Nothing shared is estimated too where sharing saves less than 20 tiles an SM; it takes less than its estimate, since what requests
// share lies in L2 then. (344 batches of all sizes, few rows by CTAs of their own, in items, or nothing shared: the choice takes
// 1.02 times the best of the three on average, 1.5 at most, and 0.79 of what the chunk attention takes.)
constexpr double kNone = 0.25, kClear = 20.0;  // (a quarter: no estimate, 1 us of host time; sharing won 3 us there at most)
double apart(const ChunkArgs& a) { return (a.d == 128 ? 0.85 : 0.7) + (a.box > 0 ? 0.0 : 0.15); }

// Measured: a run of few rows takes 3.5 us and 1.0 a tile of 16 keys
// of 8 heads of 128 (others 0.65; a piece 2 of them more); an item of query tiles 7.5 us and 1.5 a key tile (heads of 64: 1.25), 3 again for
// each further one of its CTA.
struct RowTimes {
  int heads;  // of a CTA of few rows
  double tile_us, row_us;
  explicit RowTimes(const ChunkArgs& a)
      : heads(row_heads(a.Hkv)), tile_us(a.d == 128 ? 1.5 : 1.25), row_us(heads == 8 && a.d == 128 ? 1.0 : 0.65) {}
  bool few(int keys) const {
    const int t = (keys + 15) / 16;
    return row_us * (t + kStart) < heads * (tile_us * t / 8 + 3.0);
  }
};

// Chunks of a launch with shared prefixes, and the CTAs of few rows; its time. The launch ends when its bytes have come, when the
// last of the prefixes' items is done or the last CTA of few rows. For each share of the SMs
// the length of the prefixes' pieces that ends soonest is taken, and the best share.
double plan_shared(const ChunkArgs& a, std::vector<Req>& reqs, int num_splits, int sms, Group& g) {
  constexpr int kTiles = 14, kKeys = 16;
  const RowTimes times(a);
  const int heads = times.heads, groups = (a.Hkv + heads - 1) / heads;
  const double tile_us = times.tile_us, row_us = times.row_us, key_bytes = 4.0 * a.d;
  int64_t row = 0;  // the tiles of few rows, one after the other
  double bytes = 0;
  int most = 1;
  for (Req& q : reqs) {
    bytes += (q.few ? (double)q.few : (double)kBN * std::max(q.first, q.last)) * a.Hkv * key_bytes;
    if (q.few) row += (q.few + kKeys - 1) / kKeys + kStart;
    else most = std::max(most, std::max(q.first, q.last));
  }
  std::vector<const Req*> by_len;  // the others, longest first
  int longest_few = 1;
  for (const Req& q : reqs)
    if (q.few) longest_few = std::max(longest_few, q.few);
    else by_len.push_back(&q);
  std::stable_sort(by_len.begin(), by_len.end(),
                   [](const Req* x, const Req* y) { return std::max(x->first, x->last) > std::max(y->first, y->last); });
  struct Cut {  // items of one length, us
    int64_t end;
    double each;
  };
  struct Tiles {  // the items of pieces of `tiles` key tiles: the times of the longest one, of all and of the merge, us
    int tiles;
    int64_t items;
    double longest, work, merge;
    size_t c0;  // its first among the cuts
  } t[kTiles];
  std::vector<Cut> cuts;
  cuts.reserve(kTiles * by_len.size());
  int nt = 0;
  for (int tiles = most; nt < kTiles; tiles = std::max(2, tiles * 3 / 4)) {
    Tiles& x = t[nt++];
    x = Tiles{tiles, 0, 0, 0, 0, cuts.size()};
    int pieces = 0;
    for (const Req* r : by_len) {
      const Req& q = *r;
      const int len = std::max(q.first, q.last), ns = num_splits ? num_splits : std::min(kMaxAuto, (len + tiles - 1) / tiles);
      const int64_t items = (int64_t)q.units * a.Hkv * ns;
      const double each = tile_us * 0.5 * (q.first + q.last) / ns + 3.0;
      x.items += items;
      if (cuts.size() > x.c0 && cuts.back().each == each) cuts.back().end = x.items;
      else cuts.push_back(Cut{x.items, each});
      x.work += each * (double)items;
      x.merge += (double)q.n * a.Hq * ns * 4.0 * (a.d + 1) / 5e6;
      x.longest = std::max(x.longest, tile_us * len / ns);
      pieces = std::max(pieces, ns);
    }
    x.merge += kPieceUs * pieces;
    if (tiles <= 2 || num_splits) break;
  }
  // what the CTA with the most to do of m takes: items 0, m, 2 m, ..
  auto rounds = [&](const Tiles& x, int m) {
    if (x.items > 8 * (int64_t)m) return x.work / m + 0.5 * x.longest;
    double sum = 0;
    size_t c = x.c0;
    for (int64_t i = 0; i < x.items; i += m) {
      while (cuts[c].end <= i) ++c;
      sum += cuts[c].each;
    }
    return sum;
  };
  double best = 0;
  int best_tiles = 0, best_runs = 0;
  constexpr int shares = 24;
  for (int c = 0; c < shares; ++c) {
    const int runs = std::max(1, std::min(sms - 1, sms * (c + 1) / (shares + 1)) / groups), m = std::max(1, sms - runs * groups);
    const int64_t run = (row + runs - 1) / runs;
    const double t_rows = 3.5 + row_us * (double)run, merge = kPieceUs * row_turns(a.Hkv) * ((longest_few / kKeys + kStart) / (double)run + 1.0);
    double t_tiles = 0;
    int bt = 0;
    for (int i = 0; i < nt; ++i) {
      const double end = 4.5 + std::max(t[i].longest + 3.0, rounds(t[i], m)) + t[i].merge;
      if (i == 0 || end < t_tiles) {
        t_tiles = end;
        bt = i;
      }
    }
    const double end = std::max(bytes / 6.5e6 + 5.0, std::max(t_rows, t_tiles)) + 0.05 * (t_rows + t_tiles) + merge;
    if (c == 0 || end < best) {
      best = end;
      best_tiles = bt;
      best_runs = runs;
    }
  }
  for (Req& q : reqs)
    if (!q.few && num_splits == 0)
      q.ns = std::min(kMaxAuto, std::max(1, (std::max(q.first, q.last) + t[best_tiles].tiles - 1) / t[best_tiles].tiles));
  {
    // a run longer than what a piece costs of itself; a request is cut into no more than 256 pieces
    if (num_splits) best_runs = num_splits;
    g.run = (int)std::max<int64_t>({(row + best_runs - 1) / best_runs, kStart + 1, (longest_few / kKeys + kStart) / (kMaxAuto - 2) + 1});
    g.runs = (int)((row + g.run - 1) / g.run);
    g.row_ctas = g.runs * groups;
  }
  g.ctas = (int)std::min<int64_t>(std::max(sms / 8, sms - g.row_ctas), t[best_tiles].items);
  return 1.1 * best;  // (what it took against this and the other estimate, in the batches of apart())
}

// Chunks of a launch without CTAs of few rows, and its time in us. The launch ends when the SM with the most to do does: with
// the items sorted by length and handed out one by one that is about the largest of an SM's share, the longest item, and
// k times the item number (k - 1) * SMs + 1 (some SM has k items of at least that length). Cutting shortens items
// and adds to the share: a prologue each, fp32 partials written and read, and a merge. Lengths of
// pieces from the longest list down are tried and the best estimate is kept. (64 single tokens over
// 522,892 cached ones: 345 us whole, 333 in the pieces found, 421 in 16 pieces each; a 2048-token
// prompt: 79 us in pieces of 8 tiles, 40 whole.)
double plan_items(const ChunkArgs& a, std::vector<Req>& reqs, bool shared, int sms) {
  const double tile_us = RowTimes(a).tile_us;
  int most = 0;
  struct Same {  // requests of one length (beside shared prefixes the short ones are counted together: most of 64 are)
    int tiles;
    double len;
    int64_t units, rows;
    bool part;
  };
  std::vector<Same> all;
  all.reserve(reqs.size());
  constexpr int kShort = 64;
  int at[2 * kShort];
  std::fill(at, at + 2 * kShort, -1);
  for (const Req& q : reqs) {
    const int tiles = std::max(q.first, q.last);
    most = std::max(most, tiles);
    if (shared && q.first == q.last && tiles < kShort) {
      int& i = at[tiles + (q.pre != -1 ? kShort : 0)];
      if (i >= 0) {
        all[i].units += q.units;
        all[i].rows += q.n;
        continue;
      }
      i = (int)all.size();
    }
    all.push_back(Same{tiles, 0.5 * (q.first + q.last), q.units, q.n, q.pre != -1});
  }
  auto chunks = [&](int tiles, int piece) {  // (piece is 0 where no token sees a key)
    return std::min(kMaxAuto, std::max(1, (tiles + piece - 1) / std::max(1, piece)));
  };
  auto estimate = [&](int piece) {
    constexpr int kBins = 32;
    double work = 0, longest = 0;
    int pieces = 1;
    int64_t bins[kBins] = {0};  // items by length, in steps of the longest possible one / 32
    const double step = (std::min(piece, most) + kItem) / kBins;
    bool cut = false;
    for (const Same& q : all) {
      const int ns = chunks(q.tiles, piece);
      const int64_t items = q.units * a.Hkv * ns;
      const double len = q.len / ns + kItem;
      work += len * (double)items;
      longest = std::max(longest, (double)q.tiles / ns + kItem);
      bins[std::min(kBins - 1, (int)(len / step))] += items;
      if (ns > 1 || q.part) {
        cut = true;
        pieces = std::max(pieces, ns);
        work += (double)q.rows * a.Hq * ns * 8.0 * (a.d + 1) / 65536.0;  // (a tile of K and V is 64 KB at most)
      }
    }
    double end = std::max(work / sms, longest);
    int64_t before = 0, k = 1;
    for (int b = kBins - 1; b >= 0 && k <= 8; --b) {
      for (; k <= 8 && (k - 1) * sms < before + bins[b]; ++k) end = std::max(end, (double)k * (b + 0.5) * step);
      before += bins[b];
    }
    return end + (cut ? kMerge : 0.0) + (shared ? kPieceUs * pieces / tile_us : 0.0);
  };
  int best = most;
  double best_end = estimate(most);
  for (int piece = most; piece > 2;) {
    piece = std::max(2, piece * 2 / 3);
    const double end = estimate(piece);
    if (end < 0.97 * best_end) {
      best = piece;
      best_end = end;
    }
  }
  for (Req& q : reqs) q.ns = chunks(std::max(q.first, q.last), best);
  return 4.5 + tile_us * best_end;
}

sta_status plan_group(const ChunkArgs& a, const int32_t* qi, const int32_t* ki, const Prefixes& pf, int r0, int r1,
                      int num_splits, int sms, Group& g) {
  std::vector<Req> reqs;
  reqs.reserve(pf.n > 0 ? 2 * (size_t)(r1 - r0) : (size_t)(r1 - r0));
  g.r0 = r0;
  // What it saves to compute a group's prefix once, in the time of key tiles of a pair of query tiles; kNot: there is
  // nothing to share. An item takes 3 more beside its tiles, few rows 0.4 for 16 keys and twice that more a piece.
  constexpr double kNot = -1e300;
  auto saves = [&](int r, int end, int64_t skip) -> double {
    int some = 0, n = 0;
    double apart = 0, own = 0;
    auto items = [&](int m, int64_t keys) {  // of m tokens over keys: a single query tile takes half of a pair's time
      const int q = (m + a.TQ - 1) / a.TQ;
      return a.Hkv * (0.5 * q * (double)((keys + kBN - 1) / kBN) + 3.0 * ((q + 1) / 2));
    };
    for (int x = r; x < end; ++x) {
      const int m = qi[x + 1] - qi[x];
      if (m == 0) continue;
      const int64_t len = (int64_t)ki[x + 1] - ki[x];
      ++some;
      n += m;
      apart += items(m, len);
      own += (int64_t)m * a.G <= 16 && a.row_box > 0 ? 0.4 * (double)((len - skip + 15) / 16 + kStart) * ((a.Hkv + 7) / 8) : items(m, len - skip);
    }
    if (some < 2 || skip == 0) return kNot;
    return apart - own - items(n, skip) - 2.0 * n * a.Hq * 8.0 * (a.d + 1) / 65536.0;
  };
  double sum = 0;
  for (int i = 0; i < pf.n; ++i) {
    const int from = std::max(r0, (int)pf.indptr[i]), to = std::min(r1, (int)pf.indptr[i + 1]);
    if (from < to) sum += std::max(0.0, saves(from, to, pf.prefix[i]));
  }
  auto tiles_of = [&](int n, int64_t len, int u) {  // key tiles of pair u
    int gt, wl;
    const int64_t t0 = (int64_t)2 * u * a.TQ, te = std::min<int64_t>(n, t0 + 2 * a.TQ), p0 = len - n;
    return tile_list(seen(a, p0 + t0, p0 + te - 1, len), gt, wl);
  };
  auto units_of = [&](int n) { return ((n + a.TQ - 1) / a.TQ + 1) / 2; };
  auto add = [&](int r, int64_t skip, int pre, int lead) {  // request r's keys from token `skip` on
    const int n = qi[r + 1] - qi[r], units = units_of(n);
    const int64_t len = (int64_t)ki[r + 1] - ki[r] - skip;
    reqs.push_back(Req{r - r0, n, units, tiles_of(n, len, 0), tiles_of(n, len, units - 1), std::max(num_splits, 1), (int)skip, pre,
                       r - r0 + 1, lead, (int64_t)n * a.G <= 16 ? (int)len : 0});
  };
  auto fill = [&](bool share) {
    reqs.clear();
    g.shared = false;
    for (int r = r0, i = 0; r < r1;) {
      int end = r + 1;
      if (pf.n > 0) {
        while (pf.indptr[i + 1] <= r) ++i;
        end = std::min(r1, (int)pf.indptr[i + 1]);  // (a group that two launches meet in is two groups)
        if (const double saved = share ? saves(r, end, pf.prefix[i]) : kNot; num_splits > 0 ? saved > kNot : saved > 0) {
          int lead = r;
          while (qi[lead + 1] == qi[lead]) ++lead;
          const int n = qi[end] - qi[r], tiles = (pf.prefix[i] + kBN - 1) / kBN, me = (int)reqs.size();
          reqs.push_back(Req{r - r0, n, units_of(n), tiles, tiles, std::max(num_splits, 1), pf.prefix[i], -2, end - r0, lead - r0, 0});
          g.shared = true;
          for (; r < end; ++r)
            if (qi[r + 1] > qi[r]) add(r, pf.prefix[i], me, lead - r0);
          continue;
        }
      }
      for (; r < end; ++r)
        if (qi[r + 1] > qi[r]) add(r, 0, -1, 0);
    }
  };
  fill(num_splits > 0 ? pf.n > 0 : sum > kNone * sms);
  // Few rows: pages that hold no boxes of 8 tokens are copied token by token (44 us for a case that takes 33 in items); and
  // a request takes the time of a tile of 16 keys of all of its CTA's heads, or an item for each.
  const RowTimes times(a);
  bool rows = false;
  int64_t items = 0;
  for (Req& q : reqs) {
    if (!g.shared || a.row_box == 0 || (num_splits == 0 && !times.few(q.few))) q.few = 0;
    rows = rows || q.few > 0;
    items += q.few ? 0 : (int64_t)q.units * a.Hkv;
  }
  if (num_splits > 0) {
    if (rows) plan_shared(a, reqs, num_splits, sms, g);
  } else {
    double end = plan_items(a, reqs, g.shared, sms);
    // three rounds of items and more: those of few rows are dealt out with them, by CTAs that take over one another's
    rows = rows && items <= 3 * sms;
    if (rows) {
      const std::vector<Req> whole = reqs;
      const double t = plan_shared(a, reqs, 0, sms, g);
      rows = t < end;
      if (rows) end = t;
      else reqs = whole;
    }
    if (!rows) {
      for (Req& q : reqs) q.few = 0;
      g.run = g.runs = g.row_ctas = g.ctas = 0;
    }
    if (g.shared && sum < kClear * sms) {  // or nothing shared
      std::vector<Req> shared;
      reqs.swap(shared);
      fill(false);
      for (Req& q : reqs) q.few = 0;
      if (apart(a) * plan_items(a, reqs, false, sms) > end) {
        reqs.swap(shared);
        g.shared = true;
      } else {
        g.run = g.runs = g.row_ctas = g.ctas = 0;
      }
    }
  }
  auto longest = [](const Req& q) { return q.few ? 1e9 : (double)std::max(q.first, q.last) / q.ns; };
  std::vector<int> order(reqs.size()), rank(reqs.size());
  std::iota(order.begin(), order.end(), 0);
  std::stable_sort(order.begin(), order.end(), [&](int x, int y) { return longest(reqs[x]) > longest(reqs[y]); });
  for (int i : order) {
    Req& q = reqs[i];
    const int64_t part = g.parts;
    const int64_t tiles = q.few ? (q.few + 15) / 16 + kStart : 0;  // (first in the order: base counts tiles so far)
    if (q.few) q.ns = (int)((g.items + tiles - 1) / g.run - g.items / g.run + 1) * row_turns(a.Hkv);
    if (q.ns > 1 || q.pre != -1) {
      if (q.pre != -2) g.rows += (int64_t)q.n * a.Hq;
      g.parts += (int64_t)q.n * a.Hq * q.ns;
    }
    rank[i] = (int)g.ranks.size();
    g.ranks.push_back(Group::Rank{q.req, q.n, q.ns, g.items, g.rows, part, q.skip, q.pre, q.end, q.lead});
    if (q.few) {
      ++g.n_rows;
      g.items += tiles;
    } else {
      g.items += (int64_t)q.units * a.Hkv * q.ns;
    }
  }
  for (Group::Rank& k : g.ranks)
    if (k.pre >= 0) k.pre = rank[k.pre];
  if (g.items > INT32_MAX || g.parts > INT32_MAX / 2) return STA_ERR_UNSUPPORTED;
  return STA_OK;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

constexpr unsigned kManyRows = 152 * 4;  // CTAs of the merge that an SM takes at once, with four partials on their way

struct Maps {
  CUtensorMap q, k, v, k4, v4;  // k4, v4: boxes of 32 tokens, beside those of 8
  RowMaps<true> rows;
};

// A launch that may start while the one before it on the stream ends (see grid_wait).
template <class... F, class... T>
cudaError_t launch_early(void (*kern)(F...), unsigned grid, int threads, int smem, cudaStream_t st, const T&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, int CAP, bool SHARED>
sta_status launch_group(const Maps& m, const ChunkArgs& a, const Group& g, cudaStream_t st) {
  Plan<CAP, SHARED> p;
  p.n = (int)g.ranks.size();
  for (int i = 0; i < p.n; ++i) {
    const Group::Rank& k = g.ranks[i];
    p.base[i] = (int32_t)k.base;
    p.rows[i] = (int32_t)k.row1;
    if constexpr (SHARED) {
      p.rank[i] = Rank{(int32_t)k.part, k.qn, k.skip, (uint16_t)k.req, (uint16_t)k.ns, (uint16_t)k.end, (uint16_t)k.lead, (int16_t)k.pre, 0};
    } else {
      p.part[i] = (int32_t)k.part;
      p.qn[i] = k.qn;
      p.req[i] = (uint16_t)k.req;
      p.ns[i] = (uint16_t)k.ns;
    }
  }
  p.base[p.n] = (int32_t)g.items;
  unsigned grid = (unsigned)g.items;
  if constexpr (SHARED) {
    p.n_rows = g.n_rows;
    p.row_ctas = g.row_ctas;
    p.ctas = g.ctas;
    p.runs = g.runs;
    p.run = g.run;
    if (g.row_ctas > 0) grid = (unsigned)(g.row_ctas + g.ctas);
  }
  auto kern = chunk_kernel<D, CAP, SHARED>;
  STA_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM));
  if constexpr (SHARED) {
    STA_CUDA_TRY(launch_early(kern, grid, kThreads, Cfg<D>::SMEM, st, m.q, m.k, m.v, m.k4, m.v4, m.rows, a, p, g.r0));
  } else {
    kern<<<grid, kThreads, Cfg<D>::SMEM, st>>>(m.q, m.k, m.v, m.k4, m.v4, RowMaps<false>{}, a, p, g.r0);
    STA_LAUNCH_CHECK();
  }
  if (g.rows > 0) {
    if constexpr (SHARED) {
      const unsigned ctas = (unsigned)cdiv(g.rows, 16);
      const auto merge = ctas > kManyRows && g.parts <= 3 * g.rows ? chunk_merge_shared_kernel<D, CAP, 2> : chunk_merge_shared_kernel<D, CAP, 4>;
      STA_CUDA_TRY(launch_early(merge, ctas, 128, 0, st, a, p, g.r0, (int)g.rows));
    } else {
      chunk_merge_kernel<D, CAP><<<(unsigned)cdiv(g.rows, 8), 256, 0, st>>>(a, p, g.r0, (int)g.rows);
      STA_LAUNCH_CHECK();
    }
  }
  return STA_OK;
}

template <int D>
sta_status launch_any(const Maps& m, const ChunkArgs& a, const Group& g, cudaStream_t st) {
  if (g.shared)
    return g.ranks.size() <= kSmallShared ? launch_group<D, kSmallShared, true>(m, a, g, st)
                                          : launch_group<D, kLargeShared, true>(m, a, g, st);
  return g.ranks.size() <= kSmallPlan ? launch_group<D, kSmallPlan, false>(m, a, g, st) : launch_group<D, kLargePlan, false>(m, a, g, st);
}

// The two calls: with groups of requests that share their first tokens, or none of them.
sta_status chunk_fwd(const void* q, int64_t q_stride, const void* k_pages, const void* v_pages, int page_size, int n_pages,
                     const int32_t* page_indptr_dev, const int32_t* page_indices_dev, const int32_t* q_indptr_dev,
                     const int32_t* q_indptr_host, const int32_t* kv_indptr_dev, const int32_t* kv_indptr_host, int n_req,
                     int Hq, int Hkv, int d, sta_dtype dtype, float scale, const sta_mask_src* pattern, const Prefixes& pf,
                     int num_splits, void* o, float* lse, void* workspace, size_t* workspace_bytes, sta_stream stream) {
  constexpr int64_t kFar = (int64_t)1 << 31;  // beyond any distance between two tokens
  if (!workspace_bytes || !q_indptr_host || !kv_indptr_host || n_req < 1 || Hq < 1 || Hkv < 1 || page_size < 1 ||
      n_pages < 1 || num_splits < 0 || num_splits > 1024)
    return STA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0 || !(scale > 0.f) || !std::isfinite(scale)) return STA_ERR_INVALID_ARG;
  if (dtype != STA_BF16 || (d != 64 && d != 128) || Hq / Hkv > kBM || Hq > 65535) return STA_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * page_size > INT32_MAX) return STA_ERR_UNSUPPORTED;
  if (q_indptr_host[0] != 0 || kv_indptr_host[0] != 0) return STA_ERR_INVALID_ARG;
  for (int r = 0; r < n_req; ++r)
    if (q_indptr_host[r + 1] < q_indptr_host[r] || kv_indptr_host[r + 1] < kv_indptr_host[r]) return STA_ERR_INVALID_ARG;
  if (kv_indptr_host[n_req] > INT32_MAX - 2 * kBN) return STA_ERR_UNSUPPORTED;
  for (int i = 0; i < pf.n; ++i) {  // every new token lies behind its group's prefix
    if (pf.prefix[i] < 0 || pf.prefix[i] % page_size != 0) return STA_ERR_INVALID_ARG;
    for (int r = pf.indptr[i]; r < pf.indptr[i + 1]; ++r) {
      const int n = q_indptr_host[r + 1] - q_indptr_host[r];
      if (n > 0 && (int64_t)kv_indptr_host[r + 1] - kv_indptr_host[r] - n < pf.prefix[i]) return STA_ERR_INVALID_ARG;
    }
  }
  ChunkArgs a{};
  a.causal = 1;
  a.win_lo = -kFar;
  a.win_hi = kFar;
  if (pattern) {
    if (pattern->kind != STA_MASK_PATTERN || pattern->n_global_cols < 0) return STA_ERR_INVALID_ARG;
    a.causal = pattern->causal != 0;
    a.win_lo = std::max(-kFar, std::min(kFar, pattern->win_lo));
    a.win_hi = std::max(-kFar, std::min(kFar, pattern->win_hi));
    a.n_global = std::min(kFar, pattern->n_global_cols);
  }
  if (q_stride == 0) q_stride = (int64_t)Hq * d;
  if (q_stride < (int64_t)Hq * d || (q_stride & 7)) return q_stride & 7 ? STA_ERR_UNSUPPORTED : STA_ERR_INVALID_ARG;
  a.N = q_indptr_host[n_req];
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.G = Hq / Hkv;
  a.TQ = kBM / a.G;
  a.page_size = page_size;
  a.n_pages = n_pages;
  // n / P for 0 <= n < 2^31: with 2^l >= P > 2^(l-1) and m = ceil(2^(31+l) / P) < 2^32 it is n m >> (31 + l),
  // since n (m - 2^(31+l) / P) < 2^31 <= 2^(31+l) / P
  int l = 0;
  while (((int64_t)1 << l) < page_size) ++l;
  a.page_mul = (uint32_t)((((uint64_t)1 << (31 + l)) + page_size - 1) / page_size);
  a.page_shift = l - 1;
  const int box = std::gcd(page_size, kBN);
  a.box = box % 8 == 0 ? box : 0;
  a.row_box = std::min(a.box, 16);
  a.scale_log2 = scale * kLog2e;
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaGetLastError();  // a size query also works where there is no device
  std::vector<Group> groups;
  int64_t parts = 0;
  const int batch = pf.n > 0 ? kLargeShared * 2 / 3 : kLargePlan;  // (a prefix has two requests at least)
  for (int r0 = 0; r0 < n_req; r0 += batch) {
    Group g;
    const sta_status st = plan_group(a, q_indptr_host, kv_indptr_host, pf, r0, std::min(n_req, r0 + batch), num_splits, sms, g);
    if (st != STA_OK) return st;
    parts = std::max(parts, g.parts);
    groups.push_back(std::move(g));
  }
  const size_t o_bytes = align256((size_t)parts * d * sizeof(float));
  const size_t need = std::max<size_t>(256, o_bytes + align256((size_t)parts * sizeof(float)));
  if (!workspace) {
    *workspace_bytes = need;
    return STA_OK;
  }
  if (*workspace_bytes < need) {
    *workspace_bytes = need;
    return STA_ERR_WORKSPACE;
  }
  if ((uintptr_t)workspace & 255) return STA_ERR_UNSUPPORTED;
  if (a.N == 0) return STA_OK;
  if (!q || !k_pages || !v_pages || !page_indptr_dev || !q_indptr_dev || !kv_indptr_dev || !o) return STA_ERR_INVALID_ARG;
  if (!page_indices_dev && kv_indptr_host[n_req] > 0) return STA_ERR_INVALID_ARG;  // (no sequence holds a page)
  if (((uintptr_t)q | (uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)o) & 15) return STA_ERR_UNSUPPORTED;
  if (((uintptr_t)page_indptr_dev | (uintptr_t)page_indices_dev | (uintptr_t)q_indptr_dev | (uintptr_t)kv_indptr_dev |
       (uintptr_t)lse) & 3)
    return STA_ERR_UNSUPPORTED;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.lse = lse;
  a.k = static_cast<const __nv_bfloat16*>(k_pages);
  a.v = static_cast<const __nv_bfloat16*>(v_pages);
  a.page_indptr = page_indptr_dev;
  a.page_indices = page_indices_dev;
  a.q_indptr = q_indptr_dev;
  a.kv_indptr = kv_indptr_dev;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + o_bytes);
  a.err = device_error_word();
  Maps m;
  const int64_t rows = (int64_t)n_pages * page_size, kv_stride = (int64_t)Hkv * d;
  const int kv_box = a.box > 0 ? a.box : 8;
  bool maps = make_map(&m.q, q, d, Hq, a.N, q_stride, a.G, a.TQ) && make_map(&m.k, k_pages, d, Hkv, rows, kv_stride, 1, kv_box) &&
              make_map(&m.v, v_pages, d, Hkv, rows, kv_stride, 1, kv_box);
  if (a.box == 0) {
    maps = maps && make_map(&m.k4, k_pages, d, Hkv, rows, kv_stride, 1, 32) && make_map(&m.v4, v_pages, d, Hkv, rows, kv_stride, 1, 32);
  } else {
    m.k4 = m.k;
    m.v4 = m.v;
  }
  bool few = false;
  for (const Group& g : groups) few = few || g.row_ctas > 0;
  if (few)
    maps = maps && make_row_map(&m.rows.k, k_pages, d, Hkv, rows, a.row_box) && make_row_map(&m.rows.v, v_pages, d, Hkv, rows, a.row_box);
  else
    m.rows.k = m.rows.v = m.k;  // not used
  if (!maps) {
    note_cuda_error(cudaErrorInvalidValue);  // tensor-map encoding refused
    return STA_ERR_CUDA;
  }
  const cudaStream_t s = (cudaStream_t)stream;
  for (const Group& g : groups) {
    if (g.items == 0) continue;
    const sta_status st = d == 64 ? launch_any<64>(m, a, g, s) : launch_any<128>(m, a, g, s);
    if (st != STA_OK) return st;
  }
  return STA_OK;
}

}  // namespace
}  // namespace sta

using namespace sta;

extern "C" sta_status sta_chunk_fwd_paged(const void* q, int64_t q_stride, const void* k_pages, const void* v_pages,
                                          int page_size, int n_pages, const int32_t* page_indptr_dev,
                                          const int32_t* page_indices_dev, const int32_t* q_indptr_dev,
                                          const int32_t* q_indptr_host, const int32_t* kv_indptr_dev,
                                          const int32_t* kv_indptr_host, int n_req, int Hq, int Hkv, int d,
                                          sta_dtype dtype, float scale, const sta_mask_src* pattern, int num_splits,
                                          void* o, float* lse, void* workspace, size_t* workspace_bytes,
                                          sta_stream stream) try {
  return chunk_fwd(q, q_stride, k_pages, v_pages, page_size, n_pages, page_indptr_dev, page_indices_dev, q_indptr_dev,
                   q_indptr_host, kv_indptr_dev, kv_indptr_host, n_req, Hq, Hkv, d, dtype, scale, pattern, Prefixes{},
                   num_splits, o, lse, workspace, workspace_bytes, stream);
} catch (...) {  // no memory for the plan
  return STA_ERR_INVALID_ARG;
}

extern "C" sta_status sta_prefix_fwd_paged(const void* q, int64_t q_stride, const void* k_pages, const void* v_pages,
                                           int page_size, int n_pages, const int32_t* page_indptr_dev,
                                           const int32_t* page_indices_dev, const int32_t* q_indptr_dev,
                                           const int32_t* q_indptr_host, const int32_t* kv_indptr_dev,
                                           const int32_t* kv_indptr_host, int n_req, const int32_t* group_indptr_host,
                                           const int32_t* prefix_host, int n_groups, int Hq, int Hkv, int d,
                                           sta_dtype dtype, float scale, int num_splits, void* o, float* lse,
                                           void* workspace, size_t* workspace_bytes, sta_stream stream) try {
  if (n_req < 1 || n_groups < 1 || !group_indptr_host || !prefix_host) return STA_ERR_INVALID_ARG;
  if (group_indptr_host[0] != 0 || group_indptr_host[n_groups] != n_req) return STA_ERR_INVALID_ARG;
  for (int i = 0; i < n_groups; ++i)
    if (group_indptr_host[i + 1] < group_indptr_host[i]) return STA_ERR_INVALID_ARG;
  return chunk_fwd(q, q_stride, k_pages, v_pages, page_size, n_pages, page_indptr_dev, page_indices_dev, q_indptr_dev,
                   q_indptr_host, kv_indptr_dev, kv_indptr_host, n_req, Hq, Hkv, d, dtype, scale, nullptr,
                   Prefixes{n_groups, group_indptr_host, prefix_host}, num_splits, o, lse, workspace, workspace_bytes, stream);
} catch (...) {  // no memory for the plan
  return STA_ERR_INVALID_ARG;
}
