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
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <numeric>
#include <vector>

#include "internal.h"
#include "ptx.cuh"

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
  float scale_log2;
  int causal;
  int64_t win_lo, win_hi, n_global;
  int* err;
};

// What the host planned: the requests with new tokens, longest key lists first. Rank k has the items
// base[k] .. base[k+1]-1: ((pair of query tiles, from the last down) * Hkv + KV head) * ns + chunk.
template <int CAP>
struct Plan {
  int n;                // ranks
  int32_t base[CAP + 1];
  int32_t rows[CAP];    // merged rows up to and with the rank's (those of requests that are cut)
  int32_t part[CAP];    // first partial row
  int32_t qn[CAP];      // new tokens of the request on the host
  uint16_t req[CAP];    // request, from the launch's first
  uint16_t ns[CAP];     // chunks
};

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

template <int CAP>
__device__ __forceinline__ bool get_item(const ChunkArgs& A, const Plan<CAP>& P, int req0, int item, Item& it) {
  int lo = 0, hi = P.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (P.base[mid] <= item) lo = mid;
    else hi = mid;
  }
  it.end = 0;
  it.rank = lo;
  it.ns = P.ns[lo];
  const int x = item - P.base[lo], per_u = A.Hkv * it.ns, units = (P.base[lo + 1] - P.base[lo]) / per_u;
  const int u = units - 1 - x / per_u, y = x - (x / per_u) * per_u;
  it.hk = y / it.ns;
  it.c = y - it.hk * it.ns;
  it.r = req0 + P.req[lo];
  const int q0 = __ldg(A.q_indptr + it.r), q1 = __ldg(A.q_indptr + it.r + 1);
  const int64_t len = (int64_t)__ldg(A.kv_indptr + it.r + 1) - __ldg(A.kv_indptr + it.r);
  it.pb = __ldg(A.page_indptr + it.r);  // (with the lengths, not later by the loaders: a 2048-token prompt 36 us, 39)
  it.pe = __ldg(A.page_indptr + it.r + 1);
  int n = q1 - q0;
  if (n > P.qn[lo]) {
    record_error(A.err, 0x606);
    n = P.qn[lo];
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
  it.pos0 = (int)(len - (q1 - q0));
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

template <int D, int CAP>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k4,
                 const __grid_constant__ CUtensorMap tm_v4, const __grid_constant__ ChunkArgs A,
                 const __grid_constant__ Plan<CAP> P, int req0) {
  using C = Cfg<D>;
  constexpr int ST = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<ST>& sh = *reinterpret_cast<Shared<ST>*>(smem + C::OFF_S);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(smem) & 1023) {  // swizzle atoms start on 1024-byte boundaries
    record_error(A.err, 0x607);
    return;
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
      Item it;
      for (int n = 0; ok && item >= 0; ++n) {
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
        clc_request(&sh.clc, &sh.clc_full);
        item = mbar_wait(&sh.clc_full, n & 1u, A.err, 0x62c) ? clc_answer(&sh.clc) : -1;
        fence_proxy_async_smem();  // the answer has been read before the next one is written
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
      return o >= 0 && o < pe && A.page_indices ? __ldg(A.page_indices + o) : -1;
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
        int pg = nj > 0 && b < boxes ? page_at(it.tile(it.j0) * kBN + off) : -1;
        for (; i < nj; ++i) {
          const int y = 2 * (T + i) + is_v, s = y % ST, tok0 = it.tile(it.j0 + i) * kBN, page = pg;
          if (i + 1 < nj && b < boxes) pg = page_at(it.tile(it.j0 + i + 1) * kBN + off);
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
        const int64_t prow = it.ns > 1 ? P.part[it.rank] + ((int64_t)it.c * P.qn[it.rank] + t) * A.Hq + h : 0;
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
                store32(A.part_o + prow * D + c0 + e, reinterpret_cast<const uint32_t*>(o) + e);
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
                                                          const __grid_constant__ Plan<CAP> P, int req0, int n_rows) {
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

// Requests from r0 on as one launch: its ranks, and how much scratch they need.
struct Group {
  int r0 = 0;
  int64_t items = 0, rows = 0, parts = 0;  // items; merged rows; partial rows
  struct Rank {
    int req, qn, ns;
    int64_t base, row1, part;
  };
  std::vector<Rank> ranks;
};

// Ranks of a launch: the plan travels in the launch's parameters, 1.2 KB of them for up to 64 requests,
// 18 KB for more (copied at each launch: 58 us of host time a call of 64 requests, 88 with the large one).
constexpr int kSmallPlan = 64, kLargePlan = 1024;

sta_status plan_group(const ChunkArgs& a, const int32_t* qi, const int32_t* ki, int r0, int r1, int num_splits, int sms,
                      Group& g) {
  constexpr int kMaxAuto = 256;
  constexpr double kItem = 2.0;    // an item's prologue and epilogue, in key tiles
  constexpr double kMerge = 4.0;   // the merge launch
  struct Req {
    int req, n, units, first, last, ns;  // new tokens, pairs of query tiles, key tiles of the first and last pair
  };
  std::vector<Req> reqs;
  g.r0 = r0;
  auto tiles_of = [&](int n, int64_t len, int u) {  // key tiles of pair u
    int gt, wl;
    const int64_t t0 = (int64_t)2 * u * a.TQ, te = std::min<int64_t>(n, t0 + 2 * a.TQ), p0 = len - n;
    return tile_list(seen(a, p0 + t0, p0 + te - 1, len), gt, wl);
  };
  int most = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = qi[r + 1] - qi[r];
    if (n == 0) continue;
    const int64_t len = (int64_t)ki[r + 1] - ki[r];
    const int units = ((n + a.TQ - 1) / a.TQ + 1) / 2;
    reqs.push_back(Req{r - r0, n, units, tiles_of(n, len, 0), tiles_of(n, len, units - 1), std::max(num_splits, 1)});
    most = std::max(most, std::max(reqs.back().first, reqs.back().last));
  }
  // Chunks. The launch ends when the SM with the most to do does: with the items sorted by length and
  // handed out one by one that is about the largest of an SM's share, the longest item, and k times the
  // item number (k - 1) * SMs + 1 (some SM has k items of at least that length). Cutting shortens items
  // and adds to the share: a prologue each, fp32 partials written and read, and a merge. Lengths of
  // pieces from the longest list down are tried and the best estimate is kept. (64 single tokens over
  // 522,892 cached ones: 345 us whole, 333 in the pieces found, 421 in 16 pieces each; a 2048-token
  // prompt: 79 us in pieces of 8 tiles, 40 whole.)
  if (num_splits == 0 && most > 2) {
    auto chunks = [&](int tiles, int piece) { return std::min(kMaxAuto, std::max(1, (tiles + piece - 1) / piece)); };
    auto estimate = [&](int piece) {
      constexpr int kBins = 32;
      double work = 0, longest = 0;
      int64_t bins[kBins] = {0};  // items by length, in steps of the longest possible one / 32
      const double step = (std::min(piece, most) + kItem) / kBins;
      bool cut = false;
      for (const Req& q : reqs) {
        const int tiles = std::max(q.first, q.last), ns = chunks(tiles, piece);
        const int64_t items = (int64_t)q.units * a.Hkv * ns;
        const double len = 0.5 * (q.first + q.last) / ns + kItem;
        work += len * (double)items;
        longest = std::max(longest, (double)tiles / ns + kItem);
        bins[std::min(kBins - 1, (int)(len / step))] += items;
        if (ns > 1) {
          cut = true;
          work += (double)q.n * a.Hq * ns * 8.0 * (a.d + 1) / 65536.0;  // (a tile of K and V is 64 KB at most)
        }
      }
      double end = std::max(work / sms, longest);
      int64_t before = 0, k = 1;
      for (int b = kBins - 1; b >= 0 && k <= 8; --b) {
        for (; k <= 8 && (k - 1) * sms < before + bins[b]; ++k) end = std::max(end, (double)k * (b + 0.5) * step);
        before += bins[b];
      }
      return end + (cut ? kMerge : 0.0);
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
  }
  auto longest = [](const Req& q) { return (double)std::max(q.first, q.last) / q.ns; };
  std::stable_sort(reqs.begin(), reqs.end(), [&](const Req& x, const Req& y) { return longest(x) > longest(y); });
  for (const Req& q : reqs) {
    const int64_t part = g.parts;
    if (q.ns > 1) {
      g.rows += (int64_t)q.n * a.Hq;
      g.parts += (int64_t)q.n * a.Hq * q.ns;
    }
    g.ranks.push_back(Group::Rank{q.req, q.n, q.ns, g.items, g.rows, part});
    g.items += (int64_t)q.units * a.Hkv * q.ns;
  }
  if (g.items > INT32_MAX || g.parts > INT32_MAX / 2) return STA_ERR_UNSUPPORTED;
  return STA_OK;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Maps {
  CUtensorMap q, k, v, k4, v4;  // k4, v4: boxes of 32 tokens, beside those of 8
};

template <int D, int CAP>
sta_status launch_group(const Maps& m, const ChunkArgs& a, const Group& g, cudaStream_t st) {
  Plan<CAP> p;
  p.n = (int)g.ranks.size();
  for (int i = 0; i < p.n; ++i) {
    const Group::Rank& k = g.ranks[i];
    p.base[i] = (int32_t)k.base;
    p.rows[i] = (int32_t)k.row1;
    p.part[i] = (int32_t)k.part;
    p.qn[i] = k.qn;
    p.req[i] = (uint16_t)k.req;
    p.ns[i] = (uint16_t)k.ns;
  }
  p.base[p.n] = (int32_t)g.items;
  auto kern = chunk_kernel<D, CAP>;
  STA_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM));
  kern<<<(unsigned)g.items, kThreads, Cfg<D>::SMEM, st>>>(m.q, m.k, m.v, m.k4, m.v4, a, p, g.r0);
  STA_LAUNCH_CHECK();
  if (g.rows > 0) {
    chunk_merge_kernel<D, CAP><<<(unsigned)cdiv(g.rows, 8), 256, 0, st>>>(a, p, g.r0, (int)g.rows);
    STA_LAUNCH_CHECK();
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
  a.scale_log2 = scale * kLog2e;
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaGetLastError();  // a size query also works where there is no device
  std::vector<Group> groups;
  int64_t parts = 0;
  for (int r0 = 0; r0 < n_req; r0 += kLargePlan) {
    Group g;
    const sta_status st = plan_group(a, q_indptr_host, kv_indptr_host, r0, std::min(n_req, r0 + kLargePlan), num_splits, sms, g);
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
  if (!maps) {
    note_cuda_error(cudaErrorInvalidValue);  // tensor-map encoding refused
    return STA_ERR_CUDA;
  }
  const cudaStream_t s = (cudaStream_t)stream;
  for (const Group& g : groups) {
    if (g.items == 0) continue;
    const sta_status st = g.ranks.size() <= kSmallPlan ? (d == 64 ? launch_group<64, kSmallPlan>(m, a, g, s)
                                                       : launch_group<128, kSmallPlan>(m, a, g, s))
                                            : (d == 64 ? launch_group<64, kLargePlan>(m, a, g, s)
                                                       : launch_group<128, kLargePlan>(m, a, g, s));
    if (st != STA_OK) return st;
  }
  return STA_OK;
} catch (...) {  // no memory for the plan
  return STA_ERR_INVALID_ARG;
}
