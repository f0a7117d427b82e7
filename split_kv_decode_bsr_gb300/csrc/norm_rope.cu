// Root-mean-square norms of query and key heads with the rotary positions in the same pass: alone
// (sta_norm_rope), its gradient (sta_norm_rope_bwd) and fused with the write of new tokens into a
// paged KV cache (sta_norm_rope_append_paged).
//
//   y = R_t (x r w),  r = 1 / sqrt(mean(x^2) + eps)
//   g = R_t' dy,  dx = r (g w - x r mean(g w x r)),  dw = sum over tokens and heads of g x r
//
// L lanes of a warp (a power of two) share a head: each holds the 16-byte vectors (half layout: pairs
// of them, half a rotation apart) that the rotary kernel calls units, so that the turn needs no exchange
// and the sums over a head are log2 L shuffles; the warp's 32 / L neighbouring heads of one tensor and token are
// a piece of work. Warps work on their own: each takes an equal run of the pieces (tokens, then the heads of q,
// k and v), copies its next pieces to shared memory ahead of its work (16-byte copies that the same lane reads
// again), and puts the cosines and sines of the token that it has come to into a table of its own. A head is read once
// and written once; the products in between stay in fp32 and are rounded once. The turns are exact at any position, as
// in the rotary kernel.
//
// What bounds it (8192 tokens of 32 + 8 heads of 128 in bf16, graph of calls back to back). Forward 29.6 us, 5.7 TB/s of the
// 168 MB it has to move where a copy reaches 6.78 (24.7 us); HBM, with 64 % of the issue slots taken. Backward 51.5 us
// (37.1 at copy speed): 125 registers allow 16 warps an SM, which take 58 % of the issue slots, and each waits for its
// loads, its sums' shuffles and its results in turn (3 CTAs an SM spill: 84; 20 warps with the weights in shared memory 54). The 11975 tokens of 24 prompts, 32 + 4 + 4
// heads, into pages of 100: 45.9 (36.2). Small calls are the launch: 64 tokens into the cache 4.0 us, one step's norms 2.5.
#include <type_traits>

#include "rope.inl"
#include "shares.h"

namespace sta {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
template <typename T> constexpr int kMany = sizeof(T) == 2 ? 2 : 4;  // units of a lane where a head has more than 32 (at most 64, 128)
constexpr int kMaxGrid = 152 * 2;  // CTAs of a backward pass, each with a row of partial sums for dw
// What a lane holds of a head's turning part: vectors half a rotation apart; neighbouring pairs; those where the rotation
// ends inside a vector (looked at in kPairs too, that costs 3 of 30 us); or vectors as they come, whose partners half a
// rotation away, where that is no whole number of vectors, it reads from the other lanes' copies.
enum Layout { kHalves, kPairs, kPairsEnd, kPlain };
template <int NU> constexpr int kSlots = NU <= 2 ? 3 : 2;  // pieces that a warp has on their way
template <int W, int LY, int NU>
constexpr int ctas_an_sm(bool backward) {
  return W == 1 || NU * (LY == kHalves ? 2 : 1) > 2 ? 1 : (backward || (LY == kPlain && NU == 2) ? 2 : 3);
}
enum Mode { kForward, kAppend, kBackward };

struct NormArgs {
  const uint8_t* src[3];  // q, k, v (v: to pages alone)
  uint8_t* dst[3];        // backward: dq, dk
  const uint8_t* dy[2];   // backward: the gradients of the results
  int64_t src_stride[3], dst_stride[3], dy_stride[2];  // bytes between tokens (k, v pages: of a page)
  const float* weight[2];
  int heads[3];
  int pieces[3];          // of a token: 32 / L heads of q, k or v each
  int64_t n_tokens;
  int d, rot;
  int units, rot_units;   // units of a head; the first rot_units turn
  int log_l;              // lanes of a head
  int warp_bytes;         // shared memory of a warp
  float eps, inv_d, mscale;
  const int32_t* positions;
  // paged destination of k and v
  const int32_t* q_indptr;
  const int32_t* kv_indptr;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  int n_req, page_size, n_pages;
  int* err;
  int ctas_q;             // backward: the CTAs of q, then those of k
  float* part;            // backward: [CTAs, d]
};

// Where new tokens go, found by a whole warp. The next token of a request is looked for only where a page ends.
struct Place {
  int pos = 0;        // the token's position
  int64_t row = -1;   // its cache row, -1 when it goes nowhere
  bool live = false;  // false: padding
  int64_t end = -1;   // tokens of the request end here
  int64_t list = 0, list_end = 0;
  int left = 0;       // rows of the page behind this one

  __device__ __forceinline__ void find_page(const NormArgs& A, int lane) {
    const int64_t e = list + pos / A.page_size;
    const int in = pos % A.page_size;
    row = -1;
    left = A.page_size - 1 - in;
    if (e < 0 || e >= list_end) {
      if (lane == 0) record_error(A.err, 0x604);
      return;
    }
    const int page = A.page_indices[e];
    if (page < 0 || page >= A.n_pages) {
      if (lane == 0) record_error(A.err, 0x110);
      return;
    }
    row = (int64_t)page * A.page_size + in;
  }
  // 128 requests are looked at at once, where one thread's binary search would take a round trip to memory for
  // each of its steps
  __device__ __forceinline__ void find(const NormArgs& A, int64_t t, int lane) {
    pos = 0;
    row = -1;
    left = 0;
    const int first = A.q_indptr[0], all = A.q_indptr[A.n_req];
    int lo = 0, n = A.n_req;  // the last request that starts at or before t is among lo .. lo + n - 1
    while (n > 1) {
      const int step = (n + 127) >> 7;
      int c = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = (lane + 32 * k) * step;
        c += __popc(__ballot_sync(0xffffffffu, at < n && A.q_indptr[lo + at] <= t));
      }
      c = max(c - 1, 0) * step;
      lo += c;
      n = min(step, n - c);
    }
    live = t >= first && t < all;
    end = -1;
    if (!live) return;
    const int64_t q1 = A.q_indptr[lo + 1], len = (int64_t)A.kv_indptr[lo + 1] - A.kv_indptr[lo];
    list = A.page_indptr[lo];
    list_end = A.page_indptr[lo + 1];
    const int64_t p = len - (q1 - t);
    if (p < 0 || t >= q1) {  // the sequence is shorter than its chunk: this token is not in it
      pos = (int)(p < INT32_MIN ? INT32_MIN : p);
      return;
    }
    end = q1;
    pos = (int)p;
    find_page(A, lane);
  }
  __device__ __forceinline__ void next(const NormArgs& A, int64_t t, int lane) {  // t - 1 was the last one
    if (t >= end) {
      find(A, t, lane);
      return;
    }
    ++pos;
    if (left == 0) {
      find_page(A, lane);
    } else {
      --left;
      row += row >= 0;
    }
  }
};

__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_both(float x) { return f32x2_pack(x, x); }
__device__ __forceinline__ float f32x2_sum(uint64_t x) {
  float a, b;
  f32x2_unpack(x, a, b);
  return a + b;
}

// 16 bytes to shared memory, or 16 zero bytes where `some` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A weight, by a plain load: the kernel before this one may have written it (a gradient, say) while this one had started. It
// keeps its place behind the wait for that kernel (both are volatile), but not behind the results that have been stored before
// it, which no weight is (as a load of C++ 30.4 us where this takes 29.6).
__device__ __forceinline__ float weight_at(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// A thread's units of its heads: the same elements of every head it works on. In fp32 a unit is NP
// couples of pairs, first elements in A and second ones in B, for the packed instructions (twice the
// products of an issue slot, which is what bounds these kernels first: 8192 tokens x 40 heads of 128 in
// bf16 took 36.9 us with scalar ones). A unit that does not turn has its elements there just so (half layout: in A).
template <typename T, int W, int LY, int NU>
struct Units {
  static constexpr bool IL = LY != kHalves, PL = LY == kPlain;  // a vector a unit; with partners elsewhere
  static constexpr int WI = IL && W == 1 ? 2 : W;  // elements of a vector: whole pairs when interleaved
  static constexpr int PP = IL ? WI / 2 : WI;      // pairs of a unit
  static constexpr int NP = (PP + 1) / 2;
  int unit[NU];  // -1: none
  int off[NU];   // first element
  bool turn[NU];
  int half, d;
  int partner[PL ? NU : 1][PL ? W : 1];  // byte of an element's partner in a slot
  static constexpr int V = NU * (IL ? 1 : 2);      // vectors of a head that a lane holds
  struct Row {  // elements that are not there are 0
    Vec<T, WI> a[NU], b[IL ? 1 : NU];
  };
  struct Half2 {
    uint64_t a[NP], b[NP];
  };
  __device__ __forceinline__ void set(const NormArgs& A) {
    const int l = threadIdx.x & ((1 << A.log_l) - 1);
    half = A.rot >> 1;
    d = A.d;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int u = l + (j << A.log_l);
      turn[j] = u < A.rot_units;
      unit[j] = u < A.units ? u : -1;
      off[j] = IL || turn[j] ? u * WI : A.rot + (u - A.rot_units) * WI;
      if (unit[j] < 0) off[j] = 0;
      if constexpr (PL) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const int p = partner_of(off[j] + e, A.rot), v = p / W;
          partner[j][e] = (v >> A.log_l) * 512 + ((threadIdx.x & 31) - l + (v & ((1 << A.log_l) - 1))) * 16 + p % W * (int)sizeof(T);
        }
      }
    }
  }
  static __device__ __forceinline__ int partner_of(int e, int rot) {
    return e >= rot ? e : (e < rot >> 1 ? e + (rot >> 1) : e - (rot >> 1));
  }
  // the partners of unit j's elements, out of a slot that the warp has filled
  __device__ __forceinline__ Half2 partners(const uint8_t* slot, int j) const {
    auto at = [&](int e) { return to_f(*reinterpret_cast<const T*>(slot + partner[PL ? j : 0][PL ? e : 0])); };
    Half2 x;
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      x.a[m] = f32x2_pack(at(4 * m), at(4 * m + 2));
      x.b[m] = f32x2_pack(at(4 * m + 1), at(4 * m + 3));
    }
    return x;
  }
  // x turned with its partners p, or back: [NP][cosines, signed sines][units that turn] of 4
  __device__ __forceinline__ void rotate(const NormArgs& A, const float2* s_cs, int j, Half2& x, const Half2& p, bool back) const {
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      const float4 c = reinterpret_cast<const float4*>(s_cs)[2 * m * A.rot_units + unit[j]];
      float4 s = reinterpret_cast<const float4*>(s_cs)[(2 * m + 1) * A.rot_units + unit[j]];
      if (back) s = make_float4(-s.x, -s.y, -s.z, -s.w);
      const int e = off[j] + 4 * m;
      x.a[m] = turned(f32x2_fma(p.a[m], f32x2_pack(s.x, s.y), f32x2_mul(x.a[m], f32x2_pack(c.x, c.y))), x.a[m], e, A.rot);
      x.b[m] = turned(f32x2_fma(p.b[m], f32x2_pack(s.z, s.w), f32x2_mul(x.b[m], f32x2_pack(c.z, c.w))), x.b[m], e + 1, A.rot);
    }
  }
  // Elements e and e + 2 after the turn: as they were where they lie past the rotation (0 times an
  // infinite partner would not be 0).
  static __device__ __forceinline__ uint64_t turned(uint64_t to, uint64_t was, int e, int rot) {
    if (LY < kPairsEnd || e + 2 < rot) return to;
    float t0, t1, w0, w1;
    f32x2_unpack(to, t0, t1);
    f32x2_unpack(was, w0, w1);
    return f32x2_pack(e < rot ? t0 : w0, w1);
  }
  // places in the head of a unit's couple m: first and second element of its pairs (-1: there is none)
  struct Places {
    int a0, a1, b0, b1;
  };
  static __device__ __forceinline__ Places places(int off, bool turn, int m, int half, int d) {
    Places p;
    if (IL) p = Places{off + 4 * m, PP == 1 ? -1 : off + 4 * m + 2, off + 4 * m + 1, PP == 1 ? -1 : off + 4 * m + 3};
    else p = Places{off + 2 * m, PP == 1 ? -1 : off + 2 * m + 1, turn ? off + half + 2 * m : -1,
                    turn && PP > 1 ? off + half + 2 * m + 1 : -1};
    if (p.b0 >= d) p.b0 = -1;
    return p;
  }
  // a head's vectors to this lane's places in shared memory, 32 lanes of 16 bytes a vector; zeros where there are none
  __device__ __forceinline__ void copy(uint32_t to, const uint8_t* head, bool some) const {
    const T* src = reinterpret_cast<const T*>(head);  // (not read where some is false)
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      copy16(to + j * 512, src + off[j], some && unit[j] >= 0);
      if (!IL) copy16(to + (NU + j) * 512, src + off[j] + half, some && turn[j]);
    }
  }
  static __device__ __forceinline__ void take(const uint8_t* from, Row& r) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      *reinterpret_cast<uint4*>(r.a[j].v) = *reinterpret_cast<const uint4*>(from + j * 512);
      if (!IL) *reinterpret_cast<uint4*>(r.b[IL ? 0 : j].v) = *reinterpret_cast<const uint4*>(from + (NU + j) * 512);
    }
  }
  // element by element, straight from memory
  __device__ __forceinline__ void load(const T* src, bool some, Row& r) const {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const Places p = places(off[j], turn[j], 0, half, d);
      auto at = [&](int x) { return some && unit[j] >= 0 && x >= 0 ? src[x] : from_f<T>(0.f); };
      r.a[j].v[0] = at(p.a0);
      if (IL) r.a[j].v[WI - 1] = at(p.b0);
      else r.b[IL ? 0 : j].v[0] = at(p.b0);
    }
  }
  __device__ __forceinline__ void store(T* dst, const Row& r) const {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if (unit[j] < 0) continue;
      if (W == 1 && IL && !turn[j]) {
        dst[off[j]] = r.a[j].v[0];
        if (off[j] + 1 < d) dst[off[j] + 1] = r.a[j].v[1];
      } else {
        r.a[j].store(dst + off[j]);
      }
      if (!IL && turn[j]) r.b[j].store(dst + off[j] + half);
    }
  }
  static __device__ __forceinline__ Half2 get(const Row& r, int j) {
    Half2 x;
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      if constexpr (PP == 1) {
        x.a[m] = f32x2_pack(to_f(r.a[j].v[0]), 0.f);
        x.b[m] = f32x2_pack(to_f(IL ? r.a[j].v[WI - 1] : r.b[IL ? 0 : j].v[0]), 0.f);
      } else if constexpr (sizeof(T) == 2) {  // (by words: an element at a time costs an instruction more each)
        const uint32_t *a = reinterpret_cast<const uint32_t*>(r.a[j].v), *b = reinterpret_cast<const uint32_t*>(r.b[IL ? 0 : j].v);
        if constexpr (IL) {
          x.a[m] = f32x2_pack(bf16lo(a[2 * m]), bf16lo(a[2 * m + 1]));
          x.b[m] = f32x2_pack(bf16hi(a[2 * m]), bf16hi(a[2 * m + 1]));
        } else {
          x.a[m] = f32x2_pack(bf16lo(a[m]), bf16hi(a[m]));
          x.b[m] = f32x2_pack(bf16lo(b[m]), bf16hi(b[m]));
        }
      } else if constexpr (IL) {
        x.a[m] = f32x2_pack(to_f(r.a[j].v[4 * m]), to_f(r.a[j].v[4 * m + 2]));
        x.b[m] = f32x2_pack(to_f(r.a[j].v[4 * m + 1]), to_f(r.a[j].v[4 * m + 3]));
      } else {
        x.a[m] = f32x2_pack(to_f(r.a[j].v[2 * m]), to_f(r.a[j].v[2 * m + 1]));
        x.b[m] = f32x2_pack(to_f(r.b[j].v[2 * m]), to_f(r.b[j].v[2 * m + 1]));
      }
    }
    return x;
  }
  static __device__ __forceinline__ void put(Row& r, int j, const Half2& x) {
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      float a0, a1, b0, b1;
      f32x2_unpack(x.a[m], a0, a1);
      f32x2_unpack(x.b[m], b0, b1);
      if constexpr (PP == 1) {
        r.a[j].v[0] = from_f<T>(a0);
        if (IL) r.a[j].v[WI - 1] = from_f<T>(b0);
        else r.b[IL ? 0 : j].v[0] = from_f<T>(b0);
      } else if constexpr (sizeof(T) == 2) {
        if constexpr (IL) {
          reinterpret_cast<uint32_t*>(r.a[j].v)[2 * m] = pack_bf16x2(a0, b0);
          reinterpret_cast<uint32_t*>(r.a[j].v)[2 * m + 1] = pack_bf16x2(a1, b1);
        } else {
          reinterpret_cast<uint32_t*>(r.a[j].v)[m] = pack_bf16x2(a0, a1);
          reinterpret_cast<uint32_t*>(r.b[j].v)[m] = pack_bf16x2(b0, b1);
        }
      } else if constexpr (IL) {
        r.a[j].v[4 * m] = a0;
        r.a[j].v[4 * m + 1] = b0;
        r.a[j].v[4 * m + 2] = a1;
        r.a[j].v[4 * m + 3] = b1;
      } else {
        r.a[j].v[2 * m] = a0;
        r.a[j].v[2 * m + 1] = a1;
        r.b[j].v[2 * m] = b0;
        r.b[j].v[2 * m + 1] = b1;
      }
    }
  }
  // the weights of this lane's elements (1 where there is none)
  __device__ __forceinline__ void weights(const float* w, Half2* to, bool of_partners = false) const {
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        const Places p = places(off[j], turn[j], m, half, d);
        auto at = [&](int x) {
          return w && unit[j] >= 0 && x >= 0 ? weight_at(w + (PL && of_partners ? partner_of(x, 2 * half) : x)) : 1.f;
        };
        to[j].a[m] = f32x2_pack(at(p.a0), at(p.a1));
        to[j].b[m] = f32x2_pack(at(p.b0), at(p.b1));
      }
  }
  // x turned by the token's angles, or back. Of a couple of pairs the two cosines and the two sines lie in 16
  // bytes, [NP][units that turn].
  __device__ __forceinline__ void rotate(const NormArgs& A, const float2* s_cs, int j, Half2& x, bool back) const {
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      uint64_t c, s, n;
      if constexpr (PP == 1) {
        const float2 v = s_cs[IL ? off[j] >> 1 : off[j]];
        c = f32x2_pack(v.x, 0.f);
        s = f32x2_pack(v.y, 0.f);
        n = f32x2_pack(-v.y, 0.f);
      } else {
        const float4 v = reinterpret_cast<const float4*>(s_cs)[m * A.rot_units + unit[j]];
        c = f32x2_pack(v.x, v.y);
        s = f32x2_pack(v.z, v.w);
        n = f32x2_pack(-v.z, -v.w);
      }
      const int e = off[j] + 4 * m;
      const uint64_t t = f32x2_fma(x.b[m], back ? s : n, f32x2_mul(x.a[m], c));
      x.b[m] = turned(f32x2_fma(x.a[m], back ? n : s, f32x2_mul(x.b[m], c)), x.b[m], e + 1, A.rot);
      x.a[m] = turned(t, x.a[m], e, A.rot);
    }
  }
  // The cosines and sines (times the magnitude) of a position, by a warp; 1 and 0 for what a unit holds past the rotation.
  static __device__ __forceinline__ void table(const NormArgs& A, const RopeTable& tab, int pos, float2* s_cs) {
    const int pairs = A.rot >> 1, all = PP == 1 || !IL ? pairs : (PL ? A.rot_units * W - pairs : A.rot_units * PP);
    for (int p = threadIdx.x & 31; p < all; p += 32) {
      float s = 0.f, c = 1.f;
      if (p < pairs) {
        const uint64_t phase = (uint64_t)(int64_t)pos * tab.turn[p];
        sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
        c *= A.mscale;
        s *= A.mscale;
      }
      float* to = reinterpret_cast<float*>(s_cs);
      if constexpr (PL) {
        // element e of a unit: couple e / 4, place (0, 2, 1, 3)[e % 4] of its four
        auto put = [&](int e, float sine) {
          const int in = e % W;
          float* at = to + ((in >> 2) * 2 * A.rot_units + e / W) * 4 + ((in & 1) * 2 + ((in >> 1) & 1));
          at[0] = c;
          at[A.rot_units * 4] = sine;
        };
        if (p < pairs) {
          put(p, -s);
          put(p + pairs, s);
        } else {
          put(p + pairs, 0.f);
        }
      } else if constexpr (PP == 1) {
        s_cs[p] = make_float2(c, s);
      } else {
        const int e = p % PP;  // place of the pair in its unit
        to += ((e >> 1) * A.rot_units + p / PP) * 4 + (e & 1);
        to[0] = c;
        to[2] = s;
      }
    }
  }
};

// Sums over the lanes of a head.
template <int N>
__device__ __forceinline__ void lanes_sum(float* x, int log_l) {
#pragma unroll
  for (int o = 4; o >= 0; --o)
    if (log_l > o) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], 1 << o);
    }
}

// W: elements of a vector (1: unaligned data, element by element); LY: layout; NU: units of a lane.
// Backward: a thread's part of dw stays in registers throughout.
template <typename T, int W, int LY, int NU, int MODE>
__global__ void __launch_bounds__(kThreads, ctas_an_sm<W, LY, NU>(MODE == kBackward))
    norm_rope_kernel(const __grid_constant__ NormArgs A, const __grid_constant__ RopeTable tab) {
  using U = Units<T, W, LY, NU>;
  constexpr bool BWD = MODE == kBackward;
  constexpr int S = W == 1 ? 0 : kSlots<NU>, SLOT = U::V * 512 * (BWD ? 2 : 1);
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* mine = smem + warp * A.warp_bytes;  // S slots, then the table
  const uint32_t ring = smem_u32(mine) + lane * 16;
  float2* s_cs = reinterpret_cast<float2*>(mine + S * SLOT);
  U u;
  u.set(A);
  // the kernel before this one has ended; the next one may start, and wait
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
  const int role = BWD && (int)blockIdx.x >= A.ctas_q;  // backward: the tensor of this CTA
  const int n_pieces = BWD ? A.pieces[role] : A.pieces[0] + A.pieces[1] + (MODE == kAppend ? A.pieces[2] : 0);
  const int64_t total = A.n_tokens * n_pieces;
  const int64_t nw = (int64_t)kWarps * (BWD ? (role ? (int)gridDim.x - A.ctas_q : A.ctas_q) : (int)gridDim.x);
  const int64_t w0 = (int64_t)kWarps * (blockIdx.x - (role ? A.ctas_q : 0)) + warp;
  const int64_t each = total / nw, over = total - each * nw, begin = w0 * each + min(w0, over);
  const int count = (int)(each + (w0 < over));
  // A place in the run: its token, piece, tensor, this lane's head, and the piece at which the next tensor begins.
  struct At {
    int64_t t;
    int piece, g, h, edge;
  };
  const int heads = 32 >> A.log_l, stride = heads * A.d * (int)sizeof(T);  // heads of a piece, their bytes
  auto settle = [&](At& a) {
    a.g = BWD ? role : (a.piece < A.pieces[0] ? 0 : (MODE != kAppend || a.piece < A.pieces[0] + A.pieces[1] ? 1 : 2));
    const int from = BWD ? 0 : (a.g > 0 ? A.pieces[0] : 0) + (a.g > 1 ? A.pieces[1] : 0);
    a.h = (a.piece - from) * heads + (lane >> A.log_l);
    a.edge = from + A.pieces[a.g];
  };
  auto head = [&](const uint8_t* base, int64_t token_stride, const At& a) {
    return base + a.t * token_stride + (int64_t)a.h * A.d * (int)sizeof(T);
  };
  At at;  // where the work is
  at.t = begin / n_pieces;
  at.piece = (int)(begin - at.t * n_pieces);
  settle(at);
  At ahead = at;  // where the copies are, and from where
  const uint8_t *from = head(A.src[at.g], A.src_stride[at.g], at), *from_dy = BWD ? head(A.dy[role], A.dy_stride[role], at) : nullptr;
  int to_copy = count;
  uint32_t slot = 0;
  auto copy = [&](uint32_t to) {
    if (to_copy > 0) {
      --to_copy;
      const bool some = ahead.h < A.heads[ahead.g];
      u.copy(ring + to * SLOT, from, some);
      if (BWD) u.copy(ring + to * SLOT + U::V * 512, from_dy, some);
      ahead.h += heads;
      from += stride;
      if (BWD) from_dy += stride;
      if (++ahead.piece == ahead.edge) {
        if (ahead.piece == n_pieces) {
          ahead.piece = 0;
          ++ahead.t;
        }
        settle(ahead);
        from = head(A.src[ahead.g], A.src_stride[ahead.g], ahead);
        if (BWD) from_dy = head(A.dy[role], A.dy_stride[role], ahead);
      }
    }
    copy_commit();  // (an empty one at the end, so that the waits count the same)
  };
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < S; ++i) copy(i);
  }
  constexpr bool PL = U::PL;
  typename U::Half2 w[NU], wp[PL && !BWD ? NU : 1], dw[BWD ? NU : 1] = {};
  if (BWD) u.weights(A.weight[role], w);
  Place place;
  uint8_t* out = nullptr;  // where this lane's head goes
  // a token, or a tensor of it, begins
  auto enter = [&](bool token) {
    if (token) {
      int pos = 0;
      if constexpr (MODE == kAppend) {
        place.next(A, at.t, lane);
        pos = place.pos;
      }
      if (A.positions) pos = A.positions[at.t];
      __syncwarp();  // the last token's angles have been read
      U::table(A, tab, pos, s_cs);
      __syncwarp();
    }
    if (!BWD && at.g < 2) {
      u.weights(A.weight[at.g], w);
      if constexpr (PL && !BWD) u.weights(A.weight[at.g], wp, true);
    }
    out = A.dst[at.g] + (MODE == kAppend && at.g > 0 ? place.row : at.t) * A.dst_stride[at.g] + (int64_t)at.h * A.d * (int)sizeof(T);
  };
  if (count > 0) enter(true);
  for (int k = 0; k < count; ++k) {
    const int g = at.g;
    const bool some = at.h < A.heads[g];
    typename U::Row x, dy;
    if constexpr (W > 1) {
      copy_wait<S - 1>();
      if (PL) __syncwarp();  // the other lanes' copies
      U::take(mine + lane * 16 + slot * SLOT, x);
      if (BWD) U::take(mine + lane * 16 + slot * SLOT + U::V * 512, dy);
    } else {
      u.load(reinterpret_cast<const T*>(head(A.src[g], A.src_stride[g], at)), some, x);
      if (BWD) u.load(reinterpret_cast<const T*>(head(A.dy[g], A.dy_stride[g], at)), some, dy);
    }
    uint64_t sa = 0, sb = 0, ga = 0, gb = 0;
    typename U::Half2 gr[BWD ? NU : 1];  // R' dy
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const typename U::Half2 v = U::get(x, j);
      if (BWD) {
        gr[j] = U::get(dy, j);
        if constexpr (PL) {
          if (u.turn[j]) u.rotate(A, s_cs, j, gr[j], u.partners(mine + slot * SLOT + U::V * 512, j), true);
        } else {
          if (u.turn[j]) u.rotate(A, s_cs, j, gr[j], true);
        }
      }
#pragma unroll
      for (int m = 0; m < U::NP; ++m) {
        sa = f32x2_fma(v.a[m], v.a[m], sa);
        sb = f32x2_fma(v.b[m], v.b[m], sb);
        if (BWD) {
          ga = f32x2_fma(f32x2_mul(gr[j].a[m], w[j].a[m]), v.a[m], ga);
          gb = f32x2_fma(f32x2_mul(gr[j].b[m], w[j].b[m]), v.b[m], gb);
        }
      }
    }
    float sums[2] = {f32x2_sum(f32x2_add(sa, sb)), BWD ? f32x2_sum(f32x2_add(ga, gb)) : 0.f};
    lanes_sum<BWD ? 2 : 1>(sums, A.log_l);
    typename U::Half2 xp[PL && !BWD ? NU : 1];
    if constexpr (PL && !BWD) {
#pragma unroll
      for (int j = 0; j < NU; ++j) xp[j] = u.partners(mine + slot * SLOT, j);
    }
    if constexpr (W > 1) {  // x and dy have been read
      if (PL) __syncwarp();
      copy(slot);
      slot = slot + 1 == S ? 0 : slot + 1;
    }
    const float r = rsqrtf(fmaf(sums[0], A.inv_d, A.eps));
    const uint64_t rms = f32x2_both(r);
    if (BWD) {
      const uint64_t mean = f32x2_both(-(r * (sums[1] * A.inv_d)));
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        typename U::Half2 v = U::get(x, j);
        auto one = [&](uint64_t& x2, uint64_t g2, uint64_t w2, uint64_t& dw2) {
          const uint64_t xh = f32x2_mul(x2, rms);
          if (some) dw2 = f32x2_fma(g2, xh, dw2);
          x2 = f32x2_mul(f32x2_fma(xh, mean, f32x2_mul(g2, w2)), rms);
        };
#pragma unroll
        for (int m = 0; m < U::NP; ++m) {
          one(v.a[m], gr[j].a[m], w[j].a[m], dw[j].a[m]);
          one(v.b[m], gr[j].b[m], w[j].b[m], dw[j].b[m]);
        }
        U::put(x, j, v);
      }
      if (some) u.store(reinterpret_cast<T*>(out), x);
    } else {
      if (g < 2) {
#pragma unroll
        for (int j = 0; j < NU; ++j) {
          typename U::Half2 v = U::get(x, j);
#pragma unroll
          for (int m = 0; m < U::NP; ++m) {
            v.a[m] = f32x2_mul(f32x2_mul(v.a[m], rms), w[j].a[m]);
            v.b[m] = f32x2_mul(f32x2_mul(v.b[m], rms), w[j].b[m]);
          }
          if constexpr (PL && !BWD) {
#pragma unroll
            for (int m = 0; m < U::NP; ++m) {
              xp[j].a[m] = f32x2_mul(f32x2_mul(xp[j].a[m], rms), wp[j].a[m]);
              xp[j].b[m] = f32x2_mul(f32x2_mul(xp[j].b[m], rms), wp[j].b[m]);
            }
            if (u.turn[j]) u.rotate(A, s_cs, j, v, xp[j], false);
          } else if constexpr (!PL) {
            if (u.turn[j]) u.rotate(A, s_cs, j, v, false);
          }
          U::put(x, j, v);
        }
      }
      const bool there = MODE != kAppend || (place.live && (g == 0 || place.row >= 0));
      if (some && there) u.store(reinterpret_cast<T*>(out), x);
    }
    at.h += heads;
    out += stride;
    if (++at.piece == at.edge && k + 1 < count) {
      const bool token = at.piece == n_pieces;
      if (token) {
        at.piece = 0;
        ++at.t;
      }
      settle(at);
      enter(token);
    }
  }
  if constexpr (W > 1) copy_wait<0>();
  if constexpr (BWD) {
    // the CTA's sums: over the heads of a warp by shuffles, then over the warps in order
    float* s_red = reinterpret_cast<float*>(smem);  // [warps][d]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int m = 0; m < U::NP; ++m) {
        float v[4];
        f32x2_unpack(dw[j].a[m], v[0], v[1]);
        f32x2_unpack(dw[j].b[m], v[2], v[3]);
        const typename U::Places p = U::places(u.off[j], u.turn[j], m, u.half, A.d);
        const int to[4] = {p.a0, p.a1, p.b0, p.b1};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          for (int o = 1 << A.log_l; o < 32; o <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
          if (u.unit[j] >= 0 && to[e] >= 0 && lane < (1 << A.log_l)) s_red[warp * A.d + to[e]] = v[e];
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < A.d; i += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int y = 0; y < kWarps; ++y) v += s_red[y * A.d + i];
      A.part[(int64_t)blockIdx.x * A.d + i] = v;
    }
  }
}

// dw from the CTAs' sums, always in the same order: 32 columns a block, 32 slices of the CTAs; q, then k. It starts while they
// are still at work and waits for them (8192 tokens 51.8 us, one after the other 52.8; 1999 tokens of 16 heads of 64 in fp32 9.7, 10.0).
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int nq, int nk, int d, float* dqw, float* dkw) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  float* out = blockIdx.y ? dkw : dqw;
  const int n = blockIdx.y ? nk : nq;
  if (blockIdx.y) part += (int64_t)nq * d;
  float v = 0.f;
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
  if (col < d) {
#pragma unroll 4
    for (int i = y; i < n; i += 32) v += part[(int64_t)i * d + col];
  }
  s[y][c] = v;
  __syncthreads();
  if (y == 0 && col < d && out) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][c];
    out[col] = v;
  }
}

// A launch that may start while the kernel before it on the stream ends, and waits for that before it reads anything (one
// step's norms after one another 2.4 us, 2.9 without; the gradient of 1999 tokens of 16 heads of 64 9.0, 9.6).
template <class... F, class... T>
cudaError_t launch_early(void (*kern)(F...), dim3 grid, int threads, size_t smem, cudaStream_t st, const T&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_dw(cudaStream_t st, const float* part, int nq, int nk, int d, float* dqw, float* dkw) {
  return launch_early(norm_dw_kernel, dim3((unsigned)cdiv(d, 32), 2), 1024, 0, st, part, nq, nk, d, dqw, dkw);
}

// Shape of a launch: vectors, layout, units and lanes, the pieces of a token, and the shared memory of a warp.
void set_shape(NormArgs& a, int size, bool interleaved, bool backward, int& layout, int& nu) {
  const int W = 16 / size;
  // 16-byte vectors when heads are whole numbers of them that start on 16-byte boundaries; else element by element (8192
  // tokens of 32 + 8 heads of 128 in bf16, 42 elements of which turn, forward: 44 us; element by element 456; backward 57
  // and 1377). The half layout takes pairs of vectors where half a rotation is a whole number of them (30 us), else plain
  // ones with the partners out of shared memory (the 44).
  bool wide = a.d % W == 0;
  for (int g = 0; g < 3; ++g)
    if (a.heads[g]) {
      wide = wide && !(((uintptr_t)a.src[g] | (uintptr_t)a.dst[g] | (uint64_t)a.src_stride[g] | (uint64_t)a.dst_stride[g]) & 15);
      if (backward) wide = wide && !(((uintptr_t)a.dy[g] | (uint64_t)a.dy_stride[g]) & 15);
    }
  layout = interleaved ? (wide && a.rot % W != 0 ? kPairsEnd : kPairs) : (!wide || a.rot / 2 % W == 0 ? kHalves : kPlain);
  const bool halves = layout == kHalves;
  const int wi = wide ? W : (interleaved ? 2 : 1);
  a.rot_units = halves ? a.rot / 2 / wi : (int)cdiv(a.rot, wi);
  a.units = halves ? a.rot_units + (a.d - a.rot + wi - 1) / wi : (int)cdiv(a.d, wi);
  a.log_l = 0;
  while (a.log_l < 5 && (1 << a.log_l) < a.units) ++a.log_l;
  nu = !wide ? 16 : (a.units <= 32 ? 1 : (size == 2 ? kMany<__nv_bfloat16> : kMany<float>));
  // two vectors a lane where a unit is one, and half the lanes (pairs of neighbours, forward: 30.5 us against 35.5)
  if (wide && !halves && size == 2 && a.units > 8) {
    nu = 2;
    a.log_l -= a.units <= 32;
  }
  if (!wide) a.log_l = 5;
  for (int g = 0; g < 3; ++g) a.pieces[g] = (int)cdiv(a.heads[g], 32 >> a.log_l);
  a.inv_d = 1.f / (float)a.d;
  const int slots = !wide ? 0 : (nu <= 2 ? kSlots<1> : kSlots<4>);
  const int angles = halves || !wide ? a.rot / 2 : a.rot_units * (layout == kPlain ? W : W / 2);
  a.warp_bytes = slots * nu * (halves ? 2 : 1) * 512 * (backward ? 2 : 1) + ((angles * (int)sizeof(float2) + 15) & ~15);
}

template <typename T, int MODE>
sta_status launch_norm(NormArgs& a, const RopeTable& tab, bool il, cudaStream_t st, int* ctas = nullptr) {
  constexpr int W = 16 / (int)sizeof(T);
  int layout, nu;
  set_shape(a, (int)sizeof(T), il, MODE == kBackward, layout, nu);
  const bool light = nu * (layout == kHalves ? 2 : 1) <= 2;  // (registers: ctas_an_sm)
  const int64_t H = MODE == kAppend ? 3 : 2;
  int64_t pieces = 0;
  for (int g = 0; g < H; ++g) pieces += a.pieces[g];
  size_t smem = (size_t)kWarps * a.warp_bytes;
  unsigned grid;
  if (MODE == kBackward) {
    int n[2];
    norm_ctas(light ? kMaxGrid : kMaxGrid / 2, a.pieces, a.n_tokens, kWarps, n);
    a.ctas_q = n[0];
    ctas[0] = n[0];
    ctas[1] = n[1];
    grid = (unsigned)(n[0] + n[1]);
    smem = std::max(smem, (size_t)kWarps * a.d * sizeof(float));
  } else {
    grid = (unsigned)std::min<int64_t>(152 * (!light ? 1 : (layout == kPlain && nu == 2 ? 2 : 3)), cdiv(a.n_tokens * pieces, kWarps));
  }
  if (a.n_tokens * pieces / ((int64_t)grid * kWarps) >= INT32_MAX) return STA_ERR_INVALID_ARG;
  auto go = [&](auto kern) -> sta_status {
    if (smem > 48 * 1024) STA_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    STA_CUDA_TRY(launch_early(kern, dim3(grid), kThreads, smem, st, a, tab));
    return STA_OK;
  };
  if (nu == 16) return il ? go(norm_rope_kernel<T, 1, kPairs, 16, MODE>) : go(norm_rope_kernel<T, 1, kHalves, 16, MODE>);
  auto of = [&](auto n) -> sta_status {
    constexpr int NU = decltype(n)::value;
    if (layout == kPairs) return go(norm_rope_kernel<T, W, kPairs, NU, MODE>);
    if (layout == kPairsEnd) return go(norm_rope_kernel<T, W, kPairsEnd, NU, MODE>);
    if (layout == kPlain) return go(norm_rope_kernel<T, W, kPlain, NU, MODE>);
    return go(norm_rope_kernel<T, W, kHalves, NU, MODE>);
  };
  return nu == 1 ? of(std::integral_constant<int, 1>{}) : of(std::integral_constant<int, kMany<T>>{});
}

template <typename T>
sta_status launch_bwd(NormArgs& a, const RopeTable& tab, bool il, float* dqw, float* dkw, cudaStream_t st) {
  int ctas[2];
  const sta_status status = launch_norm<T, kBackward>(a, tab, il, st, ctas);
  if (status != STA_OK) return status;
  if (dqw || dkw) {
    STA_CUDA_TRY(launch_dw(st, a.part, ctas[0], ctas[1], a.d, dqw, dkw));
  }
  return STA_OK;
}

// Sizes and the rotation, common to the three calls.
sta_status check_heads(int64_t n_tokens, int Hq, int Hk, int d, float eps, const sta_rope_params* rope, RopeTable& tab) {
  if (n_tokens < 0 || Hq < 0 || Hq > 65536 || Hk < 0 || Hk > 65536 || Hq + Hk < 1 || d < 2) return STA_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !std::isfinite(eps)) return STA_ERR_INVALID_ARG;
  if (d > 2 * kMaxPairs) return STA_ERR_UNSUPPORTED;
  return rope ? rope_table(rope, d, tab) : STA_OK;
}

}  // namespace
}  // namespace sta

using namespace sta;

extern "C" sta_status sta_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride, void* q_out,
                                    void* k_out, int64_t q_out_stride, int64_t k_out_stride, const float* q_weight,
                                    const float* k_weight, float eps, const int32_t* positions_dev,
                                    const sta_rope_params* rope, int64_t n_tokens, int Hq, int Hk, int d, sta_dtype dtype,
                                    sta_stream stream) {
  if (dtype != STA_BF16 && dtype != STA_F32) return STA_ERR_INVALID_ARG;
  RopeTable tab;
  const sta_status st = check_heads(n_tokens, Hq, Hk, d, eps, rope, tab);
  if (st != STA_OK) return st;
  const void* src[2] = {q, k};
  void* dst[2] = {q_out, k_out};
  const int64_t ss[2] = {q_stride, k_stride}, ds[2] = {q_out_stride, k_out_stride};
  const float* weight[2] = {q_weight, k_weight};
  const int heads[2] = {Hq, Hk}, size = dtype == STA_BF16 ? 2 : 4;
  for (int g = 0; g < 2; ++g) {
    if (heads[g] == 0 && (src[g] || dst[g])) return STA_ERR_INVALID_ARG;
    if (heads[g] && (ss[g] < (int64_t)heads[g] * d || ds[g] < (int64_t)heads[g] * d)) return STA_ERR_INVALID_ARG;
  }
  if (n_tokens == 0) return STA_OK;
  if (rope && !positions_dev) return STA_ERR_INVALID_ARG;
  NormArgs a{};
  for (int g = 0; g < 2; ++g) {
    if (!heads[g]) continue;
    if (!src[g] || !dst[g] || (src[g] == dst[g] && ss[g] != ds[g])) return STA_ERR_INVALID_ARG;
    if (((uintptr_t)src[g] | (uintptr_t)dst[g]) & (size - 1) || (uintptr_t)weight[g] & 3) return STA_ERR_UNSUPPORTED;
    a.src[g] = static_cast<const uint8_t*>(src[g]);
    a.dst[g] = static_cast<uint8_t*>(dst[g]);
    a.src_stride[g] = ss[g] * size;
    a.dst_stride[g] = ds[g] * size;
    a.heads[g] = heads[g];
    a.weight[g] = weight[g];
  }
  if ((uintptr_t)positions_dev & 3) return STA_ERR_UNSUPPORTED;
  a.n_tokens = n_tokens;
  a.d = d;
  a.rot = rope ? rope->rot_dim : 0;
  a.mscale = rope ? rope->mscale : 1.f;
  a.eps = eps;
  a.positions = rope ? positions_dev : nullptr;
  const bool il = rope && rope->layout == STA_ROPE_INTERLEAVED;
  return dtype == STA_BF16 ? launch_norm<__nv_bfloat16, kForward>(a, tab, il, (cudaStream_t)stream)
                           : launch_norm<float, kForward>(a, tab, il, (cudaStream_t)stream);
}

extern "C" sta_status sta_norm_rope_bwd(const void* dq_out, const void* dk_out, int64_t dq_out_stride,
                                        int64_t dk_out_stride, const void* q, const void* k, int64_t q_stride,
                                        int64_t k_stride, void* dq, void* dk, int64_t dq_stride, int64_t dk_stride,
                                        const float* q_weight, const float* k_weight, float* dq_weight, float* dk_weight,
                                        float eps, const int32_t* positions_dev, const sta_rope_params* rope,
                                        int64_t n_tokens, int Hq, int Hk, int d, sta_dtype dtype, void* workspace,
                                        size_t* workspace_bytes, sta_stream stream) {
  if (dtype != STA_BF16 && dtype != STA_F32) return STA_ERR_INVALID_ARG;
  RopeTable tab;
  const sta_status st = check_heads(n_tokens, Hq, Hk, d, eps, rope, tab);
  if (st != STA_OK) return st;
  if (!workspace_bytes) return STA_ERR_INVALID_ARG;
  const void* src[2] = {q, k};
  const void* dy[2] = {dq_out, dk_out};
  void* dst[2] = {dq, dk};
  const int64_t ss[2] = {q_stride, k_stride}, ys[2] = {dq_out_stride, dk_out_stride}, ds[2] = {dq_stride, dk_stride};
  const float* weight[2] = {q_weight, k_weight};
  float* dw[2] = {dq_weight, dk_weight};
  const int heads[2] = {Hq, Hk}, size = dtype == STA_BF16 ? 2 : 4;
  for (int g = 0; g < 2; ++g) {
    const int64_t row = (int64_t)heads[g] * d;
    if (heads[g] == 0 && (src[g] || dst[g] || dy[g] || dw[g])) return STA_ERR_INVALID_ARG;
    if (heads[g] && (ss[g] < row || ds[g] < row || ys[g] < row)) return STA_ERR_INVALID_ARG;
  }
  const size_t need = (size_t)kMaxGrid * d * sizeof(float);
  if (!workspace) {
    *workspace_bytes = need;
    return STA_OK;
  }
  if (*workspace_bytes < need) {
    *workspace_bytes = need;
    return STA_ERR_WORKSPACE;
  }
  if ((uintptr_t)workspace & 255) return STA_ERR_UNSUPPORTED;
  if (n_tokens > 0 && rope && !positions_dev) return STA_ERR_INVALID_ARG;
  NormArgs a{};
  for (int g = 0; g < 2; ++g) {
    if (!heads[g]) continue;
    if ((uintptr_t)dw[g] & 3) return STA_ERR_UNSUPPORTED;
    a.heads[g] = heads[g];
    if (n_tokens == 0) continue;
    if (!src[g] || !dst[g] || !dy[g]) return STA_ERR_INVALID_ARG;
    if ((src[g] == dst[g] && ss[g] != ds[g]) || (dy[g] == dst[g] && ys[g] != ds[g])) return STA_ERR_INVALID_ARG;
    if (((uintptr_t)src[g] | (uintptr_t)dst[g] | (uintptr_t)dy[g]) & (size - 1) || (uintptr_t)weight[g] & 3)
      return STA_ERR_UNSUPPORTED;
    a.src[g] = static_cast<const uint8_t*>(src[g]);
    a.dst[g] = static_cast<uint8_t*>(dst[g]);
    a.dy[g] = static_cast<const uint8_t*>(dy[g]);
    a.src_stride[g] = ss[g] * size;
    a.dst_stride[g] = ds[g] * size;
    a.dy_stride[g] = ys[g] * size;
    a.weight[g] = weight[g];
  }
  if ((uintptr_t)positions_dev & 3) return STA_ERR_UNSUPPORTED;
  a.d = d;
  a.part = static_cast<float*>(workspace);
  const cudaStream_t s = (cudaStream_t)stream;
  if (n_tokens == 0) {  // no rows: the weights' gradients are 0
    if (dq_weight || dk_weight) {
      STA_CUDA_TRY(launch_dw(s, a.part, 0, 0, d, dq_weight, dk_weight));
    }
    return STA_OK;
  }
  a.n_tokens = n_tokens;
  a.rot = rope ? rope->rot_dim : 0;
  a.mscale = rope ? rope->mscale : 1.f;
  a.eps = eps;
  a.positions = rope ? positions_dev : nullptr;
  const bool il = rope && rope->layout == STA_ROPE_INTERLEAVED;
  return dtype == STA_BF16 ? launch_bwd<__nv_bfloat16>(a, tab, il, dq_weight, dk_weight, s)
                           : launch_bwd<float>(a, tab, il, dq_weight, dk_weight, s);
}

extern "C" sta_status sta_norm_rope_append_paged(const void* q, const void* k, const void* v, int64_t q_stride,
                                                 int64_t k_stride, int64_t v_stride, void* q_out, void* k_pages,
                                                 void* v_pages, int page_size, int n_pages,
                                                 const int32_t* page_indptr_dev, const int32_t* page_indices_dev,
                                                 const int32_t* q_indptr_dev, const int32_t* kv_indptr_dev,
                                                 const int32_t* positions_dev, const float* q_weight,
                                                 const float* k_weight, float eps, const sta_rope_params* rope,
                                                 int64_t n_tokens, int n_req, int Hq, int Hkv, int d, sta_dtype dtype,
                                                 sta_stream stream) {
  if (n_req < 1 || Hkv < 1 || page_size < 1 || n_pages < 1) return STA_ERR_INVALID_ARG;
  RopeTable tab;
  const sta_status st = check_heads(n_tokens, Hq, Hkv, d, eps, rope, tab);
  if (st != STA_OK) return st;
  if ((Hq == 0) != (q == nullptr && q_out == nullptr)) return STA_ERR_INVALID_ARG;
  if (dtype != STA_BF16) return STA_ERR_UNSUPPORTED;
  if ((Hq > 0 && q_stride < (int64_t)Hq * d) || k_stride < (int64_t)Hkv * d || v_stride < (int64_t)Hkv * d)
    return STA_ERR_INVALID_ARG;
  if (n_tokens == 0) return STA_OK;
  if ((Hq > 0 && (!q || !q_out)) || !k || !v || !k_pages || !v_pages || !page_indptr_dev || !page_indices_dev ||
      !q_indptr_dev || !kv_indptr_dev)
    return STA_ERR_INVALID_ARG;
  const uintptr_t bits2 = (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)k_pages | (uintptr_t)v_pages;
  const uintptr_t bits4 = (uintptr_t)page_indptr_dev | (uintptr_t)page_indices_dev | (uintptr_t)q_indptr_dev |
                          (uintptr_t)kv_indptr_dev | (uintptr_t)positions_dev | (uintptr_t)q_weight | (uintptr_t)k_weight;
  if ((bits2 & 1) || (bits4 & 3)) return STA_ERR_UNSUPPORTED;
  if (q && q == q_out && q_stride != (int64_t)Hq * d) return STA_ERR_INVALID_ARG;
  NormArgs a{};
  const void* src[3] = {q, k, v};
  void* dst[3] = {q_out, k_pages, v_pages};
  const int64_t stride[3] = {q_stride, k_stride, v_stride};
  const int heads[3] = {Hq, Hkv, Hkv};
  for (int g = 0; g < 3; ++g) {
    a.src[g] = static_cast<const uint8_t*>(src[g]);
    a.dst[g] = static_cast<uint8_t*>(dst[g]);
    a.src_stride[g] = stride[g] * 2;
    a.dst_stride[g] = (int64_t)heads[g] * d * 2;
    a.heads[g] = heads[g];
  }
  a.weight[0] = q_weight;
  a.weight[1] = k_weight;
  a.n_tokens = n_tokens;
  a.d = d;
  a.rot = rope ? rope->rot_dim : 0;
  a.mscale = rope ? rope->mscale : 1.f;
  a.eps = eps;
  a.positions = positions_dev;
  a.q_indptr = q_indptr_dev;
  a.kv_indptr = kv_indptr_dev;
  a.page_indptr = page_indptr_dev;
  a.page_indices = page_indices_dev;
  a.n_req = n_req;
  a.page_size = page_size;
  a.n_pages = n_pages;
  a.err = device_error_word();
  return launch_norm<__nv_bfloat16, kAppend>(a, tab, rope && rope->layout == STA_ROPE_INTERLEAVED, (cudaStream_t)stream);
}
