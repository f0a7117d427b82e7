// Rotary positions, alone (sta_rope) and fused with the write of new tokens into a paged KV
// cache (sta_rope_append_paged).
//
// Pair p of a head at position t is turned by the angle t * f_p. The turn is taken exactly:
// f_p / 2pi is held as a 64-bit fraction of a turn, so t * fraction mod 2^64 is the position
// within the turn with no rounding at any t, and only its top 32 bits go on to fp32 (an
// error of 2^-25 of a half turn). An fp32 product t * f_p would be off by 2^-24 of the whole
// angle: 0.06 radians at t = 2^20.
//
// A CTA takes a few tokens: it puts their cosines and sines (times the magnitude) into shared
// memory once, then its threads run over the tokens' heads, a unit of work being the 16-byte
// vector (half layout: the two vectors half a rotation apart) that one thread turns. All
// loads of a thread's first two units are issued before the table is computed. Every element
// is read and written once, so HBM bounds it: 16384 tokens x 40 heads x 128 bf16 (336 MB moved)
// take 55.3 us back to back, 90 % of the copy rate (all of it: 49.6 us at the measured 6.77 TB/s). A few new
// tokens are bound by latency: one thread a token finds its place by dependent loads while the CTA waits
// for it (whether it is padding, a binary search for the request, which is six steps for 64, then lengths and
// list together, then the page), before the table, the turn and the stores. 64 tokens of 48 heads with their
// cache write take 11.4 us. (That and the times below are of a CUDA graph replayed from a cold L2, some 4 to 5
// us of events and graph launch included; so taken, the 16384 tokens are 58.5 us.)
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace sta {
namespace {

constexpr int kMaxPairs = 256;    // head size at most 512
constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;    // tokens of a CTA

struct RopeTable {
  uint64_t turn[kMaxPairs];  // f_p / 2pi mod 1, as a fraction of 2^64
};

struct RopeArgs {
  const uint8_t* src[3];  // q, k, v (sta_rope: src[0] alone)
  uint8_t* dst[3];
  int64_t src_stride[3];  // bytes between tokens
  int64_t dst_stride[3];  // bytes between tokens; k, v pages: bytes between a page's tokens
  int heads[3];           // heads of q, k, v
  int H;                  // their sum
  int64_t n_tokens;
  int d, rot;             // elements of a head; the leading rot of them turn
  int tokens;             // tokens of a CTA
  int transpose;
  float mscale;
  int units, rot_units;   // work units of a head; the first rot_units turn
  const int32_t* positions;
  // paged destination of k and v
  const int32_t* q_indptr;
  const int32_t* kv_indptr;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  int n_req, page_size, n_pages;
  int* err;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ float from_f(float v) { return v; }

// W consecutive elements, moved as one vector (W * sizeof(T) = 16) or one by one.
template <typename T, int W>
struct alignas(W * sizeof(T) == 16 ? 16 : sizeof(T)) Vec {
  T v[W];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (W * sizeof(T) == 16) *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(p));
    else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = p[i];
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (W * sizeof(T) == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    else {
#pragma unroll
      for (int i = 0; i < W; ++i) p[i] = v[i];
    }
  }
};

// Where a new token goes: its position and its cache row, -1 when it goes nowhere. False for padding.
__device__ __forceinline__ bool token_place(const RopeArgs& A, int64_t t, int& pos, int64_t& row) {
  pos = 0;
  row = -1;
  if (t < __ldg(A.q_indptr) || t >= __ldg(A.q_indptr + A.n_req)) return false;
  int lo = 0, hi = A.n_req - 1;  // the last request that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(A.q_indptr + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  // (all at once: each of these is a round trip to memory at first)
  const int64_t q1 = __ldg(A.q_indptr + lo + 1), len = (int64_t)__ldg(A.kv_indptr + lo + 1) - __ldg(A.kv_indptr + lo);
  const int64_t list = __ldg(A.page_indptr + lo), list_end = __ldg(A.page_indptr + lo + 1);
  const int64_t p = len - (q1 - t);
  if (p < 0 || t >= q1) {  // the sequence is shorter than its chunk: this token is not in it
    pos = (int)(p < INT32_MIN ? INT32_MIN : p);
    return true;
  }
  pos = (int)p;
  const int64_t e = list + p / A.page_size;
  if (e < 0 || e >= list_end) {
    record_error(A.err, 0x604);
    return true;
  }
  const int page = __ldg(A.page_indices + e);
  if (page < 0 || page >= A.n_pages) {
    record_error(A.err, 0x110);
    return true;
  }
  row = (int64_t)page * A.page_size + p % A.page_size;
  return true;
}

// W: elements of a vector (1: unaligned data, element by element); IL: interleaved pairs;
// APPEND: q, k, v with k and v going to pages.
template <typename T, int W, bool IL, bool APPEND>
__global__ void __launch_bounds__(kThreads, 6) rope_kernel(const RopeArgs A, const __grid_constant__ RopeTable tab) {
  constexpr int WI = IL && W == 1 ? 2 : W;  // elements of a vector: whole pairs when interleaved
  // units of a thread in flight: 2, and 6 CTAs an SM (16384 x 40 x 128 in bf16: 58.5 us; 4 with 3 CTAs 67)
  constexpr int U = 2;
  constexpr int PP = IL ? WI / 2 : WI;      // pairs of a unit
  // cosine and sine, two pairs in 16 bytes: [tokens][PP / 2][units][2], so that neighbouring threads
  // read neighbouring words (a unit's pairs side by side would meet in the same banks four times)
  extern __shared__ __align__(16) float2 s_cs[];
  __shared__ int64_t s_row[kMaxTokens];
  __shared__ int s_pos[kMaxTokens];
  __shared__ int s_live[kMaxTokens];
  const int half = A.rot >> 1;
  const int64_t t0 = (int64_t)blockIdx.x * A.tokens;
  const int nt = (int)min((int64_t)A.tokens, A.n_tokens - t0);
  const int per_token = A.H * A.units, total = nt * per_token;
  Vec<T, WI> a[U], b[U];
  int at[U];           // token << 20 | head (of q, k and v together); -1: none
  int off[U];          // first element of the vector
  bool turn[U];
  // One round of U units a thread: their loads, and, once the table is there, the turn and the stores.
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      at[u] = -1;
      if (i >= total) continue;
      const int t = i / per_token, x = i - t * per_token, h = x / A.units, unit = x - h * A.units;
      at[u] = (t << 20) | h;
      turn[u] = unit < A.rot_units;
      off[u] = turn[u] ? unit * WI : A.rot + (unit - A.rot_units) * WI;
      const int g = !APPEND || h < A.heads[0] ? 0 : (h < A.heads[0] + A.heads[1] ? 1 : 2);
      const int hg = h - (g > 0 ? A.heads[0] : 0) - (g > 1 ? A.heads[1] : 0);
      const T* src = reinterpret_cast<const T*>(A.src[g] + (t0 + t) * A.src_stride[g]) + (int64_t)hg * A.d + off[u];
      if (W == 1 && IL && !turn[u]) {  // the last element of an odd rest is alone
        a[u].v[0] = src[0];
        if (off[u] + 1 < A.d) a[u].v[1] = src[1];
      } else {
        a[u].load(src);
      }
      if (!IL && turn[u]) b[u].load(src + half);
    }
  };
  auto store = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at[u] < 0) continue;
      const int t = at[u] >> 20, h = at[u] & 0xfffff;
      const int g = !APPEND || h < A.heads[0] ? 0 : (h < A.heads[0] + A.heads[1] ? 1 : 2);
      const int hg = h - (g > 0 ? A.heads[0] : 0) - (g > 1 ? A.heads[1] : 0);
      if (APPEND && (!s_live[t] || (g > 0 && s_row[t] < 0))) continue;
      T* out = reinterpret_cast<T*>(A.dst[g] + (g ? s_row[t] : t0 + t) * A.dst_stride[g]) + (int64_t)hg * A.d + off[u];
      if (W == 1 && IL && !turn[u]) {
        out[0] = a[u].v[0];
        if (off[u] + 1 < A.d) out[1] = a[u].v[1];
        continue;
      }
      if (turn[u] && g < 2) {
        float2 cs[PP];
        if constexpr (PP == 1) {
          cs[0] = s_cs[t * half + (IL ? off[u] >> 1 : off[u])];
        } else {
          const float4* c4 = reinterpret_cast<const float4*>(s_cs + t * half) + off[u] / WI;
#pragma unroll
          for (int j = 0; j < PP / 2; ++j) {
            const float4 w = c4[j * A.rot_units];
            cs[2 * j] = make_float2(w.x, w.y);
            cs[2 * j + 1] = make_float2(w.z, w.w);
          }
        }
        if constexpr (IL) {
#pragma unroll
          for (int e = 0; e < WI / 2; ++e) {
            const float x = to_f(a[u].v[2 * e]), y = to_f(a[u].v[2 * e + 1]);
            a[u].v[2 * e] = from_f<T>(x * cs[e].x - y * cs[e].y);
            a[u].v[2 * e + 1] = from_f<T>(x * cs[e].y + y * cs[e].x);
          }
        } else {
#pragma unroll
          for (int e = 0; e < WI; ++e) {
            const float x = to_f(a[u].v[e]), y = to_f(b[u].v[e]);
            a[u].v[e] = from_f<T>(x * cs[e].x - y * cs[e].y);
            b[u].v[e] = from_f<T>(x * cs[e].y + y * cs[e].x);
          }
        }
      }
      a[u].store(out);
      if (!IL && turn[u]) b[u].store(out + half);
    }
  };
  load(threadIdx.x);  // under the table's latency
  if ((int)threadIdx.x < nt) {
    int pos;
    int64_t row = 0;
    bool live = true;
    if constexpr (APPEND) {
      live = token_place(A, t0 + threadIdx.x, pos, row);
      if (A.positions) pos = __ldg(A.positions + t0 + threadIdx.x);
    } else {
      pos = __ldg(A.positions + t0 + threadIdx.x);
    }
    s_pos[threadIdx.x] = pos;
    s_row[threadIdx.x] = row;
    s_live[threadIdx.x] = live;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, p = i - t * half;
    const uint64_t phase = (uint64_t)(int64_t)s_pos[t] * tab.turn[p];
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
    const int e = p % PP;  // place of the pair in its unit
    const int at_cs = PP == 1 ? p : ((e >> 1) * A.rot_units + p / PP) * 2 + (e & 1);
    s_cs[t * half + at_cs] = make_float2(c * A.mscale, (A.transpose ? -s : s) * A.mscale);
  }
  __syncthreads();
  store();
  for (int i0 = threadIdx.x + U * kThreads; i0 < total; i0 += U * kThreads) {
    load(i0);
    store();
  }
}

// The pairs' turns a token, from the parameters.
sta_status rope_table(const sta_rope_params* r, int d, RopeTable& tab) {
  if (!r || r->rot_dim < 2 || (r->rot_dim & 1) || r->rot_dim > d) return STA_ERR_INVALID_ARG;
  if (r->layout != STA_ROPE_HALF && r->layout != STA_ROPE_INTERLEAVED) return STA_ERR_INVALID_ARG;
  if (!(r->mscale > 0.f) || !std::isfinite(r->mscale)) return STA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  if (!r->freqs) {
    if (!(r->base > 1.0) || !std::isfinite(r->base)) return STA_ERR_INVALID_ARG;
    if (r->scaling < STA_ROPE_SCALE_NONE || r->scaling > STA_ROPE_SCALE_BLEND) return STA_ERR_INVALID_ARG;
    if (r->scaling != STA_ROPE_SCALE_NONE && (!(r->factor > 0.0) || !std::isfinite(r->factor))) return STA_ERR_INVALID_ARG;
    if (r->scaling == STA_ROPE_SCALE_BLEND &&
        (!(r->orig_len > 0.0) || !std::isfinite(r->orig_len) || !std::isfinite(r->low_turns) ||
         !std::isfinite(r->high_turns) || !(r->high_turns > r->low_turns)))
      return STA_ERR_INVALID_ARG;
  }
  for (int p = 0; p < r->rot_dim / 2; ++p) {
    double f;
    if (r->freqs) {
      f = r->freqs[p];
      if (!std::isfinite(f)) return STA_ERR_INVALID_ARG;
    } else {
      f = std::pow(r->base, -2.0 * p / r->rot_dim);
      if (r->scaling == STA_ROPE_SCALE_LINEAR) {
        f /= r->factor;
      } else if (r->scaling == STA_ROPE_SCALE_BLEND) {
        double g = (r->orig_len * f / two_pi - r->low_turns) / (r->high_turns - r->low_turns);
        g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
        f = g * f + (1.0 - g) * f / r->factor;
      }
    }
    double turns = std::fmod(f / two_pi, 1.0);
    if (turns < 0.0) turns += 1.0;
    if (turns >= 1.0) turns = 0.0;  // a tiny negative turn rounds up to a whole one
    tab.turn[p] = (uint64_t)std::ldexp(turns, 64);
  }
  return STA_OK;
}

template <typename T, bool APPEND>
sta_status launch_rope(RopeArgs& a, const RopeTable& tab, bool interleaved, cudaStream_t st) {
  constexpr int W = 16 / (int)sizeof(T);
  // 16-byte vectors when every vector lies whole on one side of each border and starts on a
  // 16-byte boundary; else element by element (16384 x 40 x 128 bf16: 58.5 us, 201 element by element)
  bool wide = a.d % W == 0 && (interleaved ? a.rot % W == 0 : (a.rot / 2) % W == 0);
  for (int g = 0; g < 3; ++g)
    if (a.heads[g])
      wide = wide && !(((uintptr_t)a.src[g] | (uintptr_t)a.dst[g] | (uint64_t)a.src_stride[g] | (uint64_t)a.dst_stride[g]) & 15);
  const int w = wide ? W : 1;
  const int wi = interleaved && w == 1 ? 2 : w;
  a.rot_units = interleaved ? a.rot / wi : a.rot / 2 / wi;
  a.units = a.rot_units + (a.d - a.rot + wi - 1) / wi;
  a.H = a.heads[0] + a.heads[1] + a.heads[2];
  // Tokens of a CTA: the number whose units fill rounds of 2 a thread best, the larger of two as good,
  // while two CTAs are left to every SM; two rounds only where six are. (16384 x 40 x 128 bf16: 58.5 us
  // by the rule, 64.6 with one token a CTA, 79 with 16; 64 new tokens with their cache write: 11.4 by
  // the rule and with one, 15.5 with 4, 32 with 16.)
  const int64_t per_token = (int64_t)a.H * a.units, round = 2 * kThreads;
  int tokens = 1;
  double best = 0;
  for (int t = 1; t <= kMaxTokens; ++t) {
    const int64_t rounds = cdiv(t * per_token, round);
    if (t > 1 && (rounds > 2 || a.n_tokens < (int64_t)t * 152 * (rounds > 1 ? 6 : 2))) break;
    const double fill = (double)(t * per_token) / (double)(rounds * round);
    if (fill >= best) {
      best = fill;
      tokens = t;
    }
  }
  a.tokens = tokens;
  const int64_t blocks = cdiv(a.n_tokens, tokens);
  if (blocks > INT32_MAX || (int64_t)tokens * a.H * a.units > INT32_MAX / 2) return STA_ERR_INVALID_ARG;
  const size_t smem = (size_t)tokens * (a.rot / 2) * sizeof(float2);
  if (wide) {
    if (interleaved) rope_kernel<T, W, true, APPEND><<<(unsigned)blocks, kThreads, smem, st>>>(a, tab);
    else rope_kernel<T, W, false, APPEND><<<(unsigned)blocks, kThreads, smem, st>>>(a, tab);
  } else {
    if (interleaved) rope_kernel<T, 1, true, APPEND><<<(unsigned)blocks, kThreads, smem, st>>>(a, tab);
    else rope_kernel<T, 1, false, APPEND><<<(unsigned)blocks, kThreads, smem, st>>>(a, tab);
  }
  STA_LAUNCH_CHECK();
  return STA_OK;
}

}  // namespace
}  // namespace sta

using namespace sta;

extern "C" sta_status sta_rope(const void* x, void* y, const int32_t* positions_dev, const sta_rope_params* rope,
                               int64_t n_tokens, int H, int d, int64_t x_stride, int64_t y_stride, int transpose,
                               sta_dtype dtype, sta_stream stream) {
  if (n_tokens < 0 || H < 1 || H > 65536 || d < 2) return STA_ERR_INVALID_ARG;
  if (dtype != STA_BF16 && dtype != STA_F32) return STA_ERR_INVALID_ARG;
  if (d > 2 * kMaxPairs) return STA_ERR_UNSUPPORTED;
  if (x_stride < (int64_t)H * d || y_stride < (int64_t)H * d || (transpose != 0 && transpose != 1)) return STA_ERR_INVALID_ARG;
  RopeTable tab;
  const sta_status st = rope_table(rope, d, tab);
  if (st != STA_OK) return st;
  if (n_tokens == 0) return STA_OK;
  if (!x || !y || !positions_dev) return STA_ERR_INVALID_ARG;
  if (x == y && x_stride != y_stride) return STA_ERR_INVALID_ARG;
  const int size = dtype == STA_BF16 ? 2 : 4;
  if (((uintptr_t)x | (uintptr_t)y) & (size - 1) || (uintptr_t)positions_dev & 3) return STA_ERR_UNSUPPORTED;
  RopeArgs a{};
  a.src[0] = static_cast<const uint8_t*>(x);
  a.dst[0] = static_cast<uint8_t*>(y);
  a.src_stride[0] = x_stride * size;
  a.dst_stride[0] = y_stride * size;
  a.heads[0] = H;
  a.n_tokens = n_tokens;
  a.d = d;
  a.rot = rope->rot_dim;
  a.transpose = transpose;
  a.mscale = rope->mscale;
  a.positions = positions_dev;
  const bool il = rope->layout == STA_ROPE_INTERLEAVED;
  return dtype == STA_BF16 ? launch_rope<__nv_bfloat16, false>(a, tab, il, (cudaStream_t)stream)
                           : launch_rope<float, false>(a, tab, il, (cudaStream_t)stream);
}

extern "C" sta_status sta_rope_append_paged(const void* q, const void* k, const void* v, int64_t q_stride,
                                            int64_t k_stride, int64_t v_stride, void* q_out, void* k_pages,
                                            void* v_pages, int page_size, int n_pages, const int32_t* page_indptr_dev,
                                            const int32_t* page_indices_dev, const int32_t* q_indptr_dev,
                                            const int32_t* kv_indptr_dev, const int32_t* positions_dev,
                                            const sta_rope_params* rope, int64_t n_tokens, int n_req, int Hq, int Hkv,
                                            int d, sta_dtype dtype, sta_stream stream) {
  if (n_tokens < 0 || n_req < 1 || Hkv < 1 || Hkv > 65536 || d < 2 || page_size < 1 || n_pages < 1) return STA_ERR_INVALID_ARG;
  if (Hq < 0 || Hq > 65536 || (Hq == 0) != (q == nullptr && q_out == nullptr)) return STA_ERR_INVALID_ARG;
  if (dtype != STA_BF16) return STA_ERR_UNSUPPORTED;
  if (d > 2 * kMaxPairs) return STA_ERR_UNSUPPORTED;
  if ((Hq > 0 && q_stride < (int64_t)Hq * d) || k_stride < (int64_t)Hkv * d || v_stride < (int64_t)Hkv * d)
    return STA_ERR_INVALID_ARG;
  RopeTable tab;
  if (rope) {
    const sta_status st = rope_table(rope, d, tab);
    if (st != STA_OK) return st;
  }
  if (n_tokens == 0) return STA_OK;
  if ((Hq > 0 && (!q || !q_out)) || !k || !v || !k_pages || !v_pages || !page_indptr_dev || !page_indices_dev ||
      !q_indptr_dev || !kv_indptr_dev)
    return STA_ERR_INVALID_ARG;
  const uintptr_t bits2 = (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)k_pages | (uintptr_t)v_pages;
  const uintptr_t bits4 = (uintptr_t)page_indptr_dev | (uintptr_t)page_indices_dev | (uintptr_t)q_indptr_dev |
                          (uintptr_t)kv_indptr_dev | (uintptr_t)positions_dev;
  if ((bits2 & 1) || (bits4 & 3)) return STA_ERR_UNSUPPORTED;
  if (q && q == q_out && q_stride != (int64_t)Hq * d) return STA_ERR_INVALID_ARG;
  RopeArgs a{};
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
  a.n_tokens = n_tokens;
  a.d = d;
  a.rot = rope ? rope->rot_dim : 0;
  a.mscale = rope ? rope->mscale : 1.f;
  a.positions = positions_dev;
  a.q_indptr = q_indptr_dev;
  a.kv_indptr = kv_indptr_dev;
  a.page_indptr = page_indptr_dev;
  a.page_indices = page_indices_dev;
  a.n_req = n_req;
  a.page_size = page_size;
  a.n_pages = n_pages;
  a.err = device_error_word();
  return launch_rope<__nv_bfloat16, true>(a, tab, rope && rope->layout == STA_ROPE_INTERLEAVED, (cudaStream_t)stream);
}
