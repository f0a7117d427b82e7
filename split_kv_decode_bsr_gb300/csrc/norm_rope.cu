// Root-mean-square norms of query and key heads with the rotary positions in the same pass: alone
// (sta_norm_rope), its gradient (sta_norm_rope_bwd) and fused with the write of new tokens into a
// paged KV cache (sta_norm_rope_append_paged).
//
//   y = R_t (x r w),  r = 1 / sqrt(mean(x^2) + eps)
//   g = R_t' dy,  dx = r (g w - x r mean(g w x r)),  dw = sum over tokens and heads of g x r
//
// L lanes of a warp (a power of two) share a head: each holds the 16-byte vectors (half layout: pairs
// of them, half a rotation apart) that the rotary kernel calls units, so that the turn needs no exchange
// and the sums over a head are log2 L shuffles. A head is read once and written once; the products in
// between stay in fp32 and are rounded once. The cosines and sines of a CTA's tokens go through
// shared memory, and the turns are exact at any position, as in the rotary kernel.
#include "rope.inl"

namespace sta {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens of a CTA (backward: of one of its steps)
template <typename T> constexpr int kMany = sizeof(T) == 2 ? 2 : 4;  // units of a lane where a head has more than 32 (at most 64, 128)
constexpr int kMaxGrid = 152 * 4;  // CTAs of a backward pass, each with a row of partial sums for dw

struct NormArgs {
  const uint8_t* src[3];  // q, k, v (v: to pages alone)
  uint8_t* dst[3];        // backward: dq, dk
  const uint8_t* dy[2];   // backward: the gradients of the results
  int64_t src_stride[3], dst_stride[3], dy_stride[2];  // bytes between tokens (k, v pages: of a page)
  const float* weight[2];
  int heads[3];
  int H;                  // their sum
  uint32_t h_mul;         // n / H for n < 2^31: high word of n h_mul, shifted right by h_shift (-1: H is 1)
  int h_shift;
  int64_t n_tokens;
  int d, rot;
  int tokens;             // tokens of a CTA (or step)
  int units, rot_units;   // units of a head; the first rot_units turn
  int log_l;              // lanes of a head
  int w_at;               // byte offset of the weights in shared memory
  float eps, inv_d, mscale;
  const int32_t* positions;
  // paged destination of k and v
  const int32_t* q_indptr;
  const int32_t* kv_indptr;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  int n_req, page_size, n_pages;
  int* err;
  float* part;            // backward: [CTAs, 2, d]
};

// Where a new token goes, found by a whole warp: its position and its cache row, -1 when it goes
// nowhere. False for padding. 128 requests are looked at at once, where one thread's binary search would
// take a round trip to memory for each of its steps.
__device__ __forceinline__ bool token_place_warp(const NormArgs& A, int64_t t, int lane, int& pos, int64_t& row) {
  pos = 0;
  row = -1;
  const int first = __ldg(A.q_indptr), end = __ldg(A.q_indptr + A.n_req);
  int lo = 0, n = A.n_req;  // the last request that starts at or before t is among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 127) >> 7;
    int c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = (lane + 32 * k) * step;
      c += __popc(__ballot_sync(0xffffffffu, at < n && __ldg(A.q_indptr + lo + at) <= t));
    }
    c = max(c - 1, 0) * step;
    lo += c;
    n = min(step, n - c);
  }
  if (t < first || t >= end) return false;
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
    if (lane == 0) record_error(A.err, 0x604);
    return true;
  }
  const int page = __ldg(A.page_indices + e);
  if (page < 0 || page >= A.n_pages) {
    if (lane == 0) record_error(A.err, 0x110);
    return true;
  }
  row = (int64_t)page * A.page_size + p % A.page_size;
  return true;
}

// A thread's units of its heads: the same elements of every head it works on.
template <typename T, int W, bool IL, int NU>
struct Units {
  static constexpr int WI = IL && W == 1 ? 2 : W;  // elements of a vector: whole pairs when interleaved
  static constexpr int PP = IL ? WI / 2 : WI;      // pairs of a unit
  static constexpr int E = IL ? WI : 2 * WI;       // elements of a unit that turns
  int unit[NU];  // -1: none
  int off[NU];   // first element
  bool turn[NU];
  int half, d;
  __device__ __forceinline__ void set(const NormArgs& A) {
    const int l = threadIdx.x & ((1 << A.log_l) - 1);
    half = A.rot >> 1;
    d = A.d;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int u = l + (j << A.log_l);
      turn[j] = u < A.rot_units;
      unit[j] = u < A.units ? u : -1;
      off[j] = turn[j] ? u * WI : A.rot + (u - A.rot_units) * WI;
    }
  }
  struct Row {
    Vec<T, WI> a[NU], b[IL ? 1 : NU];
  };
  // elements that are not there stay as they are
  __device__ __forceinline__ void load(const T* src, Row& r) const {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if (unit[j] < 0) continue;
      if (W == 1 && IL && !turn[j]) {  // the last element of an odd rest is alone
        r.a[j].v[0] = src[off[j]];
        if (off[j] + 1 < d) r.a[j].v[1] = src[off[j] + 1];
      } else {
        r.a[j].load(src + off[j]);
      }
      if (!IL && turn[j]) r.b[j].load(src + off[j] + half);
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
  // element e of unit j: its place in the head, -1 when there is none
  __device__ __forceinline__ int place(int j, int e) const {
    if (unit[j] < 0 || (!turn[j] && e >= WI)) return -1;
    const int p = off[j] + (e < WI ? e : half + e - WI);
    return p < d ? p : -1;
  }
  // the E elements of unit j in fp32, 0 where there is none
  __device__ __forceinline__ void get(const Row& r, int j, float* x) const {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool some = unit[j] >= 0 && (e < WI || turn[j]) && (W > 1 || !IL || e == 0 || off[j] + e < d);
      x[e] = some ? to_f(e < WI ? r.a[j].v[e] : r.b[IL ? 0 : j].v[e - WI]) : 0.f;
    }
  }
  __device__ __forceinline__ void put(Row& r, int j, const float* x) const {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (e < WI) r.a[j].v[e] = from_f<T>(x[e]);
      else r.b[IL ? 0 : j].v[e - WI] = from_f<T>(x[e]);
    }
  }
  // The weights of unit j. In shared memory four at a time, [q, k][E / 4][units], so that neighbouring
  // lanes read neighbouring words; straight from memory where heads go element by element.
  static __device__ __forceinline__ void stage(const NormArgs& A, float4* s_w) {
    if constexpr (W > 1) {
      float* s = reinterpret_cast<float*>(s_w);
      const int each = A.units * E;
      for (int i = threadIdx.x; i < 2 * each; i += kThreads) {
        const int g = i >= each, x = i - g * each, u = (x >> 2) % A.units, e = (x >> 2) / A.units * 4 + (x & 3);
        const bool turns = u < A.rot_units;
        const int o = turns ? u * WI : A.rot + (u - A.rot_units) * WI, p = e < WI ? o + e : o + (A.rot >> 1) + e - WI;
        s[i] = A.weight[g] && (e < WI || turns) ? __ldg(A.weight[g] + p) : 1.f;
      }
    }
  }
  __device__ __forceinline__ void weights(const NormArgs& A, const float4* s_w, int g, int j, float* w) const {
    if constexpr (W > 1) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 v = s_w[(g * (E / 4) + e / 4) * A.units + max(unit[j], 0)];
        w[e] = v.x;
        w[e + 1] = v.y;
        w[e + 2] = v.z;
        w[e + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int p = place(j, e);
        w[e] = A.weight[g] && p >= 0 ? __ldg(A.weight[g] + p) : 1.f;
      }
    }
  }
  // cosine and sine of unit j's pairs, two pairs in 16 bytes: [PP / 2][units that turn][2]
  __device__ __forceinline__ void angles(const NormArgs& A, const float2* s_cs, int j, float2* cs) const {
    if constexpr (PP == 1) {
      cs[0] = s_cs[IL ? off[j] >> 1 : off[j]];
    } else {
      const float4* c4 = reinterpret_cast<const float4*>(s_cs) + unit[j];
#pragma unroll
      for (int i = 0; i < PP / 2; ++i) {
        const float4 v = c4[i * A.rot_units];
        cs[2 * i] = make_float2(v.x, v.y);
        cs[2 * i + 1] = make_float2(v.z, v.w);
      }
    }
  }
  // pairs (a, b) of x turned: (a cos - b sin, b cos + a sin), or back
  static __device__ __forceinline__ void turn_pairs(float* x, const float2* cs, bool back) {
#pragma unroll
    for (int p = 0; p < PP; ++p) {
      float &a = x[IL ? 2 * p : p], &b = x[IL ? 2 * p + 1 : WI + p];
      const float c = cs[p].x, s = back ? -cs[p].y : cs[p].y, t = a;
      a = t * c - b * s;
      b = t * s + b * c;
    }
  }
  // The cosines and sines (times the magnitude) of nt tokens.
  static __device__ __forceinline__ void table(const NormArgs& A, const RopeTable& tab, const int* s_pos, int nt, float2* s_cs) {
    const int half = A.rot >> 1;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int t = i / half, p = i - t * half;
      const uint64_t phase = (uint64_t)(int64_t)s_pos[t] * tab.turn[p];
      float s, c;
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
      const int e = p % PP;  // place of the pair in its unit
      const int at = PP == 1 ? p : ((e >> 1) * A.rot_units + p / PP) * 2 + (e & 1);
      s_cs[t * half + at] = make_float2(c * A.mscale, s * A.mscale);
    }
  }
};

__device__ __forceinline__ float lanes_sum(float x, int log_l) {
  for (int o = 1 << log_l >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ int token_of(const NormArgs& A, int row) {
  return A.h_shift < 0 ? row : (int)(__umulhi((uint32_t)row, A.h_mul) >> A.h_shift);
}

// W: elements of a vector (1: unaligned data, element by element); IL: interleaved pairs; NU: units of a
// lane; APPEND: q, k, v with k and v going to pages.
template <typename T, int W, bool IL, int NU, bool APPEND>
__global__ void __launch_bounds__(kThreads, NU == 1 ? 5 : 2)
    norm_rope_kernel(const __grid_constant__ NormArgs A, const __grid_constant__ RopeTable tab) {
  using U = Units<T, W, IL, NU>;
  constexpr int R = NU == 1 ? 2 : 1;  // heads of a lane in flight
  extern __shared__ __align__(16) uint8_t smem[];
  float2* s_cs = reinterpret_cast<float2*>(smem);
  float4* s_w = reinterpret_cast<float4*>(smem + A.w_at);
  __shared__ int64_t s_row[kMaxTokens];
  __shared__ int s_pos[kMaxTokens];
  __shared__ int s_live[kMaxTokens];
  const int half = A.rot >> 1, each = kThreads >> A.log_l;  // heads of a round
  const int64_t t0 = (int64_t)blockIdx.x * A.tokens;
  const int nt = (int)min((int64_t)A.tokens, A.n_tokens - t0), total = nt * A.H;
  U u;
  u.set(A);
  typename U::Row x[R];
  int tok[R], hd[R];  // token, -1: none; head of q, k and v together
  auto group = [&](int h) { return h < A.heads[0] ? 0 : (!APPEND || h < A.heads[0] + A.heads[1] ? 1 : 2); };
  auto in_group = [&](int h, int g) { return h - (g > 0 ? A.heads[0] : 0) - (g > 1 ? A.heads[1] : 0); };
  auto load = [&](int i0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = i0 + r * each + (threadIdx.x >> A.log_l);
      tok[r] = -1;
      if (i >= total) continue;
      const int t = token_of(A, i), h = i - t * A.H, g = group(h);
      tok[r] = t;
      hd[r] = h;
      u.load(reinterpret_cast<const T*>(A.src[g] + (t0 + t) * A.src_stride[g]) + (int64_t)in_group(h, g) * A.d, x[r]);
    }
  };
  auto finish = [&]() {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int g = tok[r] < 0 ? 2 : group(hd[r]);
      float ss = 0.f;
      if (g < 2) {
#pragma unroll
        for (int j = 0; j < NU; ++j) {
          float v[U::E], s4[4] = {0.f, 0.f, 0.f, 0.f};
          u.get(x[r], j, v);
#pragma unroll
          for (int e = 0; e < U::E; ++e) s4[e & 3] = fmaf(v[e], v[e], s4[e & 3]);
          ss += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        }
      }
      ss = lanes_sum(ss, A.log_l);  // (of a whole warp: lanes without a head take part)
      if (tok[r] < 0) continue;
      const int t = tok[r];
      if (APPEND && (!s_live[t] || (g > 0 && s_row[t] < 0))) continue;
      if (g < 2) {
        const float rms = rsqrtf(fmaf(ss, A.inv_d, A.eps));
#pragma unroll
        for (int j = 0; j < NU; ++j) {
          float v[U::E], w[U::E];
          u.get(x[r], j, v);
          u.weights(A, s_w, g, j, w);
#pragma unroll
          for (int e = 0; e < U::E; ++e) v[e] = v[e] * rms * w[e];
          if (u.turn[j]) {
            float2 cs[U::PP];
            u.angles(A, s_cs + t * half, j, cs);
            U::turn_pairs(v, cs, false);
          }
          u.put(x[r], j, v);
        }
      }
      const int64_t at = APPEND && g > 0 ? s_row[t] : t0 + t;
      u.store(reinterpret_cast<T*>(A.dst[g] + at * A.dst_stride[g]) + (int64_t)in_group(hd[r], g) * A.d, x[r]);
    }
  };
  load(0);  // under the table's latency
  if constexpr (APPEND) {
    const int lane = threadIdx.x & 31;
    for (int t = threadIdx.x >> 5; t < nt; t += kThreads / 32) {
      int pos;
      int64_t row;
      const bool live = token_place_warp(A, t0 + t, lane, pos, row);
      if (lane == 0) {
        s_pos[t] = A.positions ? __ldg(A.positions + t0 + t) : pos;
        s_row[t] = row;
        s_live[t] = live;
      }
    }
  } else if ((int)threadIdx.x < nt) {
    s_pos[threadIdx.x] = A.positions ? __ldg(A.positions + t0 + threadIdx.x) : 0;
  }
  U::stage(A, s_w);
  __syncthreads();
  U::table(A, tab, s_pos, nt, s_cs);
  __syncthreads();
  finish();
  for (int i0 = R * each; i0 < total; i0 += R * each) {
    load(i0);
    finish();
  }
}

// Persistent CTAs over steps of A.tokens tokens; a thread's part of dw stays in registers throughout.
template <typename T, int W, bool IL, int NU>
__global__ void __launch_bounds__(kThreads, NU == 1 ? 2 : 1)
    norm_rope_bwd_kernel(const __grid_constant__ NormArgs A, const __grid_constant__ RopeTable tab) {
  using U = Units<T, W, IL, NU>;
  extern __shared__ __align__(16) uint8_t smem[];
  float2* s_cs = reinterpret_cast<float2*>(smem);
  float4* s_w = reinterpret_cast<float4*>(smem + A.w_at);
  __shared__ int s_pos[kMaxTokens];
  const int half = A.rot >> 1, each = kThreads >> A.log_l;
  U u;
  u.set(A);
  float dw[2][NU][U::E] = {};
  U::stage(A, s_w);
  for (int64_t t0 = (int64_t)blockIdx.x * A.tokens; t0 < A.n_tokens; t0 += (int64_t)gridDim.x * A.tokens) {
    const int nt = (int)min((int64_t)A.tokens, A.n_tokens - t0), total = nt * A.H;
    typename U::Row x, dy;
    int tok, hd;
    auto load = [&](int i0) {
      const int i = i0 + (threadIdx.x >> A.log_l);
      tok = -1;
      if (i >= total) return;
      tok = token_of(A, i);
      hd = i - tok * A.H;
      const int g = hd >= A.heads[0], h = hd - (g ? A.heads[0] : 0);
      u.load(reinterpret_cast<const T*>(A.src[g] + (t0 + tok) * A.src_stride[g]) + (int64_t)h * A.d, x);
      u.load(reinterpret_cast<const T*>(A.dy[g] + (t0 + tok) * A.dy_stride[g]) + (int64_t)h * A.d, dy);
    };
    auto finish = [&]() {
      const bool some = tok >= 0;
      const int g = some && hd >= A.heads[0];
      float ss = 0.f, sg = 0.f;
      float gr[NU][U::E];  // R' dy
      if (some) {
#pragma unroll
        for (int j = 0; j < NU; ++j) {
          float v[U::E], w[U::E];
          u.get(x, j, v);
          u.get(dy, j, gr[j]);
          if (u.turn[j]) {
            float2 cs[U::PP];
            u.angles(A, s_cs + tok * half, j, cs);
            U::turn_pairs(gr[j], cs, true);
          }
          u.weights(A, s_w, g, j, w);
          float s2[2] = {0.f, 0.f}, g2[2] = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < U::E; ++e) {
            s2[e & 1] = fmaf(v[e], v[e], s2[e & 1]);
            g2[e & 1] = fmaf(gr[j][e] * w[e], v[e], g2[e & 1]);
          }
          ss += s2[0] + s2[1];
          sg += g2[0] + g2[1];
        }
      }
      ss = lanes_sum(ss, A.log_l);
      sg = lanes_sum(sg, A.log_l);
      if (!some) return;
      const float rms = rsqrtf(fmaf(ss, A.inv_d, A.eps)), mean = rms * (sg * A.inv_d);
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        float v[U::E], w[U::E];
        u.get(x, j, v);
        u.weights(A, s_w, g, j, w);
#pragma unroll
        for (int e = 0; e < U::E; ++e) {
          const float xh = v[e] * rms, add = gr[j][e] * xh;
          if (g) dw[1][j][e] += add;
          else dw[0][j][e] += add;
          v[e] = rms * (gr[j][e] * w[e] - xh * mean);
        }
        u.put(dy, j, v);
      }
      u.store(reinterpret_cast<T*>(A.dst[g] + (t0 + tok) * A.dst_stride[g]) + (int64_t)(hd - (g ? A.heads[0] : 0)) * A.d, dy);
    };
    load(0);
    if ((int)threadIdx.x < nt) s_pos[threadIdx.x] = A.positions ? __ldg(A.positions + t0 + threadIdx.x) : 0;
    __syncthreads();
    U::table(A, tab, s_pos, nt, s_cs);
    __syncthreads();
    finish();
    for (int i0 = each; i0 < total; i0 += each) {
      load(i0);
      finish();
    }
    __syncthreads();  // the next step's positions and table
  }
  // the CTA's sums: over the heads of a warp by shuffles, then over the warps in order
  float* s_red = reinterpret_cast<float*>(smem);  // [warps][2][d]
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int e = 0; e < U::E; ++e) {
        float v = dw[g][j][e];
        for (int o = 1 << A.log_l; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int p = u.place(j, e);
        if (p >= 0 && (threadIdx.x & 31) < (1 << A.log_l)) s_red[((threadIdx.x >> 5) * 2 + g) * A.d + p] = v;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * A.d; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += s_red[w * 2 * A.d + i];
    A.part[(int64_t)blockIdx.x * 2 * A.d + i] = v;
  }
}

// dw from the CTAs' sums, always in the same order: 32 columns a block, 32 slices of the CTAs.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int n, int d, float* dqw, float* dkw) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  float v = 0.f;
  if (col < 2 * d) {
#pragma unroll 4
    for (int i = y; i < n; i += 32) v += __ldg(part + (int64_t)i * 2 * d + col);
  }
  s[y][c] = v;
  __syncthreads();
  if (y == 0 && col < 2 * d) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][c];
    float* out = col < d ? dqw : dkw;
    if (out) out[col < d ? col : col - d] = v;
  }
}

// Shape of a launch: vectors, units, lanes and tokens of a CTA. False: more heads than a CTA can number.
bool set_shape(NormArgs& a, int size, bool interleaved, bool backward, bool& wide, int& nu, size_t& smem) {
  const int W = 16 / size;
  // 16-byte vectors when every vector lies whole on one side of each border and starts on a 16-byte
  // boundary; else element by element
  wide = a.d % W == 0 && (interleaved ? a.rot % W == 0 : (a.rot / 2) % W == 0);
  for (int g = 0; g < 3; ++g)
    if (a.heads[g]) {
      wide = wide && !(((uintptr_t)a.src[g] | (uintptr_t)a.dst[g] | (uint64_t)a.src_stride[g] | (uint64_t)a.dst_stride[g]) & 15);
      if (backward) wide = wide && !(((uintptr_t)a.dy[g] | (uint64_t)a.dy_stride[g]) & 15);
    }
  const int wi = wide ? W : (interleaved ? 2 : 1);
  a.rot_units = interleaved ? a.rot / wi : a.rot / 2 / wi;
  a.units = a.rot_units + (a.d - a.rot + wi - 1) / wi;
  a.log_l = 0;
  while (a.log_l < 5 && (1 << a.log_l) < a.units) ++a.log_l;
  nu = wide ? (a.units <= 32 ? 1 : 4) : 16;
  if (nu == 16) a.log_l = 5;
  a.H = a.heads[0] + a.heads[1] + a.heads[2];
  int l = 0;
  while (((int64_t)1 << l) < a.H) ++l;
  a.h_mul = (uint32_t)((((uint64_t)1 << (31 + l)) + a.H - 1) / a.H);  // exact for rows below 2^31
  a.h_shift = l - 1;
  a.inv_d = 1.f / (float)a.d;
  // Tokens of a CTA (or step): the number whose heads fill its rounds best, the larger of two as good, while
  // two CTAs are left to every SM; more than one round only where six are.
  const int64_t round = (int64_t)(kThreads >> a.log_l) * (!backward && nu == 1 ? 2 : 1);
  int tokens = 1;
  double best = 0;
  const int most = backward ? 8 : 2;  // rounds
  for (int t = 1; t <= kMaxTokens; ++t) {
    const int64_t rounds = cdiv((int64_t)t * a.H, round);
    if (t > 1 && (rounds > most || a.n_tokens < (int64_t)t * 152 * (rounds > 1 ? 6 : 2))) break;
    const double fill = (double)((int64_t)t * a.H) / (double)(rounds * round);
    if (fill >= best) {
      best = fill;
      tokens = t;
    }
  }
  a.tokens = tokens;
  a.w_at = (tokens * (a.rot / 2) * (int)sizeof(float2) + 15) & ~15;
  smem = a.w_at + (wide ? (size_t)2 * a.units * wi * (interleaved ? 1 : 2) * sizeof(float) : 0);
  if (backward) smem = std::max(smem, (size_t)(kThreads / 32) * 2 * a.d * sizeof(float));
  return cdiv(a.n_tokens, tokens) <= INT32_MAX && (int64_t)tokens * a.H <= INT32_MAX / 2;
}

template <typename T, bool APPEND>
sta_status launch_norm(NormArgs& a, const RopeTable& tab, bool il, cudaStream_t st) {
  constexpr int W = 16 / (int)sizeof(T);
  bool wide;
  int nu;
  size_t smem;
  if (!set_shape(a, (int)sizeof(T), il, false, wide, nu, smem)) return STA_ERR_INVALID_ARG;
  const unsigned blocks = (unsigned)cdiv(a.n_tokens, a.tokens);
  auto go = [&](auto kern) { kern<<<blocks, kThreads, smem, st>>>(a, tab); };
  if (nu == 1) il ? go(norm_rope_kernel<T, W, true, 1, APPEND>) : go(norm_rope_kernel<T, W, false, 1, APPEND>);
  else if (nu == 4) il ? go(norm_rope_kernel<T, W, true, kMany<T>, APPEND>) : go(norm_rope_kernel<T, W, false, kMany<T>, APPEND>);
  else il ? go(norm_rope_kernel<T, 1, true, 16, APPEND>) : go(norm_rope_kernel<T, 1, false, 16, APPEND>);
  STA_LAUNCH_CHECK();
  return STA_OK;
}

template <typename T>
sta_status launch_bwd(NormArgs& a, const RopeTable& tab, bool il, float* dqw, float* dkw, cudaStream_t st) {
  constexpr int W = 16 / (int)sizeof(T);
  bool wide;
  int nu;
  size_t smem;
  if (!set_shape(a, (int)sizeof(T), il, true, wide, nu, smem)) return STA_ERR_INVALID_ARG;
  const unsigned blocks = (unsigned)std::min<int64_t>(kMaxGrid, cdiv(a.n_tokens, a.tokens));
  auto go = [&](auto kern) { kern<<<blocks, kThreads, smem, st>>>(a, tab); };
  if (nu == 1) il ? go(norm_rope_bwd_kernel<T, W, true, 1>) : go(norm_rope_bwd_kernel<T, W, false, 1>);
  else if (nu == 4) il ? go(norm_rope_bwd_kernel<T, W, true, kMany<T>>) : go(norm_rope_bwd_kernel<T, W, false, kMany<T>>);
  else il ? go(norm_rope_bwd_kernel<T, 1, true, 16>) : go(norm_rope_bwd_kernel<T, 1, false, 16>);
  STA_LAUNCH_CHECK();
  if (dqw || dkw) {
    norm_dw_kernel<<<(unsigned)cdiv(2 * a.d, 32), 1024, 0, st>>>(a.part, (int)blocks, a.d, dqw, dkw);
    STA_LAUNCH_CHECK();
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
  return dtype == STA_BF16 ? launch_norm<__nv_bfloat16, false>(a, tab, il, (cudaStream_t)stream)
                           : launch_norm<float, false>(a, tab, il, (cudaStream_t)stream);
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
  const size_t need = (size_t)kMaxGrid * 2 * d * sizeof(float);
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
      norm_dw_kernel<<<(unsigned)cdiv(2 * d, 32), 1024, 0, s>>>(a.part, 0, d, dq_weight, dk_weight);
      STA_LAUNCH_CHECK();
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
  return launch_norm<__nv_bfloat16, true>(a, tab, rope && rope->layout == STA_ROPE_INTERLEAVED, (cudaStream_t)stream);
}
