// Attention of chunks of new tokens over a paged KV cache.
//
// First form: one warp per (new token, query head). The lanes share the head's elements; the
// keys that the token may see are visited one by one with the online softmax
// m' = max(m, s), l' = l e^(m - m') + e^(s - m'), O' = O e^(m - m') + e^(s - m') v.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace sta {
namespace {

struct ChunkArgs {
  const __nv_bfloat16* q;  // [N, Hq, d], q_stride elements between tokens
  const __nv_bfloat16* k;  // [n_pages, page_size, Hkv, d]
  const __nv_bfloat16* v;
  __nv_bfloat16* o;        // [N, Hq, d]
  float* lse;              // [N, Hq] or null
  const int32_t* page_indptr;
  const int32_t* page_indices;
  const int32_t* q_indptr;
  const int32_t* kv_indptr;
  int64_t q_stride;
  int n_tokens, n_req, Hq, Hkv, d, page_size, n_pages;
  float scale_log2;
  int causal;
  int64_t win_lo, win_hi, n_global;  // key j of position p: (win_lo <= j - p <= win_hi or j < n_global) and, if causal, j <= p
  int* err;
};

template <int D>
__global__ void __launch_bounds__(256) chunk_kernel(const ChunkArgs A) {
  constexpr int E = D / 32;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= (int64_t)A.n_tokens * A.Hq) return;
  const int t = (int)(row / A.Hq), h = (int)(row % A.Hq), hk = h / (A.Hq / A.Hkv);
  int lo = 0, hi = A.n_req - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(A.q_indptr + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  const int r = lo, q1 = __ldg(A.q_indptr + r + 1);
  if (t >= q1) return;
  const int64_t len = max((int64_t)0, (int64_t)__ldg(A.kv_indptr + r + 1) - __ldg(A.kv_indptr + r));
  const int64_t pos = len - (q1 - t);
  const int64_t jmax = min(len - 1, A.causal ? pos : len - 1);
  const int64_t w0 = max((int64_t)0, pos + A.win_lo), w1 = min(jmax, pos + A.win_hi);
  const int64_t g1 = min(A.n_global - 1, jmax);
  const int pb = __ldg(A.page_indptr + r), pe = __ldg(A.page_indptr + r + 1);
  float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(A.q[t * A.q_stride + (int64_t)h * D + lane * E + e]) * A.scale_log2;
    acc[e] = 0.f;
  }
  for (int64_t j = g1 >= 0 ? 0 : w0; j <= max(g1, w1); ++j) {
    if (j > g1 && j < w0) j = w0;
    if (j > g1 && j > w1) break;
    const int64_t ord = pb + j / A.page_size;
    int page = ord < pe ? __ldg(A.page_indices + ord) : -1;
    if (page < 0 || page >= A.n_pages) {
      record_error(A.err, 0x110);
      page = 0;
    }
    const int64_t at = (((int64_t)page * A.page_size + j % A.page_size) * A.Hkv + hk) * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(A.k[at + e]), s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), a = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * a + p;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + p * __bfloat162float(A.v[at + e]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) A.o[row * D + lane * E + e] = __float2bfloat16_rn(acc[e] * inv);
  if (A.lse && lane == 0) A.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
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
                                          sta_stream stream) {
  constexpr int64_t kFar = (int64_t)1 << 31;  // beyond any distance between two tokens
  if (!workspace_bytes || !q_indptr_host || !kv_indptr_host || n_req < 1 || Hq < 1 || Hkv < 1 || page_size < 1 ||
      n_pages < 1 || num_splits < 0 || num_splits > 1024)
    return STA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0 || !(scale > 0.f) || !std::isfinite(scale)) return STA_ERR_INVALID_ARG;
  if (dtype != STA_BF16 || (d != 64 && d != 128) || Hq / Hkv > 128 || Hq > 65535) return STA_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * page_size > INT32_MAX) return STA_ERR_UNSUPPORTED;
  if (q_indptr_host[0] != 0 || kv_indptr_host[0] != 0) return STA_ERR_INVALID_ARG;
  for (int r = 0; r < n_req; ++r)
    if (q_indptr_host[r + 1] < q_indptr_host[r] || kv_indptr_host[r + 1] < kv_indptr_host[r]) return STA_ERR_INVALID_ARG;
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
  const size_t need = 256;
  if (!workspace) {
    *workspace_bytes = need;
    return STA_OK;
  }
  if (*workspace_bytes < need) return STA_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255) return STA_ERR_UNSUPPORTED;
  const int N = q_indptr_host[n_req];
  if (N == 0) return STA_OK;
  if (!q || !k_pages || !v_pages || !page_indptr_dev || !page_indices_dev || !q_indptr_dev || !kv_indptr_dev || !o)
    return STA_ERR_INVALID_ARG;
  if (((uintptr_t)q | (uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)o) & 15) return STA_ERR_UNSUPPORTED;
  if (((uintptr_t)page_indptr_dev | (uintptr_t)page_indices_dev | (uintptr_t)q_indptr_dev | (uintptr_t)kv_indptr_dev |
       (uintptr_t)lse) & 3)
    return STA_ERR_UNSUPPORTED;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k_pages);
  a.v = static_cast<const __nv_bfloat16*>(v_pages);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.page_indptr = page_indptr_dev;
  a.page_indices = page_indices_dev;
  a.q_indptr = q_indptr_dev;
  a.kv_indptr = kv_indptr_dev;
  a.q_stride = q_stride;
  a.n_tokens = N;
  a.n_req = n_req;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.page_size = page_size;
  a.n_pages = n_pages;
  a.scale_log2 = scale * kLog2e;
  a.err = device_error_word();
  const int64_t blocks = cdiv((int64_t)N * Hq, 8);
  if (blocks > INT32_MAX) return STA_ERR_UNSUPPORTED;
  if (d == 64) chunk_kernel<64><<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(a);
  else chunk_kernel<128><<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(a);
  STA_LAUNCH_CHECK();
  return STA_OK;
}
