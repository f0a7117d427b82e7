// What the kernels with rotary positions share: the pairs' turns, the vectors that a thread moves.
#pragma once
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace sta {
namespace {

constexpr int kMaxPairs = 256;    // head size at most 512

struct RopeTable {
  uint64_t turn[kMaxPairs];  // f_p / 2pi mod 1, as a fraction of 2^64
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
    double turns = f / two_pi;
    if (!(turns >= 0.0 && turns < 1.0)) turns = std::fmod(turns, 1.0);
    if (turns < 0.0) turns += 1.0;
    if (turns >= 1.0) turns = 0.0;  // a tiny negative turn rounds up to a whole one
    tab.turn[p] = (uint64_t)(turns * 0x1p64);
  }
  return STA_OK;
}

}  // namespace
}  // namespace sta
