// Shares of a launch by which its kernels stay within their buffers: plain arithmetic on the host, without CUDA, so that a
// test can go through all sizes.
#pragma once
#include <algorithm>
#include <cstdint>

namespace sta {

// CTAs of the norms' backward pass for q (ctas[0]) and k (ctas[1]) by the pieces of a token that each has: `most` at most
// together, for each CTA has a row of partial sums; one a tensor at least, and none without a piece for each of its warps.
inline void norm_ctas(int most, const int pieces[2], int64_t n_tokens, int warps, int ctas[2]) {
  // q's share, rounded, and what it leaves: each rounded by itself, two halves would make one CTA too many (31 + 1 pieces)
  int share[2] = {most, most};
  if (pieces[0] && pieces[1]) {
    share[0] = (int)(most * (double)pieces[0] / ((double)pieces[0] + (double)pieces[1]) + 0.5);
    share[0] = std::min(std::max(share[0], 1), most - 1);
    share[1] = most - share[0];
  }
  for (int g = 0; g < 2; ++g)
    ctas[g] = pieces[g] ? (int)std::min<int64_t>(share[g], (n_tokens * pieces[g] + warps - 1) / warps) : 0;
}

}  // namespace sta
