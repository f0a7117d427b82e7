// Shares of a launch by which its kernels stay within their buffers: plain arithmetic on the host, without CUDA, so that a
// test can go through all sizes. (What the device uses too is constexpr.)
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

// Few rows beside shared prefixes: KV heads of a CTA, warps of a head, which take tiles of 16 keys by turns, and the stages of
// the CTA's ring, a tile's K and V of all its heads each.
constexpr int kRowRing = 192 * 1024;
constexpr int row_heads(int Hkv) { return Hkv < 8 ? Hkv : 8; }
constexpr int row_turns(int Hkv) { return 8 / row_heads(Hkv); }
constexpr int row_stages(int d, int heads) {
  const int n = kRowRing / (heads * d * 64);
  return n < 16 ? n : 16;
}
// The first tile of a piece that a turn takes, counted in the piece, which begins with the CTA's tile t0. Turns go by the tile's
// number in the CTA's run, not in the piece, so that all tiles of a stage are one warp's (turns, a power of two, divide the
// stages): it has waited for a stage's last tile when it waits for the next one, whose wait would pass, the parity being
// the same, while the tile before that is still being copied.
constexpr int row_first(unsigned t0, int turn, int turns) { return (int)((unsigned)turn - t0) & (turns - 1); }

}  // namespace sta
