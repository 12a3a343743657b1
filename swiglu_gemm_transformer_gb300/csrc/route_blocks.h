// route_blocks.h -- how the one-launch form of the routers shares its tokens out.
// Plain arithmetic without CUDA headers: k_route.cu and the host tests include it.
#pragma once

namespace swiglu {

constexpr int kOneTokens = 256;  // most tokens of the one-launch form,
constexpr int kOneBlocks = 8;    // blocks of its cluster, at most

// Most tokens that one block takes alone, and tokens of a block, at least, where there
// are several.  Counts that cross blocks cost 0.8 us, a second turn of a block's warps
// more the more lanes a token has.  In a graph, us, one block | blocks of 8 | of 16:
//   4 to 8 lanes (64 experts, k = 8)  16 tokens 3.4 | 4.2, 32 tokens 4.2 | 4.4 | 4.4,
//                                     64 tokens - | 4.5 | 4.3
//   16 lanes (128 experts)            16 tokens 4.2 | 4.5, 24 tokens 4.8 | 4.6
//   32 lanes (256 experts)            12 tokens 4.8 | 5.2, 13 tokens 5.3 | 5.2
//   by scores, 64 experts             16 tokens 4.9 | 5.1, 20 tokens 5.2 | 5.1
//   by scores, 256 experts            12 tokens 5.6 | 6.2, 15 tokens 6.2 | 6.2
//   by scores, 1024 experts           15 tokens 13.6 | 13.9, 16 tokens 18.8 | 14.1
//   by scores, 256 experts, k = 32    13 tokens 11.2 | 9.9
struct OneLaunch {
  int alone, least;
};
constexpr OneLaunch one_by_logit(int lanes) {
  return lanes <= 8 ? OneLaunch{32, 16} : lanes <= 16 ? OneLaunch{16, 8} : OneLaunch{12, 8};
}
constexpr OneLaunch one_by_score(int experts_of_a_lane, int k) {
  return {k > 16 ? 8 : experts_of_a_lane <= 2 ? 18 : 15, 8};
}

// Tokens of a block of T <= kOneTokens: all of them, or the least power of two times
// `least` that leaves no more than kOneBlocks blocks.
constexpr int one_block_tokens(int T, OneLaunch how) {
  if (T <= how.alone) return T;
  int n = how.least;
  while (n * kOneBlocks < T) n *= 2;
  return n;
}
// Blocks, a power of two.
constexpr int one_blocks(int T, int tokens) {
  int n = 1;
  while (n * tokens < T) n *= 2;
  return n;
}

}  // namespace swiglu
