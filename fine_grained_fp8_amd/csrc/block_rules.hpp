// Which kernel, cut and grid the block operators take, from the sizes alone: plain host
// arithmetic, which host programs compile too.  The figures are for 256 CUs, a whole MI355X.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace fp8bs {

// ---- the gated product for few tokens or few tiles (kernels: gated.hip) ----
// M tokens, N = I channels, K; fp32: FP32 results, or codes of them

constexpr int kGatedExactTokens = 64;            // up to so many: FP32 values and codes from exact products (up to 16: BF16 ones too)
constexpr int kGatedMaxCuts = 8;
constexpr int64_t kMaxLds = 163840;
constexpr int64_t kRowBlockLds = 2048 + 64;      // the kernel for up to 16 tokens, LDS of one K block: their codes and scales

// The kernel for up to 16 tokens and the other one, one token, us: 7168 x 8192 24.0 / 25.6; 7168 x
// 9216 27.2 / 26.5; 7168 x 12288 34.6 / 32.4; 7168 x 18432 50 / 47.7; 7168 x 24576 81 / 62; 2048 x 10240
// 11.4 / 10.4; 16 tokens, 7168 x 8192 26.1 / 26.7; 7168 x 18432 51.6 / 47.5.
inline bool by_rows(int64_t M, int64_t N) { return M <= 16 && N <= 8192; }

// all results of up to 16 tokens, FP32 results and codes of up to 64
inline bool exact_products(int64_t M, bool fp32) { return M <= 16 || (M <= kGatedExactTokens && fp32); }
inline int64_t groups_of_64(int64_t M, int64_t N) { return (M + 63) / 64 * (N / 64); }
// Workgroups of four waves with two tiles each, 128 channels, which also have whole 1x128
// tiles of codes: where four waves of one tile give more workgroups than CUs (1333 tokens,
// 2048 x 1408: 15.0 us for 15.9; 1024, 7168 x 2048 39 for 44; 256 tokens, 7168 x 4096, 256 workgroups
// of 64 channels: 37 for 29).  Eight waves of one tile were as fast in one round of the
// CUs and slower in two (700, 7168 x 5632: 75 for 68).
inline bool whole_tiles(int64_t M, int64_t N, bool fp32) { return !exact_products(M, fp32) && groups_of_64(M, N) > 256; }
// Waves of one tile: five or six where they make one round of the CUs and four do not
// (us with 4 / 5 / 6, or four of two tiles: 48 tokens, 7168 x 18432 66 / 48 / 49, 57; its codes
// 71 / 54 / 55; 7168 x 24576 71 / 83 / 63, 75; 700 tokens, 7168 x 2048 38 / 57 / 33, 36).
inline int few_waves(int64_t M, int64_t N) {
  const int64_t blocks = (M + 63) / 64;
  for (const int w : {4, 5, 6})
    if ((N / 16 + w - 1) / w * blocks <= 256) return w;
  return 4;
}

// Which kernel.  The block GEMM's tiles are 128 tokens x 128 channels, one a CU; with
// few of them most CUs idle, and just above 256 the second round is a short one.  There
// workgroups of up to 64 tokens and 64 or 128 channels are faster: while those of 128
// channels are one round of the CUs, and up to 640 of them where the GEMM takes two.
// Measured, us, GEMM / these (tiles; workgroups of 128): 128 tokens, 7168 x 2048 (16; 32) 55 / 16;
// 300, 2048 x 1408 (33; 55) 19 / 10; 1333, 2048 x 1408 (121; 231) 20 / 15; 1024, 7168 x 2048
// (128; 256) 53 / 39; 300, 7168 x 6400 (150; 250) 55 / 39; 450, 7168 x 4608 (144; 288) 52 / 57;
// 65, 7168 x 18432 (144; 288) 64 / 83; 1333, 2048 x 2048 (176; 336) 20 / 21; 512, 7168 x 7168
// (224; 448) 59 / 67; 2700, 2048 x 1408 (242; 473) 22 / 25; 700, 7168 x 5632 (264; 484) 89 / 68;
// 192, 7168 x 18432 (288; 432) 107 / 82; 1333, 2048 x 3840 (330; 630) 40 / 33; 640, 2048 x 8192
// (320; 640) 38 / 38; 4096, 2048 x 1408 (352; 704) 36 / 34; 800, 2048 x 8192 (448; 832) 38 / 44.
// K is cut so that every CU has a workgroup; a cut adds partial sums and the
// finishing launch, about what 6 to 8 blocks of K take: 48 tokens, 7168 x 2048, with 1 / 2
// / 4 / 8 cuts 26 / 18 / 15 / 14; 256 tokens 29 / 24 / 24 / 30; 300 tokens, 2048 x 1408 11 / 14 / 18.
// Codes of tiles that no workgroup has whole take that launch anyway, and cuts of four
// blocks pay: 48 tokens, 2048 x 1408, 1 / 2 / 4 / 8 cuts 14.9 / 11.4 / 10.5 / 12; 64 tokens, 1024 x 512,
// 1 / 2 / 4 11.4 / 9.6 / 9.4; 128 tokens, 2048 x 1408 13.4 / 11.8 / 11.9; 300 tokens 13.7 / 14.1 / 18.
// FP32 results follow them, so that the codes are those of that result (64 tokens,
// 2048 x 1408: 10.5 for 10.9; 17 tokens, 1024 x 1024 7.6 for 6.3).
inline int gated_cuts(int64_t M, int64_t N, int64_t K, bool fp32) {
  if (M == 0) return 0;      // no tokens: nothing to share out (the quotients below divide by their groups)
  const int64_t kb = K / 128;
  if (by_rows(M, N)) return (int)((kb + kMaxLds / kRowBlockLds - 1) / (kMaxLds / kRowBlockLds));
  const int64_t tiles = (M + 127) / 128 * (N / 128), wide = (M + 63) / 64 * (N / 128);
  if (M > 64 && wide > 256 && (tiles <= 256 || wide > 640)) return 0;
  const int64_t groups = groups_of_64(M, N), worth = fp32 ? kb / 4 : (kb - 8) / 6;
  const int64_t c = std::min({256 / groups, worth, (int64_t)kGatedMaxCuts});
  return (int)(c > 1 ? c : 1);
}

// FP32 arrays [M][N] that a call needs: both sums of each cut, or h where its tiles of codes
// are spread over workgroups
inline int64_t gated_parts(int64_t M, int64_t N, int64_t K, bool fp32, bool codes) {
  const int cuts = gated_cuts(M, N, K, fp32);
  if (cuts > 1) return 2 * cuts;
  return cuts == 1 && codes && !whole_tiles(M, N, fp32) ? 1 : 0;
}

// ---- norms of heads with the position rotation (kernels: heads.hip) ----

constexpr int kHW = 4;                     // waves of a workgroup
constexpr int kMaxGradParts = 1280;        // workgroups of the backward pass: see divide()
constexpr int kForwardBlocks = 1280;       // and of the forward pass

// passes of a wave over the heads of a set, 64 / G heads each
constexpr int passes(int64_t heads, int G) { return (int)((heads * G + 63) / 64); }

// How a set is divided: a token's passes into `cuts` units of `per`, the units of all
// tokens dealt to the waves of `blocks` workgroups in the order of memory, so that
// what is in flight lies close together (8192 tokens of 64 + 8 heads of 128, forward 62 us
// for 66, backward 91 for 100, where each wave had a token of its own).
struct Shares {
  int per, cuts, blocks;
};
struct GradGrid {
  Shares set[2];
};

// A lane has 2 R elements.  With 8 instead of 16 the backward pass's sums, weights and
// heads in flight take about 100 registers instead of 160 - 190 (8192 tokens of 32 + 8
// heads of 128, BF16: 56 us for 62; 5003 tokens of 16 + 16 heads of 80, FP32: 39 for 46),
// and FP32 heads are still moved in 16-byte pieces (their forward pass 26 us for 31), BF16 ones
// in the backward pass in pieces of 8.  BF16 forward keeps 16, pieces of 16 bytes.  Heads over 512 would take more than a wave
// with 8.
inline int run_of(bool back, bool x_fp32, int64_t dim) { return (back || x_fp32) && dim <= 512 ? 4 : 8; }
// lanes of a head
inline int lanes_of(int64_t dim, int R) {
  int g = 4;
  while (g * 2 * R < dim) g *= 2;
  return g;
}

// A set of n passes a token for at most `most` workgroups.
inline Shares share_out(int64_t T, int64_t n, int64_t most, int64_t per) {
  if (n * T <= most * kHW) per = 1;
  const int64_t cuts = (n + per - 1) / per, blocks = (T * cuts + kHW - 1) / kHW;
  return Shares{(int)per, (int)cuts, (int)(blocks < most ? blocks : most)};
}
// The forward pass
inline Shares forward_shares(int64_t T, int64_t q_heads, int64_t k_heads, int64_t dim, bool x_fp32) {
  const int G = lanes_of(dim, run_of(false, x_fp32, dim));
  return share_out(T, passes(q_heads, G) + passes(k_heads, G), kForwardBlocks, 2);
}

// The backward pass: as many workgroups as run at once on 256 CUs, five a CU by their
// registers, dealt to the sets by their heads.  Measured with 768 / 1024 / 1280 / 2048, us:
// BF16, 8192 tokens of 32 + 8 heads of 128 60 / 58 / 54 / 60; 20000 tokens of 16 + 4 heads of 64
// 52 / 47 / 44 / 49; FP32, 5003 tokens of 16 + 16 heads of 80 39.4 / 39.3 / 38.5 / 38.7.
inline GradGrid divide(int64_t T, int64_t q_heads, int64_t k_heads, int64_t dim) {
  constexpr int64_t all = kMaxGradParts;
  const int G = lanes_of(dim, run_of(true, true, dim));
  const int64_t n[2] = {passes(q_heads, G), passes(k_heads, G)};
  GradGrid g{};
  for (int i = 0; i < 2; ++i) {
    if (n[i] == 0 || T == 0) continue;
    int64_t most = all * n[i] / (n[0] + n[1]);
    if (most < 1) most = 1;
    if (most > all - 1 && n[1 - i] > 0) most = all - 1;
    g.set[i] = share_out(T, n[i], most, 2);
  }
  return g;
}

}  // namespace fp8bs
