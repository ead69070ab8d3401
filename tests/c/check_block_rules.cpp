// Host check of the size rules of the block operators (block_rules.hpp) over their
// range, empty batches and the largest sizes among them: counts violations of what the
// launches rely on.
//  * no tokens: no launch and no workspace
//  * up to 64 tokens a kernel of few tokens takes the call; every cut has a K block, and a share's
//    codes fit LDS
//  * the workspace is the sums of all cuts, or one array where codes' tiles are spread
//  * every pass over the heads of a token is in a unit, no set has more workgroups than
//    it may, both together no more than the sums of the backward pass are read for
// Built with g++ and the undefined-behaviour sanitizer; no device code.
#include <cstdio>

#include "block_rules.hpp"

using namespace fp8bs;

static long cases = 0, violations = 0;
static void need(bool ok, const char* what, int64_t a, int64_t b, int64_t c) {
  if (ok) return;
  ++violations;
  printf("%s: %ld %ld %ld\n", what, (long)a, (long)b, (long)c);
}

static bool whole_share(const Shares& s, int64_t n, int64_t most) {
  return s.per >= 1 && s.blocks >= 1 && s.blocks <= most && (int64_t)s.per * s.cuts >= n && (int64_t)s.per * (s.cuts - 1) < n;
}

int main() {
  const int64_t tokens[] = {0, 1, 15, 16, 17, 48, 64, 65, 128, 129, 300, 700, 1333, 4096, 42000, int64_t{1} << 31};
  const int64_t channels[] = {128, 256, 1408, 2048, 4096, 8064, 8192, 8320, 10240, 18432, 24576, (int64_t{1} << 24) - 256};
  const int64_t ks[] = {128, 256, 1024, 7168, 9856, 9984, 18432, 131072, (int64_t{1} << 23) - 128};
  for (int64_t M : tokens)
    for (int64_t N : channels)
      for (int64_t K : ks)
        for (int fp32 = 0; fp32 < 2; ++fp32) {
          ++cases;
          const int cuts = gated_cuts(M, N, K, fp32);
          const int64_t parts = gated_parts(M, N, K, fp32, false);
          if (M == 0) {
            if (!by_rows(M, N)) need(cuts == 0, "cuts of nothing", M, N, K);
            continue;
          }
          need(cuts >= 0 && cuts <= K / 128 && (M > 64 || cuts > 0), "cuts", M, N, K);
          need(by_rows(M, N) ? (K / 128 + cuts - 1) / cuts * kRowBlockLds <= kMaxLds : cuts <= kGatedMaxCuts, "share", M, N, K);
          need(parts == (cuts > 1 ? 2 * cuts : 0), "sums", M, N, K);
          if (fp32)
            need(gated_parts(M, N, K, true, true) == (cuts > 1 ? 2 * cuts : cuts == 1 && !whole_tiles(M, N, true)), "codes", M, N, K);
          const int w = few_waves(M, N);
          need(w >= 4 && w <= 6, "waves", M, N, K);
        }
  const int64_t heads[] = {0, 1, 2, 3, 8, 64, 1000, int64_t{1} << 20};
  const int64_t rows[] = {0, 1, 3, 64, 5003, 20000, int64_t{1} << 25};
  const int64_t dims[] = {2, 16, 64, 72, 128, 512, 514, 1024};
  for (int64_t T : rows)
    for (int64_t q : heads)
      for (int64_t k : heads)
        for (int64_t dim : dims) {
          if (q + k == 0) continue;
          ++cases;
          const GradGrid g = divide(T, q, k, dim);
          const int G = lanes_of(dim, run_of(true, true, dim));
          need(G <= 64 && G * 2 * run_of(true, true, dim) >= dim, "lanes", q, k, dim);
          need(g.set[0].blocks + g.set[1].blocks <= kMaxGradParts, "sums", q, k, T);
          const int64_t n[2] = {q, k};
          for (int i = 0; i < 2; ++i) {
            if (T == 0 || n[i] == 0) need(g.set[i].blocks == 0, "no heads", T, q, k);
            else need(whole_share(g.set[i], passes(n[i], G), kMaxGradParts), "backward", T, q, k);
          }
          if (T == 0) continue;
          for (int fp32 = 0; fp32 < 2; ++fp32) {
            const int F = lanes_of(dim, run_of(false, fp32, dim));
            need(whole_share(forward_shares(T, q, k, dim, fp32), passes(q, F) + passes(k, F), kForwardBlocks), "forward", T, q, k);
          }
        }
  printf("cases=%ld violations=%ld\n", cases, violations);
  return violations == 0 ? 0 : 1;
}
