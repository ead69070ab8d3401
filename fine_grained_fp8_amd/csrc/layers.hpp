// Host-side launchers of the layer operators around the FP8 products (layer
// norm, the few-token expert layer, adapters beside a projection), internal
// to libfp8bs.so.  Arguments are already validated by api_layers.cpp; each
// launcher only sizes its grids and enqueues on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"

namespace fp8bs {

struct LayerNormProblem {
  const void* x;        // BF16 or FP32 [rows][ldx]
  int64_t rows, cols, ldx;
  const void* w;        // [cols] or null (ones)
  const void* b;        // [cols] or null (zeros)
  int x_fp32, w_fp32;
  float eps;
  void* y;              // [rows][ldy] in x's type, or null (then q is set)
  int64_t ldy;
  float* mean;          // [rows] or null
  float* rstd;          // [rows] or null
  uint8_t* q;           // E4M3 codes [rows][ldq], or null
  int64_t ldq;
  float* s;             // scales [cols/128][ld_s], or null
  int64_t ld_s;
};
hipError_t launch_layer_norm(const LayerNormProblem& p, hipStream_t stream);

struct LayerNormGradProblem {
  const void* dy;       // BF16 or FP32 [rows][lddy]
  const void* x;        // the same type [rows][ldx]
  int64_t rows, cols, lddy, ldx;
  const float* mean;    // [rows]
  const float* rstd;    // [rows]
  const void* w;        // [cols] or null (ones)
  int x_fp32, w_fp32;
  void* dx;             // x's type [rows][lddx]
  int64_t lddx;
  float* dw;            // [cols] or null
  float* db;            // [cols] or null
  float* partial;       // [layer_norm_grad_parts][2][cols]
};
// workgroups of the backward pass, each with its share of the column sums
int64_t layer_norm_grad_parts(int64_t rows, int64_t cols);
hipError_t launch_layer_norm_backward(const LayerNormGradProblem& p, hipStream_t stream);

// the longest row the layer norm holds in registers
constexpr int64_t kNormMaxCols = 16384;

// ---- the few-token expert layer ----
constexpr int kMoeMaxTokens = 64, kMoeMaxTopK = 16, kMoeMaxExperts = 1024;
constexpr int kMoeSplits = 8;
// workgroups that share a 16-channel tile of the down product, so that there
// are about two for every compute unit
inline int moe_cuts(int64_t H) {
  const int64_t c = (512 + H / 16 - 1) / (H / 16);
  return H / 16 >= 256 ? 1 : (int)(c < 8 ? c : 8);
}
// shares of a row of K that small dot products are cut into: eight waves with
// about a 128-wide block each
inline int dot_splits(int64_t K, int most) {
  const int64_t s = (K / 128 + 7) / 8;
  return (int)(s < most ? s : most);
}
struct MoeProblem {
  int T, H, I, E, first, local, top_k;
  const uint16_t* x;          // BF16 [T][ldx]
  int64_t ldx;
  const uint16_t* router;     // BF16 [E][ld_r]
  int64_t ld_r;
  const float* bias;          // [E] or null
  int sigmoid, normalize;
  float gate_scale;
  const uint8_t* w13;         // operand-tiled codes [local][2 I][H]: gate rows, then up rows
  const float* s13;           // [local][2 I / 128][H / 128]
  const uint8_t* w2;          // operand-tiled codes [local][H][I]
  const float* s2;            // [local][H / 128][I / 128]
  void* y;                    // [T][ldy]
  int64_t ldy;
  int y_fp32;
  // workspace
  int splits;                 // shares of H that the logits are summed over
  float* logits;              // [splits][T][E]: partial sums
  uint8_t* xq;                // [T][H]
  float* xs;                  // [T][H / 128]
  int32_t* slot_expert;       // [T][top_k]: chosen experts, best first
  float* slot_gate;           // [T][top_k]
  float* h;                   // [T top_k][I]
  uint8_t* hq;                // [T top_k][I]
  float* hs;                  // [T top_k][I / 128]
  int32_t* counts;            // [local]: slots that chose each held expert
  int32_t* lists;             // [local][kMoeMaxTokens]: those slots (token top_k + place), in token order
  float* parts;               // [H / 16][moe_cuts(H)][T][16]: the down kernel's sums, if a tile is cut
  int32_t* plan;              // [2 + 2 parts + 2 T top_k]: see make_plan; parts <= T top_k (1 + 1/16)
};
hipError_t launch_moe_few_tokens(const MoeProblem& p, hipStream_t stream);

// ---- adapters beside a shared projection ----
constexpr int kAdapterFewTokens = 64;   // the most tokens of the few-token form
constexpr int kAdapterMaxRank = 128;
constexpr int kAdapterSplits = 8;
// Shares of K of the shrink.  Prompts: about four 128-wide blocks each, so that
// a wave has one or two blocks' loads to wait for.  Measured at rank 64 with 1 /
// 2 / 4 / 8 shares, us of a call with 1024 outputs: K = 2048, 1333 tokens 47 / 41
// / 40 / 41; K = 7168, 4096 tokens 114 / 113 / 110 / 103; K = 18432, 8192 tokens
// 484 / 450 / 407 / 396.  (One share that writes z itself and saves the launch
// that adds the shares: the first of each.)
inline int adapter_splits(int64_t T, int64_t K) {
  if (T <= kAdapterFewTokens) return dot_splits(K, kAdapterSplits);
  const int64_t s = (K / 128 + 3) / 4;
  return (int)(s < kAdapterSplits ? s : kAdapterSplits);
}
struct AdapterProblem {
  int64_t T, N, K;
  int r, n;
  const uint16_t* x;          // BF16 [T][ldx]
  int64_t ldx;
  const uint8_t* W;           // operand-tiled codes [N][K]
  const float* sW;            // [N / 128][ld_sw]
  int64_t ld_sw;
  const uint16_t* A;          // BF16 [n][r][K]
  const uint16_t* B;          // BF16 [n][N][r]
  const int32_t* ids;         // [T]
  const float* scales;        // [n] or null (ones)
  void* C;                    // [T][ldc]
  int64_t ldc;
  int out_fp32;
  // workspace
  uint8_t* xq;                // few: operand tiles of 16 tokens; otherwise [T][K]
  float* xs;                  // few: [T][K / 128]; otherwise [K / 128][round_up(T, 4)]
  int splits;                 // adapter_splits(T, K)
  float* zp;                  // [splits][T][r]: partial sums of A x
  uint16_t* z;                // prompts: [T][r / 8][16]: A x as BF16 terms hi[8], lo[8] for every 8 ranks
};
// the few-token form (T <= kAdapterFewTokens): quantization, shrink, projection and expand
hipError_t launch_adapter_few(const AdapterProblem& p, hipStream_t stream);
// codes and scales of x (MN-major, leading dimension ld_s) and z for any number of tokens
hipError_t launch_adapter_prompt(const AdapterProblem& p, int64_t ld_s, hipStream_t stream);

// The split-K workspace of the persistent GEMM on `stream` (api.cpp)
void attach_gemm_workspace(GemmProblem& p, hipStream_t stream);

}  // namespace fp8bs
