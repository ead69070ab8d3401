// Host-side launchers of the operators between a layer's FP8 products (the
// gated feed-forward product for a few tokens and its backward pass, the head
// norms with the position rotation), internal to libfp8bs.so.  Arguments are
// already validated by api_blocks.cpp; each launcher only sizes its grids and
// enqueues on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"

namespace fp8bs {

// ---- the gated product for few tokens or few tiles ----
// Workgroups that share the K blocks of a tile of channels, for FP32 results and codes
// or for BF16 results; 0: the block GEMM is faster
int gated_few_cuts(int64_t M, int64_t N, int64_t K, bool fp32);
int64_t gated_few_parts(int64_t M, int64_t N, int64_t K, bool fp32, bool codes);
struct GatedFewProblem {
  int M;
  int64_t N, K;
  const uint8_t* A;       // codes [M][lda]
  int64_t lda;
  const float* sA;        // [K / 128][ld_sa]
  int64_t ld_sa;
  const uint8_t* W;       // operand-tiled codes [2 N][K]: gate rows, then up rows
  const float* sW;        // [2 N / 128][ld_sw]
  int64_t ld_sw;
  void* C;                // [M][ldc], or null (then gated.q is set)
  int64_t ldc;
  int out_fp32;
  GatedEpilogue gated;
  // workspace
  int cuts;               // gated_few_cuts of the result
  float* parts;           // [cuts][M][2 N] if cuts > 1; otherwise [M][N], h of a call for codes
};
hipError_t launch_gated_few(const GatedFewProblem& p, hipStream_t stream);

// ---- its backward pass ----
struct GatedGradProblem {
  int64_t T, I;
  int gelu;
  const uint16_t* dh;       // BF16 [T][ld_dh]
  int64_t ld_dh;
  const uint16_t* gate_up;  // BF16 [T][ld_gu]: gate, then up
  int64_t ld_gu;
  uint16_t* d;              // optional: BF16 [T][ld_d], d gate and then d up
  int64_t ld_d;
  uint8_t* q;               // optional: codes [T][ldq], scales [2 I / 128][ld_s]
  int64_t ldq;
  float* s;
  int64_t ld_s;
  uint8_t* qt;              // optional: transposed codes [2 I][ldqt], scales [ceil(T / 128)][ld_st]
  int64_t ldqt;
  float* st;
  int64_t ld_st;
  uint8_t* ht;              // optional: operand-tiled transposed codes of h [I][round_up(T, 128)], scales [..][ld_hst]
  float* hst;
  int64_t ld_hst;
};
hipError_t launch_gated_backward(const GatedGradProblem& p, hipStream_t stream);

// ---- norms of heads with the position rotation ----
constexpr int kHeadMaxDim = 1024, kHeadMaxAxes = 4;
struct HeadSet {
  const void* x;             // [T][heads][dim] at the strides
  int64_t heads, ld_token, ld_head;
  const void* w;             // [dim] or null (ones)
  void* y;
  int64_t ldy_token, ldy_head;
  // backward: dy at (lddy_token, lddy_head), dx in y; dw FP32 [dim] or null
  const void* dy;
  int64_t lddy_token, lddy_head;
  float* dw;
};
struct HeadProblem {
  int64_t T;
  int dim, rot, axes;
  int section_end[kHeadMaxAxes];   // pairs [.., end) take the positions of that axis
  int x_fp32, w_fp32, norm, adjacent, pos64;
  float eps;
  const void* positions;           // int32 or int64 [T][axes]
  const double* freq;              // [rot / 2] or null (rot == 0)
  HeadSet set[2];                  // queries, keys (heads == 0: none)
  float* partial;                  // backward: [head_grad_parts][dim]
};
enum HeadNorm { kHeadNone = 0, kHeadRms = 1, kHeadLayer = 2 };
hipError_t launch_head_norm_rotary(const HeadProblem& p, hipStream_t stream);
// workgroups of the backward pass at most, each with its share of a weight's gradient
int64_t head_grad_parts(int64_t T, int64_t q_heads, int64_t k_heads, int64_t dim);
hipError_t launch_head_norm_rotary_backward(const HeadProblem& p, hipStream_t stream);

// The split-K workspace of the persistent GEMM on `stream` (api.cpp)
void attach_gemm_workspace(GemmProblem& p, hipStream_t stream);

}  // namespace fp8bs
