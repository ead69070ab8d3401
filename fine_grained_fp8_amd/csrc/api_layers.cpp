// C ABI of the layer operators around the FP8 products: layer norm, the
// few-token expert layer, adapters beside a projection.  Host-side
// validation, workspace layout, dispatch.  Contracts: include/fp8bs.h.
#include "fp8bs.h"

#include <hip/hip_runtime.h>

#include "host_checks.hpp"
#include "layers.hpp"

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxLd = int64_t{1} << 28;
constexpr int64_t kMaxBlocks = int64_t{1} << 23;   // a launch holds less than 2^32 threads, here 512 a workgroup

// consecutive 256-byte aligned parts of a caller's workspace
struct Carver {
  int64_t used = 0;
  int64_t take(int64_t bytes) {
    const int64_t at = used;
    used += (bytes + 255) / 256 * 256;
    return at;
  }
};
template <typename T>
T* at(void* ws, int64_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

struct MoeLayout {
  int64_t logits, xq, xs, expert, gate, h, hq, hs, counts, lists, plan, parts, bytes;
};
MoeLayout moe_layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t local, int64_t k) {
  Carver c;
  MoeLayout l{};
  l.logits = c.take(fp8bs::dot_splits(H, fp8bs::kMoeSplits) * T * E * 4);
  l.xq = c.take(T * H);
  l.xs = c.take(T * (H / 128) * 4);
  l.expert = c.take(T * k * 4);
  l.gate = c.take(T * k * 4);
  l.h = c.take(T * k * I * 4);
  l.hq = c.take(T * k * I);
  l.hs = c.take(T * k * (I / 128) * 4);
  l.counts = c.take(local * 4);
  l.lists = c.take(local * fp8bs::kMoeMaxTokens * 4);
  l.parts = c.take(fp8bs::moe_cuts(H) > 1 ? H / 16 * fp8bs::moe_cuts(H) * T * 64 : 0);
  l.plan = c.take((2 + 2 * (T * k + T * k / 16) + 2 * T * k) * 4);
  l.bytes = c.used;
  return l;
}

struct AdapterLayout {
  int64_t xq, xs, zp, z, bytes;
};
AdapterLayout adapter_layout(int64_t T, int64_t K, int64_t r) {
  Carver c;
  AdapterLayout l{};
  if (T == 0) return l;
  l.xq = c.take((T + 15) / 16 * 16 * K);
  l.xs = c.take((K / 128) * ((T + 3) / 4 * 4) * 4);
  l.zp = c.take(fp8bs::adapter_splits(T, K) * T * r * 4);
  l.z = c.take(T * r * 4);
  l.bytes = c.used;
  return l;
}

fp8_status moe_shape(int64_t T, int64_t H, int64_t I, int64_t E, int64_t first, int64_t local, int64_t k) {
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || local <= 0 || first < 0 || first + local > E || k < 1 || k > E)
    return FP8_ERR_SHAPE;
  if (H % 128 != 0 || I % 128 != 0) return FP8_ERR_SHAPE;
  if (T > fp8bs::kMoeMaxTokens || k > fp8bs::kMoeMaxTopK || E > fp8bs::kMoeMaxExperts || H > (1 << 20) ||
      I > (1 << 20))
    return FP8_ERR_UNSUPPORTED;
  // the up product's launch: 512 threads for 16 channels of an expert, and for the routing
  if (local * (I / 16) + 1 >= kMaxBlocks) return FP8_ERR_UNSUPPORTED;
  return FP8_OK;
}

fp8_status adapter_shape(int64_t T, int64_t N, int64_t K, int64_t r, int64_t n) {
  if (T < 0 || N <= 0 || K <= 0 || r <= 0 || n <= 0) return FP8_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0 || r % 8 != 0) return FP8_ERR_SHAPE;
  if (r > fp8bs::kAdapterMaxRank || N > (1 << 23) || K > (1 << 22) || n > (1 << 20) || T > (int64_t{1} << 24))
    return FP8_ERR_UNSUPPORTED;
  // the GEMM's limits: 32-bit scale-table offsets and tile numbers
  if ((K / 128) * ((T + 3) / 4 * 4) * 4 >= (int64_t{1} << 31)) return FP8_ERR_UNSUPPORTED;
  if (((T + 127) / 128) * ((N + 255) / 256) >= (int64_t{1} << 31)) return FP8_ERR_UNSUPPORTED;
  // the prompts' shrink: 512 threads for 16 tokens and a share of K
  if ((T + 15) / 16 * fp8bs::adapter_splits(T, K) >= kMaxBlocks) return FP8_ERR_UNSUPPORTED;
  return FP8_OK;
}

}  // namespace

extern "C" {

fp8_status fp8_layer_norm(const void* x, int64_t rows, int64_t cols, int64_t ldx, fp8_out_dtype x_dtype,
                          const void* weight, const void* bias, fp8_out_dtype w_dtype, float eps, void* y,
                          int64_t ldy, float* mean, float* rstd, uint8_t* q, int64_t ldq, float* scales,
                          int64_t ld_s, void* stream) {
  if ((x_dtype != FP8_OUT_BF16 && x_dtype != FP8_OUT_FP32) || (w_dtype != FP8_OUT_BF16 && w_dtype != FP8_OUT_FP32))
    return FP8_ERR_UNSUPPORTED;
  if (rows < 0 || cols < 0 || (q && cols % 128 != 0)) return FP8_ERR_SHAPE;
  if (!(eps >= 0.0f)) return FP8_ERR_SHAPE;
  if (cols > fp8bs::kNormMaxCols || rows > kMaxRows) return FP8_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return FP8_OK;
  if (!x || (!y && !q) || ((q == nullptr) != (scales == nullptr))) return FP8_ERR_NULL;
  if (ldx < cols || (y && ldy < cols) || (q && (ldq < cols || ld_s < rows))) return FP8_ERR_LD;
  if (ldx > kMaxLd || (y && ldy > kMaxLd) || (q && (ldq > kMaxLd || ld_s > int64_t{1} << 40))) return FP8_ERR_UNSUPPORTED;
  const int64_t e = x_dtype == FP8_OUT_FP32 ? 4 : 2, we = w_dtype == FP8_OUT_FP32 ? 4 : 2;
  const uintptr_t em = static_cast<uintptr_t>(e - 1), wm = static_cast<uintptr_t>(we - 1);
  if ((reinterpret_cast<uintptr_t>(x) & em) || (reinterpret_cast<uintptr_t>(y) & em) ||
      (reinterpret_cast<uintptr_t>(weight) & wm) || (reinterpret_cast<uintptr_t>(bias) & wm) || !aligned4(mean) ||
      !aligned4(rstd) || !aligned4(scales))
    return FP8_ERR_ALIGN;
  // with codes every row is moved in 16-byte pieces
  if (q && (!aligned16(x) || (ldx * e) % 16 != 0 || !aligned16(q) || ldq % 16 != 0 || !aligned16(weight) ||
            !aligned16(bias) || (y && (!aligned16(y) || (ldy * e) % 16 != 0))))
    return FP8_ERR_ALIGN;
  const Range in[3] = {span(x, rows, cols * e, ldx * e), span(weight, weight ? 1 : 0, cols * we, 0),
                       span(bias, bias ? 1 : 0, cols * we, 0)};
  const Range out[5] = {span(y, y ? rows : 0, cols * e, ldy * e), span(mean, mean ? 1 : 0, rows * 4, 0),
                        span(rstd, rstd ? 1 : 0, rows * 4, 0), span(q, q ? rows : 0, cols, ldq),
                        span(scales, scales ? cols / 128 : 0, rows * 4, ld_s * 4)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 3; ++j)
      if (overlap(out[i], in[j])) return FP8_ERR_ALIAS;
    for (int j = i + 1; j < 5; ++j)
      if (overlap(out[i], out[j])) return FP8_ERR_ALIAS;
  }
  const fp8_status dev = check_device();
  if (dev != FP8_OK) return dev;
  fp8bs::LayerNormProblem p{};
  p.x = x; p.rows = rows; p.cols = cols; p.ldx = ldx;
  p.w = weight; p.b = bias;
  p.x_fp32 = e == 4; p.w_fp32 = we == 4;
  p.eps = eps;
  p.y = y; p.ldy = ldy; p.mean = mean; p.rstd = rstd;
  p.q = q; p.ldq = ldq; p.s = scales; p.ld_s = ld_s;
  return launched(fp8bs::launch_layer_norm(p, reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8_layer_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols > fp8bs::kNormMaxCols) return -1;
  return fp8bs::layer_norm_grad_parts(rows, cols) * 2 * cols * 4;
}

fp8_status fp8_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, int64_t rows,
                                   int64_t cols, fp8_out_dtype x_dtype, const float* mean, const float* rstd,
                                   const void* weight, fp8_out_dtype w_dtype, void* dx, int64_t lddx,
                                   float* dweight, float* dbias, void* workspace, int64_t workspace_bytes,
                                   void* stream) {
  if ((x_dtype != FP8_OUT_BF16 && x_dtype != FP8_OUT_FP32) || (w_dtype != FP8_OUT_BF16 && w_dtype != FP8_OUT_FP32))
    return FP8_ERR_UNSUPPORTED;
  if (rows < 0 || cols < 0) return FP8_ERR_SHAPE;
  if (cols > fp8bs::kNormMaxCols || rows > kMaxRows) return FP8_ERR_UNSUPPORTED;
  if (cols == 0 || (rows == 0 && !dweight && !dbias)) return FP8_OK;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx || !workspace)) return FP8_ERR_NULL;
  if (rows > 0 && (lddy < cols || ldx < cols || lddx < cols)) return FP8_ERR_LD;
  if (lddy > kMaxLd || ldx > kMaxLd || lddx > kMaxLd) return FP8_ERR_UNSUPPORTED;
  const int64_t need = fp8_layer_norm_backward_workspace(rows, cols);
  if (workspace_bytes < need) return FP8_ERR_SHAPE;
  const int64_t e = x_dtype == FP8_OUT_FP32 ? 4 : 2, we = w_dtype == FP8_OUT_FP32 ? 4 : 2;
  const uintptr_t em = static_cast<uintptr_t>(e - 1), wm = static_cast<uintptr_t>(we - 1);
  if ((reinterpret_cast<uintptr_t>(x) & em) || (reinterpret_cast<uintptr_t>(dy) & em) ||
      (reinterpret_cast<uintptr_t>(dx) & em) || (reinterpret_cast<uintptr_t>(weight) & wm) || !aligned4(mean) ||
      !aligned4(rstd) || !aligned4(dweight) || !aligned4(dbias) || !aligned16(workspace))
    return FP8_ERR_ALIGN;
  const Range in[5] = {span(x, rows, cols * e, ldx * e), span(dy, rows, cols * e, lddy * e),
                       span(mean, 1, rows * 4, 0), span(rstd, 1, rows * 4, 0),
                       span(weight, weight ? 1 : 0, cols * we, 0)};
  const Range out[4] = {span(dx, rows, cols * e, lddx * e), span(dweight, dweight ? 1 : 0, cols * 4, 0),
                        span(dbias, dbias ? 1 : 0, cols * 4, 0), span(workspace, 1, need, 0)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 5; ++j)
      if (overlap(out[i], in[j])) return FP8_ERR_ALIAS;
    for (int j = i + 1; j < 4; ++j)
      if (overlap(out[i], out[j])) return FP8_ERR_ALIAS;
  }
  const fp8_status dev = check_device();
  if (dev != FP8_OK) return dev;
  fp8bs::LayerNormGradProblem p{};
  p.dy = dy; p.x = x; p.rows = rows; p.cols = cols; p.lddy = lddy; p.ldx = ldx;
  p.mean = mean; p.rstd = rstd; p.w = weight;
  p.x_fp32 = e == 4; p.w_fp32 = we == 4;
  p.dx = dx; p.lddx = lddx; p.dw = dweight; p.db = dbias;
  p.partial = static_cast<float*>(workspace);
  return launched(fp8bs::launch_layer_norm_backward(p, reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8_moe_few_tokens_workspace(int64_t T, int64_t H, int64_t I, int32_t E, int32_t local, int32_t top_k) {
  if (moe_shape(T, H, I, E, 0, local, top_k) != FP8_OK) return -1;
  return moe_layout(T, H, I, E, local, top_k).bytes;
}

fp8_status fp8_moe_few_tokens(int64_t T, int64_t H, int64_t I, int32_t E, int32_t first, int32_t local,
                              int32_t top_k, const void* x, int64_t ldx, const void* router, int64_t ld_r,
                              const float* bias, fp8_moe_gate gate, int normalize, float gate_scale,
                              const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2, void* y,
                              fp8_out_dtype y_dtype, int64_t ldy, int32_t* ids, float* gates, void* workspace,
                              int64_t workspace_bytes, void* stream) {
  if ((gate != FP8_MOE_SOFTMAX && gate != FP8_MOE_SIGMOID) || (y_dtype != FP8_OUT_BF16 && y_dtype != FP8_OUT_FP32))
    return FP8_ERR_UNSUPPORTED;
  if (bias && gate != FP8_MOE_SIGMOID) return FP8_ERR_UNSUPPORTED;
  const fp8_status st = moe_shape(T, H, I, E, first, local, top_k);
  if (st != FP8_OK) return st;
  if (T == 0) return FP8_OK;
  if (!x || !router || !w13 || !s13 || !w2 || !s2 || !y || !workspace) return FP8_ERR_NULL;
  if (ldx < H || ld_r < H || ldy < H) return FP8_ERR_LD;
  if (ldx > kMaxLd || ld_r > kMaxLd || ldy > kMaxLd) return FP8_ERR_UNSUPPORTED;
  const MoeLayout l = moe_layout(T, H, I, E, local, top_k);
  if (workspace_bytes < l.bytes) return FP8_ERR_SHAPE;
  const int64_t e = y_dtype == FP8_OUT_FP32 ? 4 : 2;
  if (!aligned16(x) || ldx % 8 != 0 || !aligned16(router) || ld_r % 8 != 0 || !aligned16(w13) || !aligned16(w2) ||
      !aligned16(y) || (ldy * e) % 16 != 0 || !aligned4(bias) || !aligned4(s13) || !aligned4(s2) || !aligned4(ids) ||
      !aligned4(gates) || !aligned16(workspace))
    return FP8_ERR_ALIGN;
  const int64_t hi = H * I * local, bi = (H / 128) * (I / 128) * local;
  const Range in[7] = {span(x, T, H * 2, ldx * 2), span(router, E, H * 2, ld_r * 2), span(bias, bias ? 1 : 0, E * 4, 0),
                       span(w13, 1, 2 * hi, 0), span(s13, 1, 2 * bi * 4, 0), span(w2, 1, hi, 0), span(s2, 1, bi * 4, 0)};
  const Range out[4] = {span(y, T, H * e, ldy * e), span(ids, ids ? 1 : 0, T * top_k * 4, 0),
                        span(gates, gates ? 1 : 0, T * top_k * 4, 0), span(workspace, 1, l.bytes, 0)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 7; ++j)
      if (overlap(out[i], in[j])) return FP8_ERR_ALIAS;
    for (int j = i + 1; j < 4; ++j)
      if (overlap(out[i], out[j])) return FP8_ERR_ALIAS;
  }
  const fp8_status dev = check_device();
  if (dev != FP8_OK) return dev;
  fp8bs::MoeProblem p{};
  p.T = (int)T; p.H = (int)H; p.I = (int)I; p.E = E; p.first = first; p.local = local; p.top_k = top_k;
  p.x = static_cast<const uint16_t*>(x); p.ldx = ldx;
  p.router = static_cast<const uint16_t*>(router); p.ld_r = ld_r;
  p.bias = bias; p.sigmoid = gate == FP8_MOE_SIGMOID; p.normalize = normalize != 0; p.gate_scale = gate_scale;
  p.w13 = w13; p.s13 = s13; p.w2 = w2; p.s2 = s2;
  p.y = y; p.ldy = ldy; p.y_fp32 = e == 4;
  p.logits = at<float>(workspace, l.logits);
  p.splits = fp8bs::dot_splits(H, fp8bs::kMoeSplits);
  p.xq = at<uint8_t>(workspace, l.xq);
  p.xs = at<float>(workspace, l.xs);
  p.slot_expert = ids ? ids : at<int32_t>(workspace, l.expert);
  p.slot_gate = gates ? gates : at<float>(workspace, l.gate);
  p.h = at<float>(workspace, l.h);
  p.hq = at<uint8_t>(workspace, l.hq);
  p.hs = at<float>(workspace, l.hs);
  p.counts = at<int32_t>(workspace, l.counts);
  p.lists = at<int32_t>(workspace, l.lists);
  p.plan = at<int32_t>(workspace, l.plan);
  p.parts = at<float>(workspace, l.parts);
  return launched(fp8bs::launch_moe_few_tokens(p, reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8_adapter_linear_workspace(int64_t T, int64_t N, int64_t K, int32_t rank, int32_t adapters) {
  if (adapter_shape(T, N, K, rank, adapters) != FP8_OK) return -1;
  return adapter_layout(T, K, rank).bytes;
}

fp8_status fp8_adapter_linear(int64_t T, int64_t N, int64_t K, int32_t rank, int32_t adapters, const void* x,
                              int64_t ldx, const uint8_t* W, const float* sW, int64_t ld_sw, const void* A,
                              const void* B, const int32_t* ids, const float* scales, void* C,
                              fp8_out_dtype c_dtype, int64_t ldc, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  if (c_dtype != FP8_OUT_BF16 && c_dtype != FP8_OUT_FP32) return FP8_ERR_UNSUPPORTED;
  const fp8_status st = adapter_shape(T, N, K, rank, adapters);
  if (st != FP8_OK) return st;
  if (T == 0) return FP8_OK;
  if (!x || !W || !sW || !A || !B || !ids || !C || !workspace) return FP8_ERR_NULL;
  if (ldx < K || ld_sw < K / 128 || ldc < N) return FP8_ERR_LD;
  if (ldx > kMaxLd || ldc > kMaxLd || (N / 128) * ld_sw >= (int64_t{1} << 29)) return FP8_ERR_UNSUPPORTED;
  const AdapterLayout l = adapter_layout(T, K, rank);
  if (workspace_bytes < l.bytes) return FP8_ERR_SHAPE;
  const int64_t e = c_dtype == FP8_OUT_FP32 ? 4 : 2;
  if (!aligned16(x) || ldx % 8 != 0 || !aligned16(W) || !aligned16(A) || !aligned16(B) || !aligned16(C) ||
      (ldc * e) % 16 != 0 || !aligned4(sW) || !aligned4(ids) || !aligned4(scales) || !aligned16(workspace))
    return FP8_ERR_ALIGN;
  const int64_t n = adapters, r = rank;
  const Range in[7] = {span(x, T, K * 2, ldx * 2), span(W, 1, N * K, 0), span(sW, N / 128, (K / 128) * 4, ld_sw * 4),
                       span(A, 1, n * r * K * 2, 0), span(B, 1, n * r * N * 2, 0), span(ids, 1, T * 4, 0),
                       span(scales, scales ? 1 : 0, n * 4, 0)};
  const Range out[2] = {span(C, T, N * e, ldc * e), span(workspace, 1, l.bytes, 0)};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 7; ++j)
      if (overlap(out[i], in[j])) return FP8_ERR_ALIAS;
  if (overlap(out[0], out[1])) return FP8_ERR_ALIAS;
  const fp8_status dev = check_device();
  if (dev != FP8_OK) return dev;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  fp8bs::AdapterProblem p{};
  p.T = T; p.N = N; p.K = K; p.r = rank; p.n = adapters;
  p.x = static_cast<const uint16_t*>(x); p.ldx = ldx;
  p.W = W; p.sW = sW; p.ld_sw = ld_sw;
  p.A = static_cast<const uint16_t*>(A);
  p.B = static_cast<const uint16_t*>(B);
  p.ids = ids; p.scales = scales;
  p.C = C; p.ldc = ldc; p.out_fp32 = e == 4;
  p.xq = at<uint8_t>(workspace, l.xq);
  p.xs = at<float>(workspace, l.xs);
  p.splits = fp8bs::adapter_splits(T, K);
  p.zp = at<float>(workspace, l.zp);
  p.z = at<uint16_t>(workspace, l.z);
  if (T <= fp8bs::kAdapterFewTokens) return launched(fp8bs::launch_adapter_few(p, s));
  const int64_t ld_s = (T + 3) / 4 * 4;
  const hipError_t err = fp8bs::launch_adapter_prompt(p, ld_s, s);
  if (err != hipSuccess) return launched(err);
  fp8bs::GemmProblem g{};
  g.layout = fp8bs::kFprop;
  g.M = T; g.N = N; g.K = K;
  g.A = p.xq; g.lda = K; g.sA = p.xs; g.ld_sa = ld_s;
  g.B = W; g.ldb = K; g.sB = sW; g.ld_sb = ld_sw;
  g.C = C; g.ldc = ldc; g.out_fp32 = p.out_fp32;
  g.b_tiled = 1;
  g.adapters = fp8bs::AdapterEpilogue{ids, p.z, p.B, p.r, p.n};
  fp8bs::attach_gemm_workspace(g, s);
  return launched(fp8bs::launch_gemm(g, s));
}

}  // extern "C"
