// C ABI of the operators between a layer's FP8 products: the gated
// feed-forward product and its backward pass, the column quantizer for any
// number of rows, the head norms with the position rotation.  Host-side
// validation, workspace sizes, dispatch.  Contracts: include/fp8bs.h.
#include "fp8bs.h"

#include <hip/hip_runtime.h>

#include "blocks.hpp"
#include "host_checks.hpp"

namespace {

constexpr int64_t kMaxLd = int64_t{1} << 28;
constexpr int64_t kMaxBlocks = int64_t{1} << 22;   // a launch holds less than 2^32 threads, here up to 1024 a workgroup
constexpr int64_t kMaxTokens = int64_t{1} << 31;

// Rows at a stride that would end past 2^45 elements: more than any memory, and byte
// offsets stay far from 2^63.
bool too_far(int64_t rows, int64_t ld) { return ld > (int64_t{1} << 45) / (rows > 1 ? rows : 1); }

bool aligned_to(const void* p, int64_t bytes) { return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) == 0; }
int64_t up128(int64_t n) { return (n + 127) / 128 * 128; }

// outputs against inputs and each other
template <int kIn, int kOut>
bool aliased(const Range (&in)[kIn], const Range (&out)[kOut]) {
  for (int i = 0; i < kOut; ++i) {
    for (int j = 0; j < kIn; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = i + 1; j < kOut; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

fp8_status gated_shape(int64_t M, int64_t I, int64_t K) {
  if (M < 0 || I <= 0 || K <= 0 || I % 128 != 0 || K % 128 != 0) return FP8_ERR_SHAPE;
  // 32-bit offsets from a tile's rows of W1 to the end of its rows of W3
  if (I > (int64_t{1} << 24) || K > (int64_t{1} << 23) || (I + 128) * K >= (int64_t{1} << 31)) return FP8_ERR_UNSUPPORTED;
  // tile numbers are 32-bit
  if (M > kMaxTokens || (M + 127) / 128 * (I / 128) >= (int64_t{1} << 31)) return FP8_ERR_UNSUPPORTED;
  return FP8_OK;
}

// ---- heads ----

// Element (t, h, e) at t lt + h lh + e: token by token or head by head, nothing twice.
bool heads_nested(int64_t T, int64_t heads, int64_t dim, int64_t lt, int64_t lh) {
  if (lt < 0 || lh < 0) return false;
  const bool by_token = (heads == 1 || lh >= dim) && (T == 1 || lt >= (heads - 1) * lh + dim);
  const bool by_head = (T == 1 || lt >= dim) && (heads == 1 || lh >= (T - 1) * lt + dim);
  return by_token || by_head;
}
Range heads_span(const void* p, int64_t T, int64_t heads, int64_t dim, int64_t lt, int64_t lh, int64_t e) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  if (p == nullptr || T <= 0 || heads <= 0) return {b, b};
  return {b, b + static_cast<uintptr_t>(((T - 1) * lt + (heads - 1) * lh + dim) * e)};
}

// A set of heads in memory; rows: bytes that a token takes where tokens follow
// each other at `step` bytes (0: not token by token).
struct Placed {
  Range all;
  int64_t rows, step;
};
Placed placed(const void* p, int64_t T, int64_t heads, int64_t dim, int64_t lt, int64_t lh, int64_t e) {
  const int64_t row = (heads - 1) * lh + dim;
  return {heads_span(p, T, heads, dim, lt, lh, e), row * e, p != nullptr && heads > 0 && lt >= row ? lt * e : 0};
}
// Two sets that share memory.  Sets that lie side by side within rows of the same
// step do not, though their ranges overlap.
bool share(const Placed& a, const Placed& b) {
  if (!overlap(a.all, b.all)) return false;
  if (a.step == 0 || a.step != b.step) return true;
  const int64_t apart = static_cast<int64_t>((b.all.lo > a.all.lo ? b.all.lo - a.all.lo : a.all.lo - b.all.lo) % static_cast<uintptr_t>(a.step));
  const Placed& low = b.all.lo > a.all.lo ? a : b;
  const Placed& high = b.all.lo > a.all.lo ? b : a;
  return apart < low.rows || apart + high.rows > a.step;
}

struct HeadArgs {
  int64_t T, dim;
  int x_dtype, w_dtype, norm;   // as given, perhaps no value of their enums
  float eps;
  int64_t rot;
  const void* positions;
  int32_t position_bytes, axes;
  const int64_t* sections;
  const double* freq;
  int32_t adjacent;
};

bool head_sizes(int64_t T, int64_t heads_q, int64_t heads_k, int64_t dim) {
  return T >= 0 && heads_q >= 0 && heads_k >= 0 && heads_q + heads_k > 0 && dim >= 2 && dim % 2 == 0;
}
bool head_limits(int64_t T, int64_t heads_q, int64_t heads_k, int64_t dim) {
  constexpr int64_t kMost = int64_t{1} << 20;
  // a wave a token at most T >= 4096, four a workgroup of 256 threads
  return T <= (int64_t{1} << 25) && heads_q <= kMost && heads_k <= kMost && dim <= fp8bs::kHeadMaxDim;
}

// everything but the sets' own pointers; fills p
fp8_status head_common(const HeadArgs& a, int64_t heads_q, int64_t heads_k, fp8bs::HeadProblem& p) {
  if ((a.x_dtype != FP8_OUT_BF16 && a.x_dtype != FP8_OUT_FP32) || (a.w_dtype != FP8_OUT_BF16 && a.w_dtype != FP8_OUT_FP32) ||
      (a.norm != FP8_HEAD_NONE && a.norm != FP8_HEAD_RMS && a.norm != FP8_HEAD_LAYER))
    return FP8_ERR_UNSUPPORTED;
  if (!head_sizes(a.T, heads_q, heads_k, a.dim) || a.rot < 0 || a.rot > a.dim || a.rot % 2 != 0 || !(a.eps >= 0.0f)) return FP8_ERR_SHAPE;
  if (!head_limits(a.T, heads_q, heads_k, a.dim)) return FP8_ERR_UNSUPPORTED;
  p.axes = 1;
  for (int i = 0; i < fp8bs::kHeadMaxAxes; ++i) p.section_end[i] = static_cast<int>(a.rot / 2);
  if (a.rot > 0) {
    if (a.position_bytes != 4 && a.position_bytes != 8) return FP8_ERR_UNSUPPORTED;
    if (a.axes < 1 || a.axes > fp8bs::kHeadMaxAxes) return FP8_ERR_UNSUPPORTED;
    if (a.axes > 1 && !a.sections) return FP8_ERR_NULL;
    if (a.sections) {
      int64_t sum = 0;
      for (int i = 0; i < a.axes; ++i) {
        if (a.sections[i] < 0 || a.sections[i] > a.rot / 2) return FP8_ERR_SHAPE;
        sum += a.sections[i];
        p.section_end[i] = static_cast<int>(sum);
      }
      if (sum != a.rot / 2) return FP8_ERR_SHAPE;
    }
    p.axes = a.axes;
    if (a.T > 0 && (!a.positions || !a.freq)) return FP8_ERR_NULL;
    if (!aligned_to(a.positions, a.position_bytes) || !aligned_to(a.freq, 8)) return FP8_ERR_ALIGN;
  }
  p.T = a.T;
  p.dim = static_cast<int>(a.dim);
  p.rot = static_cast<int>(a.rot);
  p.x_fp32 = a.x_dtype == FP8_OUT_FP32;
  p.w_fp32 = a.w_dtype == FP8_OUT_FP32;
  p.norm = a.norm;
  p.adjacent = a.adjacent != 0;
  p.pos64 = a.position_bytes == 8;
  p.eps = a.eps;
  p.positions = a.positions;
  p.freq = a.freq;
  return FP8_OK;
}

}  // namespace

extern "C" {

int64_t fp8_block_gemm_gated_workspace(int64_t M, int64_t I, int64_t K, fp8_out_dtype h_dtype, int32_t codes) {
  if (gated_shape(M, I, K) != FP8_OK || (h_dtype != FP8_OUT_BF16 && h_dtype != FP8_OUT_FP32)) return -1;
  return fp8bs::gated_few_parts(M, I, K, codes != 0 || h_dtype == FP8_OUT_FP32, codes != 0) * M * I * 4;
}

fp8_status fp8_block_gemm_gated(int64_t M, int64_t I, int64_t K, const uint8_t* A, int64_t lda, const float* sA,
                                int64_t ld_sa, const uint8_t* W13, const float* s13, int64_t ld_s13,
                                fp8_activation act, void* h, fp8_out_dtype h_dtype, int64_t ldh, void* gate_up,
                                int64_t ld_gu, uint8_t* q, int64_t ldq, float* scales, int64_t ld_s,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  if ((act != FP8_ACT_SILU && act != FP8_ACT_GELU) || (h_dtype != FP8_OUT_BF16 && h_dtype != FP8_OUT_FP32))
    return FP8_ERR_UNSUPPORTED;
  const fp8_status st = gated_shape(M, I, K);
  if (st != FP8_OK) return st;
  if (M == 0) return FP8_OK;
  if (h && q) return FP8_ERR_UNSUPPORTED;
  if (!A || !sA || !W13 || !s13 || (!h && !q) || ((q == nullptr) != (scales == nullptr))) return FP8_ERR_NULL;
  if (lda < K || ld_sa < M || ld_s13 < K / 128 || (h && ldh < I) || (gate_up && ld_gu < 2 * I) ||
      (q && (ldq < I || ld_s < M)))
    return FP8_ERR_LD;
  if (lda > (int64_t{1} << 23) || ld_s13 > kMaxLd || ld_sa > kMaxLd || (h && ldh > kMaxLd) || (gate_up && ld_gu > kMaxLd) ||
      (q && (ldq > kMaxLd || ld_s > int64_t{1} << 40)))
    return FP8_ERR_UNSUPPORTED;
  // the scale tables are read through 32-bit byte offsets
  if ((K / 128) * ld_sa * 4 >= (int64_t{1} << 31) || (2 * I / 128) * ld_s13 * 4 >= (int64_t{1} << 31)) return FP8_ERR_UNSUPPORTED;
  const int64_t need = fp8_block_gemm_gated_workspace(M, I, K, h_dtype, q != nullptr);
  if (need > 0 && !workspace) return FP8_ERR_NULL;
  if (workspace_bytes < need) return FP8_ERR_SHAPE;
  const int64_t e = h_dtype == FP8_OUT_FP32 ? 4 : 2;
  if (!aligned16(A) || lda % 16 != 0 || !aligned16(W13) || !aligned4(sA) || !aligned4(s13) || !aligned16(h) ||
      (h && (ldh * e) % 16 != 0) || !aligned16(gate_up) || (gate_up && ld_gu % 8 != 0) || !aligned16(q) ||
      (q && ldq % 16 != 0) || !aligned4(scales) || (need > 0 && !aligned16(workspace)))
    return FP8_ERR_ALIGN;
  const Range in[4] = {span(A, M, K, lda), span(sA, K / 128, M * 4, ld_sa * 4), span(W13, 1, 2 * I * K, 0),
                       span(s13, 2 * I / 128, (K / 128) * 4, ld_s13 * 4)};
  const Range out[5] = {span(h, h ? M : 0, I * e, ldh * e), span(gate_up, gate_up ? M : 0, 4 * I, ld_gu * 2),
                        span(q, q ? M : 0, I, ldq), span(scales, scales ? I / 128 : 0, M * 4, ld_s * 4),
                        span(workspace, need > 0 ? 1 : 0, need, 0)};
  if (aliased(in, out)) return FP8_ERR_ALIAS;
  const fp8_status dev = check_device();
  if (dev != FP8_OK) return dev;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  fp8bs::GatedEpilogue ge{};
  ge.on = 1;
  ge.gelu = act == FP8_ACT_GELU;
  ge.gate_up = static_cast<uint16_t*>(gate_up);
  ge.ld_gu = ld_gu;
  ge.q = q; ge.ldq = ldq; ge.s = scales; ge.ld_s = ld_s;
  if (const int cuts = fp8bs::gated_few_cuts(M, I, K, q != nullptr || e == 4); cuts > 0) {
    fp8bs::GatedFewProblem p{};
    p.M = static_cast<int>(M); p.N = I; p.K = K;
    p.A = A; p.lda = lda; p.sA = sA; p.ld_sa = ld_sa;
    p.W = W13; p.sW = s13; p.ld_sw = ld_s13;
    p.C = h; p.ldc = ldh; p.out_fp32 = e == 4;
    p.gated = ge;
    p.cuts = cuts;
    p.parts = static_cast<float*>(workspace);
    return launched(fp8bs::launch_gated_few(p, s));
  }
  fp8bs::GemmProblem g{};
  g.layout = fp8bs::kFprop;
  g.M = M; g.N = I; g.K = K;
  g.A = A; g.lda = lda; g.sA = sA; g.ld_sa = ld_sa;
  g.B = W13; g.ldb = K; g.sB = s13; g.ld_sb = ld_s13;
  g.C = h; g.ldc = ldh; g.out_fp32 = e == 4;
  g.b_tiled = 1;
  g.gated = ge;
  // The split workspace belongs to the stream.  A captured launch does without:
  // two graphs captured on one stream may be replayed on two.
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(s, &cap) != hipSuccess) (void)hipGetLastError();
  else if (cap == hipStreamCaptureStatusNone) fp8bs::attach_gemm_workspace(g, s);
  return launched(fp8bs::launch_gemm(g, s));
}

fp8_status fp8_gated_backward(int64_t T, int64_t I, const void* dh, int64_t ld_dh, const void* gate_up,
                              int64_t ld_gu, fp8_activation act, void* d, int64_t ld_d, uint8_t* q, int64_t ldq,
                              float* scales, int64_t ld_s, uint8_t* qt, int64_t ldqt, float* scales_t, int64_t ld_st,
                              uint8_t* ht, float* scales_ht, int64_t ld_sht, void* stream) {
  if (act != FP8_ACT_SILU && act != FP8_ACT_GELU) return FP8_ERR_UNSUPPORTED;
  if (T < 0 || I < 0 || I % 128 != 0) return FP8_ERR_SHAPE;
  if (T > kMaxTokens || I > (int64_t{1} << 27) || up128(T) / 128 * (I / 128) >= kMaxBlocks) return FP8_ERR_UNSUPPORTED;
  if (T == 0 || I == 0) return FP8_OK;
  if (!dh || !gate_up || (!d && !q && !qt && !ht) || ((q == nullptr) != (scales == nullptr)) ||
      ((qt == nullptr) != (scales_t == nullptr)) || ((ht == nullptr) != (scales_ht == nullptr)))
    return FP8_ERR_NULL;
  const int64_t Tp = up128(T);
  if (ld_dh < I || ld_gu < 2 * I || (d && ld_d < 2 * I) || (q && (ldq < 2 * I || ld_s < T)) ||
      (qt && (ldqt < Tp || ld_st < 2 * I)) || (ht && ld_sht < I))
    return FP8_ERR_LD;
  if (too_far(T, ld_dh) || too_far(T, ld_gu) || (d && too_far(T, ld_d)) || (q && (too_far(T, ldq) || too_far(2 * I / 128, ld_s))) ||
      (qt && (too_far(2 * I, ldqt) || too_far(Tp / 128, ld_st))) || (ht && too_far(Tp / 128, ld_sht)))
    return FP8_ERR_UNSUPPORTED;
  if (!aligned16(dh) || ld_dh % 8 != 0 || !aligned16(gate_up) || ld_gu % 8 != 0 || !aligned16(d) || (d && ld_d % 8 != 0) ||
      !aligned16(q) || (q && ldq % 16 != 0) || !aligned16(qt) || (qt && ldqt % 16 != 0) || !aligned16(ht) ||
      !aligned4(scales) || !aligned4(scales_t) || !aligned4(scales_ht))
    return FP8_ERR_ALIGN;
  const Range in[2] = {span(dh, T, I * 2, ld_dh * 2), span(gate_up, T, 4 * I, ld_gu * 2)};
  const Range out[7] = {span(d, d ? T : 0, 4 * I, ld_d * 2), span(q, q ? T : 0, 2 * I, ldq),
                        span(scales, q ? 2 * I / 128 : 0, T * 4, ld_s * 4), span(qt, qt ? 2 * I : 0, Tp, ldqt),
                        span(scales_t, qt ? Tp / 128 : 0, 8 * I, ld_st * 4), span(ht, ht ? 1 : 0, I * Tp, 0),
                        span(scales_ht, ht ? Tp / 128 : 0, 4 * I, ld_sht * 4)};
  if (aliased(in, out)) return FP8_ERR_ALIAS;
  const fp8_status dev = check_device();
  if (dev != FP8_OK) return dev;
  fp8bs::GatedGradProblem p{};
  p.T = T; p.I = I; p.gelu = act == FP8_ACT_GELU;
  p.dh = static_cast<const uint16_t*>(dh); p.ld_dh = ld_dh;
  p.gate_up = static_cast<const uint16_t*>(gate_up); p.ld_gu = ld_gu;
  p.d = static_cast<uint16_t*>(d); p.ld_d = ld_d;
  p.q = q; p.ldq = ldq; p.s = scales; p.ld_s = ld_s;
  p.qt = qt; p.ldqt = ldqt; p.st = scales_t; p.ld_st = ld_st;
  p.ht = ht; p.hst = scales_ht; p.ld_hst = ld_sht;
  return launched(fp8bs::launch_gated_backward(p, reinterpret_cast<hipStream_t>(stream)));
}

fp8_status fp8_quant_act_cols(const void* x, int64_t rows, int64_t cols, int64_t ldx, uint8_t* q, float* scales,
                              int64_t ld_s, void* stream) {
  if (rows < 0 || cols < 0 || cols % 128 != 0) return FP8_ERR_SHAPE;
  if (rows > kMaxTokens || cols > (int64_t{1} << 27) || up128(rows) / 128 * (cols / 64) >= 2 * kMaxBlocks)
    return FP8_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return FP8_OK;
  if (!x || !q || !scales) return FP8_ERR_NULL;
  if (ldx < cols || ld_s < cols) return FP8_ERR_LD;
  if (too_far(rows, ldx) || too_far(up128(rows) / 128, ld_s)) return FP8_ERR_UNSUPPORTED;
  if (!aligned16(x) || ldx % 8 != 0 || !aligned16(q) || !aligned4(scales)) return FP8_ERR_ALIGN;
  const Range in[1] = {span(x, rows, cols * 2, ldx * 2)};
  const Range out[2] = {span(q, 1, cols * up128(rows), 0), span(scales, up128(rows) / 128, cols * 4, ld_s * 4)};
  if (aliased(in, out)) return FP8_ERR_ALIAS;
  const fp8_status dev = check_device();
  if (dev != FP8_OK) return dev;
  return launched(fp8bs::launch_quant_cols(static_cast<const uint16_t*>(x), rows, cols, ldx, q, up128(rows), scales, ld_s,
                                           nullptr, true, reinterpret_cast<hipStream_t>(stream)));
}

fp8_status fp8_head_norm_rotary(int64_t tokens, int64_t dim, fp8_out_dtype x_dtype, const fp8_heads* q,
                                const fp8_heads* k, fp8_out_dtype w_dtype, fp8_head_norm norm, float eps, int64_t rot,
                                const void* positions, int32_t position_bytes, int32_t axes, const int64_t* sections,
                                const double* freq, int32_t adjacent, void* stream) {
  const fp8_heads none{};
  const fp8_heads* const sets[2] = {q ? q : &none, k ? k : &none};
  fp8bs::HeadProblem p{};
  const HeadArgs args{tokens, dim, x_dtype, w_dtype, norm, eps, rot, positions, position_bytes, axes, sections, freq, adjacent};
  const fp8_status st = head_common(args, sets[0]->heads, sets[1]->heads, p);
  if (st != FP8_OK) return st;
  if (tokens == 0) return FP8_OK;
  const int64_t e = x_dtype == FP8_OUT_FP32 ? 4 : 2, we = w_dtype == FP8_OUT_FP32 ? 4 : 2;
  Placed x[2]{}, y[2]{};
  Range w[2]{};
  for (int i = 0; i < 2; ++i) {
    const fp8_heads& h = *sets[i];
    if (h.heads == 0) continue;
    if (!h.x || !h.y) return FP8_ERR_NULL;
    if (h.weight && norm == FP8_HEAD_NONE) return FP8_ERR_UNSUPPORTED;
    if (too_far(tokens, h.ld_token) || too_far(h.heads, h.ld_head) || too_far(tokens, h.ldy_token) || too_far(h.heads, h.ldy_head))
      return FP8_ERR_UNSUPPORTED;
    if (!heads_nested(tokens, h.heads, dim, h.ld_token, h.ld_head) || !heads_nested(tokens, h.heads, dim, h.ldy_token, h.ldy_head))
      return FP8_ERR_LD;
    if (!aligned_to(h.x, e) || !aligned_to(h.y, e) || !aligned_to(h.weight, we)) return FP8_ERR_ALIGN;
    x[i] = placed(h.x, tokens, h.heads, dim, h.ld_token, h.ld_head, e);
    y[i] = placed(h.y, tokens, h.heads, dim, h.ldy_token, h.ldy_head, e);
    w[i] = span(h.weight, h.weight ? 1 : 0, dim * we, 0);
    p.set[i].x = h.x; p.set[i].heads = h.heads; p.set[i].ld_token = h.ld_token; p.set[i].ld_head = h.ld_head;
    p.set[i].w = h.weight;
    p.set[i].y = h.y; p.set[i].ldy_token = h.ldy_token; p.set[i].ldy_head = h.ldy_head;
  }
  const Range pos = span(positions, rot > 0 ? 1 : 0, tokens * p.axes * position_bytes, 0);
  const Range fr = span(freq, rot > 0 ? 1 : 0, rot / 2 * 8, 0);
  for (int i = 0; i < 2; ++i) {
    if (sets[i]->heads == 0) continue;
    for (int j = 0; j < 2; ++j)
      if (sets[j]->heads > 0 && (share(y[i], x[j]) || overlap(y[i].all, w[j]))) return FP8_ERR_ALIAS;
    if (overlap(y[i].all, pos) || overlap(y[i].all, fr)) return FP8_ERR_ALIAS;
  }
  if (sets[0]->heads > 0 && sets[1]->heads > 0 && share(y[0], y[1])) return FP8_ERR_ALIAS;
  const fp8_status dev = check_device();
  if (dev != FP8_OK) return dev;
  return launched(fp8bs::launch_head_norm_rotary(p, reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8_head_norm_rotary_backward_workspace(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim) {
  if (!head_sizes(tokens, q_heads, k_heads, dim) || !head_limits(tokens, q_heads, k_heads, dim)) return -1;
  return fp8bs::head_grad_parts(tokens, q_heads, k_heads, dim) * dim * 4;
}

fp8_status fp8_head_norm_rotary_backward(int64_t tokens, int64_t dim, fp8_out_dtype x_dtype, const fp8_heads_grad* q,
                                         const fp8_heads_grad* k, fp8_out_dtype w_dtype, fp8_head_norm norm, float eps,
                                         int64_t rot, const void* positions, int32_t position_bytes, int32_t axes,
                                         const int64_t* sections, const double* freq, int32_t adjacent,
                                         void* workspace, int64_t workspace_bytes, void* stream) {
  const fp8_heads_grad none{};
  const fp8_heads_grad* const sets[2] = {q ? q : &none, k ? k : &none};
  fp8bs::HeadProblem p{};
  const HeadArgs args{tokens, dim, x_dtype, w_dtype, norm, eps, rot, positions, position_bytes, axes, sections, freq, adjacent};
  const fp8_status st = head_common(args, sets[0]->heads, sets[1]->heads, p);
  if (st != FP8_OK) return st;
  const bool normed = norm != FP8_HEAD_NONE;
  for (const fp8_heads_grad* h : sets)
    if (!normed && ((h->heads > 0 && h->weight) || h->dweight)) return FP8_ERR_UNSUPPORTED;
  if (tokens == 0 && !sets[0]->dweight && !sets[1]->dweight) return FP8_OK;
  const int64_t need = normed ? fp8_head_norm_rotary_backward_workspace(tokens, sets[0]->heads, sets[1]->heads, dim) : 0;
  if (need > 0 && !workspace) return FP8_ERR_NULL;
  if (workspace_bytes < need) return FP8_ERR_SHAPE;
  if (need > 0 && !aligned16(workspace)) return FP8_ERR_ALIGN;
  const int64_t e = x_dtype == FP8_OUT_FP32 ? 4 : 2, we = w_dtype == FP8_OUT_FP32 ? 4 : 2;
  Placed in[2][2]{}, dx[2]{};
  Range w[2]{}, dw[2]{};
  for (int i = 0; i < 2; ++i) {
    const fp8_heads_grad& h = *sets[i];
    if (h.heads == 0) {                       // no heads, but a gradient of zeros may be asked for
      if (!aligned4(h.dweight)) return FP8_ERR_ALIGN;
      dw[i] = span(h.dweight, h.dweight ? 1 : 0, dim * 4, 0);
      p.set[i].dw = h.dweight;
      continue;
    }
    if (tokens > 0) {
      if ((normed && !h.x) || !h.dy || !h.dx) return FP8_ERR_NULL;
      if ((normed && (too_far(tokens, h.ld_token) || too_far(h.heads, h.ld_head))) || too_far(tokens, h.lddy_token) ||
          too_far(h.heads, h.lddy_head) || too_far(tokens, h.lddx_token) || too_far(h.heads, h.lddx_head))
        return FP8_ERR_UNSUPPORTED;
      if ((normed && !heads_nested(tokens, h.heads, dim, h.ld_token, h.ld_head)) ||
          !heads_nested(tokens, h.heads, dim, h.lddy_token, h.lddy_head) ||
          !heads_nested(tokens, h.heads, dim, h.lddx_token, h.lddx_head))
        return FP8_ERR_LD;
      if ((normed && !aligned_to(h.x, e)) || !aligned_to(h.dy, e) || !aligned_to(h.dx, e)) return FP8_ERR_ALIGN;
      if (normed) in[i][0] = placed(h.x, tokens, h.heads, dim, h.ld_token, h.ld_head, e);
      in[i][1] = placed(h.dy, tokens, h.heads, dim, h.lddy_token, h.lddy_head, e);
      dx[i] = placed(h.dx, tokens, h.heads, dim, h.lddx_token, h.lddx_head, e);
    }
    if (!aligned_to(h.weight, we) || !aligned4(h.dweight)) return FP8_ERR_ALIGN;
    w[i] = span(h.weight, h.weight ? 1 : 0, dim * we, 0);
    dw[i] = span(h.dweight, h.dweight ? 1 : 0, dim * 4, 0);
    fp8bs::HeadSet& s = p.set[i];
    s.x = normed ? h.x : nullptr; s.heads = h.heads; s.ld_token = h.ld_token; s.ld_head = h.ld_head;
    s.w = h.weight;
    s.dy = h.dy; s.lddy_token = h.lddy_token; s.lddy_head = h.lddy_head;
    s.y = h.dx; s.ldy_token = h.lddx_token; s.ldy_head = h.lddx_head;
    s.dw = h.dweight;
  }
  const Range pos = span(positions, rot > 0 ? 1 : 0, tokens * p.axes * position_bytes, 0);
  const Range fr = span(freq, rot > 0 ? 1 : 0, rot / 2 * 8, 0), ws = span(workspace, need > 0 ? 1 : 0, need, 0);
  if (overlap(ws, pos) || overlap(ws, fr) || overlap(dw[0], dw[1])) return FP8_ERR_ALIAS;
  for (int i = 0; i < 2; ++i) {
    if (overlap(dx[i].all, pos) || overlap(dx[i].all, fr) || overlap(dx[i].all, ws) || overlap(dw[i], pos) ||
        overlap(dw[i], fr) || overlap(dw[i], ws) || overlap(ws, w[i]))
      return FP8_ERR_ALIAS;
    for (int j = 0; j < 2; ++j) {
      for (const Placed& x : in[j])
        if (share(dx[i], x) || overlap(dw[i], x.all) || (i == 0 && overlap(ws, x.all))) return FP8_ERR_ALIAS;
      if (overlap(dx[i].all, w[j]) || overlap(dw[i], w[j]) || overlap(dx[i].all, dw[j])) return FP8_ERR_ALIAS;
    }
  }
  if (share(dx[0], dx[1])) return FP8_ERR_ALIAS;
  const fp8_status dev = check_device();
  if (dev != FP8_OK) return dev;
  p.partial = static_cast<float*>(workspace);
  return launched(fp8bs::launch_head_norm_rotary_backward(p, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
