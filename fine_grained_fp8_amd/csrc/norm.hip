// Layer norm for gfx950: forward (optionally with the 1x128 FP8 quantization
// of its result as the epilogue) and backward with the reduction of the
// weight's and the bias's gradients.
//
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   xhat = (x - mean) rstd,  y = xhat w + b
//   g = dy w,  dx = rstd (g - sum g / C - xhat sum(g xhat) / C)
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// All of it is bound by memory: one read of every input, one write of every
// output.  A row lives in the registers of the lanes that own it, so the
// variance is taken of the differences from the mean (a second sweep over
// registers, not memory) with no cancellation, and the quantizer's tile
// maximum, scale and codes come from the FP32 result without a pass through
// BF16.  All sums are FP32 in a fixed order: results do not change from run
// to run.
#include "device.hpp"
#include "layers.hpp"

namespace fp8bs {

namespace {

typedef int nv4i __attribute__((ext_vector_type(4)));
typedef int nv2i __attribute__((ext_vector_type(2)));

// A row is owned by G lanes (16, 64, or the whole workgroup of B), each
// holding NV runs of 8 values.  Vector form: run i of lane l is columns
// (i G + l) 8 .. + 7, moved as 16-byte accesses.  Scalar form (rows that are
// not 16-byte aligned, or C % 8 != 0): value v of run i is column
// (8 i + v) G + l, so the accesses of a wave stay contiguous.
template <bool kVec, int G>
__device__ __forceinline__ int column(int i, int v, int l) {
  return kVec ? (i * G + l) * 8 + v : (8 * i + v) * G + l;
}

__device__ __forceinline__ float to_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ float to_f32(float f) { return f; }

__device__ __forceinline__ uint16_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return (uint32_t)bf16_bits(a) | ((uint32_t)bf16_bits(b) << 16);
}

// 8 values of run i (zeros past the last column)
template <bool kVec, int G, typename T>
__device__ __forceinline__ void load8(const T* __restrict__ row, int i, int l, int cols, float (&v)[8]) {
  if constexpr (kVec) {
    const int c = column<true, G>(i, 0, l);
    if (c >= cols) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.f;
      return;
    }
    if constexpr (sizeof(T) == 2) {
      const nv4i d = *reinterpret_cast<const nv4i*>(row + c);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf16_lo((uint32_t)d[k]);
        v[2 * k + 1] = bf16_hi((uint32_t)d[k]);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(row + c);
      const float4 b = *reinterpret_cast<const float4*>(row + c + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = column<false, G>(i, k, l);
      v[k] = c < cols ? to_f32(row[c]) : 0.f;
    }
  }
}

template <bool kVec, int G, typename T>
__device__ __forceinline__ void store8(T* __restrict__ row, int i, int l, int cols, const float (&v)[8]) {
  if constexpr (kVec) {
    const int c = column<true, G>(i, 0, l);
    if (c >= cols) return;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<nv4i*>(row + c) = nv4i{(int)bf16_pair(v[0], v[1]), (int)bf16_pair(v[2], v[3]),
                                               (int)bf16_pair(v[4], v[5]), (int)bf16_pair(v[6], v[7])};
    } else {
      *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = column<false, G>(i, k, l);
      if (c < cols) {
        if constexpr (sizeof(T) == 2) row[c] = bf16_bits(v[k]);
        else row[c] = v[k];
      }
    }
  }
}

// weight or bias of run i as FP32 (null: the neutral value)
template <bool kVec, int G>
__device__ __forceinline__ void load_affine(const void* p, int is_f32, float neutral, int i, int l, int cols,
                                            float (&v)[8]) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = neutral;
  } else if (is_f32) {
    load8<kVec, G>(static_cast<const float*>(p), i, l, cols, v);
  } else {
    load8<kVec, G>(static_cast<const uint16_t*>(p), i, l, cols, v);
  }
}

template <int kCtrl>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xF, 0xF, true));
}
// sum over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ float row16_sum(float v) {
  v = add_dpp<0xB1>(v);    // quad_perm 1,0,3,2
  v = add_dpp<0x4E>(v);    // quad_perm 2,3,0,1
  v = add_dpp<0x141>(v);   // row_half_mirror
  return add_dpp<0x140>(v);   // row_mirror
}

// Sum over the G lanes that own a row, in each of them.  For rows owned by
// the whole workgroup `slot` (one float per wave) is written before a
// barrier and read after it; a slot may be used again once another barrier
// has passed.
template <int G, int B>
__device__ __forceinline__ float group_sum(float v, float* slot) {
  v = row16_sum(v);
  if constexpr (G >= 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  if constexpr (G > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < B / 64; ++w) v += slot[w];
  }
  return v;
}

template <typename T, bool kVec, int G, int B, int NV, bool kQuant>
__global__ __launch_bounds__(B) void layer_norm_kernel(LayerNormProblem p) {
  constexpr int kRows = B / G;
  __shared__ float red[2][16];
  const int l = threadIdx.x % G, grp = threadIdx.x / G;
  const int cols = (int)p.cols;
  float w[NV][8], b[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_affine<kVec, G>(p.w, p.w_fp32, 1.f, i, l, cols, w[i]);
    load_affine<kVec, G>(p.b, p.w_fp32, 0.f, i, l, cols, b[i]);
  }
  const float fc = (float)cols;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = r0 + grp;
    const bool on = row < p.rows;
    float x[NV][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on) {
        load8<kVec, G>(static_cast<const T*>(p.x) + row * p.ldx, i, l, cols, x[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s += x[i][k];
    }
    const float mean = group_sum<G, B>(s, red[0]) / fc;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[i][k] = column<kVec, G>(i, k, l) < cols ? x[i][k] - mean : 0.f;
        ss = __builtin_fmaf(x[i][k], x[i][k], ss);
      }
    const float rstd = 1.0f / sqrtf(group_sum<G, B>(ss, red[1]) / fc + p.eps);
    if (!on) continue;
    if (l == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = __builtin_fmaf(x[i][k] * rstd, w[i][k], b[i][k]);
      if (!kQuant || p.y != nullptr) store8<kVec, G>(static_cast<T*>(p.y) + row * p.ldy, i, l, cols, y);
      if constexpr (kQuant) {
        // the run of 16 lanes is one 1x128 tile
        uint32_t t = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) t = max(t, __float_as_uint(y[k]) & 0x7FFFFFFFu);
        t = row16_max_u32(t);
        const int c = column<true, G>(i, 0, l);
        if (c < cols) {
          float sc;
          const uint2 q = quant8_f32(y, t, sc);
          *reinterpret_cast<nv2i*>(p.q + row * p.ldq + c) = nv2i{(int)q.x, (int)q.y};
          if ((l & 15) == 0) p.s[(int64_t)(c >> 7) * p.ld_s + row] = sc;
        }
      }
    }
  }
}

template <typename T, bool kVec, int G, int B, int NV>
__global__ __launch_bounds__(B) void layer_norm_backward_kernel(LayerNormGradProblem p) {
  constexpr int kRows = B / G;
  __shared__ float red[2][2][16];
  const int l = threadIdx.x % G, grp = threadIdx.x / G;
  const int cols = (int)p.cols;
  const float fc = (float)cols;
  float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_affine<kVec, G>(p.w, p.w_fp32, 1.f, i, l, cols, w[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = db[i][k] = 0.f;
  }
  int par = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = r0 + grp;
    const bool on = row < p.rows;
    float x[NV][8], d[NV][8];
    float mean = 0.f, rstd = 0.f;
    if (on) {
      mean = p.mean[row];
      rstd = p.rstd[row];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        load8<kVec, G>(static_cast<const T*>(p.x) + row * p.ldx, i, l, cols, x[i]);
        load8<kVec, G>(static_cast<const T*>(p.dy) + row * p.lddy, i, l, cols, d[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] = d[i][k] = 0.f;
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // columns past the last one hold dy = 0 and add nothing anywhere
        const bool in = column<kVec, G>(i, k, l) < cols;
        x[i][k] = in ? (x[i][k] - mean) * rstd : 0.f;
        dw[i][k] = __builtin_fmaf(d[i][k], x[i][k], dw[i][k]);
        db[i][k] += d[i][k];
        d[i][k] *= w[i][k];
        s1 += d[i][k];
        s2 = __builtin_fmaf(d[i][k], x[i][k], s2);
      }
    // both sums through one barrier: the first one's slot is published by
    // the second one's barrier
    if constexpr (G > 64) {
      s1 = group_sum<64, 64>(s1, nullptr);
      if ((threadIdx.x & 63) == 0) red[par][0][threadIdx.x >> 6] = s1;
      s2 = group_sum<G, B>(s2, red[par][1]);
      s1 = 0.f;
#pragma unroll
      for (int k = 0; k < B / 64; ++k) s1 += red[par][0][k];
      par ^= 1;
    } else {
      s1 = group_sum<G, B>(s1, nullptr);
      s2 = group_sum<G, B>(s2, nullptr);
    }
    if (!on) continue;
    const float c1 = s1 / fc, c2 = s2 / fc;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = rstd * (d[i][k] - c1 - x[i][k] * c2);
      store8<kVec, G>(static_cast<T*>(p.dx) + row * p.lddx, i, l, cols, o);
    }
  }
  // this workgroup's share of the column sums: [workgroup][dw, db][cols]
  float* part = p.partial + (int64_t)blockIdx.x * 2 * cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = column<kVec, G>(i, k, l);
        if (c < cols) {
          part[c] = dw[i][k];
          part[cols + c] = db[i][k];
        }
      }
  } else {
    // the row groups of the workgroup first, in order
    constexpr int kCols = G * 8 * NV;
    __shared__ float sum[kRows][kCols];
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[grp][column<kVec, G>(i, k, l)] = pass == 0 ? dw[i][k] : db[i][k];
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += B) {
        float t = sum[0][c];
#pragma unroll
        for (int g = 1; g < kRows; ++g) t += sum[g][c];
        part[pass * cols + c] = t;
      }
    }
  }
}

// Sum of the workgroups' shares: 16 columns x 16 slices of the shares per
// workgroup, blockIdx.y = 0 for dw and 1 for db.
__global__ __launch_bounds__(256) void layer_norm_grad_sum_kernel(const float* __restrict__ partial, int parts,
                                                                  int cols, float* __restrict__ dw,
                                                                  float* __restrict__ db) {
  __shared__ float sum[16][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), sl = threadIdx.x >> 4;
  float* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  float t = 0.f;
  if (c < cols)
    for (int q = sl; q < parts; q += 16) t += partial[((int64_t)q * 2 + blockIdx.y) * cols + c];
  sum[sl][threadIdx.x & 15] = t;
  __syncthreads();
  if (sl == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 16; ++k) t += sum[k][threadIdx.x & 15];
    out[c] = t;
  }
}

template <typename T, bool kVec, int G, int B, int NV>
void norm_cfg(const LayerNormProblem& p, hipStream_t stream) {
  constexpr int kRows = B / G;
  const int64_t groups = (p.rows + kRows - 1) / kRows;
  const int64_t most = 256 * (2048 / B);
  const dim3 grid((unsigned)(groups < most ? groups : most));
  if constexpr (kVec) {
    if (p.q != nullptr) {
      hipLaunchKernelGGL((layer_norm_kernel<T, kVec, G, B, NV, true>), grid, dim3(B), 0, stream, p);
      return;
    }
  }
  hipLaunchKernelGGL((layer_norm_kernel<T, kVec, G, B, NV, false>), grid, dim3(B), 0, stream, p);
}

template <typename T, bool kVec, int G, int B, int NV>
void grad_cfg(const LayerNormGradProblem& p, int64_t parts, hipStream_t stream) {
  hipLaunchKernelGGL((layer_norm_backward_kernel<T, kVec, G, B, NV>), dim3((unsigned)parts), dim3(B), 0, stream, p);
}

// rows owned by one workgroup at a time, by the row length
int rows_per_workgroup(int64_t cols) { return cols <= 128 ? 16 : cols <= 1024 ? 4 : 1; }

#define FP8BS_NORM_DISPATCH(FN, T, VEC, ...)                        \
  do {                                                              \
    if (p.cols <= 128) FN<T, VEC, 16, 256, 1>(__VA_ARGS__);         \
    else if (p.cols <= 512) FN<T, VEC, 64, 256, 1>(__VA_ARGS__);    \
    else if (p.cols <= 1024) FN<T, VEC, 64, 256, 2>(__VA_ARGS__);   \
    else if (p.cols <= 2048) FN<T, VEC, 256, 256, 1>(__VA_ARGS__);  \
    else if (p.cols <= 4096) FN<T, VEC, 256, 256, 2>(__VA_ARGS__);  \
    else if (p.cols <= 8192) FN<T, VEC, 256, 256, 4>(__VA_ARGS__);  \
    else FN<T, VEC, 512, 512, 4>(__VA_ARGS__);                      \
  } while (0)

bool aligned_rows(const void* p, int64_t ld, int64_t esz) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * esz) % 16 == 0;
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormProblem& p, hipStream_t stream) {
  const int64_t e = p.x_fp32 ? 4 : 2;
  const int64_t we = p.w_fp32 ? 4 : 2;
  const bool vec = p.cols % 8 == 0 && aligned_rows(p.x, p.ldx, e) && (!p.y || aligned_rows(p.y, p.ldy, e)) &&
                   aligned_rows(p.w, 16 / we, we) && aligned_rows(p.b, 16 / we, we);
  if (p.x_fp32) {
    if (vec) FP8BS_NORM_DISPATCH(norm_cfg, float, true, p, stream);
    else FP8BS_NORM_DISPATCH(norm_cfg, float, false, p, stream);
  } else {
    if (vec) FP8BS_NORM_DISPATCH(norm_cfg, uint16_t, true, p, stream);
    else FP8BS_NORM_DISPATCH(norm_cfg, uint16_t, false, p, stream);
  }
  return hipGetLastError();
}

int64_t layer_norm_grad_parts(int64_t rows, int64_t cols) {
  const int64_t g = (rows + rows_per_workgroup(cols) - 1) / rows_per_workgroup(cols);
  return g < 512 ? g : 512;
}

hipError_t launch_layer_norm_backward(const LayerNormGradProblem& p, hipStream_t stream) {
  const int64_t e = p.x_fp32 ? 4 : 2;
  const int64_t we = p.w_fp32 ? 4 : 2;
  const int64_t parts = layer_norm_grad_parts(p.rows, p.cols);
  const bool vec = p.cols % 8 == 0 && aligned_rows(p.x, p.ldx, e) && aligned_rows(p.dy, p.lddy, e) &&
                   aligned_rows(p.dx, p.lddx, e) && aligned_rows(p.w, 16 / we, we);
  if (parts > 0) {
    if (p.x_fp32) {
      if (vec) FP8BS_NORM_DISPATCH(grad_cfg, float, true, p, parts, stream);
      else FP8BS_NORM_DISPATCH(grad_cfg, float, false, p, parts, stream);
    } else {
      if (vec) FP8BS_NORM_DISPATCH(grad_cfg, uint16_t, true, p, parts, stream);
      else FP8BS_NORM_DISPATCH(grad_cfg, uint16_t, false, p, parts, stream);
    }
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  if (p.dw == nullptr && p.db == nullptr) return hipSuccess;
  hipLaunchKernelGGL(layer_norm_grad_sum_kernel, dim3((unsigned)((p.cols + 15) / 16), 2), dim3(256), 0, stream,
                     p.partial, (int)parts, (int)p.cols, p.dw, p.db);
  return hipGetLastError();
}

}  // namespace fp8bs
