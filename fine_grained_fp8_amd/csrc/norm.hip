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
#include "rows.hpp"

namespace fp8bs {

namespace {

// workgroups of the backward pass at most (one per CU of 1024 threads each)
constexpr int kMaxParts = 256;

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
      *reinterpret_cast<nv4i*>(row + c) = nv4i{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                                               bf16_pair(v[6], v[7])};
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

// Sum of the per-wave floats slot[0..n) of the calling wave's row group (n
// waves), in every lane: a lane reads one of them.
template <int n>
__device__ __forceinline__ float slots_sum(const float* slot) {
  return lanes_sum<n>(slot[(threadIdx.x & 63) & (n - 1)]);
}

// Sum over the G lanes that own a row, in each of them.  For rows owned by
// several waves `slot` (one float per wave) is written before a barrier and
// read after it; it may be used again once another barrier has passed.
template <int G>
__device__ __forceinline__ float group_sum(float v, float* slot) {
  v = lanes_sum<(G < 64 ? G : 64)>(v);
  if constexpr (G > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slots_sum<G / 64>(slot + threadIdx.x / G * (G / 64));
  }
  return v;
}

// Forward.  Each lane keeps one run of 8 values (two for rows over 8192), so a
// row of 7168 takes a workgroup of 1024 lanes and two of them fill a CU: with
// more runs a lane, fewer rows are in flight per CU and the registers of w and b
// double.  Bound by memory for plain output (8192 x 7168 BF16: 44.4 us, 5.3
// TB/s; a copy of the same bytes reaches 4.9 - 5.2) and about evenly by memory
// and the vector unit with codes (44.2 us, 178 MB; with the quotient y r, up to two
// FP32 places off, 42.4).  Measured against it at that size with that quotient,
// us plain / with codes: the next row loaded ahead - / 44.6 for 43.4, two runs and
// 512 lanes 45.6 / 42.8, four and 256 lanes 59 / 77, a wave a row with w and b in
// LDS 61 / 52.
// The codes are those of the FP32 result: where its sums' rounding moves a value
// over the middle between two codes it gets the other one (2-norm over whole
// 4096 - 8192 x 7168 arrays against 64 bits 3.4e-5 - 8.4e-5, an FP32 layer norm
// followed by a division 3.9e-5 - 9.2e-5).  The row's sums, y and the quotient in
// FP64 would settle those: 81 us.
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
  const float fc = (float)cols, inv_c = 1.0f / fc;
  // workgroups are dealt to the 8 XCDs in turn: each XCD's take neighbouring
  // rows, whose scales then meet in its L2 and leave as whole lines (at 8192 x
  // 7168 60.6 MB are written; in the plain order 73.4, and 0.5 us more)
  const int64_t first = kQuant && gridDim.x % 8 == 0 ? blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8 : blockIdx.x;
  for (int64_t r0 = first * kRows; r0 < p.rows; r0 += (int64_t)gridDim.x * kRows) {
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
    // sum / C with one correction (where it is finite): a row of one value
    // keeps that value as its mean
    s = group_sum<G>(s, red[0]);
    float mean = s * inv_c;
    if (fabsf(mean) < INFINITY) mean = __builtin_fmaf(__builtin_fmaf(-mean, fc, s), inv_c, mean);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (kVec && column<kVec, G>(i, 0, l) >= cols) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[i][k] = kVec || column<kVec, G>(i, k, l) < cols ? x[i][k] - mean : 0.f;
        ss = __builtin_fmaf(x[i][k], x[i][k], ss);
      }
    }
    const float rstd = rsqrt_refined(group_sum<G>(ss, red[1]) * inv_c + p.eps);
    if (!on) continue;
    if (l == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (kVec && column<kVec, G>(i, 0, l) >= cols) continue;   // whole 16-lane tiles
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = __builtin_fmaf(x[i][k] * rstd, w[i][k], b[i][k]);
      if (!kQuant || p.y != nullptr) store8<kVec, G>(static_cast<T*>(p.y) + row * p.ldy, i, l, cols, y);
      if constexpr (kQuant) {
        // the run of 16 lanes is one 1x128 tile
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) a = __builtin_elementwise_maximum(a, fabsf(y[k]));   // NaN stays
        const uint32_t t = row16_max_u32(__float_as_uint(a) & 0x7FFFFFFFu);
        const int c = column<true, G>(i, 0, l);
        float sc;
        const uint2 q = quant8_f32(y, t, sc);
        *reinterpret_cast<nv2i*>(p.q + row * p.ldq + c) = nv2i{(int)q.x, (int)q.y};
        if ((l & 15) == 0) p.s[(int64_t)(c >> 7) * p.ld_s + row] = sc;
      }
    }
  }
}

// A run of 8 values as loaded (BF16 stays packed: half the registers).  pin()
// hides the value's origin from the compiler, so that a later sweep unpacks
// the run again instead of keeping 8 unpacked values alive from the first.
template <typename T>
struct Run;
template <>
struct Run<uint16_t> {
  nv4i d;
  __device__ __forceinline__ void load(const uint16_t* p) { d = *reinterpret_cast<const nv4i*>(p); }
  __device__ __forceinline__ void zero() { d = nv4i{0, 0, 0, 0}; }
  __device__ __forceinline__ void pin() { __asm__ volatile("" : "+v"(d)); }
  __device__ __forceinline__ float get(int k) const {
    return (k & 1) ? bf16_hi((uint32_t)d[k >> 1]) : bf16_lo((uint32_t)d[k >> 1]);
  }
};
template <>
struct Run<float> {
  nv4i d, e;
  __device__ __forceinline__ void load(const float* p) {
    d = *reinterpret_cast<const nv4i*>(p);
    e = *reinterpret_cast<const nv4i*>(p + 4);
  }
  __device__ __forceinline__ void zero() { d = e = nv4i{0, 0, 0, 0}; }
  __device__ __forceinline__ void pin() { __asm__ volatile("" : "+v"(d), "+v"(e)); }
  __device__ __forceinline__ float get(int k) const { return __int_as_float(k < 4 ? d[k] : e[k - 4]); }
};

// Backward.  A workgroup walks rows and keeps the column sums of its lanes' 8
// columns in registers; one per CU of 1024 lanes, so that the shares it leaves
// (256 x 2 x C floats) stay small beside dy, x and dx.  8192 x 7168 BF16: 84 us for
// both launches, 352 MB (4.2 TB/s).  With two runs a lane (512 lanes) 125 us,
// with four (256 lanes) 192: the sums, w and the rows in flight no longer fit
// the registers that two rows a CU need.
template <typename T, bool kVec, int G, int B, int NV>
__global__ __launch_bounds__(B) void layer_norm_backward_kernel(LayerNormGradProblem p) {
  constexpr int kRows = B / G;
  constexpr int kWaves = G / 64;              // waves of a row (0: less than one)
  __shared__ float red[2][2][16];
  const int l = threadIdx.x % G, grp = threadIdx.x / G;
  const int cols = (int)p.cols;
  const float inv_c = 1.0f / (float)cols;
  float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_affine<kVec, G>(p.w, p.w_fp32, 1.f, i, l, cols, w[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = db[i][k] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * kRows;
  // Aligned rows stay in registers as loaded, and BF16 ones are loaded one row
  // ahead, so that loads are in flight across the two row sums' barrier (for
  // FP32 rows the second set of registers would spill).
  constexpr bool kPacked = kVec && NV == 1;
  constexpr bool kAhead = kPacked && sizeof(T) == 2;
  Run<T> rx[NV], rd[NV], nx[NV], nd[NV];   // kPacked: this row, the next
  float x[NV][8], d[NV][8];                // otherwise
  auto fetch = [&](int64_t row, Run<T> (&fx)[NV], Run<T> (&fd)[NV]) {
    const T* px = static_cast<const T*>(p.x) + row * p.ldx;
    const T* pd = static_cast<const T*>(p.dy) + row * p.lddy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = column<true, G>(i, 0, l);
      if (row < p.rows && c < cols) {
        fx[i].load(px + c);
        fd[i].load(pd + c);
      } else {
        fx[i].zero();
        fd[i].zero();
      }
    }
  };
  if constexpr (kAhead) fetch((int64_t)blockIdx.x * kRows + grp, nx, nd);
  int par = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + grp;
    const bool on = row < p.rows;
    const float mean = on ? p.mean[row] : 0.f, rstd = on ? p.rstd[row] : 0.f;
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        rx[i] = nx[i];
        rd[i] = nd[i];
      }
      fetch(row + step, nx, nd);
    } else if constexpr (kPacked) {
      fetch(row, rx, rd);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (on) {
          load8<kVec, G>(static_cast<const T*>(p.x) + row * p.ldx, i, l, cols, x[i]);
          load8<kVec, G>(static_cast<const T*>(p.dy) + row * p.lddy, i, l, cols, d[i]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[i][k] = d[i][k] = 0.f;
        }
      }
    }
    // xhat and dy of value (i, k); where there is no column or no row both
    // are 0 and add nothing anywhere
    auto xhat = [&](int i, int k) {
      const float v = kPacked ? rx[i].get(k) : x[i][k];
      const bool in = kVec ? column<true, G>(i, 0, l) < cols : column<false, G>(i, k, l) < cols;
      return in ? (v - mean) * rstd : 0.f;
    };
    auto grad = [&](int i, int k) { return kPacked ? rd[i].get(k) : d[i][k]; };
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = xhat(i, k), dy = grad(i, k), g = dy * w[i][k];
        dw[i][k] = __builtin_fmaf(dy, xh, dw[i][k]);
        db[i][k] += dy;
        s1 += g;
        s2 = __builtin_fmaf(g, xh, s2);
      }
      if constexpr (kPacked) {
        rx[i].pin();
        rd[i].pin();
      }
    }
    s1 = lanes_sum<(G < 64 ? G : 64)>(s1);
    s2 = lanes_sum<(G < 64 ? G : 64)>(s2);
    if constexpr (G > 64) {
      // both sums through one barrier; the two copies of the slots alternate
      const int wv = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
        red[par][0][wv] = s1;
        red[par][1][wv] = s2;
      }
      __syncthreads();
      s1 = slots_sum<kWaves>(red[par][0] + grp * kWaves);
      s2 = slots_sum<kWaves>(red[par][1] + grp * kWaves);
      par ^= 1;
    }
    if (!on) continue;
    const float c1 = s1 * inv_c, c2 = s2 * inv_c;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (kVec && column<kVec, G>(i, 0, l) >= cols) continue;
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = rstd * (grad(i, k) * w[i][k] - c1 - xhat(i, k) * c2);
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

// Sum of the workgroups' shares: 64 columns x 16 slices of the shares per
// workgroup, blockIdx.y = 0 for dw and 1 for db.  A lane's loads (at most 16)
// are independent, so that the kernel takes about one round trip.
__global__ __launch_bounds__(1024) void layer_norm_grad_sum_kernel(const float* __restrict__ partial, int parts,
                                                                   int cols, float* __restrict__ dw,
                                                                   float* __restrict__ db) {
  __shared__ float sum[16][64];
  const int l = threadIdx.x & 63, sl = threadIdx.x >> 6, c = blockIdx.x * 64 + l;
  float* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  float t = 0.f;
  if (c < cols) {
    float v[kMaxParts / 16];
#pragma unroll
    for (int k = 0; k < kMaxParts / 16; ++k) {
      const int q = sl + 16 * k;
      v[k] = q < parts ? partial[((int64_t)q * 2 + blockIdx.y) * cols + c] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kMaxParts / 16; ++k) t += v[k];
  }
  sum[sl][l] = t;
  __syncthreads();
  if (sl == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 16; ++k) t += sum[k][l];
    out[c] = t;
  }
}

template <typename T, bool kVec, int G, int B, int NV>
void norm_cfg(const LayerNormProblem& p, hipStream_t stream) {
  constexpr int kRows = B / G;
  const int64_t groups = (p.rows + kRows - 1) / kRows;
  const int64_t most = 256 * (2048 / B) / NV;   // what runs at once: 2048 lanes a CU with one run each
  const dim3 grid((unsigned)(groups < most ? groups : most));
  if constexpr (kVec) {
    if (p.q != nullptr) {
      hipLaunchKernelGGL((layer_norm_kernel<T, kVec, G, B, NV, true>), grid, dim3(B), 0, stream, p);
      return;
    }
  }
  hipLaunchKernelGGL((layer_norm_kernel<T, kVec, G, B, NV, false>), grid, dim3(B), 0, stream, p);
}
template <typename T, bool kVec>
void norm_any(const LayerNormProblem& p, hipStream_t stream) {
  if (p.cols <= 128) norm_cfg<T, kVec, 16, 256, 1>(p, stream);
  else if (p.cols <= 512) norm_cfg<T, kVec, 64, 256, 1>(p, stream);
  else if (p.cols <= 1024) norm_cfg<T, kVec, 128, 256, 1>(p, stream);
  else if (p.cols <= 2048) norm_cfg<T, kVec, 256, 256, 1>(p, stream);
  else if (p.cols <= 4096) norm_cfg<T, kVec, 512, 512, 1>(p, stream);
  else if (p.cols <= 8192) norm_cfg<T, kVec, 1024, 1024, 1>(p, stream);
  else norm_cfg<T, kVec, 1024, 1024, 2>(p, stream);
}

template <typename T, bool kVec, int G, int B, int NV>
void grad_cfg(const LayerNormGradProblem& p, hipStream_t stream) {
  const int64_t parts = layer_norm_grad_parts(p.rows, p.cols);
  hipLaunchKernelGGL((layer_norm_backward_kernel<T, kVec, G, B, NV>), dim3((unsigned)parts), dim3(B), 0, stream, p);
}
template <typename T, bool kVec>
void grad_any(const LayerNormGradProblem& p, hipStream_t stream) {
  if (p.cols <= 128) grad_cfg<T, kVec, 16, 1024, 1>(p, stream);
  else if (p.cols <= 512) grad_cfg<T, kVec, 64, 1024, 1>(p, stream);
  else if (p.cols <= 1024) grad_cfg<T, kVec, 128, 1024, 1>(p, stream);
  else if (p.cols <= 2048) grad_cfg<T, kVec, 256, 1024, 1>(p, stream);
  else if (p.cols <= 4096) grad_cfg<T, kVec, 512, 1024, 1>(p, stream);
  else if (p.cols <= 8192) grad_cfg<T, kVec, 1024, 1024, 1>(p, stream);
  else grad_cfg<T, kVec, 1024, 1024, 2>(p, stream);
}
// Rows a workgroup of the backward pass has in hand at a time.  Few short rows
// fill the launch unevenly: 20011 x 128 are 313 groups of 64 for 256 workgroups,
// two turns for 1.2 turns' work, and FP32 rows are not loaded ahead (10.4 us for
// 31 MB, the shares' sum 3.9 more).
int64_t grad_rows(int64_t cols) {
  return cols <= 128 ? 64 : cols <= 512 ? 16 : cols <= 1024 ? 8 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1;
}

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
    if (vec) norm_any<float, true>(p, stream);
    else norm_any<float, false>(p, stream);
  } else {
    if (vec) norm_any<uint16_t, true>(p, stream);
    else norm_any<uint16_t, false>(p, stream);
  }
  return hipGetLastError();
}

int64_t layer_norm_grad_parts(int64_t rows, int64_t cols) {
  const int64_t g = (rows + grad_rows(cols) - 1) / grad_rows(cols);
  return g < kMaxParts ? g : kMaxParts;
}

hipError_t launch_layer_norm_backward(const LayerNormGradProblem& p, hipStream_t stream) {
  const int64_t e = p.x_fp32 ? 4 : 2;
  const int64_t we = p.w_fp32 ? 4 : 2;
  const int64_t parts = layer_norm_grad_parts(p.rows, p.cols);
  const bool vec = p.cols % 8 == 0 && aligned_rows(p.x, p.ldx, e) && aligned_rows(p.dy, p.lddy, e) &&
                   aligned_rows(p.dx, p.lddx, e) && aligned_rows(p.w, 16 / we, we);
  if (parts > 0) {
    if (p.x_fp32) {
      if (vec) grad_any<float, true>(p, stream);
      else grad_any<float, false>(p, stream);
    } else {
      if (vec) grad_any<uint16_t, true>(p, stream);
      else grad_any<uint16_t, false>(p, stream);
    }
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  if (p.dw == nullptr && p.db == nullptr) return hipSuccess;
  hipLaunchKernelGGL(layer_norm_grad_sum_kernel, dim3((unsigned)((p.cols + 63) / 64), 2), dim3(1024), 0, stream,
                     p.partial, (int)parts, (int)p.cols, p.dw, p.db);
  return hipGetLastError();
}

}  // namespace fp8bs
