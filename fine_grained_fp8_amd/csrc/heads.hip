// Norms of query and key heads with the position rotation in the same pass, for
// gfx950: forward and backward.
//
//   n = (x - mean) rstd w      rstd = 1 / sqrt(sum (x - mean)^2 / D + eps); rms: mean = 0; none: n = x
//   (y1, y2) = (n1 c - n2 s, n2 c + n1 s) for each rotated pair,  c + i s = exp(i p f),
//   p the token's position on the pair's axis, f the pair's frequency
//   backward: d = dy rotated by -p f,  g = d w,
//   dx = rstd (g - sum g / D - xhat sum(g xhat) / D)   (rms: without the second term)
//   dw = sum over tokens and heads of d xhat
//
// Bound by memory: every head is read once and written once.  A head lives in
// the registers of G lanes, 8 pairs a lane: both elements of a pair meet in one
// lane for either order of pairs, so the rotation moves nothing between lanes,
// and the lane's eight angles serve all heads of the token.  A wave works on 64 / G
// heads of one token at a time, queries first and then keys.
#include "blocks.hpp"
#include "device.hpp"
#include "rows.hpp"

namespace fp8bs {

namespace {

constexpr int kHB = 256, kHW = kHB / 64;   // threads and waves of a workgroup
constexpr int kMaxGradParts = 1024;

typedef int hv4i __attribute__((ext_vector_type(4)));

// How a lane's 16 elements of a head lie: two runs of 8 moved as 16-byte accesses, its
// pairs (k, 8 + k) for halves or (2 k, 2 k + 1) for adjacent pairs; or (kScalar)
// element by element, pairs (k, 8 + k), for heads that are not 16-byte aligned or
// whose size or rotated part is no multiple of 16.
enum Mode { kHalves = 0, kAdjacent = 1, kScalar = 2 };

// cos and sin of p f.  The angle in turns is reduced in FP64 (an angle of 10^6
// radians has lost 2^-5 in FP32), then a quarter turn's Taylor polynomials:
// within 3e-9 + rounding on [-pi/4, pi/4].
__device__ __forceinline__ void rotation(double p, double f, float& c, float& s) {
  constexpr double kTurn = 0.15915494309189535, kTwoPi = 6.283185307179586;
  const double turns = p * f * kTurn;
  const double part = turns - __builtin_rint(turns);          // [-1/2, 1/2]
  const double quarter = __builtin_rint(4.0 * part);
  const float x = (float)(__builtin_fma(quarter, -0.25, part) * kTwoPi), z = x * x;
  float sn = __builtin_fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
  sn = __builtin_fmaf(z, sn, 1.0f / 120.0f);
  sn = __builtin_fmaf(z, sn, -1.0f / 6.0f);
  sn = __builtin_fmaf(z * x, sn, x);
  float cs = __builtin_fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  cs = __builtin_fmaf(z, cs, -1.0f / 720.0f);
  cs = __builtin_fmaf(z, cs, 1.0f / 24.0f);
  cs = __builtin_fmaf(z, cs, -0.5f);
  cs = __builtin_fmaf(z, cs, 1.0f);
  const int q = (int)quarter;                                  // -2 .. 2
  const float a = (q & 1) ? sn : cs, b = (q & 1) ? cs : sn;
  c = ((q + 1) & 2) ? -a : a;
  s = (q & 2) ? -b : b;
}

template <int kMode, int G>
struct Lane {
  int l, dim, half_rot;        // lane of the head, head size, rotated pairs
  int adjacent;
  // element of register v (0..15); past the head's end: >= dim
  __device__ __forceinline__ int element(int v) const {
    if constexpr (kMode == kAdjacent) return l * 16 + v;
    if constexpr (kMode == kHalves) {
      if (8 * l < half_rot) return v < 8 ? l * 8 + v : half_rot + l * 8 + v - 8;
      return l * 16 + v;
    }
    const int i = pair(v & 7), second = v >> 3;
    if (2 * i >= dim) return dim;
    if (!adjacent && i < half_rot) return i + second * half_rot;
    return 2 * i + second;
  }
  __device__ __forceinline__ int pair(int k) const { return kMode == kScalar ? k * G + l : l * 8 + k; }
  __device__ __forceinline__ bool on() const { return kMode == kScalar ? true : l * 16 < dim; }
  static __device__ __forceinline__ int first(int k) { return kMode == kAdjacent ? 2 * k : k; }
  static __device__ __forceinline__ int second(int k) { return kMode == kAdjacent ? 2 * k + 1 : 8 + k; }

  // zeros past the head's end
  template <typename T>
  __device__ __forceinline__ void load(const T* p, float (&v)[16]) const {
    if constexpr (kMode == kScalar) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int e = element(k);
        v[k] = e < dim ? value(p[e]) : 0.f;
      }
    } else {
      if (!on()) {
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = 0.f;
        return;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const T* q = p + element(8 * r);
        if constexpr (sizeof(T) == 2) {
          const hv4i d = *reinterpret_cast<const hv4i*>(q);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[8 * r + 2 * k] = bf16_lo((uint32_t)d[k]);
            v[8 * r + 2 * k + 1] = bf16_hi((uint32_t)d[k]);
          }
        } else {
          const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
          v[8 * r] = a.x; v[8 * r + 1] = a.y; v[8 * r + 2] = a.z; v[8 * r + 3] = a.w;
          v[8 * r + 4] = b.x; v[8 * r + 5] = b.y; v[8 * r + 6] = b.z; v[8 * r + 7] = b.w;
        }
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const float (&v)[16]) const {
    if constexpr (kMode == kScalar) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int e = element(k);
        if (e >= dim) continue;
        if constexpr (sizeof(T) == 2) p[e] = __builtin_bit_cast(uint16_t, (__bf16)v[k]);
        else p[e] = v[k];
      }
    } else {
      if (!on()) return;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        T* q = p + element(8 * r);
        const float* u = v + 8 * r;
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<hv4i*>(q) =
              hv4i{bf16_pair(u[0], u[1]), bf16_pair(u[2], u[3]), bf16_pair(u[4], u[5]), bf16_pair(u[6], u[7])};
        } else {
          *reinterpret_cast<float4*>(q) = make_float4(u[0], u[1], u[2], u[3]);
          *reinterpret_cast<float4*>(q + 4) = make_float4(u[4], u[5], u[6], u[7]);
        }
      }
    }
  }
  static __device__ __forceinline__ float value(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
  static __device__ __forceinline__ float value(float f) { return f; }

  // a weight vector (null: ones)
  __device__ __forceinline__ void load_weight(const void* w, int is_f32, float (&v)[16]) const {
    if (w == nullptr) {
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = 1.f;
    } else if (is_f32) {
      load(static_cast<const float*>(w), v);
    } else {
      load(static_cast<const uint16_t*>(w), v);
    }
  }

  // the angles of the lane's pairs at token t
  __device__ __forceinline__ void angles(const HeadProblem& p, int64_t t, float (&c)[8], float (&s)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = pair(k);
      c[k] = 1.f;
      s[k] = 0.f;
      if (i < half_rot) {
        int axis = 0;
#pragma unroll
        for (int a = 0; a + 1 < kHeadMaxAxes; ++a) axis += i >= p.section_end[a] && a + 1 < p.axes ? 1 : 0;
        const int64_t at = t * p.axes + axis;
        const double pos = p.pos64 ? (double)static_cast<const int64_t*>(p.positions)[at]
                                   : (double)static_cast<const int32_t*>(p.positions)[at];
        rotation(pos, p.freq[i], c[k], s[k]);
      }
    }
  }
  // rotates the pairs by the angles (kBack: against them); pairs that do not
  // rotate are left alone, infinities and NaN included
  template <bool kBack>
  __device__ __forceinline__ void rotate(float (&v)[16], const float (&c)[8], const float (&s)[8]) const {
    auto turn = [&](int k) {
      const float a = v[first(k)], b = v[second(k)], sn = kBack ? -s[k] : s[k];
      v[first(k)] = __builtin_fmaf(a, c[k], -(b * sn));
      v[second(k)] = __builtin_fmaf(b, c[k], a * sn);
    };
    if constexpr (kMode == kScalar) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (pair(k) < half_rot) turn(k);
    } else if (l * 8 < half_rot) {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn(k);
    }
  }
  // x becomes xhat; returns rstd
  __device__ __forceinline__ float normalize(float (&x)[16], int norm, float eps) const {
    const float d = (float)dim, inv_d = 1.0f / d;
    if (norm == kHeadLayer) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) sum += x[k];
      sum = lanes_sum<G>(sum);
      // sum / D with one correction (where it is finite): a head of one value keeps that value as its mean
      float mean = sum * inv_d;
      if (fabsf(mean) < INFINITY) mean = __builtin_fmaf(__builtin_fmaf(-mean, d, sum), inv_d, mean);
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = (kMode == kScalar ? element(k) < dim : on()) ? x[k] - mean : 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) ss = __builtin_fmaf(x[k], x[k], ss);
    const float rstd = rsqrt_refined(lanes_sum<G>(ss) * inv_d + eps);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= rstd;
    return rstd;
  }
};

// passes of a wave over the heads of a set, 64 / G heads each
__host__ __device__ inline int passes(int64_t heads, int G) { return (int)((heads * G + 63) / 64); }

template <typename T, int kMode, int G>
__global__ __launch_bounds__(kHB) void head_norm_rotary_kernel(HeadProblem p, int cut) {
  const int lane = threadIdx.x & 63, slot = lane / G;
  const int64_t unit = (int64_t)blockIdx.x * kHW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = unit / cut;
  if (t >= p.T) return;
  const int part = (int)(unit - t * cut);
  const Lane<kMode, G> me{lane % G, p.dim, p.rot / 2, p.adjacent};
  const int nq = passes(p.set[0].heads, G), n = nq + passes(p.set[1].heads, G);
  const int first = (int)((int64_t)n * part / cut), end = (int)((int64_t)n * (part + 1) / cut);
  float c[8], s[8];
  me.angles(p, t, c, s);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const HeadSet& hs = p.set[which];
    const int from = which == 0 ? first : max(first, nq) - nq, to = which == 0 ? min(end, nq) : end - nq;
    if (from >= to) continue;
    float w[16];
    if (p.norm != kHeadNone) me.load_weight(hs.w, p.w_fp32, w);
    const T* x = static_cast<const T*>(hs.x) + t * hs.ld_token;
    T* y = static_cast<T*>(hs.y) + t * hs.ldy_token;
    auto head_of = [&](int pass) { return min((int64_t)pass * (64 / G) + slot, hs.heads - 1); };   // past the last: that one again, not stored
    float v[16], next[16];
    me.load(x + head_of(from) * hs.ld_head, v);
#pragma unroll 1
    for (int pass = from; pass < to; ++pass) {
      me.load(x + head_of(min(pass + 1, to - 1)) * hs.ld_head, next);
      if (p.norm != kHeadNone) {
        me.normalize(v, p.norm, p.eps);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] *= w[k];
      }
      me.template rotate<false>(v, c, s);
      const int64_t h = (int64_t)pass * (64 / G) + slot;
      if (h < hs.heads) me.store(y + h * hs.ldy_head, v);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = next[k];
    }
  }
}

// Backward.  Waves walk (token, share of the heads) units; a lane keeps its
// elements' sums for both weights, a workgroup's meet in LDS at the end, and the
// workgroups' shares are added by a second launch, all in a fixed order.
template <typename T, int kMode, int G>
__global__ __launch_bounds__(kHB) void head_norm_rotary_backward_kernel(HeadProblem p, int cut) {
  const int lane = threadIdx.x & 63, slot = lane / G;
  const Lane<kMode, G> me{lane % G, p.dim, p.rot / 2, p.adjacent};
  const int nq = passes(p.set[0].heads, G), n = nq + passes(p.set[1].heads, G);
  const float inv_d = 1.0f / (float)p.dim;
  float dw[2][16];
#pragma unroll
  for (int k = 0; k < 16; ++k) dw[0][k] = dw[1][k] = 0.f;
  const int64_t units = p.T * cut;
  for (int64_t unit = (int64_t)blockIdx.x * kHW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); unit < units;
       unit += (int64_t)gridDim.x * kHW) {
    const int64_t t = unit / cut;
    const int part = (int)(unit - t * cut);
    const int first = (int)((int64_t)n * part / cut), end = (int)((int64_t)n * (part + 1) / cut);
    float c[8], s[8];
    me.angles(p, t, c, s);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const HeadSet& hs = p.set[which];
      const int from = which == 0 ? first : max(first, nq) - nq, to = which == 0 ? min(end, nq) : end - nq;
      if (from >= to) continue;
      float w[16];
      if (p.norm != kHeadNone) me.load_weight(hs.w, p.w_fp32, w);
      const T* x = static_cast<const T*>(hs.x) + t * hs.ld_token;
      const T* dy = static_cast<const T*>(hs.dy) + t * hs.lddy_token;
      T* dx = static_cast<T*>(hs.y) + t * hs.ldy_token;
#pragma unroll 1
      for (int pass = from; pass < to; ++pass) {
        const int64_t h = (int64_t)pass * (64 / G) + slot;
        const bool on = h < hs.heads;
        const int64_t at = on ? h : hs.heads - 1;
        float d[16];
        me.load(dy + at * hs.lddy_head, d);
        if (p.norm == kHeadNone) {
          me.template rotate<true>(d, c, s);
        } else {
          float xh[16];
          me.load(x + at * hs.ld_head, xh);
          me.template rotate<true>(d, c, s);
          const float rstd = me.normalize(xh, p.norm, p.eps);
          float s1 = 0.f, s2 = 0.f;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            if (on) dw[which][k] = __builtin_fmaf(d[k], xh[k], dw[which][k]);
            d[k] *= w[k];
            s1 += d[k];
            s2 = __builtin_fmaf(d[k], xh[k], s2);
          }
          const float c1 = p.norm == kHeadLayer ? lanes_sum<G>(s1) * inv_d : 0.f, c2 = lanes_sum<G>(s2) * inv_d;
#pragma unroll
          for (int k = 0; k < 16; ++k) d[k] = rstd * (d[k] - c1 - xh[k] * c2);
        }
        if (on) me.store(dx + h * hs.ldy_head, d);
      }
    }
  }
  if (p.norm == kHeadNone) return;
  // the workgroup's share of the weights' gradients: its lane groups in order
  __shared__ float sum[kHB / G][16 * G];
  float* out = p.partial + (int64_t)blockIdx.x * 2 * p.dim;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int e = me.element(k);
      if (me.on() && e < p.dim) sum[threadIdx.x / G][e] = dw[which][k];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.dim; e += kHB) {
      float v = sum[0][e];
      for (int g = 1; g < kHB / G; ++g) v += sum[g][e];
      out[which * p.dim + e] = v;
    }
  }
}

// The workgroups' shares added up: 64 columns x 16 slices of the shares a workgroup,
// blockIdx.y = 0 for queries and 1 for keys.
__global__ __launch_bounds__(1024) void head_grad_sum_kernel(const float* __restrict__ partial, int parts, int dim,
                                                             float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sum[16][64];
  const int l = threadIdx.x & 63, sl = threadIdx.x >> 6, e = blockIdx.x * 64 + l;
  float* out = blockIdx.y == 0 ? dwq : dwk;
  if (out == nullptr) return;
  float t = 0.f;
  if (e < dim) {
    for (int q0 = sl; q0 < parts; q0 += 16 * 16) {
      float v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int q = q0 + 16 * k;
        v[k] = q < parts ? partial[((int64_t)q * 2 + blockIdx.y) * dim + e] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) t += v[k];
    }
  }
  sum[sl][l] = t;
  __syncthreads();
  if (sl == 0 && e < dim) {
#pragma unroll
    for (int k = 1; k < 16; ++k) t += sum[k][l];
    out[e] = t;
  }
}

int lanes_of(int64_t dim) { return dim <= 64 ? 4 : dim <= 128 ? 8 : dim <= 256 ? 16 : dim <= 512 ? 32 : 64; }

// waves that share a token's heads: as many as give about 16 waves a CU
int token_cut(int64_t T, int64_t q_heads, int64_t k_heads, int64_t dim) {
  const int G = lanes_of(dim);
  const int64_t n = passes(q_heads, G) + passes(k_heads, G), want = (4096 + T - 1) / T;
  return (int)(want < n ? want : n);
}

bool aligned_heads(const void* p, int64_t ld_token, int64_t ld_head, int64_t esz) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld_token * esz) % 16 == 0 && (ld_head * esz) % 16 == 0;
}

template <bool kBack, typename T, int kMode, int G>
void start(const HeadProblem& p, hipStream_t stream) {
  const int cut = token_cut(p.T, p.set[0].heads, p.set[1].heads, p.dim);
  if constexpr (kBack) {
    const int64_t parts = head_grad_parts(p.T, p.set[0].heads, p.set[1].heads, p.dim);
    hipLaunchKernelGGL((head_norm_rotary_backward_kernel<T, kMode, G>), dim3((unsigned)parts), dim3(kHB), 0, stream, p, cut);
  } else {
    const int64_t blocks = (p.T * cut + kHW - 1) / kHW;
    hipLaunchKernelGGL((head_norm_rotary_kernel<T, kMode, G>), dim3((unsigned)blocks), dim3(kHB), 0, stream, p, cut);
  }
}
template <bool kBack, typename T, int kMode>
void start_dim(const HeadProblem& p, hipStream_t stream) {
  switch (lanes_of(p.dim)) {
    case 4: return start<kBack, T, kMode, 4>(p, stream);
    case 8: return start<kBack, T, kMode, 8>(p, stream);
    case 16: return start<kBack, T, kMode, 16>(p, stream);
    case 32: return start<kBack, T, kMode, 32>(p, stream);
    default: return start<kBack, T, kMode, 64>(p, stream);
  }
}
template <bool kBack, typename T>
void start_mode(const HeadProblem& p, hipStream_t stream) {
  bool vec = p.dim % 16 == 0 && p.rot % 16 == 0;
  for (const HeadSet& h : p.set) {
    if (h.heads == 0) continue;
    vec = vec && aligned_heads(h.y, h.ldy_token, h.ldy_head, sizeof(T)) && (reinterpret_cast<uintptr_t>(h.w) & 15) == 0 &&
          (h.x == nullptr || aligned_heads(h.x, h.ld_token, h.ld_head, sizeof(T))) &&
          (!kBack || aligned_heads(h.dy, h.lddy_token, h.lddy_head, sizeof(T)));
  }
  if (!vec) start_dim<kBack, T, kScalar>(p, stream);
  else if (p.adjacent) start_dim<kBack, T, kAdjacent>(p, stream);
  else start_dim<kBack, T, kHalves>(p, stream);
}

}  // namespace

hipError_t launch_head_norm_rotary(const HeadProblem& p, hipStream_t stream) {
  if (p.x_fp32) start_mode<false, float>(p, stream);
  else start_mode<false, uint16_t>(p, stream);
  return hipGetLastError();
}

int64_t head_grad_parts(int64_t T, int64_t q_heads, int64_t k_heads, int64_t dim) {
  if (T == 0) return 0;
  const int64_t blocks = (T * token_cut(T, q_heads, k_heads, dim) + kHW - 1) / kHW;
  return blocks < kMaxGradParts ? blocks : kMaxGradParts;
}

hipError_t launch_head_norm_rotary_backward(const HeadProblem& p, hipStream_t stream) {
  const int64_t parts = head_grad_parts(p.T, p.set[0].heads, p.set[1].heads, p.dim);
  if (parts > 0) {
    if (p.x_fp32) start_mode<true, float>(p, stream);
    else start_mode<true, uint16_t>(p, stream);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  if (p.norm == kHeadNone || (p.set[0].dw == nullptr && p.set[1].dw == nullptr)) return hipSuccess;
  hipLaunchKernelGGL(head_grad_sum_kernel, dim3((unsigned)((p.dim + 63) / 64), 2), dim3(1024), 0, stream, p.partial,
                     (int)parts, p.dim, p.set[0].dw, p.set[1].dw);
  return hipGetLastError();
}

}  // namespace fp8bs
