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
// Bound by memory: every head is read once and written once (8192 tokens of 64 + 8 heads of
// 128, BF16, nothing cached: forward 62 us, 302 MB; a copy of as much 57; without norm and
// rotation the same).  A head lives in
// the registers of G lanes, R pairs a lane (8, or 4: run_of()): both elements of a pair meet in one
// lane for either order of pairs, so the rotation moves nothing between lanes,
// and the lane's R angles serve all heads of the token.  A wave works on 64 / G
// heads of one token at a time, queries first and then keys.
#include "block_rules.hpp"
#include "blocks.hpp"
#include "device.hpp"
#include "rows.hpp"

namespace fp8bs {

namespace {

constexpr int kHB = kHW * 64;               // threads of a workgroup

typedef int hv4i __attribute__((ext_vector_type(4)));
typedef int hv2i __attribute__((ext_vector_type(2)));

// A lane's 2 R elements of a head as loaded: BF16 stays packed until it is used, so that
// the next head's loads take few registers.
template <typename T, int R>
struct Raw {
  static constexpr int kWords = R * (int)sizeof(T) / 4;   // dwords of a run
  int d[2 * kWords];                                      // two runs of R elements
};

// How a lane's 2 R elements of a head lie: two runs of R, neighbouring lanes' side by side,
// moved in whole accesses: R l .. and rot / 2 + R l .. with pairs (k, R + k) for halves (the
// channels that do not rotate likewise as two halves), R l .. and D / 2 + R l .. with pairs
// (2 k, 2 k + 1) for adjacent ones; or (kScalar)
// element by element, pairs (k, R + k), for heads that are not 16-byte aligned or
// whose size or rotated part is no multiple of 16 (us, forward and backward, inputs in the last-level cache:
// BF16, 8192 tokens of 32 + 8 heads of 80 22 and 40, with 40 of 80 channels rotating, in this mode, 59 and 92; of
// 72, in this mode, 54 and 95; FP32, 5003 tokens of 16 + 16 heads of 80 21 and 32, with 40
// rotating 26 and 44).
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

template <int kMode, int G, int R>
struct Lane {
  int l, dim, half_rot;        // lane of the head, head size, rotated pairs
  int adjacent;
  // element of register v (0 .. 2 R - 1); past the head's end: >= dim
  __device__ __forceinline__ int element(int v) const {
    if constexpr (kMode == kAdjacent) return (v < R ? 0 : dim / 2 - R) + l * R + v;
    if constexpr (kMode == kHalves) {
      if (R * l < half_rot) return v < R ? l * R + v : half_rot + l * R + v - R;
      return 2 * half_rot + l * R - half_rot + (v < R ? v : dim / 2 - half_rot + v - R);
    }
    const int i = pair(v % R), second = v / R;
    if (2 * i >= dim) return dim;
    if (!adjacent && i < half_rot) return i + second * half_rot;
    return 2 * i + second;
  }
  __device__ __forceinline__ int pair(int k) const {
    if constexpr (kMode == kAdjacent) return (k < R / 2 ? 0 : dim / 4 - R / 2) + l * (R / 2) + k;
    return kMode == kScalar ? k * G + l : l * R + k;
  }
  __device__ __forceinline__ bool on() const { return kMode == kScalar ? true : l * 2 * R < dim; }
  static __device__ __forceinline__ int first(int k) { return kMode == kAdjacent ? 2 * k : k; }
  static __device__ __forceinline__ int second(int k) { return kMode == kAdjacent ? 2 * k + 1 : R + k; }

  // asks for a head; lanes past its end get zeros
  template <typename T>
  __device__ __forceinline__ void fetch(const T* p, Raw<T, R>& r) const {
    constexpr int kWords = Raw<T, R>::kWords;
    if constexpr (kMode == kScalar) {
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) {
        const int e = element(k);
        const T v = e < dim ? p[e] : T(0);
        if constexpr (sizeof(T) == 4) r.d[k] = __builtin_bit_cast(int, v);
        else if (k & 1) r.d[k / 2] |= (int)((uint32_t)v << 16);
        else r.d[k / 2] = (int)(uint32_t)v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * kWords; ++i) r.d[i] = 0;
      if (!on()) return;
#pragma unroll
      for (int run = 0; run < 2; ++run) {
        const T* q = p + element(run * R);
        if constexpr (kWords == 2) {
          const hv2i v = *reinterpret_cast<const hv2i*>(q);
          r.d[run * 2] = v[0];
          r.d[run * 2 + 1] = v[1];
        } else {
#pragma unroll
          for (int i = 0; i < kWords; i += 4) {
            const hv4i v = *reinterpret_cast<const hv4i*>(q + i * 4 / (int)sizeof(T));
#pragma unroll
            for (int k = 0; k < 4; ++k) r.d[run * kWords + i + k] = v[k];
          }
        }
      }
    }
  }
  template <typename T>
  static __device__ __forceinline__ void unpack(const Raw<T, R>& r, float (&v)[2 * R]) {
#pragma unroll
    for (int k = 0; k < 2 * R; ++k) {
      if constexpr (sizeof(T) == 4) v[k] = __int_as_float(r.d[k]);
      else v[k] = (k & 1) ? bf16_hi((uint32_t)r.d[k / 2]) : bf16_lo((uint32_t)r.d[k / 2]);
    }
  }
  template <bool kStream, typename T>
  __device__ __forceinline__ void store(T* p, const float (&v)[2 * R]) const {
    constexpr int kWords = Raw<T, R>::kWords;
    if constexpr (kMode == kScalar) {
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) {
        const int e = element(k);
        if (e >= dim) continue;
        if constexpr (sizeof(T) == 2) p[e] = __builtin_bit_cast(uint16_t, (__bf16)v[k]);
        else p[e] = v[k];
      }
    } else {
      if (!on()) return;
#pragma unroll
      for (int run = 0; run < 2; ++run) {
        T* q = p + element(run * R);
        int d[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          if constexpr (sizeof(T) == 4) d[i] = __float_as_int(v[run * R + i]);
          else d[i] = bf16_pair(v[run * R + 2 * i], v[run * R + 2 * i + 1]);
        }
        if constexpr (kWords == 2) {
          if constexpr (kStream) __builtin_nontemporal_store(hv2i{d[0], d[1]}, reinterpret_cast<hv2i*>(q));
          else *reinterpret_cast<hv2i*>(q) = hv2i{d[0], d[1]};
        } else {
#pragma unroll
          for (int i = 0; i < kWords; i += 4) {
            const hv4i v = {d[i], d[i + 1], d[i + 2], d[i + 3]};
            hv4i* at = reinterpret_cast<hv4i*>(q + i * 4 / (int)sizeof(T));
            if constexpr (kStream) __builtin_nontemporal_store(v, at);
            else *at = v;
          }
        }
      }
    }
  }

  // The lane's elements of a weight in LDS.
  __device__ __forceinline__ void weight(const float* w, float (&v)[2 * R]) const {
    if constexpr (kMode == kScalar) {
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) v[k] = w[min(element(k), dim - 1)];
    } else {
#pragma unroll
      for (int k = 0; k < 2 * R; k += 4) {
        const float4 a = *reinterpret_cast<const float4*>(w + (on() ? element(k) : 0));
        v[k] = a.x; v[k + 1] = a.y; v[k + 2] = a.z; v[k + 3] = a.w;
      }
    }
  }

  // cos and sin of the lane's pairs at token t (pairs that do not rotate: whatever).  The
  // wave's lanes form the token's angles once between them and share them through
  // `shared` (one pair of floats for each rotated pair): each lane for itself, 64 / G
  // times over, cost 20000 tokens of 16 + 4 heads of
  // 64 38 us for 32 (with the walk below).
  __device__ __forceinline__ void angles(const HeadProblem& p, int64_t t, float2* shared, float (&c)[R], float (&s)[R]) const {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      c[k] = 1.f;
      s[k] = 0.f;
    }
    if (half_rot == 0) return;
    auto position = [&](int64_t at) {
      return p.pos64 ? (double)static_cast<const int64_t*>(p.positions)[at] : (double)static_cast<const int32_t*>(p.positions)[at];
    };
    const double pos0 = p.axes == 1 ? position(t) : 0.0;
    order();                           // the token before: its angles have been read
    for (int i = threadIdx.x & 63; i < half_rot; i += 64) {
      double pos = pos0;
      if (p.axes > 1) {
        int axis = 0;
#pragma unroll
        for (int a = 0; a + 1 < kHeadMaxAxes; ++a) axis += i >= p.section_end[a] && a + 1 < p.axes ? 1 : 0;
        pos = position(t * p.axes + axis);
      }
      float2 cs;
      rotation(pos, p.freq[i], cs.x, cs.y);
      shared[i] = cs;
    }
    order();
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float2 cs = shared[min(pair(k), half_rot - 1)];
      c[k] = cs.x;
      s[k] = cs.y;
    }
  }
  // Within a wave LDS accesses happen in the order of its instructions: this keeps the
  // compiler from moving them.
  static __device__ __forceinline__ void order() {
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    __asm__ volatile("" ::: "memory");
  }
  // rotates the pairs by the angles (kBack: against them); pairs that do not
  // rotate are left alone, infinities and NaN included
  template <bool kBack>
  __device__ __forceinline__ void rotate(float (&v)[2 * R], const float (&c)[R], const float (&s)[R]) const {
    auto turn = [&](int k) {
      const float a = v[first(k)], b = v[second(k)], sn = kBack ? -s[k] : s[k];
      v[first(k)] = __builtin_fmaf(a, c[k], -(b * sn));
      v[second(k)] = __builtin_fmaf(b, c[k], a * sn);
    };
    if constexpr (kMode == kScalar) {
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (pair(k) < half_rot) turn(k);
    } else if constexpr (kMode == kAdjacent) {      // a run rotates or not (rot % 16 == 0)
      if (pair(0) < half_rot) {
#pragma unroll
        for (int k = 0; k < R / 2; ++k) turn(k);
      }
      if (pair(R / 2) < half_rot) {
#pragma unroll
        for (int k = R / 2; k < R; ++k) turn(k);
      }
    } else if (l * R < half_rot) {
#pragma unroll
      for (int k = 0; k < R; ++k) turn(k);
    }
  }
  // x becomes xhat; returns rstd
  __device__ __forceinline__ float normalize(float (&x)[2 * R], int norm, float eps) const {
    const float d = (float)dim, inv_d = 1.0f / d;
    if (norm == kHeadLayer) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) sum += x[k];
      sum = lanes_sum<G>(sum);
      // sum / D with one correction (where it is finite): a head of one value keeps that value as its mean
      float mean = sum * inv_d;
      if (fabsf(mean) < INFINITY) mean = __builtin_fmaf(__builtin_fmaf(-mean, d, sum), inv_d, mean);
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) x[k] = (kMode == kScalar ? element(k) < dim : on()) ? x[k] - mean : 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 2 * R; ++k) ss = __builtin_fmaf(x[k], x[k], ss);
    const float rstd = rsqrt_refined(lanes_sum<G>(ss) * inv_d + eps);
#pragma unroll
    for (int k = 0; k < 2 * R; ++k) x[k] *= rstd;
    return rstd;
  }
};

// A weight into LDS as FP32 (null: ones), by the workgroup; a barrier publishes it.
__device__ __forceinline__ void stage_weight(const void* w, int is_f32, int dim, float* to) {
  for (int e = threadIdx.x; e < dim; e += kHB)
    to[e] = w == nullptr ? 1.f : is_f32 ? static_cast<const float*>(w)[e] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(w)[e] << 16);
}
// Barrier that waits for LDS alone: the loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));   // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}

// A wave's walk over its units: token, unit of the token, pass.
struct Walk {
  int64_t t;
  int cut, pass, end;
  int dt, dc;             // a step of all waves, in tokens and units
  Shares sh;
  int n;                  // passes of a token
  __device__ __forceinline__ Walk(const Shares& s, int n_, int block) : sh(s), n(n_) {
    const uint32_t first = (uint32_t)block * kHW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t all = (uint32_t)s.blocks * kHW, cuts = (uint32_t)s.cuts;
    t = first / cuts;
    cut = (int)(first - (uint32_t)t * cuts);
    dt = (int)(all / cuts);
    dc = (int)(all - (uint32_t)dt * cuts);
    open();
  }
  __device__ __forceinline__ void open() {
    pass = cut * sh.per;
    end = min(pass + sh.per, n);
  }
  __device__ __forceinline__ bool fresh() const { return pass == cut * sh.per; }     // a unit begins
  __device__ __forceinline__ void next() {
    if (++pass < end) return;
    t += dt;
    cut += dc;
    if (cut >= sh.cuts) {
      cut -= sh.cuts;
      ++t;
    }
    open();
  }
};
// Forward.  A wave walks over tokens with its share of their heads, queries and then
// keys; the heads of its next two passes are in flight, across tokens too.  FP32 results
// are stored past the caches (5003 x 16 + 16 heads of 80: 27.6 us for 29.5; BF16: no
// difference).
template <typename T, int kMode, int G, int R>
__global__ __launch_bounds__(kHB) void head_norm_rotary_kernel(HeadProblem p, Shares sh) {
  __shared__ float2 turn[kHW][G * R];
  __shared__ __attribute__((aligned(16))) float w[2][2 * R * G];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), slot = lane / G;
  const Lane<kMode, G, R> me{lane % G, p.dim, p.rot / 2, p.adjacent};
  const int nq = passes(p.set[0].heads, G), n = nq + passes(p.set[1].heads, G);
  // what pass `pass` of token t is about: its set, and the lane's head of it
  auto head_of = [&](int pass) { return (int64_t)(pass < nq ? pass : pass - nq) * (64 / G) + slot; };
  auto fetch = [&](int64_t t, int pass, Raw<T, R>& r) {      // past the last head: that one again, not stored
    const HeadSet& hs = p.set[pass >= nq];
    me.fetch(static_cast<const T*>(hs.x) + t * hs.ld_token + min(head_of(pass), hs.heads - 1) * hs.ld_head, r);
  };
  Walk at(sh, n, (int)blockIdx.x), ahead = at;      // the pass at hand, the next to ask for
  Raw<T, R> r0, r1;
  if (ahead.t < p.T) fetch(ahead.t, ahead.pass, r0);
  ahead.next();
  if (ahead.t < p.T) fetch(ahead.t, ahead.pass, r1);
  ahead.next();
  if (p.norm != kHeadNone) {
    stage_weight(p.set[0].w, p.w_fp32, p.dim, w[0]);
    stage_weight(p.set[1].w, p.w_fp32, p.dim, w[1]);
    lds_barrier();
  }
  float c[R], s[R];
#pragma unroll 1
  while (at.t < p.T) {
    if (at.fresh()) me.angles(p, at.t, turn[wave], c, s);
    const int which = at.pass >= nq;
    float v[2 * R];
    me.unpack(r0, v);
    r0 = r1;
    if (ahead.t < p.T) fetch(ahead.t, ahead.pass, r1);
    ahead.next();
    if (p.norm != kHeadNone) {
      me.normalize(v, p.norm, p.eps);
      float wv[2 * R];
      me.weight(w[which], wv);
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) v[k] *= wv[k];
    }
    me.template rotate<false>(v, c, s);
    const HeadSet& hs = p.set[which];
    const int64_t h = head_of(at.pass);
    if (h < hs.heads) me.template store<sizeof(T) == 4>(static_cast<T*>(hs.y) + at.t * hs.ldy_token + h * hs.ldy_head, v);
    at.next();
  }
}

// Backward.  A workgroup has one set, and one share of its heads; its waves walk over
// tokens, the next heads' loads in flight, across tokens too.  (Both sets in a
// workgroup would hold twice the sums in registers: 76 us for 71 with 16 elements a
// lane.)  A lane keeps its elements' sums for the weight, a workgroup's meet in LDS at
// the end, and the workgroups' sums are added by a second launch, all in a fixed order.
template <typename T, int kMode, int G, int R>
__global__ __launch_bounds__(kHB) void head_norm_rotary_backward_kernel(HeadProblem p, GradGrid grid) {
  __shared__ float2 turn[kHW][G * R];
  __shared__ __attribute__((aligned(16))) float w[2 * R * G];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), slot = lane / G;
  const Lane<kMode, G, R> me{lane % G, p.dim, p.rot / 2, p.adjacent};
  const int queries = grid.set[0].blocks, which = (int)blockIdx.x >= queries;
  const Shares sh = grid.set[which];
  const HeadSet& hs = p.set[which];
  const float inv_d = 1.0f / (float)p.dim;
  const bool normed = p.norm != kHeadNone;
  Raw<T, R> rd, rx;
  auto fetch = [&](int64_t t, int pass) {      // past the last head: that one again, not used
    const int64_t h = min((int64_t)pass * (64 / G) + slot, hs.heads - 1);
    me.fetch(static_cast<const T*>(hs.dy) + t * hs.lddy_token + h * hs.lddy_head, rd);
    if (normed) me.fetch(static_cast<const T*>(hs.x) + t * hs.ld_token + h * hs.ld_head, rx);
  };
  Walk at(sh, passes(hs.heads, G), (int)blockIdx.x - which * queries);
  if (at.t < p.T) fetch(at.t, at.pass);
  if (normed) {
    stage_weight(hs.w, p.w_fp32, p.dim, w);
    lds_barrier();
  }
  float dw[2 * R], c[R], s[R];
#pragma unroll
  for (int k = 0; k < 2 * R; ++k) dw[k] = 0.f;
#pragma unroll 1
  while (at.t < p.T) {
    if (at.fresh()) me.angles(p, at.t, turn[wave], c, s);
    const int64_t h = (int64_t)at.pass * (64 / G) + slot, now = at.t;
    const bool on = h < hs.heads;
    float d[2 * R], xh[2 * R];
    me.unpack(rd, d);
    me.unpack(rx, xh);
    at.next();
    if (at.t < p.T) fetch(at.t, at.pass);
    me.template rotate<true>(d, c, s);
    if (normed) {
      const float rstd = me.normalize(xh, p.norm, p.eps);
      if (on) {
#pragma unroll
        for (int k = 0; k < 2 * R; ++k) dw[k] = __builtin_fmaf(d[k], xh[k], dw[k]);
      }
      float wv[2 * R];
      me.weight(w, wv);
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) {
        d[k] *= wv[k];
        s1 += d[k];
        s2 = __builtin_fmaf(d[k], xh[k], s2);
      }
      const float c1 = p.norm == kHeadLayer ? lanes_sum<G>(s1) * inv_d : 0.f, c2 = lanes_sum<G>(s2) * inv_d;
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) d[k] = rstd * (d[k] - c1 - xh[k] * c2);
    }
    if (on) me.template store<true>(static_cast<T*>(hs.y) + now * hs.ldy_token + h * hs.ldy_head, d);
  }
  if (!normed) return;
  // the workgroup's share of the weight's gradient: its lane groups in order
  __shared__ float sum[kHB / G][2 * R * G];
#pragma unroll
  for (int k = 0; k < 2 * R; ++k) {
    const int e = me.element(k);
    if (me.on() && e < p.dim) sum[threadIdx.x / G][e] = dw[k];
  }
  __syncthreads();
  float* out = p.partial + (int64_t)blockIdx.x * p.dim;
  for (int e = threadIdx.x; e < p.dim; e += kHB) {
    float v = sum[0][e];
    for (int g = 1; g < kHB / G; ++g) v += sum[g][e];
    out[e] = v;
  }
}

// The workgroups' shares added up: 16 columns x 64 slices of the shares a workgroup (of
// 64 columns, a head of 128 would be read by two CUs a set: 5.9 us), blockIdx.y = 0 for
// queries and 1 for keys.
__global__ __launch_bounds__(1024) void head_grad_sum_kernel(const float* __restrict__ partial, int parts_q, int parts_k,
                                                             int dim, float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sum[64][17];
  const int l = threadIdx.x & 15, sl = threadIdx.x >> 4, e = blockIdx.x * 16 + l;
  float* out = blockIdx.y == 0 ? dwq : dwk;
  if (out == nullptr) return;
  if (blockIdx.y != 0) partial += (int64_t)parts_q * dim;
  const int parts = blockIdx.y == 0 ? parts_q : parts_k;
  float t = 0.f;
  if (e < dim) {
    float v[kMaxGradParts / 64];
#pragma unroll
    for (int k = 0; k < kMaxGradParts / 64; ++k) {
      const int q = sl + 64 * k;
      v[k] = q < parts ? partial[(int64_t)q * dim + e] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kMaxGradParts / 64; ++k) t += v[k];
  }
  sum[sl][l] = t;
  __syncthreads();
  if (sl == 0 && e < dim) {
    for (int k = 1; k < 64; ++k) t += sum[k][l];
    out[e] = t;
  }
}

// heads of a set that all start 16-byte aligned (a stride that no step is taken along does not count)
bool aligned_heads(const void* p, int64_t T, int64_t heads, int64_t ld_token, int64_t ld_head, int64_t esz) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (T == 1 || (ld_token * esz) % 16 == 0) && (heads == 1 || (ld_head * esz) % 16 == 0);
}

template <bool kBack, typename T, int kMode, int G, int R>
void start(const HeadProblem& p, hipStream_t stream) {
  if constexpr (kBack) {
    const GradGrid g = divide(p.T, p.set[0].heads, p.set[1].heads, p.dim);
    const int64_t parts = g.set[0].blocks + g.set[1].blocks;
    hipLaunchKernelGGL((head_norm_rotary_backward_kernel<T, kMode, G, R>), dim3((unsigned)parts), dim3(kHB), 0, stream, p, g);
  } else {
    const Shares sh = forward_shares(p.T, p.set[0].heads, p.set[1].heads, p.dim, p.x_fp32);
    hipLaunchKernelGGL((head_norm_rotary_kernel<T, kMode, G, R>), dim3((unsigned)sh.blocks), dim3(kHB), 0, stream, p, sh);
  }
}
template <bool kBack, typename T, int kMode>
void start_dim(const HeadProblem& p, hipStream_t stream) {
  if constexpr (kBack || sizeof(T) == 4) {
    if (run_of(kBack, sizeof(T) == 4, p.dim) == 4) {
      switch (lanes_of(p.dim, 4)) {
        case 4: return start<kBack, T, kMode, 4, 4>(p, stream);
        case 8: return start<kBack, T, kMode, 8, 4>(p, stream);
        case 16: return start<kBack, T, kMode, 16, 4>(p, stream);
        case 32: return start<kBack, T, kMode, 32, 4>(p, stream);
        default: return start<kBack, T, kMode, 64, 4>(p, stream);
      }
    }
    return start<kBack, T, kMode, 64, 8>(p, stream);
  } else {
    switch (lanes_of(p.dim, 8)) {
      case 4: return start<kBack, T, kMode, 4, 8>(p, stream);
      case 8: return start<kBack, T, kMode, 8, 8>(p, stream);
      case 16: return start<kBack, T, kMode, 16, 8>(p, stream);
      case 32: return start<kBack, T, kMode, 32, 8>(p, stream);
      default: return start<kBack, T, kMode, 64, 8>(p, stream);
    }
  }
}
template <bool kBack, typename T>
void start_mode(const HeadProblem& p, hipStream_t stream) {
  bool vec = p.dim % 16 == 0 && p.rot % 16 == 0;
  for (const HeadSet& h : p.set) {
    if (h.heads == 0) continue;
    vec = vec && aligned_heads(h.y, p.T, h.heads, h.ldy_token, h.ldy_head, sizeof(T)) &&
          (h.x == nullptr || aligned_heads(h.x, p.T, h.heads, h.ld_token, h.ld_head, sizeof(T))) &&
          (!kBack || aligned_heads(h.dy, p.T, h.heads, h.lddy_token, h.lddy_head, sizeof(T)));
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
  const GradGrid g = divide(T, q_heads, k_heads, dim);
  return g.set[0].blocks + g.set[1].blocks;
}

hipError_t launch_head_norm_rotary_backward(const HeadProblem& p, hipStream_t stream) {
  if (p.T > 0) {
    if (p.x_fp32) start_mode<true, float>(p, stream);
    else start_mode<true, uint16_t>(p, stream);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  if (p.norm == kHeadNone || (p.set[0].dw == nullptr && p.set[1].dw == nullptr)) return hipSuccess;
  const GradGrid g = divide(p.T, p.set[0].heads, p.set[1].heads, p.dim);
  hipLaunchKernelGGL(head_grad_sum_kernel, dim3((unsigned)((p.dim + 15) / 16), 2), dim3(1024), 0, stream, p.partial,
                     g.set[0].blocks, g.set[1].blocks, p.dim, p.set[0].dw, p.set[1].dw);
  return hipGetLastError();
}

}  // namespace fp8bs
