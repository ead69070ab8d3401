// The gated feed-forward block's own kernels for gfx950: the product for up to
// 64 tokens, and the backward pass up to the operands of Dgrad and Wgrad.
// (More tokens: the block GEMM with its gated epilogue, gemm.hip.)
//
//   a = X W1^T, u = X W3^T,  h = act(a) u,  act(a) = a logistic(v(a))
//   da = dh u act'(a),  du = dh act(a)
//   act'(a) = z + a z (1 - z) v'(a),  z = logistic(v(a))
#include "device.hpp"
#include "blocks.hpp"
#include "gate.hpp"
#include "rows.hpp"

namespace fp8bs {

namespace {

typedef int gv4i __attribute__((ext_vector_type(4)));
typedef int gv2i __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

// ===========================================================================
// Up to 64 tokens
// ===========================================================================

// 8 E4M3 codes (two dwords) as BF16, exactly
__device__ __forceinline__ v8bf codes_to_bf16(int lo, int hi) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A 128-wide K block of a 16-row operand: a lane's 32 codes (bytes 16 g.. and
// 64 + 16 g.. for lane group g).
struct Block {
  gv4i lo, hi;
};
struct Bf16Block {
  v8bf f[4];
};
__device__ __forceinline__ Bf16Block to_bf16(const Block& b) {
  return Bf16Block{{codes_to_bf16(b.lo[0], b.lo[1]), codes_to_bf16(b.lo[2], b.lo[3]),
                    codes_to_bf16(b.hi[0], b.hi[1]), codes_to_bf16(b.hi[2], b.hi[3])}};
}
__device__ __forceinline__ v4f block_product(const Bf16Block& a, const Bf16Block& b) {
  v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mfma_bf16_16x16x32(a.f[i], b.f[i], c);
  return c;
}

__device__ __forceinline__ float gated(float a, float u, int gelu) {
  return a * logistic(gelu ? gelu_argument(a) : a) * u;
}

// A workgroup has RT tiles of 16 channels, the gate rows and the up rows of
// each, for every token; its PW waves deal the K blocks of its share (`cuts`
// workgroups share a tile's), the next block's weights loaded before the
// present one's products.  The products convert the codes to BF16: exact, with
// FP32 sums.
template <int NT, int RT, int PW>
__global__ __launch_bounds__(PW * 64, 2) void gated_few_kernel(GatedFewProblem p) {
  __shared__ v4f part[PW][RT][2][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int kb_n = (int)(p.K / 128), M = p.M;
  const int cut = blockIdx.x % p.cuts, group = blockIdx.x / p.cuts;
  const int kb0 = (int)((int64_t)kb_n * cut / p.cuts), kb1 = (int)((int64_t)kb_n * (cut + 1) / p.cuts);
  const int tiles = (int)(p.N / 16);
  const uint8_t* w[RT][2];
  const float* s[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int t = min(group * RT + i, tiles - 1);      // past the last one: the last one again, not stored
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      w[i][g] = p.W + ((int64_t)g * tiles + t) * kb_n * 2048 + lane * 16;
      s[i][g] = p.sW + ((int64_t)g * (tiles / 8) + t / 8) * p.ld_sw;
    }
  }
  const uint8_t* x[NT];
  const float* sx[NT];
  v4f acc[RT][2][NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = min(j * 16 + lrow, M - 1);
    x[j] = p.A + t * p.lda + lgrp * 16;
    sx[j] = p.sA + t;
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i][0][j] = acc[i][1][j] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  auto fetch = [&](int kb, Block (&b)[RT][2]) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint8_t* at = w[i][g] + (int64_t)kb * 2048;
        b[i][g] = Block{*reinterpret_cast<const gv4i*>(at), *reinterpret_cast<const gv4i*>(at + 1024)};
      }
  };
  const int last = kb1 - 1;
  auto step = [&](int kb, const Block (&b)[RT][2], Block (&next)[RT][2]) {
    Block xb[NT];
    float c[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint8_t* at = x[j] + kb * 128;
      xb[j] = Block{*reinterpret_cast<const gv4i*>(at), *reinterpret_cast<const gv4i*>(at + 64)};
      c[j] = sx[j][(int64_t)kb * p.ld_sa];
    }
    __asm__ volatile("" ::: "memory");
    fetch(min(kb + PW, last), next);     // past the wave's last block: one that is not used
    Bf16Block xf[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xf[j] = to_bf16(xb[j]);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const Bf16Block wf = to_bf16(b[i][g]);
        const float f = s[i][g][kb];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const v4f q = block_product(wf, xf[j]);
          const float cj = c[j] * f;
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][g][j][v] = __builtin_fmaf(q[v], cj, acc[i][g][j][v]);
        }
      }
  };
  if (kb0 + wave < kb1) {
    Block b0[RT][2], b1[RT][2];
    fetch(kb0 + wave, b0);
    for (int kb = kb0 + wave;; kb += 2 * PW) {
      step(kb, b0, b1);
      if (kb + PW >= kb1) break;
      step(kb + PW, b1, b0);
      if (kb + 2 * PW >= kb1) break;
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if (j != 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      part[wave][i][0][lane] = acc[i][0][j];
      part[wave][i][1][lane] = acc[i][1][j];
    }
    __syncthreads();
    for (int i = wave; i < RT; i += PW) {
      v4f a = part[0][i][0][lane], u = part[0][i][1][lane];
#pragma unroll
      for (int q = 1; q < PW; ++q) {
        a += part[q][i][0][lane];
        u += part[q][i][1][lane];
      }
      const int t = j * 16 + lrow, tile = group * RT + i;
      if (t >= M || tile >= tiles) continue;
      const int64_t n = tile * 16 + lgrp * 4;
      if (p.cuts > 1) {
        float* at = p.parts + ((int64_t)cut * M + t) * 2 * p.N + n;
        *reinterpret_cast<v4f*>(at) = a;
        *reinterpret_cast<v4f*>(at + p.N) = u;
        continue;
      }
      if (p.gated.gate_up != nullptr) {
        uint16_t* at = p.gated.gate_up + t * p.gated.ld_gu + n;
        *reinterpret_cast<v4bf*>(at) = __builtin_convertvector(a, v4bf);
        *reinterpret_cast<v4bf*>(at + p.N) = __builtin_convertvector(u, v4bf);
      }
      v4f h;
#pragma unroll
      for (int v = 0; v < 4; ++v) h[v] = gated(a[v], u[v], p.gated.gelu);
      if (p.gated.q != nullptr) *reinterpret_cast<v4f*>(p.parts + t * p.N + n) = h;
      else if (p.out_fp32) *reinterpret_cast<v4f*>(static_cast<float*>(p.C) + t * p.ldc + n) = h;
      else *reinterpret_cast<v4bf*>(static_cast<uint16_t*>(p.C) + t * p.ldc + n) = __builtin_convertvector(h, v4bf);
    }
  }
}

// What the product's workgroups left: the sums of a cut tile, and the codes
// of h (a 1x128 tile spans eight 16-channel tiles).  16 lanes a tile.
__global__ __launch_bounds__(256) void gated_finish_kernel(GatedFewProblem p) {
  const int kb_n = (int)(p.N / 128), tile = blockIdx.x * 16 + (threadIdx.x >> 4), l16 = threadIdx.x & 15;
  if (tile >= p.M * kb_n) return;                 // whole 16-lane groups
  const int t = tile / kb_n, kb = tile - t * kb_n;
  const int64_t n = kb * 128 + l16 * 8;
  float h[8];
  if (p.cuts > 1) {
    const float* src = p.parts + (int64_t)t * 2 * p.N + n;
    const int64_t step = (int64_t)p.M * 2 * p.N;
    v4f a[2], u[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      a[k] = *reinterpret_cast<const v4f*>(src + 4 * k);
      u[k] = *reinterpret_cast<const v4f*>(src + p.N + 4 * k);
    }
    for (int c = 1; c < p.cuts; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        a[k] += *reinterpret_cast<const v4f*>(src + c * step + 4 * k);
        u[k] += *reinterpret_cast<const v4f*>(src + c * step + p.N + 4 * k);
      }
    if (p.gated.gate_up != nullptr) {
      uint16_t* at = p.gated.gate_up + t * p.gated.ld_gu + n;
      *reinterpret_cast<gv4i*>(at) = gv4i{bf16_pair(a[0][0], a[0][1]), bf16_pair(a[0][2], a[0][3]),
                                          bf16_pair(a[1][0], a[1][1]), bf16_pair(a[1][2], a[1][3])};
      *reinterpret_cast<gv4i*>(at + p.N) = gv4i{bf16_pair(u[0][0], u[0][1]), bf16_pair(u[0][2], u[0][3]),
                                                bf16_pair(u[1][0], u[1][1]), bf16_pair(u[1][2], u[1][3])};
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = gated(a[k >> 2][k & 3], u[k >> 2][k & 3], p.gated.gelu);
  } else {
    const float* src = p.parts + t * p.N + n;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = src[k];
  }
  if (p.gated.q != nullptr) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(h[k]) & 0x7FFFFFFFu);
    float sc;
    const uint2 q = quant8_f32(h, row16_max_u32(m), sc);
    *reinterpret_cast<gv2i*>(p.gated.q + t * p.gated.ldq + n) = gv2i{(int)q.x, (int)q.y};
    if (l16 == 0) p.gated.s[kb * p.gated.ld_s + t] = sc;
  } else if (p.out_fp32) {
    float* at = static_cast<float*>(p.C) + t * p.ldc + n;
    *reinterpret_cast<float4*>(at) = make_float4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<float4*>(at + 4) = make_float4(h[4], h[5], h[6], h[7]);
  } else {
    *reinterpret_cast<gv4i*>(static_cast<uint16_t*>(p.C) + t * p.ldc + n) =
        gv4i{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3]), bf16_pair(h[4], h[5]), bf16_pair(h[6], h[7])};
  }
}

template <int NT, int RT, int PW>
void few(const GatedFewProblem& p, hipStream_t stream) {
  const int64_t tiles = p.N / 16;
  hipLaunchKernelGGL((gated_few_kernel<NT, RT, PW>), dim3((unsigned)((tiles + RT - 1) / RT * p.cuts)), dim3(PW * 64), 0,
                     stream, p);
}

template <int NT>
void few_tiles(const GatedFewProblem& p, hipStream_t stream) {
  if (p.N / 16 * p.cuts <= 512) few<NT, 1, 8>(p, stream);
  else few<NT, 2, 4>(p, stream);
}

// ===========================================================================
// Backward
// ===========================================================================

// quotient y / s of the online rule, as in quant8_f32: r + l = 1 / s
struct ScaleInverse {
  float r, l;
};
// scale of a tile from its |y| maximum's bits; infinite or NaN: r = l = 0 or NaN
__device__ __forceinline__ float tile_scale_f32(uint32_t amax_bits, ScaleInverse& inv) {
  if (amax_bits >= 0x7F800000u) {
    inv.r = inv.l = amax_bits == 0x7F800000u ? 0.0f : NAN;
    return __uint_as_float(amax_bits == 0x7F800000u ? amax_bits : kCanonicalNaN);
  }
  const float s = fmaxf(div448_bf16(__uint_as_float(amax_bits)), scale_floor());
  inv.r = __uint_as_float(__float_as_uint(__builtin_amdgcn_rcpf(s)) - 2u);
  const float e = __builtin_fmaf(-s, inv.r, 1.0f);
  inv.l = inv.r * __builtin_fmaf(e, e, e);
  return s;
}
__device__ __forceinline__ float quotient(float y, const ScaleInverse& i) { return __builtin_fmaf(y, i.r, y * i.l); }

constexpr int kGB = 512, kGW = kGB / 64;   // threads and waves of a workgroup
constexpr int kGR = 4;                     // rows of a lane

// One 128 x 128 block of tokens x channels: dh, gate and up are read once, da
// and du (and h) stay in registers as FP32 for both orientations' codes.  Lane
// (sub, l16) of wave w has rows 16 w + 4 sub .. + 3 and channels 8 l16 .. + 7, so
// that a row tile is one 16-lane DPP row, and four codes of a column one
// dword; the columns' maxima and the transposed codes meet in LDS.  Tokens past
// the last one are zeros, which the transposed codes are padded with.
template <bool kH>
__global__ __launch_bounds__(kGB) void gated_backward_kernel(GatedGradProblem p) {
  constexpr int kSets = kH ? 3 : 2;                          // da, du, h
  __shared__ uint32_t most[kSets][kGW][128];
  __shared__ __attribute__((aligned(16))) float inv[kSets][2][128];
  __shared__ __attribute__((aligned(16))) uint8_t codes[kSets][128 * 128];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane >> 4, l16 = lane & 15;
  const int64_t ncb = p.I / 128, nrb = (p.T + 127) / 128;
  const int64_t rb = blockIdx.x / ncb, cb = blockIdx.x % ncb;
  const int64_t r0 = rb * 128 + wave * 16 + sub * 4, c0 = cb * 128 + l16 * 8;

  float y[kSets][kGR][8];
  {
    gv4i dh[kGR], g[kGR], u[kGR];
#pragma unroll
    for (int i = 0; i < kGR; ++i) {
      dh[i] = g[i] = u[i] = gv4i{0, 0, 0, 0};
      if (r0 + i < p.T) {
        const uint16_t* gu = p.gate_up + (r0 + i) * p.ld_gu + c0;
        dh[i] = __builtin_nontemporal_load(reinterpret_cast<const gv4i*>(p.dh + (r0 + i) * p.ld_dh + c0));
        g[i] = __builtin_nontemporal_load(reinterpret_cast<const gv4i*>(gu));
        u[i] = __builtin_nontemporal_load(reinterpret_cast<const gv4i*>(gu + p.I));
      }
    }
#pragma unroll
    for (int i = 0; i < kGR; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t gw = (uint32_t)g[i][k >> 1], uw = (uint32_t)u[i][k >> 1], dw = (uint32_t)dh[i][k >> 1];
        const float a = (k & 1) ? bf16_hi(gw) : bf16_lo(gw), b = (k & 1) ? bf16_hi(uw) : bf16_lo(uw);
        const float d = (k & 1) ? bf16_hi(dw) : bf16_lo(dw);
        const float z = logistic(p.gelu ? gelu_argument(a) : a);
        const float f = a * z;                               // act(a)
        const float slope = p.gelu ? gelu_argument_slope(a) : 1.0f;
        y[0][i][k] = d * b * __builtin_fmaf(f * (1.0f - z), slope, z);
        y[1][i][k] = d * f;
        if constexpr (kH) y[2][i][k] = f * b;
      }
  }

  // row tiles, from registers
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int64_t col = m * p.I + c0;
    if (p.d != nullptr) {
#pragma unroll
      for (int i = 0; i < kGR; ++i)
        if (r0 + i < p.T) {
          const float* v = y[m][i];
          __builtin_nontemporal_store(gv4i{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])},
                                      reinterpret_cast<gv4i*>(p.d + (r0 + i) * p.ld_d + col));
        }
    }
    if (p.q != nullptr) {
#pragma unroll
      for (int i = 0; i < kGR; ++i) {
        uint32_t t = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) t = max(t, __float_as_uint(y[m][i][k]) & 0x7FFFFFFFu);
        float s;
        const uint2 q = quant8_f32(y[m][i], row16_max_u32(t), s);
        if (r0 + i < p.T) {
          __builtin_nontemporal_store(gv2i{(int)q.x, (int)q.y}, reinterpret_cast<gv2i*>(p.q + (r0 + i) * p.ldq + col));
          if (l16 == 0) p.s[(m * ncb + cb) * p.ld_s + r0 + i] = s;
        }
      }
    }
  }
  if (p.qt == nullptr && !kH) return;

  // column tiles: their maxima over the waves
#pragma unroll
  for (int m = 0; m < kSets; ++m) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < kGR; ++i) t = max(t, __float_as_uint(y[m][i][k]) & 0x7FFFFFFFu);
      const auto a = __builtin_amdgcn_permlane16_swap(t, t, false, false);
      t = max(a[0], a[1]);
      const auto b = __builtin_amdgcn_permlane32_swap(t, t, false, false);
      t = max(b[0], b[1]);
      if (sub == 0) most[m][wave][l16 * 8 + k] = t;
    }
  }
  __syncthreads();
  if (threadIdx.x < kSets * 128) {
    const int m = threadIdx.x >> 7, c = threadIdx.x & 127;
    uint32_t t = most[m][0][c];
#pragma unroll
    for (int w = 1; w < kGW; ++w) t = max(t, most[m][w][c]);
    ScaleInverse v;
    const float s = tile_scale_f32(t, v);
    inv[m][0][c] = v.r;
    inv[m][1][c] = v.l;
    if (m == 2) p.hst[rb * p.ld_hst + cb * 128 + c] = s;
    else if (p.qt != nullptr) p.st[rb * p.ld_st + m * p.I + cb * 128 + c] = s;
  }
  __syncthreads();
  // codes: column c's 128 bytes (tokens) at c * 128, 16-byte chunks XOR-swizzled by c / 8
#pragma unroll
  for (int m = 0; m < kSets; ++m) {
    float r[8], l[8];
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const v4f a = *reinterpret_cast<const v4f*>(&inv[m][0][l16 * 8 + k]);
      const v4f b = *reinterpret_cast<const v4f*>(&inv[m][1][l16 * 8 + k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r[k + e] = a[e];
        l[k + e] = b[e];
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const ScaleInverse v{r[k], l[k]};
      float q[4];
#pragma unroll
      for (int i = 0; i < kGR; ++i) q[i] = quotient(y[m][i][k], v);
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
      if (!(r[k] > 0.0f)) w = (int)pack4_sat_nan(q[0], q[1], q[2], q[3]);   // an infinite or NaN scale
      *reinterpret_cast<uint32_t*>(&codes[m][(l16 * 8 + k) * 128 + ((wave ^ (l16 & 7)) << 4) + sub * 4]) = (uint32_t)w;
    }
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    if (p.qt == nullptr) break;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = i * kGB + threadIdx.x, c = at >> 3, ch = at & 7;
      const gv4i v = *reinterpret_cast<const gv4i*>(&codes[m][c * 128 + ((ch ^ ((c >> 3) & 7)) << 4)]);
      __builtin_nontemporal_store(v, reinterpret_cast<gv4i*>(p.qt + (m * p.I + cb * 128 + c) * p.ldqt + rb * 128 + ch * 16));
    }
  }
  if constexpr (kH) {
    // operand tiles: 16 columns x 128 tokens are 2 KB, lane 16 g + c of half h: tokens 64 h + 16 g ..
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = i * kGB + threadIdx.x, c = (at >> 7) * 16 + (at & 15), ch = (at >> 4) & 7;
      const gv4i v = *reinterpret_cast<const gv4i*>(&codes[2][c * 128 + ((ch ^ ((c >> 3) & 7)) << 4)]);
      uint8_t* tile = p.ht + ((cb * 8 + (at >> 7)) * nrb + rb) * 2048;
      __builtin_nontemporal_store(v, reinterpret_cast<gv4i*>(tile + (at & 127) * 16));
    }
  }
}

}  // namespace

int gated_few_cuts(int64_t N, int64_t K) {
  const int64_t tiles = N / 16, kb = K / 128;
  int64_t c = (256 + tiles - 1) / tiles;
  if (c > kGatedMaxCuts) c = kGatedMaxCuts;
  if (c > kb) c = kb;
  return (int)c;
}

hipError_t launch_gated_few(const GatedFewProblem& p, hipStream_t stream) {
  switch ((p.M + 15) / 16) {
    case 1: few_tiles<1>(p, stream); break;
    case 2: few_tiles<2>(p, stream); break;
    case 3: few_tiles<3>(p, stream); break;
    default: few_tiles<4>(p, stream); break;
  }
  if (p.cuts > 1 || p.gated.q != nullptr) {
    const int64_t groups = p.M * (p.N / 128);
    hipLaunchKernelGGL(gated_finish_kernel, dim3((unsigned)((groups + 15) / 16)), dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}

hipError_t launch_gated_backward(const GatedGradProblem& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + 127) / 128 * (p.I / 128)));
  if (p.ht != nullptr) hipLaunchKernelGGL(gated_backward_kernel<true>, grid, dim3(kGB), 0, stream, p);
  else hipLaunchKernelGGL(gated_backward_kernel<false>, grid, dim3(kGB), 0, stream, p);
  return hipGetLastError();
}

}  // namespace fp8bs
