// E4M3 quantisation with one fp32 scale per 128 consecutive elements of a row
// (activations) or per 128 x 128 block (weights).
//
//   s = fp32(max|block| / 448), at least 2^-126; 1 for a block of zeros
//   code = the E4M3 value nearest to x / s, ties to the even code
// The quotient is rounded once: fp32 arithmetic decides every element whose
// quotient is not within a few ulp of the middle of two codes, and the others are
// settled by the exact sign of the division's remainder.  A block that holds a
// NaN or an infinity gets the scale NaN and zero codes, so that products with it
// are NaN.
//
// Sources of a row: bf16 or fp32 rows (optionally gathered: row r from row
// token_of_row[r]), the experts' gated unit of a [gate | up] row (never stored:
// the unit's fp32 value is quantised directly), or that unit's gradient.
#include "common.cuh"
#include "moe_internal.h"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBlk = 128;
constexpr float kE4m3Max = 448.f;

struct BlockScale {
  float s, inv;
};

// amax is the block's maximum magnitude, NaN or infinite if an element is.
__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale b;
  if (!(amax < INFINITY)) {
    b.s = __int_as_float(0x7fffffff);
    b.inv = 0.f;
    return b;
  }
  b.s = amax > 0.f ? fmaxf(__fdiv_rn(amax, kE4m3Max), 1.17549435e-38f) : 1.f;
  b.inv = __frcp_rn(b.s);
  return b;
}

// The quotient x / s, moved off the middle of two codes to the side where the
// exact quotient lies.  q is the correctly rounded quotient, on the exact one's
// side of every fp32 value except itself; middles of codes have 19 zero bits, and
// there the remainder x - q s (exact in one fused operation, after both are
// scaled by a power of two so that it cannot underflow) tells the side.
__device__ __noinline__ float quotient_exact(float x, float s) {
  const float f = __int_as_float(0x7f000000 - (__float_as_int(s) & 0x7f800000));   // 2^-floor(log2 s)
  s *= f;
  x *= f;
  float q = __fdiv_rn(x, s);
  if ((__float_as_uint(q) & 0x7FFFFu) == 0 && q != 0.f) {
    const float r = fmaf(-q, s, x);
    if (r != 0.f) {
      const bool away = (r > 0.f) == (q > 0.f);   // the exact quotient is larger in magnitude
      q = __int_as_float(__float_as_int(q) + (away ? 1 : -1));
    }
  }
  return q;
}

// x * inv is within two ulp of x / s.  Codes have 3 mantissa bits, so the middle
// of two normal codes has fp32 mantissa bits 1000...0 below them (20 low bits);
// below 2^-6 the codes are multiples of 2^-9, which adding 2^-6 brings to the same
// bits.  Anything within 4 ulp of a middle takes the exact way.
__device__ __forceinline__ float code_quotient(float x, const BlockScale& b) {
  const float q = __fmul_rn(x, b.inv);
  float y = fabsf(q);
  if (y < 0.015625f) y += 0.015625f;
  const uint32_t d = (__float_as_uint(y) - 0x80000u + 4u) & 0xFFFFFu;
  return d <= 8u ? quotient_exact(x, b.s) : q;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], const BlockScale& b) {
  if (b.inv == 0.f) return make_uint2(0, 0);   // scale NaN: zero codes
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = code_quotient(v[i], b);
  return make_uint2(e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16), e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16));
}

// Maximum magnitude with NaN kept (as a bit pattern above infinity's).
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ float half_warp_max(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
  return __uint_as_float(m);
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(w[j]);
    v[2 * j + 1] = bf16_hi(w[j]);
  }
}

// The gated unit and its derivatives in fp32 (expf and the approximate division,
// about 3 ulp: the code's rounding is 2^-4).
//   SwiGLU    h = a(g) b(u), a = silu(min(g, cg)), b = clamp(u, -cu, cu)
//   SiTU-GLU  a = bg tanh(g / bg) sigmoid(g), b = bu tanh(u / bu)
// sigma = 1 / (1 + e), 1 - sigma = e sigma with e = e^-g held finite so
// that neither product meets infinity times zero.
__device__ __forceinline__ void glu_parts(float g, float u, const QuantArgs& a, bool grad, float& av, float& bv,
                                          float& da, float& db) {
  if (a.act == MOE_ACT_SITU_GLU) {
    const float e = expf(fminf(-g, 88.f));
    const float sg = __fdividef(1.f, 1.f + e);
    const float tg = tanhf(__fdiv_rn(g, a.beta_g)), tu = tanhf(__fdiv_rn(u, a.beta_u));
    av = a.beta_g * tg * sg;
    bv = a.beta_u * tu;
    if (grad) {
      da = (1.f - tg * tg) * sg + a.beta_g * tg * sg * (e * sg);
      db = 1.f - tu * tu;
    }
  } else {
    const float gc = fminf(g, a.gate_clamp);
    const float e = expf(fminf(-gc, 88.f));
    const float sg = __fdividef(1.f, 1.f + e);
    av = gc * sg;
    bv = fminf(fmaxf(u, -a.up_clamp), a.up_clamp);
    if (grad) {
      // A clamped value has no gradient; one at its bound has.
      da = g <= a.gate_clamp ? sg * (1.f + gc * (e * sg)) : 0.f;
      db = (u >= -a.up_clamp && u <= a.up_clamp) ? 1.f : 0.f;
    }
  }
  // fminf and fmaxf drop a NaN: keep it.
  if (isnan(g)) av = da = g;
  if (isnan(u)) bv = db = u;
}

// Block of 256 threads = 16 half-warps, each on one row; a half-warp takes a
// block of 128 columns (8 a lane, one 16-byte load of bf16), kUnroll of them at a
// time so that their loads are in flight together.
// Bound by memory: every element is read once and its code written once.
constexpr int kRowsPerCta = 16;
constexpr int kUnroll = 2;

template <int KIND>
__global__ void __launch_bounds__(256) k_quant_blocks(const QuantArgs a) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x * kRowsPerCta + (threadIdx.x >> 4);
  const int hl = threadIdx.x & 15;
  int limit = a.R;
  if (a.n_rows != nullptr) limit = min(limit, *a.n_rows);
  long long src = r;
  bool live = r < limit;
  if (live && a.token_of_row != nullptr) {
    src = a.token_of_row[r];
    live = src >= 0 && src < a.src_rows;
  }
  const int nkb = (a.K + kBlk - 1) / kBlk;
  const size_t row = static_cast<size_t>(src) * static_cast<size_t>(a.ld);
  const int per_y = (nkb + gridDim.y - 1) / gridDim.y;
  const int kb1 = min(nkb, static_cast<int>(blockIdx.y + 1) * per_y);
  for (int kb0 = blockIdx.y * per_y; kb0 < kb1; kb0 += kUnroll) {
    float v[kUnroll][8];
    float w[KIND == kQuantGluBackward ? kUnroll : 1][8];   // the up half's gradient
#pragma unroll
    for (int z = 0; z < kUnroll; ++z)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[z][i] = 0.f;
    if constexpr (KIND == kQuantBf16) {
      uint4 u[kUnroll];
#pragma unroll
      for (int z = 0; z < kUnroll; ++z) {
        const int c = (kb0 + z) * kBlk + hl * 8;
        u[z] = make_uint4(0, 0, 0, 0);
        if (live && kb0 + z < kb1 && c < a.K)
          u[z] = *(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + row + c));
      }
#pragma unroll
      for (int z = 0; z < kUnroll; ++z) unpack8(u[z], v[z]);
    } else if constexpr (KIND == kQuantF32) {
#pragma unroll
      for (int z = 0; z < kUnroll; ++z) {
        const int c = (kb0 + z) * kBlk + hl * 8;
        if (live && kb0 + z < kb1 && c < a.K) {
          const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + row + c);
          const float4 lo = *(p), hi = *(p + 1);
          v[z][0] = lo.x; v[z][1] = lo.y; v[z][2] = lo.z; v[z][3] = lo.w;
          v[z][4] = hi.x; v[z][5] = hi.y; v[z][6] = hi.z; v[z][7] = hi.w;
        }
      }
    } else {
      uint4 ug[kUnroll], uu[kUnroll], ud[kUnroll];
#pragma unroll
      for (int z = 0; z < kUnroll; ++z) {
        const int c = (kb0 + z) * kBlk + hl * 8;
        ug[z] = uu[z] = ud[z] = make_uint4(0, 0, 0, 0);
        if (live && kb0 + z < kb1 && c < a.K) {
          const uint16_t* p = static_cast<const uint16_t*>(a.x) + row + c;
          ug[z] = *(reinterpret_cast<const uint4*>(p));
          uu[z] = *(reinterpret_cast<const uint4*>(p + a.K));
          if (KIND == kQuantGluBackward)
            ud[z] = *(reinterpret_cast<const uint4*>(a.dh + static_cast<size_t>(r) * a.ld_dh + c));
        }
      }
#pragma unroll
      for (int z = 0; z < kUnroll; ++z) {
        float g[8], u[8], d[8];
        unpack8(ug[z], g);
        unpack8(uu[z], u);
        unpack8(ud[z], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float av, bv, da = 0.f, db = 0.f;
          glu_parts(g[i], u[i], a, KIND == kQuantGluBackward, av, bv, da, db);
          if constexpr (KIND == kQuantGluBackward) {
            v[z][i] = d[i] * bv * da;
            w[z][i] = d[i] * av * db;
          } else {
            v[z][i] = av * bv;
          }
        }
      }
    }
#pragma unroll
    for (int z = 0; z < kUnroll; ++z) {
      const int kb = kb0 + z, c = kb * kBlk + hl * 8;
      const bool in = live && kb < kb1;
      const int width = KIND == kQuantGluBackward ? 2 * a.K : a.K;
      uint8_t* out = a.codes + static_cast<size_t>(r) * width + c;
      const BlockScale b = block_scale(half_warp_max(amax8(v[z])));
      if (in && c < a.K) *reinterpret_cast<uint2*>(out) = codes8(v[z], b);
      if (in && hl == 0) a.scales[static_cast<size_t>(kb) * a.ld_s + r] = b.s;
      if constexpr (KIND == kQuantGluBackward) {
        // K is a multiple of 128 here: the up half's blocks follow the gate half's.
        const BlockScale bu = block_scale(half_warp_max(amax8(w[z])));
        if (in) *reinterpret_cast<uint2*>(out + a.K) = codes8(w[z], bu);
        if (in && hl == 0) a.scales[static_cast<size_t>(nkb + kb) * a.ld_s + r] = bu.s;
      }
    }
  }
}

// One CTA per 128 x 128 block of one group's weights: every thread holds 64
// elements, so the block is read once.
__global__ void __launch_bounds__(256) k_quant_weights_block(const uint16_t* w, uint8_t* codes,
                                                             float* scales, int N, int K) {
  griddep_wait();
  griddep_launch();
  __shared__ uint32_t wmax[8];
  const int kb = blockIdx.x, nb = blockIdx.y, g = blockIdx.z;
  const int c = kb * kBlk + (threadIdx.x & 15) * 8;
  const int n0 = nb * kBlk + (threadIdx.x >> 4);
  const size_t base = static_cast<size_t>(g) * N * K;
  uint4 u[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 16 * i;
    u[i] = make_uint4(0, 0, 0, 0);
    if (n < N && c < K) u[i] = *(reinterpret_cast<const uint4*>(w + base + static_cast<size_t>(n) * K + c));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack8(u[i], v);
    m = max(m, amax8(v));
  }
  m = __reduce_max_sync(kFull, m);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, wmax[i]);
  const BlockScale b = block_scale(__uint_as_float(m));
  if (threadIdx.x == 0) scales[(static_cast<size_t>(g) * gridDim.y + nb) * gridDim.x + kb] = b.s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 16 * i;
    if (n >= N || c >= K) continue;
    float v[8];
    unpack8(u[i], v);
    *reinterpret_cast<uint2*>(codes + base + static_cast<size_t>(n) * K + c) = codes8(v, b);
  }
}

}  // namespace

cudaError_t launch_quant_blocks(const QuantArgs& a, int kind, cudaStream_t s) {
  const int nkb = (a.K + kBlk - 1) / kBlk;
  // Every CTA takes kUnroll blocks of its rows at a time; few rows spread their
  // columns over more CTAs.
  const int gy = (nkb + kUnroll - 1) / kUnroll;
  const dim3 grid((a.R + kRowsPerCta - 1) / kRowsPerCta, gy), block(256);
  switch (kind) {
    case kQuantBf16: return launch_k(k_quant_blocks<kQuantBf16>, grid, block, 0, s, false, a);
    case kQuantF32: return launch_k(k_quant_blocks<kQuantF32>, grid, block, 0, s, false, a);
    case kQuantGlu: return launch_k(k_quant_blocks<kQuantGlu>, grid, block, 0, s, false, a);
    default: return launch_k(k_quant_blocks<kQuantGluBackward>, grid, block, 0, s, false, a);
  }
}

cudaError_t launch_quant_weights_block(const uint16_t* w, uint8_t* codes, float* scales, int G, int N, int K,
                                       cudaStream_t s) {
  const dim3 grid((K + kBlk - 1) / kBlk, (N + kBlk - 1) / kBlk, G);
  return launch_k(k_quant_weights_block, grid, dim3(256), 0, s, false, w, codes, scales, N, K);
}

}  // namespace moe
