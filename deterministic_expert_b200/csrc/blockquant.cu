// E4M3 quantisation with one fp32 scale per 128 consecutive elements of a row
// (activations) or per 128 x 128 block (weights).
//
//   s = fp32(max|block| / 448), at least 2^-126; 1 for a block of zeros
//   code = the E4M3 value nearest to x / s, ties to the even code
// The quotient is rounded once: an enclosure of it decides every element that is
// not within 2^-20 of the middle of two codes, and the others are settled by the
// exact sign of x - middle * s.  A block that holds a
// NaN or an infinity gets the scale NaN and zero codes, so that products with it
// are NaN.
//
// Sources of a row: bf16 or fp32 rows (optionally gathered: row r from row
// token_of_row[r]), the experts' gated unit of a [gate | up] row (never stored:
// the unit's fp32 value is quantised directly), or that unit's gradient.
#include <algorithm>

#include "common.cuh"
#include "moe_internal.h"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBlk = 128;
constexpr float kE4m3Max = 448.f;

// A block's scale and two reciprocals of it, one a little too small and one a
// little too large: x * lo and x * hi enclose x / s (the reciprocal is within an
// ulp, each product rounds by half of one: 2^-20 covers all of it four times).
struct BlockScale {
  float s, inv, lo, hi;
  float rem;   // amax - 448 s, exact (0 for a raised scale, whose division is by a power of two)
};

// amax is the block's maximum magnitude, NaN or infinite if an element is.
// amax / 448: an estimate plus its exact remainder times the reciprocal, rounded
// once.  448 = 7 * 64, so the quotient is at least 1/14 ulp away from the middle of
// two fp32 values, far more than the 2^-46 that the sum is off: it is the
// correctly rounded quotient.
__device__ __forceinline__ BlockScale block_scale(float amax) {
  constexpr float kInv448 = 1.f / 448.f;
  const float q = amax * kInv448;
  BlockScale b;
  b.s = fmaf(fmaf(-q, kE4m3Max, amax), kInv448, q);
  b.rem = b.s >= 1.17549435e-38f ? fmaf(-b.s, kE4m3Max, amax) : 0.f;
  b.s = amax > 0.f ? fmaxf(b.s, 1.17549435e-38f) : 1.f;
  b.inv = __fdividef(1.f, b.s);
  if (!(amax < INFINITY)) {
    b.s = __int_as_float(0x7fffffff);
    b.inv = 0.f;
  }
  b.lo = b.inv * (1.f - 0x1p-20f);
  b.hi = b.inv * (1.f + 0x1p-20f);
  return b;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Of the two neighbouring codes that enclose x / s (c and the next in magnitude)
// the nearest, the even one for a tie.  near is within 2^-19 of the middle m of the
// two, so m is near with its bits below half a code's step cut off: codes have 3
// mantissa bits, and those below 2^-6 are multiples of 2^-9, which adding 2^-6
// brings to the same bits.  x - m s is exact in sign in one fused operation, once
// a tiny s and x are scaled up.
__device__ __forceinline__ uint32_t nearest_code(float x, float s, float near, uint32_t c) {
  const float low = near < 0.015625f ? 0.015625f : 0.f;
  const float m = __uint_as_float((__float_as_uint(near + low) & 0xFFF00000u) | 0x80000u) - low;
  const float up = s < 0x1p-60f ? 0x1p64f : 1.f;
  const float r = fmaf(-m, s * up, fabsf(x) * up);
  return c + ((r > 0.f || (r == 0.f && (c & 1u))) ? 1u : 0u);
}

// Pairs of fp32 in one operation.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2(uint64_t p) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
  return e4m3x2(x, y);
}

// Codes of eight elements that are bf16 values, in a block whose maximum is one.
// With 8-bit significands a (x) and b (amax), 448 x / amax is 7 a / b times a power
// of two; it is either the middle of two codes exactly, or (numerator and
// denominator are integers, the middles' significands have 5 bits) at least 2^-13
// of its size away.  So x / s lies beside a middle only where 448 x / amax is one,
// and then on the side that the rounding of s to fp32 went away from: a
// reciprocal 2^-18 too small (s rounded up) or too large (down) takes every such
// element to its side and no other across.  Where s = amax / 448 exactly, it is a
// number of at most 6 bits times a power of two: the quotient, known to 2^-21, is a
// middle or at least 2^-10.2 of its size away from one, so that rounding it to 16 bits
// meets middles exactly, which go to the even code, and takes no other across.  (An
// exact remainder x - q s instead would underflow for tiny s.)
__device__ __forceinline__ uint2 codes8_bf16(const float (&v)[8], const BlockScale& b) {
  const float f = b.rem == 0.f ? b.inv : b.inv * (b.rem < 0.f ? 1.f - 0x1p-18f : 1.f + 0x1p-18f);
  const uint64_t f2 = pair(f, f);
  uint64_t x[4], q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = pair(v[2 * i], v[2 * i + 1]);
    q[i] = mul2(x[i], f2);
  }
  if (b.rem == 0.f) {
    // Veltkamp's split: t - (t - q) with t = 257 q.
    const uint64_t up = pair(257.f, 257.f), one = pair(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t t = mul2(q[i], up);
      q[i] = fma2(fma2(q[i], one, t), one, t);
    }
  }
  const uint2 c = make_uint2(e4m3x2(q[0]) | e4m3x2(q[1]) << 16, e4m3x2(q[2]) | e4m3x2(q[3]) << 16);
  return c;
}

// Codes of eight fp32 elements.  Rounding is monotone, so where both ends of the
// enclosure have one code, that is the quotient's: a product and half a conversion
// of each end an element.  The others (about one in 50000) are settled one by one.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const BlockScale& b) {
  const uint64_t l2 = pair(b.lo, b.lo), h2 = pair(b.hi, b.hi);
  uint32_t lo[2], hi[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint64_t p = pair(v[4 * w], v[4 * w + 1]), q = pair(v[4 * w + 2], v[4 * w + 3]);
    lo[w] = e4m3x2(mul2(p, l2)) | e4m3x2(mul2(q, l2)) << 16;
    hi[w] = e4m3x2(mul2(p, h2)) | e4m3x2(mul2(q, h2)) << 16;
  }
  if (lo[0] != hi[0] || lo[1] != hi[1]) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t diff = lo[w] ^ hi[w];
      while (diff != 0) {
        const int i = (__ffs(diff) - 1) >> 3;
        const float x = i == 0 ? v[4 * w] : (i == 1 ? v[4 * w + 1] : (i == 2 ? v[4 * w + 2] : v[4 * w + 3]));
        const uint32_t c = lo[w] >> (8 * i) & 0xFFu;
        lo[w] += (nearest_code(x, b.s, fabsf(x) * b.hi, c) - c) << (8 * i);   // the next code at most: no carry
        diff &= ~(0xFFu << (8 * i));
      }
    }
  }
  return make_uint2(lo[0], lo[1]);
}

// Maximum magnitude with NaN kept (as a bit pattern above infinity's).
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}
// The same of eight packed bf16 values, as an fp32 bit pattern.
__device__ __forceinline__ uint32_t amax8(const uint4& u) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&u);
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(p[0]), __habs2(p[1])), __hmax2_nan(__habs2(p[2]), __habs2(p[3])));
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&m) & 0x7fff7fffu;
  return max(w & 0xffff0000u, w << 16);
}
// Over the eight lanes of a block.
__device__ __forceinline__ float lanes_max(uint32_t m) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
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

// sigmoid(g) = 1 / (1 + e^-g), to 8 2^-24 relative for every g.  The power of 2 of
// g log2 e rounded to fp32 would be |g| 2^-24 off; but a gate is a bf16 value, so its
// product with a head of log2 e of 16 bits is exact, and the constant's tail goes into
// the power as 1 - g tail (|g tail| < 4.4e-4 where e^-g is a number: its square's half
// is below 10^-7).  A clamp is any fp32 value: there (ANY) what the product lost is
// added to the tail.  ex2 4 2^-24, the correction, its product and 1 + e one each at
// most, rcp 2.  Below -87.3 the result is 0.  c: 1 - sigmoid(g) = e^-g sigmoid(g), as
// accurate (1 where e^-g is infinite: the product with 0 is a NaN, which fminf drops).
// From kSure on s is 1; units that are finite for an infinite gate, or whose lost part
// would be infinite, bound the gate by it.
constexpr float kSure = 128.f;
template <bool ANY>
__device__ __forceinline__ float sigmoid_f32(float g, float& c) {
  constexpr float kHead = 47274.f / 32768.f, kTail = 4.88849515e-6f;   // tail: 1 - head ln 2
  const float t = g * -kHead;
  float w = fmaf(g, -kTail, 1.f), p, r;
  if (ANY) w = fmaf(fmaf(g, -kHead, -t), 0.693147181f, w);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(p, w, 1.f)));   // p infinite: 0
  c = fminf(p * w * r, 1.f);
  return r;
}

// The gated unit and its gradient in fp32 (the code's rounding is 2^-4):
//   SwiGLU    h = a(g) b(u), a = silu(min(g, cg)), b = clamp(u, -cu, cu)
//   SiTU-GLU  a = bg tanh(g / bg) sigmoid(g), b = bu tanh(u / bu)
//   dg = d a'(g) b(u), du = d a(g) b'(u)
// A NaN stays one; a clamped value has no gradient, one at its bound has.
enum GluKind : int { kSwiglu = 0, kSwigluClamped = 1, kSitu = 2 };

// Of a unit (g, u): h, or with GRAD dg and du from d.
template <int GLU, bool GRAD>
__device__ __forceinline__ void glu_unit(float g, float u, float d, const QuantArgs& a, float& first, float& second) {
  float c;
  if (GLU == kSitu) {
    const float sg = sigmoid_f32<false>(fminf(g, kSure), c);
    const float tg = tanhf(__fdiv_rn(g, a.beta_g)), tu = tanhf(__fdiv_rn(u, a.beta_u));
    const float av = a.beta_g * tg * sg, bv = a.beta_u * tu;
    if (GRAD) {
      // The slopes 1 - t^2 to 2^-24 of 1: of the size of d b sigmoid(g) and d a.
      first = d * bv * fmaf(1.f - tg * tg, sg, av * c);
      second = d * av * (1.f - tu * tu);
    } else {
      first = av * bv;
    }
  } else {
    float gpass = 1.f, upass = 1.f, bv = u;
    if (GLU == kSwigluClamped) {
      gpass = g > a.gate_clamp ? 0.f : 1.f;
      g = g > a.gate_clamp ? a.gate_clamp : g;
      upass = (u > a.up_clamp || u < -a.up_clamp) ? 0.f : 1.f;
      bv = u > a.up_clamp ? a.up_clamp : (u < -a.up_clamp ? -a.up_clamp : u);
    }
    const float sg = GLU == kSwigluClamped ? sigmoid_f32<true>(fminf(g, kSure), c) : sigmoid_f32<false>(g, c);
    if (GRAD) {
      // d sigmoid(g) is a factor of both (24576 x 1408, caches cold: 60.4 us; each on its own 66).
      const float ds = d * sg;
      first = ds * bv * fmaf(g, c, 1.f);
      second = ds * g;
      if (GLU == kSwigluClamped) {
        first *= gpass;
        second *= upass;
      }
    } else {
      first = g * sg * bv;
    }
  }
}

// Eight lanes take a block of 128 columns: lane i its columns 8 i .. 8 i + 7 and
// 64 + 8 i .. 64 + 8 i + 7, so that its scale costs each lane a sixteenth of a
// block and every load and store of the eight lanes is one segment.  A CTA of 256
// threads takes 32 rows (their scales of a block are one 128-byte segment) and
// walks their blocks, U at a time so that their loads are in flight together.
// Bound by memory: every element is read once and its code written once.  24576 bf16
// rows of 2048: 25.7 us (6.0 TB/s; two blocks at a time 27.3), and 21.1 us gathered from
// 4096 rows, which then come through L2.  fp32 rows 45.7 us (5.5 TB/s).  Gated unit of
// 32768 x 2048: 58.5 us (5.8 TB/s), clamped 80, SiTU 187 (two tanhf and two divisions
// an element); its gradient, 24576 x 1408: 54-57 us (4.9-5.2 TB/s), clamped 83, SiTU
// 133.
constexpr int kRowsPerCta = 32;
template <int KIND>
constexpr int kUnroll = KIND == kQuantBf16 ? 4 : 1;

template <int KIND, int GLU = kSwiglu>
__global__ void __launch_bounds__(256) k_quant_blocks(const QuantArgs a) {
  constexpr int U = kUnroll<KIND>;
  constexpr bool GRAD = KIND == kQuantGluBackward;
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x * kRowsPerCta + (threadIdx.x >> 3);
  const int l = threadIdx.x & 7;
  int limit = a.R;
  if (a.n_rows != nullptr) limit = min(limit, *a.n_rows);
  long long src = r;
  bool live = r < limit;
  if (live && a.token_of_row != nullptr) {
    src = a.token_of_row[r];
    live = src >= 0 && src < a.src_rows;
  }
  const int nkb = (a.K + kBlk - 1) / kBlk;
  const size_t row = static_cast<size_t>(src) * static_cast<size_t>(a.ld) + l * 8;
  const uint16_t* dh = GRAD ? a.dh + static_cast<size_t>(r) * a.ld_dh + l * 8 : nullptr;
  uint8_t* codes = a.codes + static_cast<size_t>(r) * (GRAD ? 2 * a.K : a.K) + l * 8;
  float* scales = a.scales + r;
  const int per_y = (nkb + gridDim.y - 1) / gridDim.y;
  const int kb1 = min(nkb, static_cast<int>(blockIdx.y + 1) * per_y);
  // Columns c .. c + 7 of the row exist (l * 8 is in the pointers).
  auto in = [&](int c) { return live && c + l * 8 < a.K; };
  // A block's codes and scale; `first`: columns before it in the written row.
  auto put = [&](const float(&v)[2][8], uint32_t m, int c, int sb, int first) {
    const BlockScale b = block_scale(lanes_max(m));
    if (live) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2 q = KIND == kQuantBf16 ? codes8_bf16(v[h], b) : codes8(v[h], b);
        if (b.inv == 0.f) q = make_uint2(0, 0);   // scale NaN: zero codes
        if (in(c + 64 * h)) *reinterpret_cast<uint2*>(codes + first + c + 64 * h) = q;
      }
      if (l == 0) scales[sb * a.ld_s] = b.s;
    }
  };
  for (int kb0 = blockIdx.y * per_y; kb0 < kb1; kb0 += U) {
    if constexpr (KIND == kQuantBf16) {
      uint4 u[U][2];
#pragma unroll
      for (int z = 0; z < U; ++z)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = (kb0 + z) * kBlk + 64 * h;
          u[z][h] = make_uint4(0, 0, 0, 0);
          if (kb0 + z < kb1 && in(c)) u[z][h] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + row + c);
        }
#pragma unroll
      for (int z = 0; z < U; ++z) {
        if (kb0 + z >= kb1) break;
        float v[2][8];
        unpack8(u[z][0], v[0]);
        unpack8(u[z][1], v[1]);
        put(v, max(amax8(u[z][0]), amax8(u[z][1])), (kb0 + z) * kBlk, kb0 + z, 0);
      }
    } else if constexpr (KIND == kQuantF32) {
      float v[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = kb0 * kBlk + 64 * h;
        float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
        if (in(c)) {
          const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + row + c);
          lo = p[0];
          hi = p[1];
        }
        v[h][0] = lo.x; v[h][1] = lo.y; v[h][2] = lo.z; v[h][3] = lo.w;
        v[h][4] = hi.x; v[h][5] = hi.y; v[h][6] = hi.z; v[h][7] = hi.w;
      }
      put(v, max(amax8(v[0]), amax8(v[1])), kb0 * kBlk, kb0, 0);
    } else {
      uint4 ug[2], uu[2], ud[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = kb0 * kBlk + 64 * h;
        ug[h] = uu[h] = ud[h] = make_uint4(0, 0, 0, 0);
        if (in(c)) {
          const uint16_t* p = static_cast<const uint16_t*>(a.x) + row + c;
          ug[h] = *reinterpret_cast<const uint4*>(p);
          uu[h] = *reinterpret_cast<const uint4*>(p + a.K);
          if (GRAD) ud[h] = *reinterpret_cast<const uint4*>(dh + c);
        }
      }
      float g[2][8], u[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float d[8];
        unpack8(ug[h], g[h]);
        unpack8(uu[h], u[h]);
        unpack8(ud[h], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) glu_unit<GLU, GRAD>(g[h][i], u[h][i], d[i], a, g[h][i], u[h][i]);
      }
      put(g, max(amax8(g[0]), amax8(g[1])), kb0 * kBlk, kb0, 0);
      // K is a multiple of 128 for the gradient: the up half's blocks follow.
      if (GRAD) put(u, max(amax8(u[0]), amax8(u[1])), kb0 * kBlk, nkb + kb0, a.K);
    }
  }
}

// One CTA per 128 x 128 block of one group's weights: every thread holds 64
// elements, so the block is read once.  Bound by memory: 8 x 4096 x 7168 in 102 us
// (6.9 TB/s).
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
  for (int i = 0; i < 8; ++i) m = max(m, amax8(u[i]));
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
    uint2 q = codes8_bf16(v, b);
    if (b.inv == 0.f) q = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(codes + base + static_cast<size_t>(n) * K + c) = q;
  }
}

}  // namespace

namespace {
template <int KIND, int GLU = kSwiglu>
cudaError_t launch_kind(const QuantArgs& a, cudaStream_t s) {
  constexpr int U = kUnroll<KIND>;
  const int nkb = (a.K + kBlk - 1) / kBlk;
  const int gx = (a.R + kRowsPerCta - 1) / kRowsPerCta;
  // A CTA walks its rows' blocks U at a time; few rows spread their columns over
  // more CTAs, until there are several for every SM.
  const int gy = std::min((nkb + U - 1) / U, std::max(1, (148 * 8 + gx - 1) / gx));
  return launch_k(k_quant_blocks<KIND, GLU>, dim3(gx, gy), dim3(256), 0, s, false, a);
}
template <int KIND>
cudaError_t launch_glu(const QuantArgs& a, cudaStream_t s) {
  if (a.act == MOE_ACT_SITU_GLU) return launch_kind<KIND, kSitu>(a, s);
  return a.clamped ? launch_kind<KIND, kSwigluClamped>(a, s) : launch_kind<KIND, kSwiglu>(a, s);
}
}  // namespace

cudaError_t launch_quant_blocks(const QuantArgs& a, int kind, cudaStream_t s) {
  switch (kind) {
    case kQuantBf16: return launch_kind<kQuantBf16>(a, s);
    case kQuantF32: return launch_kind<kQuantF32>(a, s);
    case kQuantGlu: return launch_glu<kQuantGlu>(a, s);
    default: return launch_glu<kQuantGluBackward>(a, s);
  }
}

cudaError_t launch_quant_weights_block(const uint16_t* w, uint8_t* codes, float* scales, int G, int N, int K,
                                       cudaStream_t s) {
  const dim3 grid((K + kBlk - 1) / kBlk, (N + kBlk - 1) / kBlk, G);
  return launch_k(k_quant_weights_block, grid, dim3(256), 0, s, false, w, codes, scales, N, K);
}

}  // namespace moe
