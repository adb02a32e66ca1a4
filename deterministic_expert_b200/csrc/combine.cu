// Weighted combine of expert rows back to their tokens, and its gradient.
//
//   out[t]  = (addend[t] +) sum_j w[t, j] y[row_of_slot[t, j]]
// fp32, slots in order, the addend first, one rounding at the end (the Fireworks
// parity post, Trap 3 and its case study: all k contributions in fp32).
//   dy[row] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[row]>
// A slot with no row (index outside [0, rows)) adds nothing and has dw = 0; rows
// that no slot names are left as they were.
#include "common.cuh"
#include "moe_internal.h"
#include "ops_internal.h"

namespace moe {
namespace {

template <typename T>
struct Eight;   // eight consecutive elements
template <>
struct Eight<uint16_t> {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t* p) { u = *(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[2 * j] = bf16_lo(w[j]); v[2 * j + 1] = bf16_hi(w[j]); }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *(reinterpret_cast<const float4*>(p));
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// One thread per 8 columns of a token; its slots' loads are issued four at a time
// before they are added, in slot order.
// Bound by memory: k rows read, one written.
constexpr int kSlotsAtOnce = 4;

template <typename Y, typename O>
__global__ void __launch_bounds__(256) k_combine_rows(const CombineArgs a) {
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 8;
  if (c >= a.D) return;
  const Y* y = static_cast<const Y*>(a.y) + c;
  const int32_t* rows = a.row_of_slot + static_cast<size_t>(t) * a.k;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (a.addend != nullptr) {
    Eight<uint16_t> e;
    e.load(a.addend + static_cast<size_t>(t) * a.D + c);
    e.get(acc);
  }
  for (int j0 = 0; j0 < a.k; j0 += kSlotsAtOnce) {
    Eight<Y> e[kSlotsAtOnce];
    float w[kSlotsAtOnce];
    bool ok[kSlotsAtOnce];
#pragma unroll
    for (int z = 0; z < kSlotsAtOnce; ++z) {
      const int j = j0 + z;
      const int r = j < a.k ? rows[j] : -1;
      ok[z] = r >= 0 && r < a.rows;
      w[z] = 1.f;
      if (ok[z]) {
        e[z].load(y + static_cast<size_t>(r) * a.ld_y);
        if (a.w != nullptr) w[z] = a.w[static_cast<size_t>(t) * a.k + j];
      }
    }
#pragma unroll
    for (int z = 0; z < kSlotsAtOnce; ++z) {
      if (!ok[z]) continue;
      float v[8];
      e[z].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[z], v[i], acc[i]);
    }
  }
  Eight<O>::store(static_cast<O*>(a.out) + static_cast<size_t>(t) * a.D + c, acc);
}

// One CTA per token: a thread keeps its columns of dout, slot by slot reads y,
// writes dy and adds to the slot's dot product; the products are summed over the
// CTA in a fixed tree.
// Bound by memory: k rows read, k rows written.
template <typename Y>
__global__ void __launch_bounds__(256) k_combine_rows_backward(const CombineArgs a) {
  griddep_wait();
  griddep_launch();
  __shared__ float part[kRouteMaxK][8];
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t* rows = a.row_of_slot + static_cast<size_t>(t) * a.k;
  const uint16_t* d = a.dout + static_cast<size_t>(t) * a.D;
  for (int j0 = 0; j0 < a.k; j0 += kSlotsAtOnce) {
    float dot[kSlotsAtOnce], w[kSlotsAtOnce];
    int row[kSlotsAtOnce];
#pragma unroll
    for (int z = 0; z < kSlotsAtOnce; ++z) {
      const int j = j0 + z;
      row[z] = j < a.k ? rows[j] : -1;
      if (row[z] >= a.rows) row[z] = -1;
      w[z] = (row[z] >= 0 && a.w != nullptr) ? a.w[static_cast<size_t>(t) * a.k + j] : 1.f;
      dot[z] = 0.f;
    }
    for (int c = threadIdx.x * 8; c < a.D; c += 256 * 8) {
      Eight<uint16_t> ed;
      Eight<Y> ey[kSlotsAtOnce];
      ed.load(d + c);
      if (a.dw != nullptr) {
#pragma unroll
        for (int z = 0; z < kSlotsAtOnce; ++z)
          if (row[z] >= 0) ey[z].load(static_cast<const Y*>(a.y) + static_cast<size_t>(row[z]) * a.ld_y + c);
      }
      float dv[8];
      ed.get(dv);
#pragma unroll
      for (int z = 0; z < kSlotsAtOnce; ++z) {
        if (row[z] < 0) continue;
        float v[8];
        if (a.dw != nullptr) {
          ey[z].get(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[z] = fmaf(dv[i], v[i], dot[z]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = dv[i] * w[z];
        Eight<Y>::store(static_cast<Y*>(a.dy) + static_cast<size_t>(row[z]) * a.ld_y + c, v);
      }
    }
    if (a.dw != nullptr) {
#pragma unroll
      for (int z = 0; z < kSlotsAtOnce; ++z) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[z] += __shfl_xor_sync(0xffffffffu, dot[z], o);
        if (lane == 0 && j0 + z < a.k) part[j0 + z][warp] = dot[z];
      }
    }
  }
  if (a.dw == nullptr) return;
  __syncthreads();
  if (threadIdx.x < a.k) {
    float s = part[threadIdx.x][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += part[threadIdx.x][w];
    a.dw[static_cast<size_t>(t) * a.k + threadIdx.x] = s;
  }
}

}  // namespace

cudaError_t launch_combine_rows(const CombineArgs& a, bool y_f32, bool out_f32, cudaStream_t s) {
  const dim3 grid(a.T, (a.D / 8 + 255) / 256), block(256);
  if (y_f32)
    return out_f32 ? launch_k(k_combine_rows<float, float>, grid, block, 0, s, false, a)
                   : launch_k(k_combine_rows<float, uint16_t>, grid, block, 0, s, false, a);
  return out_f32 ? launch_k(k_combine_rows<uint16_t, float>, grid, block, 0, s, false, a)
                 : launch_k(k_combine_rows<uint16_t, uint16_t>, grid, block, 0, s, false, a);
}

cudaError_t launch_combine_rows_backward(const CombineArgs& a, bool y_f32, cudaStream_t s) {
  return y_f32 ? launch_k(k_combine_rows_backward<float>, dim3(a.T), dim3(256), 0, s, false, a)
               : launch_k(k_combine_rows_backward<uint16_t>, dim3(a.T), dim3(256), 0, s, false, a);
}

}  // namespace moe
