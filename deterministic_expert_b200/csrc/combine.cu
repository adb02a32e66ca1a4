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

// One CTA per token.  Its slots' rows and weights are read once into shared memory;
// a thread then takes 8 columns at a time, kSlotsAtOnce slots' loads issued before
// they are added, in slot order.
// Bound by memory: k rows read, one written; T = 8192, k = 8, D = 7168 bf16 in 155 us,
// 6.8 TB/s.
constexpr int kSlotsAtOnce = 8;

// Threads for D columns, 8 a thread: as few passes as 256 threads need, evenly.
int row_threads(int D) {
  const int chunks = D / 8, passes = (chunks + 255) / 256;
  return ((chunks + passes - 1) / passes + 31) / 32 * 32;
}

template <typename Y, typename O>
__global__ void __launch_bounds__(256) k_combine_rows(const CombineArgs a) {
  __shared__ int s_row[kRouteMaxK];
  __shared__ float s_w[kRouteMaxK];
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x;
  if (threadIdx.x < kRouteMaxK) {
    int r = -1;
    float w = 1.f;
    if (threadIdx.x < a.k) {
      const size_t i = static_cast<size_t>(t) * a.k + threadIdx.x;
      r = a.row_of_slot[i];
      if (a.w != nullptr) w = a.w[i];
    }
    s_row[threadIdx.x] = r < a.rows ? r : -1;
    s_w[threadIdx.x] = w;
  }
  __syncthreads();
  for (int c = threadIdx.x * 8; c < a.D; c += blockDim.x * 8) {
    const Y* y = static_cast<const Y*>(a.y) + c;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.addend != nullptr) {
      Eight<uint16_t> e;
      e.load(a.addend + static_cast<size_t>(t) * a.D + c);
      e.get(acc);
    }
    for (int j0 = 0; j0 < a.k; j0 += kSlotsAtOnce) {
      Eight<Y> e[kSlotsAtOnce];
#pragma unroll
      for (int z = 0; z < kSlotsAtOnce; ++z) {
        const int r = s_row[j0 + z];
        if (r >= 0) e[z].load(y + static_cast<size_t>(r) * a.ld_y);
      }
#pragma unroll
      for (int z = 0; z < kSlotsAtOnce; ++z) {
        if (s_row[j0 + z] < 0) continue;
        const float w = s_w[j0 + z];
        float v[8];
        e[z].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[i], acc[i]);
      }
    }
    Eight<O>::store(static_cast<O*>(a.out) + static_cast<size_t>(t) * a.D + c, acc);
  }
}

// One CTA per token: a thread takes 8 columns of dout at a time, reads its slots'
// y, writes their dy and adds to their dot products; the products are summed over
// the CTA in a fixed tree.
// Bound by memory: k rows read, k rows written; T = 4096, k = 6, D = 2048 bf16 in
// 37.8 us, 5.8 TB/s.  Two slots at a time: more take registers, and with them resident CTAs.
constexpr int kSlotsBack = 2;

template <typename Y>
__global__ void __launch_bounds__(256) k_combine_rows_backward(const CombineArgs a) {
  __shared__ float part[kRouteMaxK][8];
  __shared__ int s_row[kRouteMaxK];
  __shared__ float s_w[kRouteMaxK];
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < kRouteMaxK) {
    int r = -1;
    float w = 1.f;
    if (threadIdx.x < a.k) {
      const size_t i = static_cast<size_t>(t) * a.k + threadIdx.x;
      r = a.row_of_slot[i];
      if (a.w != nullptr) w = a.w[i];
    }
    s_row[threadIdx.x] = r < a.rows ? r : -1;
    s_w[threadIdx.x] = w;
  }
  __syncthreads();
  const uint16_t* d = a.dout + static_cast<size_t>(t) * a.D;
  for (int j0 = 0; j0 < a.k; j0 += kSlotsBack) {
    float dot[kSlotsBack] = {};
    for (int c = threadIdx.x * 8; c < a.D; c += blockDim.x * 8) {
      Eight<uint16_t> ed;
      Eight<Y> ey[kSlotsBack];
      ed.load(d + c);
      if (a.dw != nullptr) {
#pragma unroll
        for (int z = 0; z < kSlotsBack; ++z) {
          const int r = s_row[j0 + z];
          if (r >= 0) ey[z].load(static_cast<const Y*>(a.y) + static_cast<size_t>(r) * a.ld_y + c);
        }
      }
      float dv[8];
      ed.get(dv);
#pragma unroll
      for (int z = 0; z < kSlotsBack; ++z) {
        const int r = s_row[j0 + z];
        if (r < 0) continue;
        const float w = s_w[j0 + z];
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = dv[i] * w;
        Eight<Y>::store(static_cast<Y*>(a.dy) + static_cast<size_t>(r) * a.ld_y + c, v);
        if (a.dw != nullptr) {
          ey[z].get(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[z] = fmaf(dv[i], v[i], dot[z]);
        }
      }
    }
    if (a.dw != nullptr) {
#pragma unroll
      for (int z = 0; z < kSlotsBack; ++z) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[z] += __shfl_xor_sync(0xffffffffu, dot[z], o);
        if (lane == 0) part[j0 + z][warp] = dot[z];
      }
    }
  }
  if (a.dw == nullptr) return;
  __syncthreads();
  if (threadIdx.x < a.k) {
    const int warps = blockDim.x >> 5;
    float s = part[threadIdx.x][0];
    for (int w = 1; w < warps; ++w) s += part[threadIdx.x][w];
    a.dw[static_cast<size_t>(t) * a.k + threadIdx.x] = s;
  }
}

}  // namespace

cudaError_t launch_combine_rows(const CombineArgs& a, bool y_f32, bool out_f32, cudaStream_t s) {
  const dim3 grid(a.T), block(row_threads(a.D));
  if (y_f32)
    return out_f32 ? launch_k(k_combine_rows<float, float>, grid, block, 0, s, false, a)
                   : launch_k(k_combine_rows<float, uint16_t>, grid, block, 0, s, false, a);
  return out_f32 ? launch_k(k_combine_rows<uint16_t, float>, grid, block, 0, s, false, a)
                 : launch_k(k_combine_rows<uint16_t, uint16_t>, grid, block, 0, s, false, a);
}

cudaError_t launch_combine_rows_backward(const CombineArgs& a, bool y_f32, cudaStream_t s) {
  const dim3 grid(a.T), block(row_threads(a.D));
  return y_f32 ? launch_k(k_combine_rows_backward<float>, grid, block, 0, s, false, a)
               : launch_k(k_combine_rows_backward<uint16_t>, grid, block, 0, s, false, a);
}

}  // namespace moe
