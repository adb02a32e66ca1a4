// Products of block-scaled E4M3 matrices on the 5th-generation tensor cores.
//
//   C[m, n] = sum_b sa[b, m] sw[n / 128, b] P_b[m, n],
//   P_b[m, n] = sum over the 128 elements k of block b of a[m, k] w[n, k]
// for one weight matrix, or for groups of rows that each meet their own (the
// experts).  Transposed, the same weights are contracted over their rows:
//   C[m, k] = sum_b sa[b, m] sw[b, k / 128] sum over the 128 n of b of a[m, n] w[n, k]
// (the gradient with respect to the product's input).
//
// The tensor core sums one block of 128 products into TMEM; the block's scale is
// fp32 and differs by row, so each P_b is read back and added in registers:
//   acc = fma(P_b, fl(sa sw), acc), b ascending.
// Every output element goes through exactly these operations whatever the tile
// shape, operand roles, group or batch, so its bits depend on its own row alone.
//
// Bound: 128 rows x 256 columns of a CTA take 512 tensor-pipe cycles a block at
// the nominal rate; reading P_b back (32 columns a load) and its 32768
// multiply-adds (packed in pairs) take the epilogue warps about half of that when
// they overlap, so two accumulator buffers of 256 TMEM columns keep both busy.
//
// A CTA pair (cta_group::2) works on 256 rows of one operand and up to 256 of the
// other:
//   full tiles     256 rows of A as the M operand (128 a CTA), 256 weight rows as N;
//                  a thread holds one row and 128 columns, so its scale is one
//                  number a block
//   the rest       256 weight rows as M, the tile's r < 256 rows as N (rounded up
//                  to 16): padding below 16 rows, so small groups and single
//                  tokens stream the weights without wasted products; a thread
//                  holds one column of C and the rows' scales come from shared
//                  memory
// Roles: warp 0 TMA, warp 1 MMA, warps 4-11 read back, scale and store (two warps
// a TMEM lane quarter, splitting the columns).  Registers move from the first
// warpgroup to the other two, whose threads hold 128 sums each.
// Every wait is bounded; on time-out the device's operator error word is set, the
// CTA's copies and MMAs drain (bounded) and TMEM is freed.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "moe_internal.h"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 384;
constexpr int kEpiW = 8;                       // epilogue warps
constexpr int kRing = 184 * 1024;              // stage ring
constexpr int kRingMost = 12;
constexpr int kWSlot = 128 * 128;              // weight bytes of a CTA's stage
constexpr int kEpiSlot = 4096;                 // per epilogue warp
constexpr int kBarSpace = 512;
constexpr int kSmem = 1024 + kRing + kBarSpace + kEpiW * kEpiSlot;
constexpr uint32_t kCols = 512;
constexpr uint32_t kBufCols = 256;
constexpr unsigned long long kDrain = 200ull * 1000 * 1000;   // 200 ms
constexpr int kAhead = 4;                      // blocks whose scales are loaded ahead

// 184 KB ring: 5 stages of 32 KB, or 9 to 10 when a tile has few rows.
static_assert(kRing / (kWSlot + 16 * 128) <= kRingMost, "stages");

// Error word of the handle-free operators on this device.
__device__ int g_operator_error;

struct BTile {
  int g, row0, rows, n0, nt;   // group, first row, valid rows, first weight row / column, N of a swapped tile
  bool swap;
};

__device__ __forceinline__ void group_range(const BlockGemmArgs& a, int g, int& lo, int& hi) {
  if (a.offsets == nullptr) { lo = 0; hi = a.M; return; }
  lo = min(max(a.offsets[g], 0), a.M);
  hi = min(max(a.offsets[g + 1], lo), a.M);
}

__device__ __forceinline__ BTile decode(const BlockGemmArgs& a, const int* start, int ntn, int t) {
  int lo = 0, hi = a.G;   // largest g with start[g] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid;
  }
  BTile ti;
  ti.g = lo;
  int r0, r1;
  group_range(a, lo, r0, r1);
  const int local = t - start[lo];
  const int m = local / ntn;
  ti.n0 = (local - m * ntn) * 256;
  ti.row0 = r0 + m * a.tile_rows;
  ti.rows = min(a.tile_rows, r1 - ti.row0);
  ti.swap = ti.rows < 256;
  ti.nt = (ti.rows + 15) & ~15;
  return ti;
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const void* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// A tile whose contiguous 128 bytes run along M or N (the transposed weights): one
// 128-byte swizzle atom spans the operand's 128 rows, 8 contraction rows are 1024
// bytes, an MMA's 32 contraction rows four of those.  Fields as in
// sw128_kmajor_desc; the leading offset is between repeats along M or N, of which
// there is one.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(16384u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
// Two independent fp32 fused multiply-adds, each rounded as a single one.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t p, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(p), "l"(s));
}

template <int TRANS, typename Out>
__global__ void __launch_bounds__(kThreads, 1) k_block_gemm(const __grid_constant__ BlockGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = min(kRingMost, kRing / (kWSlot + a.a_slot));
  uint8_t* sW = smem;                       // S x kWSlot
  uint8_t* sA = smem + S * kWSlot;          // S x a_slot
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRing);
  uint64_t* full = bars;
  uint64_t* empty = bars + kRingMost;
  uint64_t* tfull = bars + 2 * kRingMost;
  uint64_t* tempty = tfull + 2;
  uint64_t* tdone = tempty + 2;
  uint8_t* epi = smem + kRing + kBarSpace;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int s_start[kMatmulMaxGroups + 1];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 2 * kEpiW); }
    mbar_init(tdone, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(&tmem_slot, kCols);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  volatile int* abort = &abort_flag;
  int* err = &g_operator_error;
  griddep_wait();
  griddep_launch();

  const int ntn = (a.width + 255) / 256;
  const int nkb = (a.con + 127) / 128;
  // First tile of every group.
  if (warp == 2) {
    int run = 0;
    for (int b = 0; b < a.G; b += 32) {
      int n = 0;
      if (b + lane < a.G) {
        int lo, hi;
        group_range(a, b + lane, lo, hi);
        n = (hi - lo + a.tile_rows - 1) / a.tile_rows * ntn;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
      }
      if (b + lane < a.G) s_start[b + lane] = run + incl - n;
      run += __shfl_sync(kFull, incl, 31);
    }
    if (lane == 0) s_start[a.G] = run;
  }
  __syncthreads();
  const int total = s_start[a.G];
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const uint32_t full0 = mapa_shared(full, 0);
  const uint32_t tempty0 = mapa_shared(tempty, 0);

  if (warp < 4) {
    // 64 + 2 x 216 registers of the 3 x 168 a thread that the block was launched with.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- TMA producer
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, issued_phase = 0;   // stages with a copy in flight, and its parity
      bool ok = true;
      for (int t = pair; ok && t < total; t += pairs) {
        const BTile ti = decode(a, s_start, ntn, t);
        const int a_rows = ti.swap ? ti.nt / 2 : 128;
        const int box = a_rows <= 16 ? 0 : (a_rows <= 32 ? 1 : (a_rows <= 64 ? 2 : 3));
        const int y = ti.row0 + static_cast<int>(rank) * a_rows;
        const int wr = ti.n0 + static_cast<int>(rank) * 128;
        const uint32_t bytes = (16u << box) * 128u;
        // The host sizes the A slot for tile_rows rows; a larger box would overrun it.
        if (static_cast<int>(bytes) > a.a_slot) {
          atomicExch(err, kDevBadIndex);
          *abort = 1;
          ok = false;
          break;
        }
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort, err, a.timeout_ns)) { ok = false; break; }
          // The even CTA counts both CTAs' bytes.
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * (bytes + kWSlot));
          const uint32_t fb = full0 + 8 * stage;
          tma_load_2d_pair(sA + stage * a.a_slot, &a.mapA[box], kb * 128, y, fb);
          if (TRANS) tma_load_3d_pair(sW + stage * kWSlot, &a.mapW, wr, kb * 128, ti.g, fb);
          else tma_load_3d_pair(sW + stage * kWSlot, &a.mapW, kb * 128, wr, ti.g, fb);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && leader)
        for (int s = 0; s < S; ++s)
          if (issued >> s & 1u) mbar_wait_drain(&full[s], issued_phase >> s & 1u, kDrain);
    } else if (warp == 1 && lane == 0 && leader) {
      // ------------------------------------------------------ MMA issuer
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      for (int t = pair; ok && t < total; t += pairs) {
        const BTile ti = decode(a, s_start, ntn, t);
        // The transposed weights run along M (swapped: bit 15) or N (bit 16).
        const uint32_t idesc = idesc_e4m3_f32(256, ti.swap ? ti.nt : 256) |
                               (TRANS ? (ti.swap ? 1u << 15 : 1u << 16) : 0u);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&tempty[buf], bphase ^ 1u, abort, err, a.timeout_ns)) { ok = false; break; }
          if (!mbar_wait(&full[stage], phase, abort, err, a.timeout_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t ta = smem_u32(sA + stage * a.a_slot), wa = smem_u32(sW + stage * kWSlot);
          const uint32_t d = tmem_base + buf * kBufCols;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t td = sw128_kmajor_desc(ta + kk * 32);
            const uint64_t wd = TRANS ? sw128_mnmajor_desc(wa + kk * 4096) : sw128_kmajor_desc(wa + kk * 32);
            umma_e4m3_pair(d, ti.swap ? wd : td, ti.swap ? td : wd, idesc, kk != 0 ? 1u : 0u);
          }
          umma_commit_pair_mc(&empty[stage], 0x3);
          umma_commit_pair_mc(&tfull[buf], 0x3);
          if (++stage == S) { stage = 0; phase ^= 1u; }
          if (++buf == 2) { buf = 0; bphase ^= 1u; }
        }
      }
      umma_commit_pair_mc(tdone, 0x1);
      mbar_wait_drain(tdone, 0, kDrain);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // --------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 4) >> 2;
    uint8_t* stage_w = epi + (warp - 4) * kEpiSlot;
    float* s_sc = reinterpret_cast<float*>(stage_w);   // swapped: two slots of 128 scales
    int buf = 0;
    uint32_t bphase = 0;
    bool ok = true;
    for (int t = pair; ok && t < total; t += pairs) {
      const BTile ti = decode(a, s_start, ntn, t);
      const int hc = ti.nt >> 1;   // swapped: columns (rows of A) of this warp
      // Scale addresses: the row of A this lane loads for (full tile: its own row;
      // swapped: rows lane, lane + 32, ... of the warp's), the weights' block.
      const int own = ti.swap ? half * hc + lane : static_cast<int>(rank) * 128 + q * 32 + lane;
      const float* ps = a.a_scale + ti.row0 + own;
      const int oblk = ti.n0 / 128 + (ti.swap ? static_cast<int>(rank) : half);
      // Past the last block (its columns are not stored) the scale is taken as 0.
      const bool wlive = oblk * 128 < a.width;
      const float* pw = a.w_scale + ti.g * a.ws_g + (wlive ? oblk : 0) * a.ws_o;
      // Rows behind the tile's last are never read (they may lie behind the buffer).
      bool live[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        live[i] = own + 32 * i < ti.rows && (ti.swap ? lane + 32 * i < hc : i == 0);
      float sa[kAhead][4], sw[kAhead];
      auto load = [&](int slot, int kb) {
        const bool in = kb < nkb;
        sw[slot] = in && wlive ? pw[kb * a.ws_c] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) sa[slot][i] = in && live[i] ? ps[kb * a.ld_as + 32 * i] : 0.f;
      };
#pragma unroll
      for (int z = 0; z < kAhead; ++z) load(z, z);

      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      for (int kb = 0; kb < nkb; ++kb) {
        ok = mbar_wait(&tfull[buf], bphase, abort, err, a.timeout_ns);
        if (!__all_sync(kFull, ok)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kBufCols;
        if (!ti.swap) {
          const float s = __fmul_rn(sa[0][0], sw[0]);
          const uint64_t s2 = pack2(s, s);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(tb + half * 128 + c * 32, v);
            tmem_ld_wait();
            if (c == 3) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * buf);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) fma2(acc[c * 16 + i], pack2u(v[2 * i], v[2 * i + 1]), s2);
          }
        } else {
          float* sc = s_sc + (kb & 1) * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i * 32 < hc) sc[i * 32 + lane] = __fmul_rn(sa[0][i], sw[0]);
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c * 32 >= hc) continue;
            uint32_t v[32];
            tmem_ld32(tb + half * hc + c * 32, v);
            tmem_ld_wait();
            if ((c + 1) * 32 >= hc) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * buf);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 f = *reinterpret_cast<const float4*>(sc + c * 32 + 4 * i);
              fma2(acc[c * 16 + 2 * i], pack2u(v[4 * i], v[4 * i + 1]), pack2(f.x, f.y));
              fma2(acc[c * 16 + 2 * i + 1], pack2u(v[4 * i + 2], v[4 * i + 3]), pack2(f.z, f.w));
            }
          }
        }
        // Move the scales up by one block and load the one after the last.
#pragma unroll
        for (int z = 0; z + 1 < kAhead; ++z) {
          sw[z] = sw[z + 1];
#pragma unroll
          for (int i = 0; i < 4; ++i) sa[z][i] = sa[z + 1][i];
        }
        load(kAhead - 1, kb + kAhead);
        if (++buf == 2) { buf = 0; bphase ^= 1u; }
      }
      if (!ok) break;

      // ------------------------------------------------------- store
      Out* out = static_cast<Out*>(a.out);
      constexpr int kPer = 16 / sizeof(Out);           // elements of a 16-byte chunk
      constexpr int kSeg = 128 / sizeof(Out);          // columns of a 128-byte segment
      auto conv = [](float v) {
        if constexpr (sizeof(Out) == 2) return static_cast<Out>(pack_bf16x2(v, 0.f) & 0xFFFFu);
        else return v;
      };
      if (!ti.swap) {
        // A thread's row goes through the warp's staging buffer so that stores
        // cover 128-byte row segments (chunk m of row r at m ^ (r & 7)).
        const int r0 = static_cast<int>(rank) * 128 + q * 32;
        const int col0 = ti.n0 + half * 128;
#pragma unroll
        for (int p = 0; p < 128 / kSeg; ++p) {
          __syncwarp();
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            uint4 u;
            if constexpr (sizeof(Out) == 2) {
              const float2 f0 = unpack2(acc[p * 32 + m * 4]), f1 = unpack2(acc[p * 32 + m * 4 + 1]);
              const float2 f2 = unpack2(acc[p * 32 + m * 4 + 2]), f3 = unpack2(acc[p * 32 + m * 4 + 3]);
              u = make_uint4(pack_bf16x2(f0.x, f0.y), pack_bf16x2(f1.x, f1.y), pack_bf16x2(f2.x, f2.y),
                             pack_bf16x2(f3.x, f3.y));
            } else {
              const float2 f0 = unpack2(acc[p * 16 + m * 2]), f1 = unpack2(acc[p * 16 + m * 2 + 1]);
              u = make_uint4(__float_as_uint(f0.x), __float_as_uint(f0.y), __float_as_uint(f1.x), __float_as_uint(f1.y));
            }
            *reinterpret_cast<uint4*>(stage_w + lane * 128 + ((m ^ (lane & 7)) << 4)) = u;
          }
          __syncwarp();
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const int r = it * 4 + (lane >> 3), ch = lane & 7;
            const int col = col0 + p * kSeg + ch * kPer;
            const uint4 u = *reinterpret_cast<const uint4*>(stage_w + r * 128 + ((ch ^ (r & 7)) << 4));
            Out* dst = out + static_cast<size_t>(ti.row0 + r0 + r) * a.ldo + col;   // 256 valid rows in a full tile
            if (a.out_vec && col + kPer <= a.width) {
              *reinterpret_cast<uint4*>(dst) = u;
            } else {
              union { uint4 u; Out e[kPer]; } x;
              x.u = u;
#pragma unroll
              for (int z = 0; z < kPer; ++z)
                if (col + z < a.width) dst[z] = x.e[z];
            }
          }
        }
      } else {
        // A thread's column: 32 lanes write 32 neighbouring columns of one row.
        const int col = ti.n0 + static_cast<int>(rank) * 128 + q * 32 + lane;
        const int valid = min(hc, ti.rows - half * hc);
        Out* dst = out + static_cast<size_t>(ti.row0 + half * hc) * a.ldo + col;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          if (2 * i >= valid) break;
          const float2 f = unpack2(acc[i]);
          if (col < a.width) {
            dst[static_cast<size_t>(2 * i) * a.ldo] = conv(f.x);
            if (2 * i + 1 < valid) dst[static_cast<size_t>(2 * i + 1) * a.ldo] = conv(f.y);
          }
        }
      }
      __syncwarp();
    }
  }

  // Neither CTA leaves while the other may still signal it.
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kCols);
  }
}

using Kernel = void (*)(BlockGemmArgs);
Kernel kernel_of(bool transposed, bool f32) {
  if (transposed) return f32 ? k_block_gemm<1, float> : k_block_gemm<1, uint16_t>;
  return f32 ? k_block_gemm<0, float> : k_block_gemm<0, uint16_t>;
}

std::mutex g_mu;
int g_pairs[64];
bool g_ready[64];

}  // namespace

// Shared memory limit and the CTA pairs that fit at once, once per device.  The
// persistent grid is never larger, so no pair waits for another to finish.
int block_gemm_pairs() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_ready[dev]) return g_pairs[dev];
  int n = 1 << 30;
  for (int v = 0; v < 4; ++v) {
    const void* fn = reinterpret_cast<const void*>(kernel_of(v & 1, v & 2));
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) n = 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, fn, &cfg) != cudaSuccess) c = 0;
    n = std::min(n, c);
  }
  cudaGetLastError();
  if (n <= 0) return 0;
  g_pairs[dev] = n;
  g_ready[dev] = true;
  return n;
}

cudaError_t launch_block_gemm(const BlockGemmArgs& a, int max_tiles, cudaStream_t s) {
  const int pairs = block_gemm_pairs();
  if (pairs <= 0) return cudaErrorInvalidConfiguration;
  return launch_k(kernel_of(a.transposed != 0, a.out_f32 != 0), dim3(2 * std::min(pairs, max_tiles)), dim3(kThreads),
                  kSmem, s, true, a);
}

cudaError_t read_operator_error(int* value, cudaStream_t s) {
  void* p = nullptr;
  cudaError_t rc = cudaGetSymbolAddress(&p, g_operator_error);
  if (rc == cudaSuccess) rc = cudaMemcpyAsync(value, p, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (rc == cudaSuccess) rc = cudaMemsetAsync(p, 0, sizeof(int), s);
  if (rc == cudaSuccess) rc = cudaStreamSynchronize(s);
  return rc;
}

}  // namespace moe
