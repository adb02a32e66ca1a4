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
// the nominal rate, about 680 with both operands coming from shared memory.  Reading
// P_b back takes another 512 (128 KB at TMEM's rate) plus the latencies of commit,
// first load and release; the two accumulator buffers of 256 TMEM columns overlap the
// two, and the round trip of a buffer through both, about 880 cycles a block, is what
// bounds large products: 8192 x 4096 x 7168 in 212-217 us, 2220-2270 TFLOP/s, the
// tensor pipe busy half of the time.  A tile's store costs 1.3 us (all SMs write at once) and its
// start 0.5 us, which short contractions feel.  Few rows a group are bound by the
// weights' stream: 384 rows over 64 groups of 2816 x 2048 at 5.9-6.1 TB/s.
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
#include <type_traits>

#include "common.cuh"
#include "moe_internal.h"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 384;
constexpr int kEpiW = 8;                       // epilogue warps
constexpr int kRing = 168 * 1024;              // stage ring
constexpr int kRingMost = 12;
constexpr int kWSlot = 128 * 128;              // weight bytes of a CTA's stage
constexpr int kEpiSlot = 4096;                 // per epilogue warp
constexpr int kBarSpace = 512;
constexpr int kDoneBar = 2 * kRingMost + 4;  // index of the barrier of the last MMAs
constexpr int kSlotBlocks = 4;                 // blocks whose scales a slot holds
constexpr int kScaleSlots = 4;
constexpr int kSlotBytes = kSlotBlocks * 256 * 4;
constexpr uint32_t kCols = 512;
constexpr int kSwapRows = 128;                 // tiles of at most this many rows have the weights as M
constexpr unsigned long long kDrain = 200ull * 1000 * 1000;   // 200 ms
constexpr int kSmem = 1024 + kRing + kBarSpace + kEpiW * kEpiSlot + kScaleSlots * kSlotBytes;

// 168 KB ring: 5 stages of 32 KB, or up to 9 when a tile has few rows.
static_assert(kRing / (kWSlot + 16 * 128) <= kRingMost, "stages");
static_assert(kSlotBlocks == 4, "the epilogue reads a row's scales of a slot as one float4");

// Error word of the handle-free operators on this device, and what was last taken from
// it (under a lock on the host).
__device__ int g_operator_error;
__device__ int g_operator_taken;

// One exchange: an error that another stream raises meanwhile is in it or stays.
__global__ void k_take_operator_error() { g_operator_taken = atomicExch(&g_operator_error, 0); }

struct BTile {
  int g, row0, rows, n0, nt;   // group, first row, valid rows, first output column, N of the MMA
  int batch;                   // blocks of the contraction in one accumulator buffer
  bool swap;
};

__device__ __forceinline__ void group_range(const BlockGemmArgs& a, int g, int& lo, int& hi) {
  if (a.offsets == nullptr) { lo = 0; hi = a.M; return; }
  lo = min(max(a.offsets[g], 0), a.M);
  hi = min(max(a.offsets[g + 1], lo), a.M);
}

// First tile of every group (ntn tiles a row of tiles); one warp.
__device__ __forceinline__ void scan_groups(const BlockGemmArgs& a, int* start, int ntn, int lane) {
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
    if (b + lane < a.G) start[b + lane] = run + incl - n;
    run += __shfl_sync(kFull, incl, 31);
  }
  if (lane == 0) start[a.G] = run;
}

template <int COLS = 256>
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
  ti.n0 = (local - m * ntn) * COLS;
  ti.row0 = r0 + m * a.tile_rows;
  ti.rows = min(a.tile_rows, r1 - ti.row0);
  ti.swap = ti.rows <= kSwapRows;
  ti.nt = ti.swap ? (ti.rows + 15) & ~15 : 256;
  // Two buffers of 256 TMEM columns; tiles with few rows put several blocks in one,
  // since handing a buffer over costs the epilogue about 800 cycles however few its
  // columns (wait, load latency beside the running products, release).
  ti.batch = ti.nt <= 64 ? 4 : (ti.nt <= 128 ? 2 : 1);
  return ti;
}

// Index of the smallest A box (16 << index rows) that holds `rows`.
__device__ __forceinline__ int box_of(int rows) { return rows <= 16 ? 0 : (rows <= 32 ? 1 : (rows <= 64 ? 2 : 3)); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

__device__ __forceinline__ uint32_t mapa_u32(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Arrive once at `bar` in both CTAs when the pair's MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const void* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// High word of both operands' shared-memory descriptors (128-byte swizzle,
// version 1, 1024 bytes between groups of 8): as sw128_kmajor_desc.  The transposed
// weights are a tile whose contiguous 128 bytes run along M or N: one swizzle atom
// spans the operand's 128 rows, 8 contraction rows are 1024 bytes, an MMA's 32
// contraction rows 4096; the leading offset is between repeats along M or N, of
// which there is one.
constexpr uint64_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;

// True in one lane of the warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// Wait for the loads from TMEM; v is only defined after it, so it passes through.
__device__ __forceinline__ void tmem_wait32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                 "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

// CH consecutive columns of this thread's TMEM lane, and the wait for them.
template <int CH>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[CH]) {
  if constexpr (CH == 32) {
    tmem_ld32(taddr, r);
  } else if constexpr (CH == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    static_assert(CH == 8, "8, 16 or 32 columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  }
}
template <int CH>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[CH]) {
  if constexpr (CH == 32) {
    tmem_wait32(v);
  } else if constexpr (CH == 16) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
  } else {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])
                 :
                 : "memory");
  }
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

// Barriers and shared memory by 32-bit shared addresses: the epilogue's threads
// have no registers to spare for generic pointers.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ int ld_shared_i32(uint32_t p) {
  int v;
  asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t p) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t p, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(p), "f"(v) : "memory");
}
// One float by asynchronous copy, or a zero (nothing is read) unless `live`.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f32x4(uint32_t p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p));
  return v;
}
// Four floats as two packed pairs.
__device__ __forceinline__ void ld_shared_pairs(uint32_t p, uint64_t& lo, uint64_t& hi) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(lo), "=l"(hi) : "r"(p));
}

// A bounded wait: every failed try sleeps in hardware for up to about a
// microsecond, so the limit (BlockGemmArgs::tries) is of the order of seconds.  On
// time-out it raises the CTA's abort flag and the device's error word; it gives up at
// once when another role has.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t abort, int tries) {
  if (bar_try(bar, parity)) return true;
  for (int i = 0; i < tries; ++i) {
    if (bar_try(bar, parity)) return true;
    if (ld_shared_i32(abort) != 0) return false;
  }
  asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(abort) : "memory");
  atomicExch(&g_operator_error, kDevTimeout);
  return false;
}

// 32 staged rows of 128 bytes to rows that start anywhere or end inside the segment
// (`cols` columns are left): a row at a time, neighbouring lanes neighbouring
// elements, 4 bytes a lane, the shared reads of kRowsAtOnce rows in flight.
// (11562 x 1497 x 208: 40 us; eight elements a lane, one after the other, took 77.)
constexpr int kRowsAtOnce = 8;
template <typename Out>
__device__ __noinline__ void store_segment(Out* out, long long ldo, int rows, int cols, const uint8_t* stage, int lane) {
  constexpr int kPer = 16 / sizeof(Out);
  auto at = [&](int r, int c) {
    return *(reinterpret_cast<const Out*>(stage + r * 128 + (((c / kPer) ^ (r & 7)) << 4)) + c % kPer);
  };
  rows = min(rows, 32);
  for (int r0 = 0; r0 < rows; r0 += kRowsAtOnce, out += kRowsAtOnce * ldo) {
    if constexpr (sizeof(Out) == 4) {
      Out v[kRowsAtOnce];
#pragma unroll
      for (int z = 0; z < kRowsAtOnce; ++z) v[z] = at(r0 + z, lane);
#pragma unroll
      for (int z = 0; z < kRowsAtOnce; ++z)
        if (r0 + z < rows && lane < cols) out[z * ldo + lane] = v[z];
    } else {
      // Pairs from the first element on 4 bytes; an odd row's first and 64th are alone.
      Out lo[kRowsAtOnce], hi[kRowsAtOnce];
      const int odd0 = static_cast<int>(reinterpret_cast<uintptr_t>(out) >> 1 & 1), step = static_cast<int>(ldo & 1);
#pragma unroll
      for (int z = 0; z < kRowsAtOnce; ++z) {
        const int c = 2 * lane + (odd0 ^ (step & z));
        lo[z] = at(r0 + z, c);
        hi[z] = at(r0 + z, (c + 1) & 63);   // an odd row's last lane: the first element
      }
#pragma unroll
      for (int z = 0; z < kRowsAtOnce; ++z) {
        if (r0 + z >= rows) break;
        const int odd = odd0 ^ (step & z), c = 2 * lane + odd;
        Out* to = out + z * ldo;
        if (c + 1 < min(cols, 64)) {
          *reinterpret_cast<uint32_t*>(to + c) = lo[z] | static_cast<uint32_t>(hi[z]) << 16;
        } else {
          if (c < cols) to[c] = lo[z];
          if (c == 63 && cols > 0) to[0] = hi[z];
        }
      }
    }
  }
}

// The current tile of a warp, in shared memory: decoding it inline, or keeping it in
// registers, costs the epilogue's loops registers that they need (8192 x 4096 x 7168:
// 234 us decoded inline, 224 so).
__device__ __noinline__ void decode_to(const BlockGemmArgs& a, const int* start, int ntn, int t, BTile* to) {
  const BTile ti = decode(a, start, ntn, t);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) *to = ti;
  __syncwarp();
}

template <int TRANS, typename Out>
__global__ void __launch_bounds__(kThreads, 1) k_block_gemm(const __grid_constant__ BlockGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = min(kRingMost, kRing / (kWSlot + a.a_slot));
  uint8_t* sW = smem;                       // S x kWSlot
  uint8_t* sA = smem + S * kWSlot;          // S x a_slot
  __shared__ uint32_t tmem_slot;
  __shared__ BTile s_tile[kThreads / 32];
  __shared__ int abort_flag;
  __shared__ int s_start[kMatmulMaxGroups + 1];
  const uint32_t smem0 = smem_u32(smem);
  const uint32_t full = smem0 + kRing, empty = full + 8 * kRingMost;
  const uint32_t tfull = empty + 8 * kRingMost, tempty = tfull + 8 * 2, tdone = tempty + 8 * 2;
  const uint32_t sfull = tdone + 8, sempty = sfull + 8 * kScaleSlots;
  const uint32_t epi = smem0 + kRing + kBarSpace;
  const uint32_t scales = epi + kEpiW * kEpiSlot;   // kScaleSlots x kSlotBytes
  const uint32_t abort = smem_u32(&abort_flag);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRing);
    for (int s = 0; s < 2 * kRingMost; ++s) mbar_init(&bars[s], 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars[2 * kRingMost + b], 1);
      mbar_init(&bars[2 * kRingMost + 2 + b], 2 * kEpiW);
    }
    mbar_init(&bars[kDoneBar], 1);
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(&bars[kDoneBar + 1 + i], 2);   // this CTA's scale warps
      mbar_init(&bars[kDoneBar + 1 + kScaleSlots + i], kEpiW);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(&tmem_slot, kCols);
  if (threadIdx.x == 0) {
    prefetch_map(&a.mapA[box_of(a.tile_rows >= 256 ? 128 : a.tile_rows / 2)]);
    prefetch_map(&a.mapW);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  griddep_wait();
  griddep_launch();

  const int ntn = (a.width + 255) / 256;
  const int nkb = (a.con + 127) / 128;
  if (warp == 2) scan_groups(a, s_start, ntn, lane);
  __syncthreads();
  const int total = s_start[a.G];
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp < 4) {
    // 72 + 2 x 216 registers of the 3 x 168 a thread that the block was launched with.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- TMA producer
      const uint32_t full0 = mapa_u32(full, 0);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, issued_phase = 0;   // stages with a copy in flight, and its parity
      bool ok = true;
      for (int t = pair; ok && t < total; t += pairs) {
        const BTile ti = decode(a, s_start, ntn, t);
        const int a_rows = ti.swap ? ti.nt / 2 : 128;
        const int box = box_of(a_rows);
        const int y = ti.row0 + static_cast<int>(rank) * a_rows;
        const int wr = ti.n0 + static_cast<int>(rank) * 128;
        const uint32_t bytes = (16u << box) * 128u;
        // The host sizes the A slot for tile_rows rows; a larger box would overrun it.
        if (static_cast<int>(bytes) > a.a_slot) {
          atomicExch(&g_operator_error, kDevBadIndex);
          abort_flag = 1;
          ok = false;
          break;
        }
        for (int kb = 0; kb < a.load_blocks; ++kb) {
          if (!bar_wait(empty + 8 * stage, phase ^ 1u, abort, a.tries)) { ok = false; break; }
          // The even CTA counts both CTAs' bytes.
          if (leader)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full + 8 * stage),
                         "r"(2 * (bytes + kWSlot)) : "memory");
          const uint32_t fb = full0 + 8 * stage;
          tma_load_2d_pair(sA + stage * a.a_slot, &a.mapA[box], kb * 128, y, fb);
          if (TRANS) tma_load_3d_pair(sW + stage * kWSlot, &a.mapW, wr, kb * 128, ti.g, fb);
          else tma_load_3d_pair(sW + stage * kWSlot, &a.mapW, kb * 128, wr, ti.g, fb);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (a.load_blocks < nkb) ok = false;   // the self-test's
      }
      if (!ok && leader)
        for (int s = 0; s < S; ++s)
          if (issued >> s & 1u) mbar_wait_drain(reinterpret_cast<uint64_t*>(smem + kRing) + s, issued_phase >> s & 1u, kDrain);
    } else if (warp == 1 && leader) {
      // ------------------------------------------------------ MMA issuer
      // The whole warp walks the loop (its addresses stay in uniform registers); one
      // lane issues.
      const bool issuer = elect_one();
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      // Low words of the operands' descriptors: start address and leading offset, >> 4.
      const uint32_t tok_lo = (((smem0 + S * kWSlot) >> 4) & 0x3FFFu) | 1u << 16;
      const uint32_t w_lo = ((smem0 >> 4) & 0x3FFFu) | (TRANS ? 16384u >> 4 : 1u) << 16;
      const uint32_t tok_step = static_cast<uint32_t>(a.a_slot) >> 4;
      bool ok = true;
      for (int t = pair; ok && t < total; t += pairs) {
        const BTile ti = decode(a, s_start, ntn, t);
        // The transposed weights run along M (swapped: bit 15) or N (bit 16).
        const uint32_t idesc = idesc_e4m3_f32(256, ti.nt) | (TRANS ? (ti.swap ? 1u << 15 : 1u << 16) : 0u);
        int left = 0;   // blocks that the current buffer still takes
        uint32_t d = 0;
        for (int kb = 0; kb < nkb; ++kb) {
          ok = bar_wait(full + 8 * stage, phase, abort, a.tries);
          if (left == 0) {
            ok = ok && bar_wait(tempty + 8 * buf, bphase ^ 1u, abort, a.tries);
            left = ti.batch;
            d = tmem_base + buf * 256;
          }
          if (!__all_sync(kFull, ok)) { ok = false; break; }
          tc_fence_after();
          const uint32_t tlo = tok_lo + stage * tok_step, wlo = w_lo + stage * (kWSlot >> 4);
          const uint32_t alo = ti.swap ? wlo : tlo, blo = ti.swap ? tlo : wlo;
          const uint32_t astep = TRANS && ti.swap ? 4096 >> 4 : 2, bstep = TRANS && !ti.swap ? 4096 >> 4 : 2;
          --left;
          const bool last = left == 0 || kb == nkb - 1;
          if (issuer) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_e4m3_pair(d, (kDescHi << 32) | (alo + kk * astep), (kDescHi << 32) | (blo + kk * bstep), idesc,
                             kk != 0 ? 1u : 0u);
            if (last) commit_pair(tfull + 8 * buf);
            commit_pair(empty + 8 * stage);
          }
          __syncwarp();
          d += 256 / ti.batch;
          if (++stage == S) { stage = 0; phase ^= 1u; }
          if (last) {
            left = 0;
            if (++buf == 2) { buf = 0; bphase ^= 1u; }
          }
        }
      }
      if (issuer) {
      uint64_t* done = reinterpret_cast<uint64_t*>(smem + kRing) + kDoneBar;
      umma_commit_pair_mc(done, 0x1);
      mbar_wait_drain(done, 0, kDrain);
      }
    } else if (warp >= 2) {
      // ---------------------------------------------------- scale warps
      // fl(sa sw) of kSlotBlocks blocks at a time, 256 numbers a block: full tiles
      // the CTA's 128 rows under each of its two weight blocks (a row's numbers of
      // the slot side by side), swapped tiles the tile's rows under the CTA's weight
      // block.  The rows' factors come by 4-byte asynchronous copies (rows start at
      // any address) two slots ahead; the thread that copied a number multiplies
      // it.  A slot covers several blocks because every hand-over costs the
      // epilogue's warps about 100 cycles, and their round trip with the tensor
      // core is what bounds full tiles (M = 9472, N = 1024, K = 7168: 71 us now; when
      // four blocks a slot came in, it went from 94 to 76).
      const int i0 = threadIdx.x - 64;
      int slot = 0, fslot = 0;            // slot multiplied next, slot filled next
      uint32_t fphase = 0;
      bool ok = true;
      for (int t = pair; ok && t < total; t += pairs) {
        const BTile ti = decode(a, s_start, ntn, t);
        const int row = (ti.swap ? 0 : static_cast<int>(rank) * 128) + i0;
        const float* ps = a.a_scale + ti.row0 + row;
        const int ob = ti.n0 / 128 + (ti.swap ? static_cast<int>(rank) : 0);
        const float* pw = a.w_scale + ti.g * a.ws_g + ob * a.ws_o;
        // Blocks behind the last column are multiplied by 0 and not stored; rows
        // behind the tile's last are not read.
        const bool w0 = ob * 128 < a.width, w1 = !ti.swap && (ob + 1) * 128 < a.width;
        const int nsl = (nkb + kSlotBlocks - 1) / kSlotBlocks;
        // Cell of number i (rows i0 + 64 i, or i & 1 and weight block i >> 1) of block z.
        auto cell = [&](int sl, int z, int i) {
          return scales + sl * kSlotBytes +
                 (ti.swap ? (z * 256 + i * 64 + i0) * 4 : ((i * 64 + i0) * kSlotBlocks + z) * 4);
        };
        auto fill = [&](int j) {
          if (j < nsl) {
            ok = ok && bar_wait(sempty + 8 * fslot, fphase ^ 1u, abort, a.tries);
            for (int z = 0; ok && z < kSlotBlocks && j * kSlotBlocks + z < nkb; ++z) {
              const float* p = ps + static_cast<long long>(j * kSlotBlocks + z) * a.ld_as;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (ti.swap || i < 2) copy4(cell(fslot, z, i), p + 64 * i, row + 64 * i < ti.rows);
            }
            if (++fslot == kScaleSlots) { fslot = 0; fphase ^= 1u; }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
        fill(0);
        fill(1);
        for (int j = 0; j < nsl; ++j) {
          float sw[kSlotBlocks][2];
#pragma unroll
          for (int z = 0; z < kSlotBlocks; ++z) {
            const int kb = j * kSlotBlocks + z;
            sw[z][0] = kb < nkb && w0 ? pw[kb * a.ws_c] : 0.f;
            sw[z][1] = kb < nkb && w1 ? pw[kb * a.ws_c + a.ws_o] : 0.f;
          }
          fill(j + 2);
          if (!__all_sync(kFull, ok)) { ok = false; break; }
          asm volatile("cp.async.wait_group 2;" ::: "memory");
#pragma unroll
          for (int z = 0; z < kSlotBlocks; ++z) {
            if (ti.swap) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t c = cell(slot, z, i);
                st_shared_f32(c, __fmul_rn(ld_shared_f32(c), sw[z][0]));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float v = ld_shared_f32(cell(slot, z, i));
                st_shared_f32(cell(slot, z, i), __fmul_rn(v, sw[z][0]));
                st_shared_f32(cell(slot, z, i + 2), __fmul_rn(v, sw[z][1]));
              }
            }
          }
          __syncwarp();
          if (lane == 0) bar_arrive(sfull + 8 * slot);
          if (++slot == kScaleSlots) slot = 0;
        }
      }
      // No copy is in flight when the CTA goes.
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // --------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tempty0 = mapa_u32(tempty, 0);
    const uint32_t tlane = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    int buf = 0, slots = 0;   // slots read: slot and parity in one
    uint32_t bphase = 0;
    bool ok = true;
    for (int t = pair; ok && t < total; t += pairs) {
      decode_to(a, s_start, ntn, t, &s_tile[warp]);
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      // Products, and before the first read of a slot its scales: those are there long
      // before, so both are tried at once.
      auto wait_products = [&](bool scales_too) {
        const uint32_t sbar = sfull + 8 * (slots % kScaleSlots), sparity = slots / kScaleSlots & 1;
        bool there = true;
        if (scales_too) there = bar_try(sbar, sparity);
        ok = bar_wait(tfull + 8 * buf, bphase, abort, a.tries);
        if (!there) ok = ok && bar_wait(sbar, sparity, abort, a.tries);
        ok = __all_sync(kFull, ok);
        tc_fence_after();
        return ok;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * buf);
        if (++buf == 2) { buf = 0; bphase ^= 1u; }
      };
      auto give_scales = [&]() {
        __syncwarp();
        if (lane == 0) bar_arrive(sempty + 8 * (slots % kScaleSlots));
        slots = (slots + 1) % (2 * kScaleSlots);
      };
      // Full tiles: one block a buffer, four chunks of 32 columns, each one's load under
      // the multiply-adds of the one before, across blocks too: the next block's first
      // chunk is fetched before the last of this one is added.  The buffer is given back
      // as soon as its last chunk has arrived.  (Loads that start afresh with each block:
      // 8192 x 4096 x 7168 takes 247 us instead of 224.)
      auto full_tile = [&]() {
        float4 s4 = make_float4(0.f, 0.f, 0.f, 0.f);
        uint32_t v[2][32];
        auto add = [&](int c, const uint32_t(&x)[32], uint64_t s2) {
#pragma unroll
          for (int i = 0; i < 16; ++i) fma2(acc[c * 16 + i], pack2u(x[2 * i], x[2 * i + 1]), s2);
        };
        if (!wait_products(true)) return;
        tmem_ld32(tlane + buf * 256 + half * 128, v[0]);
        for (int kb = 0; kb < nkb; ++kb) {
          const int z = kb % kSlotBlocks;
          const uint32_t tb = tlane + buf * 256 + half * 128;
          if (z == 0) {
            s4 = ld_shared_f32x4(scales + slots % kScaleSlots * kSlotBytes + (half * 128 + q * 32 + lane) * 16);
            give_scales();
          }
          const uint64_t s2 = pack2(s4.x, s4.x);
          tmem_wait32(v[0]);
          tmem_ld32(tb + 32, v[1]);
          add(0, v[0], s2);
          tmem_wait32(v[1]);
          tmem_ld32(tb + 64, v[0]);
          add(1, v[1], s2);
          tmem_wait32(v[0]);
          tmem_ld32(tb + 96, v[1]);
          add(2, v[0], s2);
          tmem_wait32(v[1]);
          release();
          if (kb + 1 < nkb) {
            if (!wait_products(z == kSlotBlocks - 1)) return;
            tmem_ld32(tlane + buf * 256 + half * 128, v[0]);
          }
          add(3, v[1], s2);
          s4 = make_float4(s4.y, s4.z, s4.w, 0.f);
        }
      };
      // Swapped tiles: BATCH blocks a buffer; the 128 / BATCH columns that a warp can
      // have of a block are loaded CH at a time, all blocks' at once.
      auto swapped_tile = [&](auto batch, auto chunk, const int hc) {
        constexpr int BATCH = decltype(batch)::value, CH = decltype(chunk)::value, N = 128 / BATCH / CH;
        for (int kb = 0; kb < nkb; kb += BATCH) {
          const int z = kb % kSlotBlocks;
          if (!wait_products(z == 0)) return;
          const uint32_t tb = tlane + buf * 256 + half * hc;
          const uint32_t sc = scales + slots % kScaleSlots * kSlotBytes + (z * 256 + half * hc) * 4;
#pragma unroll
          for (int c = 0; c < N; ++c) {
            if (c * CH >= hc) break;
            uint32_t v[BATCH][CH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) tmem_ld<CH>(tb + j * (256 / BATCH) + c * CH, v[j]);
#pragma unroll
            for (int j = 0; j < BATCH; ++j) tmem_wait<CH>(v[j]);
            if ((c + 1) * CH >= hc) release();
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
              if (kb + j >= nkb) break;
#pragma unroll
              for (int i = 0; i < CH / 4; ++i) {
                uint64_t lo, hi;
                ld_shared_pairs(sc + (j * 256 + c * CH + 4 * i) * 4, lo, hi);
                fma2(acc[c * (CH / 2) + 2 * i], pack2u(v[j][4 * i], v[j][4 * i + 1]), lo);
                fma2(acc[c * (CH / 2) + 2 * i + 1], pack2u(v[j][4 * i + 2], v[j][4 * i + 3]), hi);
              }
            }
          }
          if (z + BATCH == kSlotBlocks || kb + BATCH >= nkb) give_scales();
        }
      };
      {
        const volatile BTile& ti = s_tile[warp];
        if (!ti.swap) full_tile();
        else if (ti.batch == 4) swapped_tile(std::integral_constant<int, 4>{}, std::integral_constant<int, 8>{}, ti.nt >> 1);
        else swapped_tile(std::integral_constant<int, 2>{}, std::integral_constant<int, 32>{}, ti.nt >> 1);
      }
      if (!ok) break;
      // Read again rather than kept in registers over the loop.
      asm volatile("" ::: "memory");
      const volatile BTile& ti = s_tile[warp];
      const int hc = ti.nt >> 1;
      uint8_t* stage_w = smem + kRing + kBarSpace + (warp - 4) * kEpiSlot;

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
        // cover 128-byte row segments (chunk m of row r at m ^ (r & 7)): 16 bytes a
        // lane where rows start on 16 bytes and the columns are all there.
        const int r0 = static_cast<int>(rank) * 128 + q * 32;
        const int col0 = ti.n0 + half * 128;
        const int rows = ti.rows - r0;
        const bool fast = a.out_vec && col0 + 128 <= a.width;
        Out* base = out + static_cast<size_t>(ti.row0 + r0 + (lane >> 3)) * a.ldo + col0 + (lane & 7) * kPer;
        const size_t step = static_cast<size_t>(a.ldo) * 4;
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
          Out* dst = base + p * kSeg;
          if (fast) {
#pragma unroll
            for (int it = 0; it < 8; ++it, dst += step) {
              const int r = it * 4 + (lane >> 3), ch = lane & 7;
              const uint4 u = *reinterpret_cast<const uint4*>(stage_w + r * 128 + ((ch ^ (r & 7)) << 4));
              if (r < rows) *reinterpret_cast<uint4*>(dst) = u;
            }
          } else if (a.out_vec) {
            const int col = col0 + p * kSeg + (lane & 7) * kPer;
            for (int it = 0; it < 8; ++it, dst += step) {
              const int r = it * 4 + (lane >> 3), ch = lane & 7;
              union { uint4 u; Out e[kPer]; } x;
              x.u = *reinterpret_cast<const uint4*>(stage_w + r * 128 + ((ch ^ (r & 7)) << 4));
              if (r >= rows) continue;
              if (col + kPer <= a.width) {
                *reinterpret_cast<uint4*>(dst) = x.u;
              } else {
#pragma unroll
                for (int z = 0; z < kPer; ++z)
                  if (col + z < a.width) dst[z] = x.e[z];
              }
            }
          } else {
            store_segment<Out>(out + static_cast<size_t>(ti.row0 + r0) * a.ldo + col0 + p * kSeg, a.ldo, rows,
                               a.width - col0 - p * kSeg, stage_w, lane);
          }
        }
      } else {
        // A thread's column: 32 lanes write 32 neighbouring columns of one row.
        const int col = ti.n0 + static_cast<int>(rank) * 128 + q * 32 + lane;
        const int valid = min(hc, ti.rows - half * hc);
        Out* dst = out + static_cast<size_t>(ti.row0 + half * hc) * a.ldo + col;
#pragma unroll
        for (int i = 0; i < kSwapRows / 4; ++i) {
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

// ------------------------------------------------------------ few tiles
// Products with too few tiles to fill the device with the kernel above (single
// tokens against one weight matrix): a cluster of C CTAs takes one tile of 128
// weight rows x up to 32 rows of A and divides the contraction's blocks into C runs.
// Each CTA streams its run and keeps its block sums P_b in TMEM, side by side; then
// the sums walk through the cluster: CTA 0 adds its blocks to zero, hands its
// 128 x rows fp32 sums to CTA 1 through distributed shared memory, which adds its
// own, and so on; the last one stores.  Every element is acc = fma(P_b, fl(sa sw),
// acc) with b ascending, as above: the same bits.
// Bound by the weights' stream and the walk: a CTA alone streams about 100 GB/s, so
// the split brings M = 8, N = 4096, K = 7168 from 32 busy SMs to 128 (20 -> 13.3 us);
// the walk costs about 1.5 us a CTA.
// Roles: warp 0 TMA, warp 1 MMA, warps 2-3 scales, warps 4-7 sums (a thread one
// weight row).
constexpr int kThinThreads = 256;
constexpr int kThinRing = 176 * 1024;
constexpr int kThinMost = 12;
constexpr int kThinRows = 32;
constexpr int kThinSums = kThinRows * 128 * 4;   // sum_at
constexpr int kThinSmem = 1024 + kThinRing + 512 + kThinSums + 512 * 4;

__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// bar_wait for a barrier that another CTA of the cluster arrives on after writing
// this CTA's shared memory.
__device__ __forceinline__ bool bar_wait_cluster(uint32_t bar, uint32_t parity, uint32_t abort, int tries) {
  for (int i = 0; i < tries; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (ld_shared_i32(abort) != 0) return false;
  }
  asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(abort) : "memory");
  atomicExch(&g_operator_error, kDevTimeout);
  return false;
}

// Byte of the sums of weight row `row` and rows 4 i .. 4 i + 3 of A: four numbers
// together, so that a warp moves them 16 bytes a thread without bank conflicts.
__device__ __forceinline__ uint32_t sum_at(int row, int i) { return (i * 128 + row) * 16; }

template <int TRANS, typename Out>
__global__ void __launch_bounds__(kThinThreads, 1) k_block_gemm_thin(const __grid_constant__ BlockGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = min(kThinMost, kThinRing / (kWSlot + a.a_slot));
  uint8_t* sW = smem;
  uint8_t* sA = smem + S * kWSlot;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int s_start[kMatmulMaxGroups + 1];
  const uint32_t smem0 = smem_u32(smem);
  const uint32_t full = smem0 + kThinRing, empty = full + 8 * kThinMost;
  const uint32_t tfull = empty + 8 * kThinMost, sfull = tfull + 8, sums_in = sfull + 8;
  const uint32_t sums = smem0 + kThinRing + 512;
  const uint32_t scales = sums + kThinSums;   // [block of the run][row of A]
  const uint32_t abort = smem_u32(&abort_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank()), C = a.split;
  if (threadIdx.x == 0) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kThinRing);
    for (int s = 0; s < 2 * kThinMost + 1; ++s) mbar_init(&bars[s], 1);
    mbar_init(&bars[2 * kThinMost + 1], 2);     // scales: one arrival a scale warp
    mbar_init(&bars[2 * kThinMost + 2], 4);     // sums: one arrival a warp of the CTA before
    abort_flag = 0;
    fence_barrier_init();
    prefetch_map(&a.mapA[box_of(a.tile_rows)]);
    prefetch_map(&a.mapW);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, kCols);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  griddep_wait();
  griddep_launch();

  const int ntn = (a.width + 127) / 128;
  const int nkb = (a.con + 127) / 128;
  if (warp == 0) scan_groups(a, s_start, ntn, lane);
  __syncthreads();
  const int t = blockIdx.x / C;
  if (t < s_start[a.G]) {   // the same for all CTAs of the cluster
    const BTile ti = decode<128>(a, s_start, ntn, t);
    const int per = (nkb + C - 1) / C;
    const int kb0 = min(nkb, rank * per), n = min(nkb, kb0 + per) - kb0;   // this CTA's run (may be empty)
    const int box = box_of(ti.nt);
    if (warp == 0 && lane == 0) {
      const uint32_t bytes = (16u << box) * 128u;
      bool ok = static_cast<int>(bytes) <= a.a_slot && n * ti.nt <= 512;
      if (!ok) {
        atomicExch(&g_operator_error, kDevBadIndex);
        abort_flag = 1;
      }
      int last[kThinMost];   // parity of the copy last issued to a stage
      for (int s = 0; s < S; ++s) last[s] = -1;
      for (int i = 0; ok && i < min(n, a.load_blocks); ++i) {
        const int s = i % S;
        const uint32_t ph = static_cast<uint32_t>(i / S) & 1u;
        if (!bar_wait(empty + 8 * s, ph ^ 1u, abort, a.tries)) { ok = false; break; }
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full + 8 * s),
                     "r"(bytes + kWSlot) : "memory");
        tma_load_2d(sA + s * a.a_slot, &a.mapA[box], (kb0 + i) * 128, ti.row0,
                    reinterpret_cast<uint64_t*>(smem + kThinRing) + s);
        if (TRANS) tma_load_3d(sW + s * kWSlot, &a.mapW, ti.n0, (kb0 + i) * 128, ti.g, full + 8 * s);
        else tma_load_3d(sW + s * kWSlot, &a.mapW, (kb0 + i) * 128, ti.n0, ti.g, full + 8 * s);
        last[s] = static_cast<int>(ph);
      }
      if (!ok || a.load_blocks < n)
        for (int s = 0; s < S; ++s)
          if (last[s] >= 0) mbar_wait_drain(reinterpret_cast<uint64_t*>(smem + kThinRing) + s, last[s], kDrain);
    } else if (warp == 1) {
      const bool issuer = elect_one();
      // The weights are the M operand.
      const uint32_t idesc = idesc_e4m3_f32(128, ti.nt) | (TRANS ? 1u << 15 : 0u);
      const uint32_t tok_lo = (((smem0 + S * kWSlot) >> 4) & 0x3FFFu) | 1u << 16;
      const uint32_t w_lo = ((smem0 >> 4) & 0x3FFFu) | (TRANS ? 16384u >> 4 : 1u) << 16;
      int s = 0;
      uint32_t ph = 0;
      for (int i = 0; i < n; ++i) {
        const bool ok = bar_wait(full + 8 * s, ph, abort, a.tries);
        if (!__all_sync(kFull, ok)) break;
        tc_fence_after();
        const uint32_t alo = w_lo + s * (kWSlot >> 4), blo = tok_lo + s * (static_cast<uint32_t>(a.a_slot) >> 4);
        if (issuer) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_e4m3(tmem_base + i * ti.nt, (kDescHi << 32) | (alo + kk * (TRANS ? 4096 >> 4 : 2)),
                      (kDescHi << 32) | (blo + kk * 2), idesc, kk != 0 ? 1u : 0u);
          commit_one(empty + 8 * s);
        }
        __syncwarp();
        if (++s == S) { s = 0; ph ^= 1u; }
      }
      // Also when the run was cut short: the MMAs issued are done before TMEM goes.
      if (issuer) commit_one(tfull);
    } else if (warp == 2 || warp == 3) {
      // fl(sa sw) of the run's blocks and the tile's rows (rows behind it: 0).
      const int ob = ti.n0 / 128;
      const float* pw = a.w_scale + ti.g * a.ws_g + ob * a.ws_o;
      for (int j = threadIdx.x - 64; j < n * ti.nt; j += 64) {
        const int b = j / ti.nt, r = j - b * ti.nt;
        float v = 0.f;
        if (r < ti.rows) v = __fmul_rn(a.a_scale[(kb0 + b) * a.ld_as + ti.row0 + r], pw[(kb0 + b) * a.ws_c]);
        st_shared_f32(scales + 4 * j, v);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(sfull);
    } else if (warp >= 4) {
      const int q = warp & 3, row = q * 32 + lane;   // TMEM lane = weight row
      const uint32_t tl = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      bool ok = bar_wait(sfull, 0, abort, a.tries) && bar_wait(tfull, 0, abort, a.tries);
      if (rank > 0) ok = ok && bar_wait_cluster(sums_in, 0, abort, a.tries);
      ok = __all_sync(kFull, ok);
      tc_fence_after();
      const int col = ti.n0 + row;
      const uint32_t next = rank + 1 < C ? mapa_u32(sums, rank + 1) : 0u;
      Out* out = static_cast<Out*>(a.out) + static_cast<size_t>(ti.row0) * a.ldo + col;
      for (int c = 0; ok && c < ti.nt; c += 16) {
        uint64_t acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[i] = 0;
        }
        if (rank > 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) ld_shared_pairs(sums + sum_at(row, c / 4 + i), acc[2 * i], acc[2 * i + 1]);
        }
        uint32_t v[2][16];
        if (n > 0) tmem_ld<16>(tl + c, v[0]);
        // Two blocks a turn, the second's load under the first's multiply-adds.
        for (int b = 0; b < n; b += 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (b + h >= n) break;
            tmem_wait<16>(v[h]);
            if (b + h + 1 < n) tmem_ld<16>(tl + (b + h + 1) * ti.nt + c, v[h ^ 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint64_t lo, hi;
              ld_shared_pairs(scales + ((b + h) * ti.nt + c + 4 * i) * 4, lo, hi);
              fma2(acc[2 * i], pack2u(v[h][4 * i], v[h][4 * i + 1]), lo);
              fma2(acc[2 * i + 1], pack2u(v[h][4 * i + 2], v[h][4 * i + 3]), hi);
            }
          }
        }
        if (rank + 1 < C) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(next + sum_at(row, c / 4 + i)), "l"(acc[2 * i]),
                         "l"(acc[2 * i + 1])
                         : "memory");
        } else if (col < a.width) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 f = unpack2(acc[i / 2]);
            const float x = i & 1 ? f.y : f.x;
            if (c + i < ti.rows) {
              if constexpr (sizeof(Out) == 2)
                out[static_cast<size_t>(c + i) * a.ldo] = static_cast<Out>(pack_bf16x2(x, 0.f) & 0xFFFFu);
              else
                out[static_cast<size_t>(c + i) * a.ldo] = x;
            }
          }
        }
      }
      // After a time-out the next CTA is told all the same; it has its own error
      // to find, or passes on what it has: the error word says the output is not whole.
      __syncwarp();
      if (rank + 1 < C && lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_u32(sums_in, rank + 1))
                     : "memory");
      tc_fence_before();
    }
  }
  // No CTA leaves while another may still write to it; TMEM is free of running MMAs:
  // the sums' warps waited for them (or, after a time-out, this one does).
  if (warp == 1 && t < s_start[a.G]) mbar_wait_drain(reinterpret_cast<uint64_t*>(smem + kThinRing) + 2 * kThinMost, 0, kDrain);
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kCols);
  }
}

using Kernel = void (*)(BlockGemmArgs);
Kernel kernel_of(bool transposed, bool f32) {
  if (transposed) return f32 ? k_block_gemm<1, float> : k_block_gemm<1, uint16_t>;
  return f32 ? k_block_gemm<0, float> : k_block_gemm<0, uint16_t>;
}

Kernel thin_kernel_of(bool transposed, bool f32) {
  if (transposed) return f32 ? k_block_gemm_thin<1, float> : k_block_gemm_thin<1, uint16_t>;
  return f32 ? k_block_gemm_thin<0, float> : k_block_gemm_thin<0, uint16_t>;
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
    const void* thin = reinterpret_cast<const void*>(thin_kernel_of(v & 1, v & 2));
    if (cudaFuncSetAttribute(thin, cudaFuncAttributeMaxDynamicSharedMemorySize, kThinSmem) != cudaSuccess) n = 0;
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
  if (a.split > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(max_tiles) * a.split);
    cfg.blockDim = dim3(kThinThreads);
    cfg.dynamicSmemBytes = kThinSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, thin_kernel_of(a.transposed != 0, a.out_f32 != 0), a);
  }
  return launch_k(kernel_of(a.transposed != 0, a.out_f32 != 0), dim3(2 * std::min(pairs, max_tiles)), dim3(kThreads),
                  kSmem, s, true, a);
}

cudaError_t read_operator_error(int* value, cudaStream_t s) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  void* p = nullptr;
  cudaError_t rc = cudaGetSymbolAddress(&p, g_operator_taken);
  if (rc != cudaSuccess) return rc;
  k_take_operator_error<<<1, 1, 0, s>>>();
  rc = cudaGetLastError();
  if (rc == cudaSuccess) rc = cudaMemcpyAsync(value, p, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (rc == cudaSuccess) rc = cudaStreamSynchronize(s);
  return rc;
}

}  // namespace moe
