// Declarations of the handle-free expert-layer operators: routing, grouping,
// E4M3 quantisation with one scale per 128 elements, block-scaled products and
// the weighted combine.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"

namespace moe {

constexpr int kRouteMaxE = 1024;     // experts of moe_route
constexpr int kRouteMaxK = 32;       // one slot per lane
constexpr int kRouteMaxPerLane = 32; // experts one lane owns
constexpr int kMatmulMaxGroups = 1024;

// ---------------------------------------------------------------- routing
struct RouteOpArgs {
  const void* logits;   // [T, ld]
  long long ld;
  const float* bias;    // [E] or NULL
  int T, E, k;
  int softmax;          // 1 softmax scores, 0 sigmoid
  int n_groups, topk_groups, group_top;
  int gs;               // experts per group
  int lpg;              // lanes per group (a power of two)
  int cpl;              // experts per lane
  int vec;              // rows may be read 16 bytes at a time (cpl * size a multiple of 16)
  int vec_bias;         // the same for the bias
  int renorm;
  float scale;
  int32_t* idx;         // [T, k]
  float* w;             // [T, k]
};
cudaError_t launch_route(const RouteOpArgs& a, bool bf16, cudaStream_t s);

struct RouteBackArgs {
  const void* logits;   // [T, ld]
  long long ld;
  const int32_t* idx;   // [T, k]
  const float* dw;      // [T, k]
  void* dlogits;        // [T, ld_out], type of logits
  long long ld_out;
  int T, E, k, softmax, renorm;
  int vec;              // 4-element vectors
  float scale;
};
cudaError_t launch_route_backward(const RouteBackArgs& a, bool bf16, cudaStream_t s);

cudaError_t launch_group_rows(const int32_t* idx, int T, int k, int E, int32_t* offsets, int32_t* token_of_row,
                              int32_t* row_of_slot, cudaStream_t s);

// ----------------------------------------------------------- quantisation
struct QuantArgs {
  const void* x;               // [*, ld] bf16 or fp32; gated units: [R, 2I] bf16, gate columns then up
  long long ld;
  const int32_t* token_of_row; // [R] source row of each row (negative: row left as it is), or NULL
  int src_rows;                // rows of x when token_of_row is given
  const int32_t* n_rows;       // device count of rows to write (<= R), or NULL
  int R, K;                    // rows and columns written (gated unit: K = I; its gradient: K = I, 2I written)
  const uint16_t* dh;          // gradient of the gated unit's output [R, ld_dh]
  long long ld_dh;
  uint8_t* codes;              // [R, K] (gradient: [R, 2I])
  float* scales;               // [blocks of 128, ld_s]
  long long ld_s;
  int act;
  int clamped;                 // a SwiGLU clamp is finite
  float gate_clamp, up_clamp, beta_g, beta_u;
};
enum QuantKind : int { kQuantBf16 = 0, kQuantF32 = 1, kQuantGlu = 2, kQuantGluBackward = 3 };
cudaError_t launch_quant_blocks(const QuantArgs& a, int kind, cudaStream_t s);
cudaError_t launch_quant_weights_block(const uint16_t* w, uint8_t* codes, float* scales, int G, int N, int K,
                                       cudaStream_t s);

// --------------------------------------------------------------- products
struct BlockGemmArgs {
  CUtensorMap mapA[4];    // A operand [M, con] E4M3, boxes of 128 codes x 16 / 32 / 64 / 128 rows
  CUtensorMap mapW;       // weights [G, N, K] E4M3, box 128 x 128 of one group
  const int32_t* offsets; // [G + 1] rows of each group, or NULL: one group of M rows
  int G;
  int M;
  int con;                // contraction extent (K, or N when transposed)
  int width;              // output columns (N, or K when transposed)
  int transposed;
  int tile_rows;          // rows per tile: 256 (full tiles with the rows as the MMA's M), or fewer
                          // (every tile with the weights as M)
  int a_slot;             // A bytes per stage
  int split;              // 0, or CTAs that share a tile's contraction (products of few tiles)
  const float* a_scale;   // [con / 128, ld_as]
  long long ld_as;
  const float* w_scale;   // group g, output block o, contraction block c at g * ws_g + o * ws_o + c * ws_c
  long long ws_g, ws_o, ws_c;
  void* out;              // [M, ldo]
  long long ldo;
  int out_f32;
  int out_vec;            // rows of out start on 16-byte boundaries
  int load_blocks;        // blocks of the contraction that are loaded: all (fewer: the waits' self-test)
  int tries;              // limit of a wait
};
cudaError_t launch_block_gemm(const BlockGemmArgs& a, int max_tiles, cudaStream_t s);
int block_gemm_pairs();                       // CTA pairs resident at once (0: the device cannot run it)
cudaError_t read_operator_error(int* value, cudaStream_t s);   // read and clear; synchronises s

// ---------------------------------------------------------------- combine
struct CombineArgs {
  const void* y;               // [rows, ld_y] bf16 or fp32
  long long ld_y;
  int rows;                    // rows of y (indexes outside [0, rows) add nothing)
  const int32_t* row_of_slot;  // [T, k]
  const float* w;              // [T, k] or NULL (all 1)
  const uint16_t* addend;      // [T, D] bf16 or NULL
  int T, k, D;
  void* out;                   // forward: [T, D]
  const uint16_t* dout;        // backward: [T, D] bf16
  void* dy;                    // backward: [rows, ld_y], type of y
  float* dw;                   // backward: [T, k] or NULL
};
cudaError_t launch_combine_rows(const CombineArgs& a, bool y_f32, bool out_f32, cudaStream_t s);
cudaError_t launch_combine_rows_backward(const CombineArgs& a, bool y_f32, cudaStream_t s);

}  // namespace moe
