// Launch interface of the FP8 tile kernel (fp8_tile.cu).
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace nvfp4moe {

struct TileParams {
  int M, N;                  // dense: rows of A and B; down: N = H
  int nkb;                   // 128-blocks of K
  int nsb;                   // 128-blocks of B's rows (of one matrix)
  int n_mt, n_nt;            // row tiles (dense), column tiles
  int a_box;                 // rows of one TMA box of A
  int split;                 // CTAs that share a tile's K
  const int4* tiles;         // grouped: [0].x row tiles, then {expert, first row, rows, -} each
  const float* sa;           // scales of A: row pitch lda_s
  const float* sb;           // scales of B: 128-row block pitch ldb_s, matrix pitch sb_e
  int64_t lda_s, ldb_s, sb_e;
  void* D;
  int64_t ldd;
  int d_f32, d_vec;
  uint8_t* h_codes;          // gate/up: h in E4M3, rows of A
  float* h_scale;
  int64_t ldh, ldh_s;
  int I;
  uint32_t* status;
};

// Columns of a tile, CTAs that split its K, and whether a pair of CTAs runs a tile of 256 rows.
struct DensePlan {
  int bn, split;
  bool pair;
};
DensePlan fp8_dense_plan(int64_t M, int64_t N, int64_t K);

nvfp4moe_status launch_fp8_dense(const uint8_t* A, int64_t lda, const float* A_scale, int64_t lda_s, const uint8_t* B,
                                 int64_t ldb, const float* B_scale, int64_t ldb_s, int64_t M, int64_t N, int64_t K,
                                 void* D, int64_t ldd, int d_f32, cudaStream_t s);

// Gate/up (SwiGLU, h in E4M3) then down over the rows of x in expert order.
struct GroupedArgs {
  int H, I, E;
  int64_t rows;              // rows of x_codes, h_codes and slots
  int max_row_tiles;         // an upper bound of tiles[0].x
  const int4* tiles;
  const uint8_t* x_codes;    // [rows][H]
  const float* x_scale;      // [rows][H / 128]
  const uint8_t* w13_codes;  // [E][2][I][H]
  const float* w13_scale;    // [E][2][I / 128][H / 128]
  const uint8_t* w2_codes;   // [E][H][I]
  const float* w2_scale;     // [E][H / 128][I / 128]
  uint8_t* h_codes;          // [rows][I]
  float* h_scale;            // [rows][I / 128]
  float* slots;              // [rows][H]
};
nvfp4moe_status launch_fp8_grouped(const GroupedArgs& g, cudaStream_t s);

// Tensor map of E4M3 matrices [mats][rows][K], rows `pitch` bytes apart and matrices `mat_pitch`; box
// 128 bytes x box_rows, 128-byte swizzle.  Rows and bytes past the ends read as zero.
nvfp4moe_status make_fp8_map(CUtensorMap* map, const void* base, int64_t K, int64_t rows, int64_t mats, int64_t pitch,
                             int64_t mat_pitch, int box_rows);

// The whole layer in one persistent launch, for batches of at most 16 tokens (fp8_layer.cu).
struct Fp8LayerSizes {
  int64_t counters, parts, slots, h_codes, h_scale, x_codes, x_scale;  // elements of their types below
};
struct Fp8LayerCall {
  const void* x;
  const float* logits;
  int T, H, I, E, k;
  const uint8_t *w13_codes, *w2_codes;
  const float *w13_scale, *w2_scale;
  int* counters;
  float* parts;
  float* slots;
  uint8_t* h_codes;
  float* h_scale;
  uint8_t* x_codes;
  float* x_scale;
  void* out;
};
// The same stream over rows in expert order, for batches whose experts get few rows each: g.tiles
// lists groups of at most kStreamRows rows; counters: as many zeros as groups.
constexpr int kStreamRows = 32;
nvfp4moe_status launch_fp8_stream(const GroupedArgs& g, int* counters, cudaStream_t s);

bool fp8_layer_fits(int T, int H, int I, int E, int k);
Fp8LayerSizes fp8_layer_sizes(int T, int H, int I, int E, int k);
nvfp4moe_status launch_fp8_layer(const Fp8LayerCall& c, cudaStream_t s);

}  // namespace nvfp4moe
