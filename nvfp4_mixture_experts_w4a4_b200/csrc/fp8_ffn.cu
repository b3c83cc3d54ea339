// fp8_moe_ffn_forward: the routed feed-forward layer on FP8 weights with a scale per 128 x 128
// block.  Batches of at most 16 tokens are one launch (fp8_layer.cu).  Otherwise routing and permutation
// are the NVFP4 layer's (one order for both), x is quantised per row and 128 columns into expert order,
// and the products run as a stream of weights (fp8_layer.cu) or in tiles of rows (fp8_tile.cu).
#include "ffn_gemv.cuh"
#include "fp8.cuh"
#include "fp8_tile.cuh"

namespace nvfp4moe {
namespace {

constexpr int kPlaceThreads = 256;
constexpr int kRowTile = 128;  // rows of a tile of the grouped products

// x [T][H] bf16 -> E4M3 rows in expert order: each 128-element group is quantised once (half a
// warp, 16 bytes a lane) and written to the k rows of its token.  Block 0 writes the list of row
// groups instead.
__global__ void __launch_bounds__(kPlaceThreads)
fp8_place_kernel(const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ pair_to_row,
                 const int32_t* __restrict__ offsets, int T, int H, int E, int k, uint8_t* __restrict__ codes,
                 float* __restrict__ scale, int group, int4* __restrict__ tiles, int* __restrict__ counters) {
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0) {
    __shared__ int s_sum[kPlaceThreads / 32];
    fp8_list_groups<kPlaceThreads>(E, group, [&](int e) { return offsets[e]; },
                                   [&](int e) { return offsets[e + 1] - offsets[e]; }, s_sum, tiles, counters);
    return;
  }
  const int nb = (H + FP8_BLOCK - 1) / FP8_BLOCK;
  const int64_t groups = int64_t(T) * nb;
  const int64_t g = (int64_t(blockIdx.x - 1) * kPlaceThreads + threadIdx.x) / 16;
  const int sub = threadIdx.x & 15;
  const int64_t t = g / nb;
  const int b = int(g - t * nb), c = b * FP8_BLOCK + sub * 8;
  const bool live = g < groups && c < H;  // H is a multiple of 16: eight elements exist or none
  const uint4 u = live ? __ldg(reinterpret_cast<const uint4*>(x + t * H + c)) : make_uint4(0u, 0u, 0u, 0u);
  uint32_t m = fp8_amax_bits(bf16x8_max(0u, u));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const Fp8ScaleBf16 f = fp8_scale_bf16(m);
  const uint2 out = fp8_encode8(u, f);
  if (!live) return;
  for (int j = 0; j < k; ++j) {
    const int64_t row = __ldg(pair_to_row + t * k + j);
    *reinterpret_cast<uint2*>(codes + row * H + c) = out;
    if (sub == 0) scale[row * nb + b] = f.scale;
  }
}

struct Layout {
  int64_t ids, w, counts, offsets, padded, pair_to_row, row_token, row_pair, tile_expert, active, scratch, groups,
      x_codes, x_scale, h_codes, h_scale, slots, counters, parts, total;
  int64_t pairs;
  int group, max_row_tiles;  // rows of a group, groups at most
  bool single, stream;
};

nvfp4moe_status check_desc(const fp8_moe_ffn_desc* d, const char* fn) {
  NVFP4_REQUIRE(d != nullptr, NVFP4MOE_INVALID_ARG, "%s: NULL descriptor", fn);
  NVFP4_REQUIRE(d->T >= 0, NVFP4MOE_INVALID_ARG, "%s: T < 0", fn);
  NVFP4_REQUIRE(d->H >= 16 && d->H % 16 == 0 && d->H <= (1 << 20), NVFP4MOE_UNSUPPORTED_SHAPE,
                "%s: H=%d is not a multiple of 16 in [16, 2^20]", fn, d->H);
  NVFP4_REQUIRE(d->I >= 16 && d->I % 16 == 0 && d->I <= (1 << 20), NVFP4MOE_UNSUPPORTED_SHAPE,
                "%s: I=%d is not a multiple of 16 in [16, 2^20]", fn, d->I);
  NVFP4_REQUIRE(d->E >= 1 && d->E <= 1024, NVFP4MOE_UNSUPPORTED_SHAPE, "%s: E=%d outside [1, 1024]", fn, d->E);
  NVFP4_REQUIRE(d->top_k >= 1 && d->top_k <= 32 && d->top_k <= d->E, NVFP4MOE_UNSUPPORTED_SHAPE,
                "%s: top_k=%d outside [1, min(E, 32)]", fn, d->top_k);
  NVFP4_REQUIRE(int64_t(d->T) * d->top_k <= (int64_t(1) << 24), NVFP4MOE_UNSUPPORTED_SHAPE, "%s: T*top_k > 2^24", fn);
  NVFP4_REQUIRE(d->launch_mode == NVFP4MOE_LAUNCH_AUTO || d->launch_mode == NVFP4MOE_LAUNCH_SINGLE ||
                    d->launch_mode == NVFP4MOE_LAUNCH_MULTI,
                NVFP4MOE_INVALID_ARG, "%s: launch_mode=%d", fn, d->launch_mode);
  NVFP4_REQUIRE(d->launch_mode != NVFP4MOE_LAUNCH_SINGLE || d->T == 0 || fp8_layer_fits(d->T, d->H, d->I, d->E, d->top_k),
                NVFP4MOE_UNSUPPORTED_SHAPE, "%s: T=%d H=%d does not fit the single launch", fn, d->T, d->H);
  return NVFP4MOE_OK;
}

// One launch for the batches it fits, unless the caller says otherwise.
bool takes_single(const fp8_moe_ffn_desc& d) {
  return d.launch_mode != NVFP4MOE_LAUNCH_MULTI && d.T > 0 && fp8_layer_fits(d.T, d.H, d.I, d.E, d.top_k);
}

// The stream of weights in groups of 32 rows: few rows an expert (20 on average at most: most experts
// are one group, and a 128-row tile would be nearly empty), and a batch short enough that an expert that
// everyone picks is read from L2 eight times at most.  Stream / tiles, us: 64 experts of 2048 x 512, top 10,
// with 10, 20 and 30 rows an expert 64 / 71, 68 / 77, 71 / 79, with 40 85 / 80; 64 experts of 4096 x 1024,
// top 8, with 16, 20, 25 and 32 rows 156 / 175, 161 / 181, 168 / 183, 191 / 186; 8 experts of 2048 x 512, top
// 2, with 15 to 40 rows within 2 %.  (So 20 is on the safe side of the crossing near 30.)  The batch is bounded
// because of popular experts: 512 tokens, 512 experts, Zipf 150 / 136.
bool takes_stream(const fp8_moe_ffn_desc& d) {
  const int64_t P = int64_t(d.T) * d.top_k, touched = P < d.E ? P : d.E;
  return d.T <= 256 && P <= 20 * touched;
}

Layout make_layout(const fp8_moe_ffn_desc& d) {
  Layout L{};
  int64_t at = 0;
  auto put = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const int64_t P = int64_t(d.T) * d.top_k, nH = fp8_blocks(d.H), nI = fp8_blocks(d.I);
  L.pairs = P;
  L.stream = takes_stream(d);
  L.group = L.stream ? kStreamRows : kRowTile;
  L.max_row_tiles = int(P / L.group + (P < d.E ? P : d.E));
  L.single = takes_single(d);
  if (L.single) {
    const Fp8LayerSizes z = fp8_layer_sizes(d.T, d.H, d.I, d.E, d.top_k);
    L.counters = put(z.counters * 4), L.parts = put(z.parts * 4), L.slots = put(z.slots * 4);
    L.h_codes = put(z.h_codes), L.h_scale = put(z.h_scale * 4);
    L.x_codes = put(z.x_codes), L.x_scale = put(z.x_scale * 4);
    L.total = at;
    return L;
  }
  L.ids = put(P * 4), L.w = put(P * 4);
  L.counts = put(d.E * 4), L.offsets = put((d.E + 1) * 4), L.padded = put((d.E + 1) * 4);
  L.pair_to_row = put(P * 4), L.row_token = put(P * 4), L.row_pair = put(P * 4), L.tile_expert = put(P * 4);
  L.active = put((d.E + 1) * 4);
  L.scratch = put(d.T > 0 ? batch_prologue_scratch_bytes(d.T, d.E) : 0);
  L.groups = put((int64_t(L.max_row_tiles) + 1) * 16);
  L.counters = L.stream ? put(int64_t(L.max_row_tiles) * 4) : 0;  // (the tiles count nothing)
  L.x_codes = put(P * d.H), L.x_scale = put(P * nH * 4);
  L.h_codes = put(P * d.I), L.h_scale = put(P * nI * 4);
  L.slots = put(P * d.H * 4);
  L.total = at;
  return L;
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

size_t fp8_moe_ffn_workspace_size(const fp8_moe_ffn_desc* d) {
  if (check_desc(d, "fp8_moe_ffn_workspace_size") != NVFP4MOE_OK) return 0;
  return size_t(make_layout(*d).total);
}

nvfp4moe_status fp8_moe_ffn_forward(const fp8_moe_ffn_desc* desc, const void* x, const float* logits, void* out,
                                    void* workspace, size_t workspace_bytes, nvfp4moe_stream_t stream) {
  const char* fn = "fp8_moe_ffn_forward";
  nvfp4moe_status st = check_desc(desc, fn);
  if (st != NVFP4MOE_OK) return st;
  const fp8_moe_ffn_desc& d = *desc;
  if (d.T == 0) return NVFP4MOE_OK;
  NVFP4_REQUIRE(x && logits && out && workspace, NVFP4MOE_INVALID_ARG, "%s: NULL pointer", fn);
  NVFP4_REQUIRE(d.w13_codes && d.w13_scale && d.w2_codes && d.w2_scale, NVFP4MOE_INVALID_ARG, "%s: NULL weights", fn);
  NVFP4_REQUIRE(aligned16(x) && aligned16(out) && aligned16(d.w13_codes) && aligned16(d.w2_codes) &&
                    reinterpret_cast<uintptr_t>(workspace) % 256 == 0,
                NVFP4MOE_INVALID_ARG, "%s: x, out and the weights need 16-byte alignment, the workspace 256", fn);
  const Layout L = make_layout(d);
  NVFP4_REQUIRE(workspace_bytes >= size_t(L.total), NVFP4MOE_WORKSPACE_TOO_SMALL, "%s: workspace %zu < %zu", fn,
                workspace_bytes, size_t(L.total));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto i32 = [&](int64_t at) { return reinterpret_cast<int32_t*>(ws + at); };
  auto f32 = [&](int64_t at) { return reinterpret_cast<float*>(ws + at); };
  if (L.single) {
    Fp8LayerCall c{};
    c.x = x, c.logits = logits, c.out = out;
    c.T = d.T, c.H = d.H, c.I = d.I, c.E = d.E, c.k = d.top_k;
    c.w13_codes = d.w13_codes, c.w2_codes = d.w2_codes, c.w13_scale = d.w13_scale, c.w2_scale = d.w2_scale;
    c.counters = i32(L.counters), c.parts = f32(L.parts), c.slots = f32(L.slots);
    c.h_codes = ws + L.h_codes, c.h_scale = f32(L.h_scale);
    c.x_codes = ws + L.x_codes, c.x_scale = f32(L.x_scale);
    return launch_fp8_layer(c, s);
  }
  int4* groups = reinterpret_cast<int4*>(ws + L.groups);
  int* counters = L.stream ? i32(L.counters) : nullptr;
  if (prologue_fits(d.T, d.E, d.top_k)) {
    // one cluster launch for routing and permutation, then x (45 tokens, 20 experts of 1040 x 336: 29.5 us, 32.1
    // with the three launches of larger batches; 33 to 64 tokens, 512 experts of 2048 x 512: within 0.5 %)
    st = launch_prologue(x, logits, d.T, d.H, d.E, d.top_k, 1, 0, nullptr, i32(L.ids), f32(L.w), i32(L.counts),
                         i32(L.offsets), i32(L.padded), i32(L.pair_to_row), i32(L.row_token), i32(L.row_pair),
                         i32(L.tile_expert), i32(L.active), nullptr, 1, nullptr, nullptr, nullptr, nullptr, 0, 0, s);
    if (st != NVFP4MOE_OK) return st;
    const int64_t x_groups = int64_t(d.T) * fp8_blocks(d.H);
    const cudaError_t e = launch_dependent(fp8_place_kernel, dim3(unsigned(1 + (x_groups * 16 + kPlaceThreads - 1) / kPlaceThreads)),
                         dim3(kPlaceThreads), 0, s, static_cast<const __nv_bfloat16*>(x),
                         static_cast<const int32_t*>(i32(L.pair_to_row)), static_cast<const int32_t*>(i32(L.offsets)),
                         int(d.T), int(d.H), int(d.E), int(d.top_k), ws + L.x_codes, f32(L.x_scale), L.group, groups,
                         counters);
    NVFP4_REQUIRE(e == cudaSuccess, NVFP4MOE_CUDA_ERROR, "%s: %s", fn, cudaGetErrorString(e));
  } else {
    const Fp8Place place{ws + L.x_codes, f32(L.x_scale), L.group, groups, counters};
    st = launch_batch_prologue(x, logits, d.T, d.H, d.E, d.top_k, 1, 0, nullptr, i32(L.ids), f32(L.w), i32(L.counts),
                               i32(L.offsets), i32(L.padded), i32(L.pair_to_row), i32(L.row_token), i32(L.row_pair),
                               i32(L.tile_expert), i32(L.active), nullptr, 1, nullptr, nullptr, ws + L.scratch, nullptr,
                               nullptr, s, &place);
    if (st != NVFP4MOE_OK) return st;
  }
  GroupedArgs g{};
  g.H = d.H, g.I = d.I, g.E = d.E;
  g.rows = L.pairs;
  g.max_row_tiles = L.max_row_tiles;
  g.tiles = groups;
  g.x_codes = ws + L.x_codes, g.x_scale = f32(L.x_scale);
  g.w13_codes = d.w13_codes, g.w13_scale = d.w13_scale, g.w2_codes = d.w2_codes, g.w2_scale = d.w2_scale;
  g.h_codes = ws + L.h_codes, g.h_scale = f32(L.h_scale), g.slots = f32(L.slots);
  st = L.stream ? launch_fp8_stream(g, counters, s) : launch_fp8_grouped(g, s);
  if (st != NVFP4MOE_OK) return st;
  return launch_combine_rows(f32(L.slots), i32(L.pair_to_row), f32(L.w), d.T, d.H, d.top_k, out, s);
}

}  // extern "C"
