// fp8_quantize: bf16 / fp32 -> E4M3 with one fp32 scale per 1 x 128 or 128 x 128 group.
//
// Each element is read once and each code written once, so the bound is memory: 3 (bf16) or 5
// (fp32) bytes an element.  A row group is held by half a warp (bf16: 16 bytes a lane) or a whole
// one (fp32), its maximum found by shuffles; four steps are loaded before the first is used.  A
// square block is held in the registers of one CTA (64 elements a thread), so it too is read once.
// Rows whose start, pitch or length does not allow 16-byte loads take scalar ones.
#include "fp8.cuh"

namespace nvfp4moe {
namespace {

struct QuantArgs {
  const void* x;
  int64_t batch, rows, K, ldx, x_batch;
  uint8_t* codes;
  int64_t ldc, c_batch;
  float* scale;
  int64_t lds, s_batch;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(v);
  else return v;
}

// VEC elements from p (n of them exist); VECTOR: p is aligned to VEC elements.
template <typename T, int VEC, bool VECTOR>
__device__ __forceinline__ void load_elements(const T* p, int n, float* v) {
  if (VECTOR && n >= VEC) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < VEC / 8; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(p) + i);
        v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}

// 4 * W codes to p (n of them exist); ALIGNED: p is aligned to 4 * W bytes.
template <int W, bool ALIGNED>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, const uint32_t* w) {
  if (ALIGNED && n >= 4 * W) {
    if constexpr (W == 1) *reinterpret_cast<uint32_t*>(p) = w[0];
    else if constexpr (W == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * W; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
}

constexpr int kThreads = 256;

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kThreads) fp8_rows_kernel(QuantArgs a) {
  constexpr int VEC = 16 / sizeof(T);      // elements a lane: one 16-byte load
  constexpr int LANES = FP8_BLOCK / VEC;   // lanes a group: 16 (bf16) or 32 (fp32)
  constexpr int DEPTH = 4;                 // groups in flight a lane
  const int64_t nb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK;
  const int64_t groups = a.batch * a.rows * nb;
  const int sub = threadIdx.x % LANES;
  const int64_t first = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / LANES;
  const int64_t step = int64_t(gridDim.x) * (kThreads / LANES);
  const T* x = static_cast<const T*>(a.x);
  // the loop's trip count is the same for the lanes of a warp: `first` less the lane's own share
  const int64_t warp_first = (int64_t(blockIdx.x) * kThreads + (threadIdx.x & ~31)) / LANES;
  for (int64_t base = 0; warp_first + base < groups; base += DEPTH * step) {
    float v[DEPTH][VEC];
    int64_t row[DEPTH];
    int b[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int64_t g = first + base + d * step;
      row[d] = -1;
      b[d] = 0;
      if (g < groups) {
        row[d] = groups <= INT32_MAX ? int64_t(uint32_t(g) / uint32_t(nb)) : g / nb;
        b[d] = int(g - row[d] * nb);
        const int64_t bi = a.batch == 1 ? 0 : row[d] / a.rows, r = row[d] - bi * a.rows;
        const int64_t c = int64_t(b[d]) * FP8_BLOCK + sub * VEC;
        load_elements<T, VEC, VECTOR>(x + bi * a.x_batch + r * a.ldx + c, int(min(a.K - c, int64_t(VEC))), v[d]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[d][i] = 0.0f;
      }
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < VEC; ++i) m = max(m, abs_bits(v[d][i]));
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const Fp8Scale f = fp8_scale(m);
      if (row[d] >= 0) {
        const int64_t bi = a.batch == 1 ? 0 : row[d] / a.rows, r = row[d] - bi * a.rows;
        const int64_t c = int64_t(b[d]) * FP8_BLOCK + sub * VEC;
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) w[i] = fp8_encode4(v[d] + 4 * i, f);
        store_codes<VEC / 4, VECTOR>(a.codes + bi * a.c_batch + r * a.ldc + c, int(min(a.K - c, int64_t(VEC))), w);
        if (sub == 0) a.scale[bi * a.s_batch + r * a.lds + b[d]] = f.scale;
      }
    }
  }
}

// One CTA per 128 x 128 block: warp w holds rows w, w + 8, ...; a lane four consecutive columns.
template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kThreads) fp8_blocks_kernel(QuantArgs a) {
  constexpr int WARPS = kThreads / 32, ROWS = FP8_BLOCK / WARPS;
  __shared__ uint32_t s_max[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t nb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK, nr = (a.rows + FP8_BLOCK - 1) / FP8_BLOCK;
  const int64_t blk = blockIdx.x;
  const int64_t bi = blk / (nb * nr), rb = blk / nb - bi * nr, b = blk % nb;
  const int64_t c = b * FP8_BLOCK + lane * 4;
  const int n = int(max(int64_t(0), min(a.K - c, int64_t(4))));
  const T* x = static_cast<const T*>(a.x) + bi * a.x_batch + c;
  float v[ROWS][4];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int64_t r = rb * FP8_BLOCK + warp + i * WARPS;
    const int m = r < a.rows ? n : 0;
    const T* p = x + r * a.ldx;
    if (VECTOR && m == 4) {
      if constexpr (sizeof(T) == 2) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        v[i][0] = __uint_as_float(u.x << 16), v[i][1] = __uint_as_float(u.x & 0xFFFF0000u);
        v[i][2] = __uint_as_float(u.y << 16), v[i][3] = __uint_as_float(u.y & 0xFFFF0000u);
      } else {
        load_elements<T, 4, true>(p, 4, v[i]);
      }
    } else {
      load_elements<T, 4, false>(p, m, v[i]);
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, abs_bits(v[i][j]));
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
  m = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) m = max(m, s_max[w]);
  const Fp8Scale f = fp8_scale(m);
  if (threadIdx.x == 0) a.scale[bi * a.s_batch + rb * a.lds + b] = f.scale;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int64_t r = rb * FP8_BLOCK + warp + i * WARPS;
    if (r < a.rows && n > 0) {
      const uint32_t w = fp8_encode4(v[i], f);
      store_codes<1, VECTOR>(a.codes + bi * a.c_batch + r * a.ldc + c, n, &w);
    }
  }
}

template <typename T>
void launch_rows(const QuantArgs& a, bool vec, cudaStream_t s) {
  const int64_t per_block = kThreads / (FP8_BLOCK / (16 / int64_t(sizeof(T))));
  const int64_t want = (a.batch * a.rows * fp8_blocks(a.K) + per_block - 1) / per_block;
  const int64_t most = int64_t(num_sms()) * 8;  // eight CTAs an SM, then a grid-wide stride
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  if (vec) fp8_rows_kernel<T, true><<<grid, kThreads, 0, s>>>(a);
  else fp8_rows_kernel<T, false><<<grid, kThreads, 0, s>>>(a);
}

template <typename T>
void launch_blocks(const QuantArgs& a, bool vec, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.batch * fp8_blocks(a.rows) * fp8_blocks(a.K)));
  if (vec) fp8_blocks_kernel<T, true><<<grid, kThreads, 0, s>>>(a);
  else fp8_blocks_kernel<T, false><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" nvfp4moe_status fp8_quantize(const void* x, int32_t x_dtype, int64_t batch, int64_t rows, int64_t K,
                                        int64_t ldx, int64_t x_batch_stride, int32_t tile, uint8_t* codes,
                                        int64_t ldc, int64_t codes_batch_stride, float* scale, int64_t lds,
                                        int64_t scale_batch_stride, nvfp4moe_stream_t stream) {
  const char* fn = "fp8_quantize";
  NVFP4_REQUIRE(x_dtype == NVFP4MOE_DTYPE_BF16 || x_dtype == NVFP4MOE_DTYPE_F32, NVFP4MOE_INVALID_ARG,
                "%s: x_dtype=%d", fn, x_dtype);
  NVFP4_REQUIRE(tile == NVFP4MOE_FP8_ROWS || tile == NVFP4MOE_FP8_BLOCKS, NVFP4MOE_INVALID_ARG, "%s: tile=%d", fn,
                tile);
  NVFP4_REQUIRE(batch >= 0 && rows >= 0 && K >= 0, NVFP4MOE_INVALID_ARG, "%s: negative size", fn);
  if (batch == 0 || rows == 0 || K == 0) return NVFP4MOE_OK;
  NVFP4_REQUIRE(K <= INT32_MAX && rows <= INT32_MAX && batch <= INT32_MAX, NVFP4MOE_UNSUPPORTED_SHAPE,
                "%s: a size above 2^31 - 1", fn);
  NVFP4_REQUIRE(x && codes && scale, NVFP4MOE_INVALID_ARG, "%s: NULL pointer", fn);
  const int64_t nb = fp8_blocks(K), srows = tile == NVFP4MOE_FP8_ROWS ? rows : fp8_blocks(rows);
  NVFP4_REQUIRE((rows == 1 || ldx >= K) && (rows == 1 || ldc >= K) && (srows == 1 || lds >= nb),
                NVFP4MOE_INVALID_ARG, "%s: a row pitch below the row's length", fn);
  NVFP4_REQUIRE(ldx >= 0 && ldc >= 0 && lds >= 0 && x_batch_stride >= 0 && codes_batch_stride >= 0 &&
                    scale_batch_stride >= 0,
                NVFP4MOE_INVALID_ARG, "%s: negative stride", fn);
  NVFP4_REQUIRE(batch * srows <= INT64_MAX / nb && batch * srows * nb <= (int64_t(1) << 31) - 1,
                NVFP4MOE_UNSUPPORTED_SHAPE, "%s: more than 2^31 - 1 groups", fn);
  const int64_t elt = x_dtype == NVFP4MOE_DTYPE_BF16 ? 2 : 4;
  NVFP4_REQUIRE(reinterpret_cast<uintptr_t>(x) % elt == 0, NVFP4MOE_INVALID_ARG, "%s: x is not aligned to its type",
                fn);
  // 16-byte loads and 8-byte code stores when every row starts where they may
  const bool vec = aligned16(x) && ldx * elt % 16 == 0 && (batch == 1 || x_batch_stride * elt % 16 == 0) &&
                   reinterpret_cast<uintptr_t>(codes) % 8 == 0 && ldc % 8 == 0 &&
                   (batch == 1 || codes_batch_stride % 8 == 0);
  const QuantArgs a{x, batch, rows, K, ldx, x_batch_stride, codes, ldc, codes_batch_stride, scale, lds,
                    scale_batch_stride};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tile == NVFP4MOE_FP8_ROWS) {
    if (elt == 2) launch_rows<__nv_bfloat16>(a, vec, s);
    else launch_rows<float>(a, vec, s);
  } else {
    if (elt == 2) launch_blocks<__nv_bfloat16>(a, vec, s);
    else launch_blocks<float>(a, vec, s);
  }
  return check_launch(fn);
}
