// fp8_quantize: bf16 / fp32 -> E4M3 with one fp32 scale per 1 x 128 or 128 x 128 group.
//
// Each element is read once and each code written once, so the bound is memory: 3 (bf16) or 5
// (fp32) bytes an element.  A row group is held by a few lanes with 64 bytes or 128 in flight each.  A
// square block is held in the registers of one CTA (32 elements a thread), so it too is read once.
// Rows whose start, pitch or length does not allow 16-byte loads take scalar ones.
#include "fp8.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace nvfp4moe {
namespace {

using namespace sm100;

struct QuantArgs {
  const void* x;
  int64_t batch, rows, K, ldx, x_batch;
  uint8_t* codes;
  int64_t ldc, c_batch;
  float* scale;
  int64_t lds, s_batch;
};

// W 32-bit words of elements (two bf16 or one fp32 each), read as they are: n elements exist, the
// others are zero.  VECTOR: p is aligned to the words' size.
template <typename T, int W, bool VECTOR>
__device__ __forceinline__ void load_words(const T* p, int n, uint32_t* u) {
  constexpr int PER = 4 / sizeof(T);
  if (VECTOR && n >= W * PER) {
    if constexpr (W == 4) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
      u[0] = q.x, u[1] = q.y, u[2] = q.z, u[3] = q.w;
    } else {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      u[0] = q.x, u[1] = q.y;
    }
  } else if constexpr (PER == 1) {
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = i < n ? __float_as_uint(__ldg(p + i)) : 0u;
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      u[i] = 2 * i < n ? __ldg(h + 2 * i) : 0u;
      if (2 * i + 1 < n) u[i] |= uint32_t(__ldg(h + 2 * i + 1)) << 16;
    }
  }
}

// The largest magnitude of the words' elements, as fp32 bits (a NaN stays above everything).
template <typename T, int W>
__device__ __forceinline__ uint32_t words_max(const uint32_t* u) {
  uint32_t m = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < W; ++i) m = max(m, u[i] & 0x7FFFFFFFu);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) m = __vmaxu2(m, u[i] & 0x7FFF7FFFu);
    m = max(m << 16, m & 0xFFFF0000u);
  }
  return m;
}

// A group's scale as its elements' type uses it.
template <typename T>
__device__ __forceinline__ auto scale_for(uint32_t m) {
  if constexpr (sizeof(T) == 2) return fp8_scale_bf16(m);
  else return fp8_scale(m);
}

template <typename T, typename S>
__device__ __forceinline__ uint32_t encode_words(const uint32_t* u, const S& f) {  // four elements
  float v[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  return fp8_encode4(v, f);
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
// Lanes that hold a row group, and groups of a lane, all loaded before the first is used.  Measured, TB/s at
// 16384 x 16384 bf16 / 8 x 4096 x 4096 fp32: 4 lanes 5.5 / -, 8 lanes and one group 4.0 / 5.7, two groups
// 4.8 / 6.4, 16 lanes - / 5.0 (fewer lanes: fewer instructions an element for the scale and the shuffles).
template <typename T>
constexpr int lanes_of() { return sizeof(T) == 2 ? 4 : 8; }
template <typename T>
constexpr int depth_of() { return sizeof(T) == 2 ? 1 : 2; }
constexpr int kBlockThreads = 512;
// 192 KB of blocks in flight an SM: three fp32 blocks of one CTA, or three bf16 ones of each of two CTAs
// (a bf16 block is half the bytes for the same arithmetic, which then needs the second CTA's overlap).
constexpr int kStages = 3;
template <typename T>
constexpr int ctas_of() { return sizeof(T) == 2 ? 2 : 1; }

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) fp8_rows_kernel(QuantArgs a) {
  griddep_wait();  // x may come from the launch before
  griddep_launch_dependents();
  constexpr int VEC = 16 / sizeof(T);                  // elements of a 16-byte load
  constexpr int kLanes = lanes_of<T>();
  constexpr int CHUNKS = FP8_BLOCK / (VEC * kLanes);   // loads a lane and group: 2 (bf16), 4 (fp32)
  constexpr int DEPTH = depth_of<T>();
  const int nb = int((a.K + FP8_BLOCK - 1) / FP8_BLOCK);
  const int64_t groups = a.rows * nb;
  const int sub = threadIdx.x % kLanes;
  // this lane's groups: first and first + half, half a CTA's share apart
  const int64_t first = int64_t(blockIdx.x) * (DEPTH * kThreads / kLanes) + threadIdx.x / kLanes;
  const int K = int(a.K) - sub * VEC;  // elements of a row from this lane's first on
  for (int64_t bi = blockIdx.y; bi < a.batch; bi += gridDim.y) {
    const T* x = static_cast<const T*>(a.x) + bi * a.x_batch + sub * VEC;
    uint8_t* codes = a.codes + bi * a.c_batch + sub * VEC;
    float* scale = a.scale + bi * a.s_batch;
    uint32_t u[DEPTH][CHUNKS][4];
    int64_t rows[DEPTH];
    int cs[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int64_t g = first + d * (kThreads / kLanes);
      rows[d] = groups <= INT32_MAX ? int64_t(uint32_t(g) / uint32_t(nb)) : g / nb;
      const int b = int(g - rows[d] * nb);
      cs[d] = g < groups ? b * FP8_BLOCK : INT32_MAX / 2;  // past the row's end: nothing is read or written
      const T* p = x + rows[d] * a.ldx + b * FP8_BLOCK;
#pragma unroll
      for (int j = 0; j < CHUNKS; ++j)
        load_words<T, 4, true>(p + j * kLanes * VEC, K - cs[d] - j * kLanes * VEC, u[d][j]);
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < CHUNKS; ++j) m = max(m, words_max<T, 4>(u[d][j]));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const auto f = scale_for<T>(m);
      uint8_t* q = codes + rows[d] * a.ldc + cs[d];
#pragma unroll
      for (int j = 0; j < CHUNKS; ++j) {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) w[i] = encode_words<T>(u[d][j] + i * sizeof(T), f);
        store_codes<VEC / 4, true>(q + j * kLanes * VEC, K - cs[d] - j * kLanes * VEC, w);
      }
      if (sub == 0 && cs[d] < K) scale[rows[d] * a.lds + cs[d] / FP8_BLOCK] = f.scale;
    }
  }
}

// The same for rows that start anywhere: a warp takes a group, its lanes every 32nd element, so that
// single loads and byte stores are still neighbours'.
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_rows_any_kernel(QuantArgs a) {
  griddep_wait();  // x may come from the launch before
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nb = int((a.K + FP8_BLOCK - 1) / FP8_BLOCK);
  const int64_t g = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / 32;
  if (g >= a.rows * nb) return;  // whole warps
  const int64_t row = g / nb;
  const int c = int(g - row * nb) * FP8_BLOCK + lane;
  for (int64_t bi = blockIdx.y; bi < a.batch; bi += gridDim.y) {
    const T* x = static_cast<const T*>(a.x) + bi * a.x_batch + row * a.ldx;
    float v[4];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 0.0f;
      if (c + 32 * i < a.K) {
        if constexpr (sizeof(T) == 2) v[i] = __bfloat162float(x[c + 32 * i]);
        else v[i] = x[c + 32 * i];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, abs_bits(v[i]));
    const auto f = scale_for<T>(__reduce_max_sync(0xffffffffu, m));
    const uint32_t w = fp8_encode4(v, f);
    uint8_t* q = a.codes + bi * a.c_batch + row * a.ldc + c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + 32 * i < a.K) q[32 * i] = static_cast<uint8_t>(w >> (8 * i));
    if (lane == 0) a.scale[bi * a.s_batch + row * a.lds + c / FP8_BLOCK] = f.scale;
  }
}

// 128 x 128 blocks, one after another in a persistent CTA: tile copies bring the next blocks to shared memory
// (192 KB in flight) while the threads hold the current one in registers, find its maximum and write
// its codes.  Warp w holds rows w, w + 16, ...; a lane four consecutive columns.  Waits are bounded: a CTA that
// gives up issues no more copies and leaves once those in flight have landed.  (Blocks loaded to
// registers by a CTA each, two CTAs an SM, waited at their barriers with nothing in flight: 4.5 TB/s at
// 17400 x 5004 fp32.)
template <typename T>
__global__ void __launch_bounds__(kBlockThreads, ctas_of<T>())
fp8_blocks_kernel(const __grid_constant__ CUtensorMap tm, QuantArgs a, int64_t blocks, uint32_t* status) {
  constexpr int WARPS = kBlockThreads / 32, ROWS = FP8_BLOCK / WARPS, W = sizeof(T);
  constexpr int STAGES = kStages, BYTES = FP8_BLOCK * FP8_BLOCK * sizeof(T);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_shared_1024(smem_raw);
  __shared__ uint64_t full[STAGES];
  __shared__ uint32_t s_max[2][WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t nb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK, nr = (a.rows + FP8_BLOCK - 1) / FP8_BLOCK;
  const int64_t mine = blocks > blockIdx.x ? (blocks - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  auto place = [&](int64_t i, int64_t& bi, int64_t& rb, int64_t& b) {
    const int64_t blk = blockIdx.x + i * gridDim.x, row = blk / nb;
    bi = row / nr, rb = row - bi * nr, b = blk - row * nb;
  };
  auto load = [&](int64_t i) {
    int64_t bi, rb, b;
    place(i, bi, rb, b);
    const int s = int(i % STAGES);
    mbar_arrive_expect_tx(&full[s], BYTES);
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(smem + s * BYTES)), "l"(reinterpret_cast<uint64_t>(&tm)), "r"(int(b * FP8_BLOCK)),
        "r"(int(rb * FP8_BLOCK)), "r"(int(bi)), "r"(smem_u32(&full[s]))
        : "memory");
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1);
    mbar_fence_init();
  }
  griddep_wait();  // x may come from the launch before
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int64_t i = 0; i < STAGES && i < mine; ++i) load(i);
  }
  __syncthreads();
  for (int64_t i = 0; i < mine; ++i) {
    const int s = int(i % STAGES);
    const bool ok = mbar_wait(&full[s], uint32_t(i / STAGES) & 1);
    uint32_t u[ROWS][W], m = 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const uint8_t* q = smem + s * BYTES + (warp + r * WARPS) * (FP8_BLOCK * int(sizeof(T))) + lane * 4 * int(sizeof(T));
      if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(q);
        u[r][0] = v.x, u[r][1] = v.y, u[r][2] = v.z, u[r][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(q);
        u[r][0] = v.x, u[r][1] = v.y;
      }
      m = max(m, words_max<T, W>(u[r]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) s_max[i & 1][warp] = m;
    // the block is in registers, and every warp's maximum is here; where a thread gave up waiting, all leave
    if (__syncthreads_or(!ok)) {
      if (threadIdx.x == 0) {
        atomicOr(status, uint32_t(NVFP4MOE_DEV_TIMEOUT));
        for (int64_t j = i; j < i + STAGES && j < mine; ++j)  // the copies land before the CTA leaves
          mbar_wait(&full[j % STAGES], uint32_t(j / STAGES) & 1, 1u << 16);
      }
      return;
    }
    if (threadIdx.x == 0 && i + STAGES < mine) load(i + STAGES);
    const auto f = scale_for<T>(__reduce_max_sync(0xffffffffu, s_max[i & 1][lane % WARPS]));
    int64_t bi, rb, b;
    place(i, bi, rb, b);
    if (threadIdx.x == 0) a.scale[bi * a.s_batch + rb * a.lds + b] = f.scale;
    const int64_t c = b * FP8_BLOCK + lane * 4;
    const int n = int(max(int64_t(0), min(a.K - c, int64_t(4))));
    uint8_t* out = a.codes + bi * a.c_batch + c;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int64_t row = rb * FP8_BLOCK + warp + r * WARPS;
      const uint32_t w = encode_words<T>(u[r], f);
      if (row < a.rows && n > 0) store_codes<1, true>(out + row * a.ldc, n, &w);
    }
  }
}

// The same for matrices that tile copies do not take: one CTA per block, single loads and stores.
template <typename T>
__global__ void __launch_bounds__(kBlockThreads) fp8_blocks_any_kernel(QuantArgs a) {
  griddep_wait();  // x may come from the launch before
  griddep_launch_dependents();
  constexpr int WARPS = kBlockThreads / 32, ROWS = FP8_BLOCK / WARPS;
  __shared__ uint32_t s_max[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t nb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK, nr = (a.rows + FP8_BLOCK - 1) / FP8_BLOCK;
  const int64_t blk = blockIdx.x;
  const int64_t bi = blk / (nb * nr), rb = blk / nb - bi * nr, b = blk % nb;
  const int64_t c = b * FP8_BLOCK + lane;  // and every 32nd column after it
  const T* x = static_cast<const T*>(a.x) + bi * a.x_batch;
  float v[ROWS][4];
  uint32_t m = 0;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = rb * FP8_BLOCK + warp + r * WARPS;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[r][i] = 0.0f;
      if (row < a.rows && c + 32 * i < a.K) {
        if constexpr (sizeof(T) == 2) v[r][i] = __bfloat162float(x[row * a.ldx + c + 32 * i]);
        else v[r][i] = x[row * a.ldx + c + 32 * i];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, abs_bits(v[r][i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
  const auto f = scale_for<T>(__reduce_max_sync(0xffffffffu, s_max[lane % WARPS]));
  if (threadIdx.x == 0) a.scale[bi * a.s_batch + rb * a.lds + b] = f.scale;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = rb * FP8_BLOCK + warp + r * WARPS;
    const uint32_t w = fp8_encode4(v[r], f);
    uint8_t* q = a.codes + bi * a.c_batch + row * a.ldc + c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row < a.rows && c + 32 * i < a.K) q[32 * i] = static_cast<uint8_t>(w >> (8 * i));
  }
}

template <typename T>
nvfp4moe_status launch_rows(const QuantArgs& a, bool vec, cudaStream_t s) {
  // no grid-wide stride: CTAs that finish early make room for the next ones, where a fixed grid's last
  // turn was a third empty at 4096 x 5120
  const int64_t per_block = vec ? depth_of<T>() * kThreads / lanes_of<T>() : kThreads / 32;
  const dim3 grid(static_cast<unsigned>((a.rows * fp8_blocks(a.K) + per_block - 1) / per_block),
                  static_cast<unsigned>(a.batch < 65535 ? a.batch : 65535));
  const cudaError_t e = launch_dependent(vec ? fp8_rows_kernel<T> : fp8_rows_any_kernel<T>, grid, dim3(kThreads), 0, s, a);
  return e == cudaSuccess ? NVFP4MOE_OK : fail(NVFP4MOE_CUDA_ERROR, "fp8_quantize: %s", cudaGetErrorString(e));
}

template <typename T>
nvfp4moe_status launch_blocks(const QuantArgs& a, bool vec, cudaStream_t s) {
  const int64_t blocks = a.batch * fp8_blocks(a.rows) * fp8_blocks(a.K);
  const int64_t pitch = a.rows > 1 ? a.ldx * int64_t(sizeof(T)) : 16;
  const int64_t batch_pitch = a.batch > 1 ? a.x_batch * int64_t(sizeof(T)) : 16;
  if (!vec || pitch >= (int64_t(1) << 40) || batch_pitch >= (int64_t(1) << 40) || batch_pitch == 0) {
    const cudaError_t e = launch_dependent(fp8_blocks_any_kernel<T>, dim3(static_cast<unsigned>(blocks)),
                                           dim3(kBlockThreads), 0, s, a);
    return e == cudaSuccess ? NVFP4MOE_OK : fail(NVFP4MOE_CUDA_ERROR, "fp8_quantize: %s", cudaGetErrorString(e));
  }
  uint32_t* status = device_status_ptr();
  auto fn = tensor_map_encoder();
  if (!status || !fn) return fail(NVFP4MOE_CUDA_ERROR, "fp8_quantize: device status word or tensor maps unavailable");
  CUtensorMap tm;
  const cuuint64_t dims[3] = {cuuint64_t(a.K), cuuint64_t(a.rows), cuuint64_t(a.batch)};
  const cuuint64_t strides[2] = {cuuint64_t(pitch), cuuint64_t(batch_pitch)};
  const cuuint32_t box[3] = {FP8_BLOCK, FP8_BLOCK, 1u}, estr[3] = {1, 1, 1};
  const CUresult r = fn(&tm, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                        const_cast<void*>(a.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(NVFP4MOE_CUDA_ERROR, "fp8_quantize: cuTensorMapEncodeTiled failed (%d)", int(r));
  constexpr int smem = 1024 + kStages * FP8_BLOCK * FP8_BLOCK * int(sizeof(T));
  cudaError_t e = set_smem_limit_once<fp8_blocks_kernel<T>>(smem);
  const int64_t most = int64_t(num_sms()) * ctas_of<T>(), grid = blocks < most ? blocks : most;
  if (e == cudaSuccess)
    e = launch_dependent(fp8_blocks_kernel<T>, dim3(static_cast<unsigned>(grid)), dim3(kBlockThreads), smem, s, tm, a,
                         blocks, status);
  return e == cudaSuccess ? NVFP4MOE_OK : fail(NVFP4MOE_CUDA_ERROR, "fp8_quantize: %s", cudaGetErrorString(e));
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
  NVFP4_REQUIRE(K <= INT32_MAX / 4 && rows <= INT32_MAX && batch <= INT32_MAX, NVFP4MOE_UNSUPPORTED_SHAPE,
                "%s: K above 2^29 or another size above 2^31 - 1", fn);
  NVFP4_REQUIRE(x && codes && scale, NVFP4MOE_INVALID_ARG, "%s: NULL pointer", fn);
  const int64_t nb = fp8_blocks(K), srows = tile == NVFP4MOE_FP8_ROWS ? rows : fp8_blocks(rows);
  NVFP4_REQUIRE((rows == 1 || ldx >= K) && (rows == 1 || ldc >= K) && (srows == 1 || lds >= nb),
                NVFP4MOE_INVALID_ARG, "%s: a row pitch below the row's length", fn);
  NVFP4_REQUIRE(ldx >= 0 && ldc >= 0 && lds >= 0 && x_batch_stride >= 0 && codes_batch_stride >= 0 &&
                    scale_batch_stride >= 0,
                NVFP4MOE_INVALID_ARG, "%s: negative stride", fn);
  NVFP4_REQUIRE(batch * srows <= INT64_MAX / nb && batch * srows * nb <= (int64_t(1) << 31) - 1,
                NVFP4MOE_UNSUPPORTED_SHAPE, "%s: more than 2^31 - 1 groups", fn);
  // matrices behind one another, or with their rows interleaved
  auto apart = [&](int64_t n, int64_t length, int64_t pitch, int64_t stride) {
    return batch == 1 || stride >= (n - 1) * pitch + length ||
           (stride >= length && (n == 1 || pitch >= (batch - 1) * stride + length));
  };
  NVFP4_REQUIRE(apart(rows, K, ldc, codes_batch_stride) && apart(srows, nb, lds, scale_batch_stride),
                NVFP4MOE_INVALID_ARG, "%s: the codes or scales of two matrices overlap", fn);
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
  const nvfp4moe_status st =
      tile == NVFP4MOE_FP8_ROWS
          ? (elt == 2 ? launch_rows<__nv_bfloat16>(a, vec, s) : launch_rows<float>(a, vec, s))
          : (elt == 2 ? launch_blocks<__nv_bfloat16>(a, vec, s) : launch_blocks<float>(a, vec, s));
  return st == NVFP4MOE_OK ? check_launch(fn) : st;
}
