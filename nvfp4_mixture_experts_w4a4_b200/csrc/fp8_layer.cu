// The whole FP8 routed layer in one persistent launch for batches of at most 16 tokens: routing,
// gate/up, SwiGLU, h in E4M3, down and the combine in slot order.  A small launch before it puts x
// in E4M3 and zeroes the counters; the layer's launch is its programmatic dependent and routes
// meanwhile.
//
// Such a batch is a stream of expert weights, 3 H I bytes per touched expert, against a few rows of
// activations: its time is those bytes over the memory's rate plus what precedes and follows the
// stream.  One CTA per SM routes the whole batch itself, so the stream starts as soon as the logits
// have been read, and keeps x in shared memory (by TMA) as the MMA's B operand; the weights are its M side (128
// rows), the batch its N side (16 columns).  A stage of the ring is two 128 x 128 tiles of
// weights (32 KB) with a scale each:
//   gate/up unit (expert, 128 columns of h): a gate and an up tile per block of H.  Its sums, with
//     the scales of both operands applied in fp32 registers after every block, give 128 columns of h:
//     one quantisation group a token, so nothing but done counters leaves the CTA.
//   down unit (expert, 128 columns of the output): two tiles per stage, blocks 2j and 2j + 1 of I.
//     Its h rows come back from L2 once the expert's gate/up units have counted up; the weights
//     never wait, so the ring keeps streaming across the change.
// Units go round-robin over the CTAs, gate/up first; CTAs with one gate/up unit less take the
// first down units.  Where few experts are touched, gate/up units are split along H (the last
// of a unit's parts to finish adds the parts in order) and down units along I (the combine adds them).
// Combine: after a grid-wide barrier every CTA sums a slice of the outputs over the k slots of a
// token, in slot order, and rounds once.
//
// GROUPED is the same stream for larger batches whose experts get few rows each: the routing and x in
// expert order come from launches before, units take at most 32 rows of an expert, x comes per stage
// as h does, and the rows of the output stay in expert order for the combine's own launch.
//
// Warps: 0 streams weights (TMA); 1 owns TMEM and issues the MMAs; 2 and 3 fetch x and its scales;
// 4..7 add and finish the first tile of every stage, 8..11 the second; 12..15 take every fourth stage
// each and fetch its scales, and h for down stages (four, because each waits out an L2 read a stage:
// one warp alone ran a stage in 1.0 us where the weights come in 0.75).  A rare stage some of whose scales do
// not multiply to an ordinary number is held back until every adding warp, waiting for it, has seen its
// number: the usual stage has no choice to make (decode 96.8 us, 95.6 without any of this, 101.6 with a choice in
// the adding loop).
// Every wait is bounded (status bit on timeout; copies in flight land before the CTA exits).
#include "fp8.cuh"
#include "fp8_tile.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"
#include "topk.cuh"

namespace nvfp4moe {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kTile = 128 * 128;         // bytes of a weight tile
constexpr int kStage = 2 * kTile;
constexpr int kMaxStages = 6, kMinStages = 3;  // (more than 8 or less than 3: see the scale warps)
constexpr int kSlots = 8;                // accumulator slots (stages in flight past the MMA)
constexpr int kMaxE = 1024;
constexpr int kPitch = 132;              // floats of a row of the exchange buffer
constexpr int kSmemLimit = 226 * 1024;   // dynamic; a few hundred bytes more are static
constexpr int kMaxSplit = 4;             // parts of a gate/up unit
constexpr uint32_t kTimeout = NVFP4MOE_DEV_TIMEOUT;
constexpr uint32_t kPolls = 1u << 22;

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct LayerArgs {
  const float* logits;
  const float* x_scale;    // [T][nH]; GROUPED: [pairs][nH]
  const int4* list;        // GROUPED: [0].x row groups, then {expert, first row, rows, -} each
  int T, H, I, E, k;
  int nH, nI;              // 128-blocks
  int stages;
  int max_parts;           // gate/up unit parts that `parts` holds
  int chunks_cap;          // K chunks per pair that `slots` holds
  const float* w13_scale;  // [E][2][nI][nH]
  const float* w2_scale;   // [E][nH][nI]
  uint8_t* h_codes;        // [pairs][I]
  float* h_scale;          // [pairs][nI]
  float* parts;            // [max_parts][2][NT][128]
  float* slots;            // [pairs][s2][H]
  int* done;               // [experts touched] finished gate/up units
  int* tickets;            // [gate/up units] finished parts, where units are split
  int* gbar;               // [1]
  __nv_bfloat16* out;
  uint32_t* status;
};

// Byte offsets in dynamic shared memory (1024-byte aligned base).
struct Smem {
  int h, x, xs, sb, hs, buf, mask, list, row0, rowof, ids, w, bars, total;
};
__host__ __device__ inline Smem smem_layout(int nt, int nH, int k, int E, int stages, bool grouped) {
  if (grouped) nH = 0, k = 0, E = 0;  // no x, no routing
  Smem m;
  int at = stages * kStage;
  auto put = [&](int bytes) {
    const int here = at;
    at += (bytes + 15) / 16 * 16;
    return here;
  };
  m.h = put(stages * 2 * nt * 128);
  m.x = put(nH * nt * 128);
  m.xs = put(nH * nt * 4);
  m.sb = put(kSlots * 2 * 4);
  m.hs = put(kSlots * 2 * nt * 4);
  m.buf = put(nt * kPitch * 4);
  const int most = nt * k < E ? nt * k : E;
  m.mask = put(E * 4);
  m.rowof = put(E * 4);
  m.list = put(most * 4);
  m.row0 = put((most + 1) * 4);
  m.ids = put(nt * k * 4);
  m.w = put(nt * k * 4);
  m.bars = put((2 * kMaxStages + 2 * kSlots + 4) * 8);
  m.total = at + 1024;
  return m;
}

// The schedule, the same in every thread of every CTA: it follows from the number of experts
// touched (A) and the grid.
struct Plan {
  int A, G, s1, s2, n1, n2, extra, light, heavy, first2;
  __device__ Plan(const LayerArgs& a, int active, int grid, int cta, bool grouped) {
    A = active, G = grid;
    s1 = 1, s2 = 1;
    const int u1 = A * a.nI, u2 = A * a.nH, st2 = ceil_div(a.nI, 2);
    // Parts of a unit: the count with the fewest stages in the fullest CTA, a split gate/up unit
    // costing six stages for the exchange of its parts and a down unit one for its end.  A lane tries one count.
    const int s = (threadIdx.x & 31) + 1;
    if (!grouped && u1 < G) {
      int cost = INT32_MAX;
      if (s <= kMaxSplit && s <= a.nH && u1 * s <= a.max_parts)
        cost = (ceil_div(u1 * s, G) * (ceil_div(a.nH, s) + (s > 1 ? 6 : 0))) * 32 + s - 1;
      s1 = (__reduce_min_sync(0xffffffffu, cost) & 31) + 1;
    }
    if (!grouped && u2 < 4 * G) {
      int cost = INT32_MAX;
      if (s <= a.chunks_cap && s <= st2) cost = ceil_div(u2 * s, G) * (ceil_div(st2, s) + 1) * 32 + s - 1;
      s2 = (__reduce_min_sync(0xffffffffu, cost) & 31) + 1;
    }
    const int U1 = u1 * s1, U2 = u2 * s2;
    heavy = U1 % G;
    light = G - heavy;
    n1 = U1 / G + (cta < heavy ? 1 : 0);
    // (with one round of gate/up units no h is ready earlier for the CTAs that have none)
    extra = heavy > 0 && U1 > G ? min(ceil_div(a.nH, s1) / ceil_div(st2, s2), U2 / light) : 0;
    const int rest = U2 - extra * light;
    first2 = (cta + G - heavy) % G;  // place among the CTAs that share the rest: light ones first
    n2 = (cta >= heavy ? extra : 0) + rest / G + (first2 < rest % G ? 1 : 0);
  }
  __device__ int units() const { return n1 + n2; }
};

struct Unit {
  bool down;
  int a;         // index of the expert among the touched
  int blk;       // 128-block of I (gate/up) or of H (down)
  int part;      // K part
  int id;        // gate/up: unit index without the part
  int j0, j1;    // stages: blocks of H, or pairs of blocks of I
};

__device__ __forceinline__ Unit unit_of(const Plan& p, const LayerArgs& a, int i, int cta) {
  Unit u;
  u.down = i >= p.n1;
  if (!u.down) {
    const int id = cta + i * p.G;
    u.id = id / p.s1;
    u.part = id - u.id * p.s1;
    u.a = u.id / a.nI;
    u.blk = u.id - u.a * a.nI;
    u.j0 = a.nH * u.part / p.s1;
    u.j1 = a.nH * (u.part + 1) / p.s1;
  } else {
    int r = i - p.n1, id;
    if (cta >= p.heavy && r < p.extra) {
      id = r * p.light + cta - p.heavy;
    } else {
      if (cta >= p.heavy) r -= p.extra;
      id = p.extra * p.light + r * p.G + p.first2;
    }
    const int v = id / p.s2, st2 = ceil_div(a.nI, 2);
    u.part = id - v * p.s2;
    u.a = v / a.nH;
    u.blk = v - u.a * a.nH;
    u.id = v;
    u.j0 = st2 * u.part / p.s2;
    u.j1 = st2 * (u.part + 1) / p.s2;
  }
  return u;
}

__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// One more at *p, releasing what this thread and those it has met at a barrier wrote before.
__device__ __forceinline__ void add_release(int* p) {
  asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p) : "memory");
}
// The same, returning the count before and acquiring what the others released.
__device__ __forceinline__ int add_acq_rel(int* p) {
  int v;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// Waits until *p >= want; false when it gave up.  The second form is a whole warp's, which gets one answer.
__device__ __forceinline__ bool wait_count(const int* p, int want) {
  for (uint32_t i = 0; i < kPolls; ++i) {
    if (load_acquire(p) >= want) return true;
    __nanosleep(32);
  }
  return false;
}
__device__ __forceinline__ bool wait_count_warp(const int* p, int want) {
  for (uint32_t i = 0; i < kPolls; ++i) {
    if (__all_sync(0xffffffffu, load_acquire(p) >= want)) return true;
    __nanosleep(32);
  }
  return false;
}
__device__ __forceinline__ void add_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void read_columns(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 32) {
    tmem_ld_32x32b_x32(taddr, r);
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
  tmem_ld_wait();
}

// x [T][H] bf16 -> E4M3 and scales (eight lanes a group of 128), and the layer's counters to zero.
__global__ void __launch_bounds__(256)
fp8_layer_prepare_kernel(const __nv_bfloat16* __restrict__ x, int T, int H, uint8_t* __restrict__ codes,
                         float* __restrict__ scale, int* __restrict__ counters, int n) {
  griddep_wait();  // the call before may still use the counters and x
  griddep_launch_dependents();
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) counters[i] = 0;
  const int nH = ceil_div(H, 128), sub = threadIdx.x & 7;
  const int g = (blockIdx.x * 256 + threadIdx.x) >> 3;
  const int t = g / nH, kb = g - t * nH;
  uint4 u[2];
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = kb * 128 + (sub + 8 * j) * 8;
    u[j] = t < T && c < H ? __ldg(reinterpret_cast<const uint4*>(x + int64_t(t) * H + c)) : make_uint4(0u, 0u, 0u, 0u);
    mx = bf16x8_max(mx, u[j]);
  }
  mx = fp8_amax_bits(mx);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const Fp8ScaleBf16 f = fp8_scale_bf16(mx);
  if (t >= T) return;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = kb * 128 + (sub + 8 * j) * 8;
    const uint2 w = fp8_encode8(u[j], f);
    if (c < H) *reinterpret_cast<uint2*>(codes + int64_t(t) * H + c) = w;
  }
  if (sub == 0) scale[t * nH + kb] = f.scale;
}

template <int NT, int PER_LANE, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 1)
fp8_layer_kernel(const __grid_constant__ CUtensorMap tm13, const __grid_constant__ CUtensorMap tm2,
                 const __grid_constant__ CUtensorMap tmh, const __grid_constant__ CUtensorMap tmx, const LayerArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_shared_1024(smem_raw);
  const Smem m = smem_layout(NT, a.nH, a.k, a.E, a.stages, GROUPED);
  float* s_xs = reinterpret_cast<float*>(smem + m.xs);          // [nH][NT]
  float* s_sb = reinterpret_cast<float*>(smem + m.sb);          // [slot][2]
  float* s_hs = reinterpret_cast<float*>(smem + m.hs);          // [slot][2][NT]
  float* s_buf = reinterpret_cast<float*>(smem + m.buf);        // [NT][kPitch]
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + m.mask);  // [E] tokens of each expert
  int* s_rowof = reinterpret_cast<int*>(smem + m.rowof);        // [E] first pair row of the expert
  int* s_list = reinterpret_cast<int*>(smem + m.list);          // touched experts, ascending
  int* s_row0 = reinterpret_cast<int*>(smem + m.row0);          // their first pair rows, then the end
  int* s_ids = reinterpret_cast<int*>(smem + m.ids);            // [T][k]
  float* s_w = reinterpret_cast<float*>(smem + m.w);            // [T][k]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + m.bars);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + kSlots;
  uint64_t* x_full = acc_empty + kSlots;
  uint64_t* drain = x_full + 1;
  __shared__ uint32_t tmem_holder;
  __shared__ volatile int abort_flag;
  // stages some of whose columns' scales do not multiply to an ordinary number: their number + 1, from the scale
  // warp that has one, and from each adding warp once it knows
  __shared__ volatile uint32_t s_rare[4], s_seen[8];
  __shared__ int s_active, s_scan[2][kThreads / 32], s_last;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
  // Scale warps: stage it is warp 12 + it % W's.  A wait on a barrier's parity is only meant for the
  // phase before it or the one before that, so a warp that skips stages has to know that the barrier
  // is not two phases back.  It waits for `empty` first: at its last visit, W stages ago, stage
  // it - W - S was consumed, which is it - 2S or later as W <= S.  Then stage it - S is consumed, so
  // the accumulators of it - S - 8 have been read, which is it - 16 or later as S <= 8.
  const int W = a.stages >= 4 ? 4 : 3;

  // ---- set-up, with the logits on their way ----
  static_assert(GROUPED || NT == kThreads / 32, "a warp routes a token");
  constexpr int TOK = GROUPED ? 0 : 1;
  float lg[TOK + GROUPED][PER_LANE];
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int t = warp + 16 * i;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      const int e = lane + 32 * j;
      lg[i][j] = t < a.T && e < a.E ? __ldg(a.logits + int64_t(t) * a.E + e) : 0.0f;
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 8);
    }
    mbar_init(x_full, 33);
    mbar_init(drain, 1);
    abort_flag = 0;
    for (int i = 0; i < 4; ++i) s_rare[i] = 0u;
    for (int i = 0; i < 8; ++i) s_seen[i] = 0u;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, kSlots * 2 * NT);
    tmem_relinquish();
  }
  if (threadIdx.x == 64) {
    prefetch_tensormap(&tm13);
    prefetch_tensormap(&tm2);
    prefetch_tensormap(&tmh);
    prefetch_tensormap(&tmx);
  }
  if constexpr (!GROUPED)
    for (int e = threadIdx.x; e < a.E; e += kThreads) s_mask[e] = 0u;
  __syncthreads();
  // Every CTA is resident and has its TMEM: the next launch may take what is left of the SM and set itself
  // up.  (Before the allocation it could not: a waiting launch that got the columns first would hold them.)
  if constexpr (!GROUPED) griddep_launch_dependents();

  // ---- routing and the list of touched experts ----
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int t = warp + 16 * i;
    if (t < a.T) {
      int id;
      float wt;
      warp_topk_regs<PER_LANE>(lg[i], a.E, a.k, &id, &wt);
      if (lane < a.k) {
        s_ids[t * a.k + lane] = id;
        s_w[t * a.k + lane] = wt;
        atomicOr(&s_mask[id], 1u << t);
      }
    }
  }
  if constexpr (GROUPED) {
    griddep_wait();  // the list, x and the counters come from the launches before
    griddep_launch_dependents();
  } else {
    __syncthreads();
    static_assert(kMaxE == 2 * kThreads, "two experts a thread");
    int n[2], act = 0, rows = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * int(threadIdx.x) + i;
      n[i] = e < a.E ? __popc(s_mask[e]) : 0;
      act += n[i] > 0;
      rows += n[i];
    }
    int ia = act, ir = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, ia, o), z = __shfl_up_sync(0xffffffffu, ir, o);
      if (lane >= o) ia += y, ir += z;
    }
    if (lane == 31) s_scan[0][warp] = ia, s_scan[1][warp] = ir;
    __syncthreads();
    ia -= act, ir -= rows;
    const bool before = lane < warp;  // the warps before this one (there are 16)
    ia += __reduce_add_sync(0xffffffffu, before ? s_scan[0][lane & 15] : 0);
    ir += __reduce_add_sync(0xffffffffu, before ? s_scan[1][lane & 15] : 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * int(threadIdx.x) + i;
      if (n[i] > 0) {
        s_list[ia] = e;
        s_row0[ia] = ir;
        s_rowof[e] = ir;
        ++ia, ir += n[i];
      }
    }
    if (threadIdx.x == kThreads - 1) {
      s_active = ia;
      s_row0[ia] = ir;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  const Plan p(a, GROUPED ? a.list[0].x : s_active, int(gridDim.x), cta, GROUPED);
  const int units = p.units();
  const int S = a.stages;
  auto abort_now = [&]() {
    abort_flag = 1;
    atomicOr(a.status, kTimeout);
  };
  auto warp_aborted = [&]() { return __any_sync(0xffffffffu, abort_flag) != 0; };  // one answer for a whole warp
  // the expert of a unit, its first row in expert order and its rows
  struct Rows {
    int e, row0, n;
  };
  auto rows_of = [&](const Unit& u) {
    if constexpr (GROUPED) {
      const int4 q = __ldg(a.list + 1 + u.a);
      return Rows{q.x, q.y, q.z};
    } else {
      return Rows{s_list[u.a], s_row0[u.a], s_row0[u.a + 1] - s_row0[u.a]};
    }
  };

  if (warp == 0) {
    if (elect_one()) {
      uint32_t it = 0;
      for (int i = 0; i < units && !abort_flag; ++i) {
        const Unit u = unit_of(p, a, i, cta);
        const int e = rows_of(u).e;
        for (int j = u.j0; j < u.j1; ++j, ++it) {
          const int s = it % S;
          if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1)) {
            abort_now();
            break;
          }
          uint8_t* dst = smem + s * kStage;
          mbar_arrive_expect_tx(&full[s], kStage);
          if (u.down) {
            load_tile(dst, &tm2, 2 * j * 128, u.blk * 128, e, &full[s]);
            load_tile(dst + kTile, &tm2, (2 * j + 1) * 128, u.blk * 128, e, &full[s]);
          } else {
            load_tile(dst, &tm13, j * 128, u.blk * 128, 2 * e, &full[s]);
            load_tile(dst + kTile, &tm13, j * 128, u.blk * 128, 2 * e + 1, &full[s]);
          }
        }
      }
      if (abort_flag)
        for (uint32_t back = 0; back < uint32_t(S) && back < it; ++back) {
          const uint32_t j = it - 1 - back;
          mbar_wait(&full[j % S], (j / S) & 1, 1u << 16);
        }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_f8(128, NT);
      uint32_t it = 0;
      bool ok = GROUPED || mbar_wait(x_full, 0);
      if (!ok) abort_now();
      for (int i = 0; i < units && ok && !abort_flag; ++i) {
        const Unit u = unit_of(p, a, i, cta);
        for (int j = u.j0; j < u.j1; ++j, ++it) {
          const int s = it % S, slot = it % kSlots;
          if (!mbar_wait(&acc_empty[slot], ((it / kSlots) & 1) ^ 1) || !mbar_wait(&full[s], (it / S) & 1)) {
            abort_now();
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t ad = desc_kmajor_sw128(smem + s * kStage + h * kTile);
            const uint8_t* b = u.down ? smem + m.h + (2 * s + h) * NT * 128
                                      : (GROUPED ? smem + m.h + 2 * s * NT * 128 : smem + m.x + j * NT * 128);
            const uint64_t bd = desc_kmajor_sw128(b);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              tc_mma_f8(tmem + (2 * slot + h) * NT, ad + 2 * q, bd + 2 * q, idesc, q != 0 ? 1u : 0u);
          }
          tc_commit(&empty[s]);
          tc_commit(&acc_full[slot]);
        }
      }
      tc_commit(drain);
      mbar_wait(drain, 0, 1u << 20);
    }
  } else if (warp == 2 && !GROUPED) {
    griddep_wait();  // x comes from the launch before
    if (elect_one()) {
      mbar_arrive_expect_tx(x_full, a.nH * NT * 128);
      for (int kb = 0; kb < a.nH; ++kb) load_tile(smem + m.x + kb * NT * 128, &tmx, kb * 128, 0, 0, x_full);
    }
  } else if (warp == 3 && !GROUPED) {
    griddep_wait();
    for (int i = lane; i < a.nH * a.T; i += 32) {
      const int t = i / a.nH, kb = i - t * a.nH;
      s_xs[kb * NT + t] = __ldg(a.x_scale + i);
    }
    mbar_arrive(x_full);
  } else if (warp >= 12) {
    // scales of the stage's two tiles, and for down stages h and its scales
    uint32_t it = 0;
    int have = -1;  // the expert whose h is known to be complete
    bool ok = true;
    griddep_wait();  // the counters are zero
    for (int i = 0; i < units && ok && !warp_aborted(); ++i) {
      const Unit u = unit_of(p, a, i, cta);
      const auto [e, row0, n] = rows_of(u);
      for (int j = u.j0; j < u.j1; ++j, ++it) {
        if (int(it % W) != warp - 12) continue;
        const int s = it % S, slot = it % kSlots;
        float sb = 0.0f, xs = 0.0f;
        if (u.down) {
          if (lane < 2 && 2 * j + lane < a.nI) sb = __ldg(a.w2_scale + (int64_t(e) * a.nH + u.blk) * a.nI + 2 * j + lane);
          if (u.a != have) {
            if (!wait_count_warp(a.done + u.a, a.nI)) {
              abort_now();
              ok = false;
              break;
            }
            have = u.a;
            asm volatile("fence.proxy.async;" ::: "memory");  // h was written by ordinary stores
          }
        } else if (lane < 2) {
          sb = __ldg(a.w13_scale + ((int64_t(e) * 2 + lane) * a.nI + u.blk) * a.nH + j);
        }
        if (!u.down && lane < (GROUPED ? n : a.T))
          xs = __ldg(a.x_scale + int64_t(GROUPED ? row0 + lane : lane) * a.nH + j);
        if (!mbar_wait_warp(&empty[s], ((it / S) & 1) ^ 1) ||
            !mbar_wait_warp(&acc_empty[slot], ((it / kSlots) & 1) ^ 1)) {
          abort_now();
          ok = false;
          break;
        }
        // the columns' scales of either tile: a lane holds a column's
        static_assert(NT <= 32, "a column a lane");
        float cs[2] = {xs, xs};
        if (u.down) {
          if (lane == 0) {
            mbar_expect_tx(&full[s], 2 * NT * 128);
            load_tile(smem + m.h + 2 * s * NT * 128, &tmh, 2 * j * 128, row0, 0, &full[s]);
            load_tile(smem + m.h + (2 * s + 1) * NT * 128, &tmh, (2 * j + 1) * 128, row0, 0, &full[s]);
          }
          if (lane < n) {
            const float* q = a.h_scale + int64_t(row0 + lane) * a.nI + 2 * j;
            cs[0] = __ldcg(q);
            if (2 * j + 1 < a.nI) cs[1] = __ldcg(q + 1);
          }
          if (lane < NT) {
            s_hs[(2 * slot) * NT + lane] = cs[0];
            s_hs[(2 * slot + 1) * NT + lane] = cs[1];
          }
        } else if constexpr (GROUPED) {
          if (lane == 0) {
            mbar_expect_tx(&full[s], NT * 128);
            load_tile(smem + m.h + 2 * s * NT * 128, &tmx, j * 128, row0, 0, &full[s]);
          }
          if (lane < NT) s_hs[(2 * slot) * NT + lane] = xs;
        }
        if (lane < 2) s_sb[2 * slot + lane] = sb;
        const bool both = fp8_needs_both(cs[0], __shfl_sync(0xffffffffu, sb, 0)) |
                          fp8_needs_both(cs[1], __shfl_sync(0xffffffffu, sb, 1));
        if (__any_sync(0xffffffffu, both)) {
          // the adding warps, held up at this stage, see its number; when all have, it may go on
          if (lane == 0) s_rare[warp - 12] = it + 1;
          bool seen = false;
          for (uint32_t k = 0; k < (1u << 22) && !seen; ++k) {
            seen = __all_sync(0xffffffffu, int32_t(s_seen[lane & 7] - (it + 1)) >= 0);
            if (!seen) __nanosleep(64);
          }
          if (!seen) {
            abort_now();
            ok = false;
            break;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
    }
  } else if (warp >= 4 && warp < 12) {
    const int half = (warp - 4) >> 2, q = warp & 3, r = q * 32 + lane;
    const uint32_t trow = tmem + (uint32_t(q * 32) << 16);
    bool ok = GROUPED || mbar_wait_warp(x_full, 0);
    if (!ok) abort_now();
    griddep_wait();  // the counters are zero
    auto is_rare = [&](uint32_t i) {
      return __any_sync(0xffffffffu, s_rare[lane & 3] == i + 1) != 0;
    };
    auto wait_sums = [&](uint32_t i) {
      for (uint32_t k = 0; k < (1u << 22); ++k) {
        if (__all_sync(0xffffffffu, mbar_try_wait(&acc_full[i % kSlots], (i / kSlots) & 1))) return true;
        if (is_rare(i)) return false;
      }
      return false;
    };
    uint32_t it = 0;
    for (int i = 0; i < units; ++i) {
      const Unit u = unit_of(p, a, i, cta);
      const auto [e, row0, n] = rows_of(u);
      float acc[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) acc[c] = 0.0f;
      for (int j = u.j0; j < u.j1 && ok; ++j, ++it) {
        const int slot = it % kSlots;
        const float4* sc = reinterpret_cast<const float4*>(
            u.down ? s_hs + (2 * slot + half) * NT : (GROUPED ? s_hs + 2 * slot * NT : s_xs + j * NT));
        constexpr int CW = NT < 32 ? NT : 32;
        if (warp_aborted() || !wait_sums(it)) {
          // gave up, or a rare stage: sums times one scale, then the other
          ok = is_rare(it);
          if (ok) {
            if (lane == 0) s_seen[warp - 4] = it + 1;
            ok = mbar_wait_warp(&acc_full[slot], (it / kSlots) & 1);
          }
          if (!ok) {
            abort_now();
            break;
          }
          tc_fence_after();
          const float sb = s_sb[2 * slot + half];
#pragma unroll
          for (int c0 = 0; c0 < NT; c0 += CW) {
            uint32_t v[CW];
            read_columns<CW>(trow + (2 * slot + half) * NT + c0, v);
#pragma unroll
            for (int c = 0; c < CW; ++c) {
              float first, second;
              fp8_factors(reinterpret_cast<const float*>(sc)[c0 + c], sb, first, second);
              acc[c0 + c] = fmaf(__uint_as_float(v[c]) * first, second, acc[c0 + c]);
            }
          }
        } else {
          tc_fence_after();
          const float sb = s_sb[2 * slot + half];
#pragma unroll
          for (int c0 = 0; c0 < NT; c0 += CW) {
            if (GROUPED && c0 >= n) break;  // columns without rows
            uint32_t v[CW];
            read_columns<CW>(trow + (2 * slot + half) * NT + c0, v);
#pragma unroll
            for (int c = 0; c < CW; c += 4) {
              const float4 f = sc[(c0 + c) / 4];
              acc[c0 + c] = fmaf(__uint_as_float(v[c]), f.x * sb, acc[c0 + c]);
              acc[c0 + c + 1] = fmaf(__uint_as_float(v[c + 1]), f.y * sb, acc[c0 + c + 1]);
              acc[c0 + c + 2] = fmaf(__uint_as_float(v[c + 2]), f.z * sb, acc[c0 + c + 2]);
              acc[c0 + c + 3] = fmaf(__uint_as_float(v[c + 3]), f.w * sb, acc[c0 + c + 3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[slot]);
      }
      if (u.down) {
        // both halves' sums are one output: the second hands its over
        if (half == 1) {
#pragma unroll
          for (int c = 0; c < NT; ++c)
            if (c < n) s_buf[c * kPitch + r] = acc[c];
        }
        if (add_barrier_any(!ok)) break;
        const int col = u.blk * 128 + r;
        if (half == 0 && col < a.H) {
          float* dst = a.slots + (int64_t(row0) * p.s2 + u.part) * a.H + col;
#pragma unroll
          for (int c = 0; c < NT; ++c)
            if (c < n) dst[int64_t(c) * p.s2 * a.H] = acc[c] + s_buf[c * kPitch + r];
        }
        add_barrier();
      } else {
        bool finish = true;
        if (!GROUPED && p.s1 > 1) {
          // this part's sums; the last part to arrive adds all of them in order
          float* dst = a.parts + ((int64_t(u.id) * p.s1 + u.part) * 2 + half) * NT * 128 + r;
#pragma unroll
          for (int c = 0; c < NT; ++c)
            if (c < a.T) __stcg(dst + c * 128, acc[c]);
          if (add_barrier_any(!ok)) break;
          if (threadIdx.x == 128) s_last = add_acq_rel(a.tickets + u.id) == p.s1 - 1;
          add_barrier();
          finish = s_last != 0;
          if (finish) {
#pragma unroll
            for (int c = 0; c < NT; ++c) acc[c] = 0.0f;
            for (int k = 0; k < p.s1; ++k) {
              const float* src = a.parts + ((int64_t(u.id) * p.s1 + k) * 2 + half) * NT * 128 + r;
#pragma unroll
              for (int c = 0; c < NT; ++c)
                if (c < a.T) acc[c] += __ldcg(src + c * 128);
            }
          }
        }
        if (finish) {
          if (half == 1) {
#pragma unroll
            for (int c = 0; c < NT; ++c) s_buf[c * kPitch + r] = acc[c];
          }
          if (add_barrier_any(!ok)) break;
          if (half == 0) {
#pragma unroll
            for (int c = 0; c < NT; ++c)
              s_buf[c * kPitch + r] = silu_times(acc[c], s_buf[c * kPitch + r]);
          }
          add_barrier();
          // a warp takes every eighth token of the expert: 128 columns, one group
          const uint32_t mask = GROUPED ? 0u : s_mask[e];
          const int i0 = u.blk * 128 + lane * 4;
          for (int c = warp - 4; c < n; c += 8) {
            const int t = GROUPED ? c : int(__fns(mask, 0, c + 1));  // the token's column
            const float4 h = *reinterpret_cast<const float4*>(s_buf + t * kPitch + lane * 4);
            const uint32_t mx = __reduce_max_sync(
                0xffffffffu, max(max(abs_bits(h.x), abs_bits(h.y)), max(abs_bits(h.z), abs_bits(h.w))));
            const Fp8Scale f = fp8_scale(mx);
            const float v[4] = {h.x, h.y, h.z, h.w};
            const uint32_t codes = fp8_encode4(v, f);
            if (i0 < a.I) *reinterpret_cast<uint32_t*>(a.h_codes + int64_t(row0 + c) * a.I + i0) = codes;
            if (lane == 0) a.h_scale[int64_t(row0 + c) * a.nI + u.blk] = f.scale;
          }
          add_barrier();
          if (threadIdx.x == 128) add_release(a.done + u.a);
        }
      }
    }
    // ---- combine ----
    if constexpr (!GROUPED) add_barrier();
    if (!GROUPED && threadIdx.x == 128) {
      add_release(a.gbar);
      if (!wait_count(a.gbar, int(gridDim.x))) abort_now();
    }
    if constexpr (!GROUPED) add_barrier();
    if (!GROUPED && !abort_flag) {
      const int per_row = a.H / 4;
      const int total = a.T * per_row, stride = int(gridDim.x) * 256;
      for (int i = cta * 256 + int(threadIdx.x) - 128; i < total; i += stride) {
        const int t = i / per_row, c = (i - t * per_row) * 4;
        const uint32_t below = (1u << t) - 1u;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int j = 0; j < a.k; ++j) {
          const int id = s_ids[t * a.k + j];
          const float w = s_w[t * a.k + j];
          const float* src = a.slots + int64_t(s_rowof[id] + __popc(s_mask[id] & below)) * p.s2 * a.H + c;
          float4 z = __ldcg(reinterpret_cast<const float4*>(src));
          for (int k = 1; k < p.s2; ++k) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src + int64_t(k) * a.H));
            z.x += v.x, z.y += v.y, z.z += v.z, z.w += v.w;
          }
          y.x = fmaf(w, z.x, y.x), y.y = fmaf(w, z.y, y.y), y.z = fmaf(w, z.z, y.z), y.w = fmaf(w, z.w, y.w);
        }
        const __nv_bfloat162 o0 = __floats2bfloat162_rn(y.x, y.y), o1 = __floats2bfloat162_rn(y.z, y.w);
        *reinterpret_cast<uint2*>(a.out + int64_t(t) * a.H + c) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&o0), *reinterpret_cast<const uint32_t*>(&o1));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kSlots * 2 * NT);
}

constexpr int kTokens = 16;  // tokens of a single launch at most (with 32, x and three stages of weights fill shared
                             // memory, and the launches below are faster: 512 experts of 2048 x 512, top 10, 17
                             // tokens 110 us against 95, 32 tokens 163 against 141; 16 tokens 86 against 95)

int stages_for(int H, int E, int k) {
  for (int s = kMaxStages; s >= kMinStages; --s)
    if (smem_layout(kTokens, int(fp8_blocks(H)), k, E, s, false).total <= kSmemLimit) return s;
  return 0;
}
// K chunks of a down unit at most: enough for the fewest units there can be (one expert)
int chunks_for(int H, int I) {
  const int st2 = int((fp8_blocks(I) + 1) / 2);
  int c = (4 * 148 + int(fp8_blocks(H)) - 1) / int(fp8_blocks(H));
  return c < 1 ? 1 : (c > st2 ? st2 : (c > 8 ? 8 : c));
}
constexpr int kMaxParts = 4 * 148;

template <int NT, int PER_LANE, bool GROUPED = false>
cudaError_t launch_one(const CUtensorMap& m13, const CUtensorMap& m2, const CUtensorMap& mh, const CUtensorMap& mx, const LayerArgs& a,
                       int grid, size_t smem, cudaStream_t s) {
  constexpr auto kern = fp8_layer_kernel<NT, PER_LANE, GROUPED>;
  const cudaError_t e = set_smem_limit_once<kern>(kSmemLimit);
  return e != cudaSuccess ? e : launch_cooperative_dependent(kern, dim3(grid), dim3(kThreads), smem, s, m13, m2, mh, mx, a);
}

}  // namespace

bool fp8_layer_fits(int T, int H, int I, int E, int k) {
  return T >= 1 && T <= kTokens && stages_for(H, E, k) > 0 && int64_t(E) * ((fp8_blocks(I) > fp8_blocks(H) ? fp8_blocks(I) : fp8_blocks(H))) < (1 << 27);
}

Fp8LayerSizes fp8_layer_sizes(int T, int H, int I, int E, int k) {
  const int64_t P = int64_t(T) * k, nI = fp8_blocks(I);
  const int64_t touched = P < E ? P : E;
  Fp8LayerSizes z;
  z.counters = touched + kMaxParts + 1;
  z.parts = int64_t(kMaxParts) * 2 * kTokens * 128;
  z.slots = P * chunks_for(H, I) * H;
  z.h_codes = P * I;
  z.h_scale = P * nI;
  z.x_codes = int64_t(T) * H;
  z.x_scale = T * fp8_blocks(H);
  return z;
}

nvfp4moe_status launch_fp8_layer(const Fp8LayerCall& c, cudaStream_t s) {
  LayerArgs a{};
  a.logits = c.logits;
  a.x_scale = c.x_scale;
  a.T = c.T, a.H = c.H, a.I = c.I, a.E = c.E, a.k = c.k;
  a.nH = int(fp8_blocks(c.H)), a.nI = int(fp8_blocks(c.I));
  a.stages = stages_for(c.H, c.E, c.k);
  a.max_parts = kMaxParts;
  a.chunks_cap = chunks_for(c.H, c.I);
  a.w13_scale = c.w13_scale, a.w2_scale = c.w2_scale;
  a.h_codes = c.h_codes, a.h_scale = c.h_scale, a.parts = c.parts, a.slots = c.slots;
  const int touched = c.T * c.k < c.E ? c.T * c.k : c.E;
  a.done = c.counters, a.tickets = c.counters + touched, a.gbar = c.counters + touched + kMaxParts;
  a.out = static_cast<__nv_bfloat16*>(c.out);
  a.status = device_status_ptr();
  if (!a.status) return fail(NVFP4MOE_CUDA_ERROR, "device status word unavailable");
  CUtensorMap m13, m2, mh, mx;
  nvfp4moe_status st = make_fp8_map(&m13, c.w13_codes, c.H, c.I, 2 * int64_t(c.E), c.H, int64_t(c.I) * c.H, 128);
  if (st == NVFP4MOE_OK) st = make_fp8_map(&m2, c.w2_codes, c.I, c.H, c.E, c.I, int64_t(c.I) * c.H, 128);
  if (st == NVFP4MOE_OK) st = make_fp8_map(&mh, c.h_codes, c.I, int64_t(c.T) * c.k, 1, c.I, c.I, kTokens);
  if (st == NVFP4MOE_OK) st = make_fp8_map(&mx, c.x_codes, c.H, c.T, 1, c.H, c.H, kTokens);
  if (st != NVFP4MOE_OK) return st;
  cudaError_t e = launch_dependent(fp8_layer_prepare_kernel, dim3((c.T * a.nH * 8 + 255) / 256), dim3(256), 0, s,
                                   static_cast<const __nv_bfloat16*>(c.x), int(c.T), int(c.H), c.x_codes, c.x_scale,
                                   c.counters, int(touched + kMaxParts + 1));
  if (e != cudaSuccess) return fail(NVFP4MOE_CUDA_ERROR, "fp8 layer (prepare): %s", cudaGetErrorString(e));
  const size_t smem = smem_layout(kTokens, a.nH, c.k, c.E, a.stages, false).total;
  const int per = (c.E + 31) / 32, grid = num_sms();
  e = per <= 1    ? launch_one<kTokens, 1>(m13, m2, mh, mx, a, grid, smem, s)
      : per <= 4  ? launch_one<kTokens, 4>(m13, m2, mh, mx, a, grid, smem, s)
      : per <= 8  ? launch_one<kTokens, 8>(m13, m2, mh, mx, a, grid, smem, s)
      : per <= 16 ? launch_one<kTokens, 16>(m13, m2, mh, mx, a, grid, smem, s)
                  : launch_one<kTokens, 32>(m13, m2, mh, mx, a, grid, smem, s);
  if (e != cudaSuccess) return fail(NVFP4MOE_CUDA_ERROR, "fp8 layer: %s", cudaGetErrorString(e));
  return check_launch("fp8 layer");
}

nvfp4moe_status launch_fp8_stream(const GroupedArgs& g, int* counters, cudaStream_t s) {
  constexpr int nt = kStreamRows;
  LayerArgs a{};
  a.x_scale = g.x_scale;
  a.list = g.tiles;
  a.H = g.H, a.I = g.I, a.E = g.E;
  a.nH = int(fp8_blocks(g.H)), a.nI = int(fp8_blocks(g.I));
  for (a.stages = kMaxStages; smem_layout(nt, 0, 0, 0, a.stages, true).total > kSmemLimit; --a.stages) {
  }
  a.w13_scale = g.w13_scale, a.w2_scale = g.w2_scale;
  a.h_codes = g.h_codes, a.h_scale = g.h_scale, a.slots = g.slots;
  a.done = counters;
  a.status = device_status_ptr();
  if (!a.status) return fail(NVFP4MOE_CUDA_ERROR, "device status word unavailable");
  CUtensorMap m13, m2, mh, mx;
  nvfp4moe_status st = make_fp8_map(&m13, g.w13_codes, g.H, g.I, 2 * int64_t(g.E), g.H, int64_t(g.I) * g.H, 128);
  if (st == NVFP4MOE_OK) st = make_fp8_map(&m2, g.w2_codes, g.I, g.H, g.E, g.I, int64_t(g.I) * g.H, 128);
  if (st == NVFP4MOE_OK) st = make_fp8_map(&mh, g.h_codes, g.I, g.rows, 1, g.I, g.I, nt);
  if (st == NVFP4MOE_OK) st = make_fp8_map(&mx, g.x_codes, g.H, g.rows, 1, g.H, g.H, nt);
  if (st != NVFP4MOE_OK) return st;
  const size_t smem = smem_layout(nt, 0, 0, 0, a.stages, true).total;
  const cudaError_t e = launch_one<nt, 1, true>(m13, m2, mh, mx, a, num_sms(), smem, s);
  if (e != cudaSuccess) return fail(NVFP4MOE_CUDA_ERROR, "fp8 stream: %s", cudaGetErrorString(e));
  return check_launch("fp8 stream");
}

}  // namespace nvfp4moe
