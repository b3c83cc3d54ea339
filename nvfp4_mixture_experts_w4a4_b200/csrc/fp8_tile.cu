// FP8 x FP8 products with a scale per block of 128, on the tensor cores: one dense GEMM
// (fp8_gemm) and the grouped gate/up and down products of the routed layer.
//
//   D[m][n] = sum over kb of sa[m][kb] * sb[n / 128][kb] * sum over k in block kb of A[m][k] B[n][k]
//
// The tensor core sums one 128-element block of K (four tcgen05.mma kind::f8f6f4 of K = 32, fp32
// accumulators in TMEM); between blocks the partial sum is multiplied by its two scales and added
// to fp32 registers.  The rows of A are the MMA's M side, so a thread of the adding warps holds one
// row: the product of both scales is one number a thread, and a column costs one FMA.  (The weights
// on the M side, an expert's rows in steps of 16 on the N side: a third fewer blocks for 256 experts
// with 128 rows on average, but a scale a column, read from shared memory for every block, and an
// epilogue across warps; 1300 us a layer of 4096 tokens against 1060.  FMAs packed in pairs: slower,
// the register pairs cost moves.)  All of TMEM is accumulators (512 / BN of them), so the MMA of block
// kb + 1 runs under the additions of block kb.  Per block an SM multiplies for 512 cycles (128 x 256 x
// 128 at 8192 MACs a cycle) while its eight adding warps read 128 KB of TMEM (256 cycles) and issue 256
// FMAs a scheduler (256 cycles).  What a block takes is 1000 to 1200 cycles.  Dense: 4096 x 5120 x 17408 in
// pairs 366 to 370 us in a burst (1990 TFLOP/s), 425 to 435 in a long run (power: 1.57 GHz).  Of a run of 391,
// 306 were left without the additions: the rest is the way between the MMA and the additions (commit, barrier,
// read, barrier).  And 320 tiles on 74 pairs are 4.32 rounds that take the time of five: in the last, 50 pairs
// have nothing to do, 13.5 % of the time.  Grouped, with experts of 128 rows and more: the loads, 10 TB/s from
// L2 of which 4.5 come from memory (4096 tokens, 256 experts of 4096 x 1024: gate/up 492 us, down 343; with
// the additions left out the layer lost 65 of 993 us, three stages were as good as four, and prefetches into L2
// cost 6 to 14 %).
//
//   warp 0      TMA producer: 128 rows of A and BN rows of B, 128 bytes of K each, per stage
//   warp 1      TMEM owner and MMA issuer
//   warps 2, 3  the products of both scales for eight blocks at a time, into shared memory (read by
//               the adding warps themselves, every eighth block waited out an L2 read: 787 -> 484 us for
//               4096 x 5120 x 17408)
//   warps 4..11 additions and epilogue: warp w reads TMEM lanes 32 * (w % 4), the first four take
//               the left half of the columns and the others the right half
// A thread that adds holds 128 sums, so the register file is split unevenly: launched with 168
// registers a thread (384 threads, 64512), warps 0..3 keep 40 and warps 4..11 take 232 (the same sum).
//
// Pairs of CTAs (cta_group::2) take 256 x 256 tiles of large dense products: each loads half of B, a
// third less to load (2048 x 4096 x 4096: 42.6 us, 46.3 unpaired).  Grouped tiles stay single: an
// expert's rows rarely fill 256 (gate/up 588 us in pairs, 490 single, 256 experts with 128 rows on
// average).  Where experts have few rows their weights come at 4.5 TB/s in these two launches; fp8_layer.cu, which
// streams gate/up and down weights in one, gets 5.5 to 6, so this is not the memory's own limit: each launch
// waits for the one before it with nothing in flight (how much of the difference that makes is not measured).
//
// Products with few tiles and a long sum split K over the CTAs of a cluster (SPLIT): each adds its
// share of the blocks, writes its tile to its own shared memory, and the cluster's CTAs sum slices
// of it in rank order through distributed shared memory, so results do not depend on timing.
// Every wait is bounded (status bit on timeout; copies in flight land before the CTA exits).
#include <cooperative_groups.h>

#include "fp8.cuh"
#include "fp8_tile.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace nvfp4moe {
namespace {

using namespace sm100;

constexpr int TM = 128;              // rows of A per tile (the MMA's M)
constexpr int TK = FP8_BLOCK;        // K per stage: one scale block, one 128-byte swizzle row
constexpr int TTHREADS = 384;
constexpr int ADD_WARPS = 8;
constexpr int A_STAGE = TM * TK;
constexpr int kMaxSplit = 8;         // CTAs of a cluster (the portable size)
constexpr uint32_t kTimeout = NVFP4MOE_DEV_TIMEOUT;

enum Mode { DENSE = 0, GATEUP = 1, DOWN = 2 };

constexpr int SC_BLOCKS = 8;                    // blocks of K whose scales are staged at once: 32 bytes of a row
constexpr int SC_FLOATS = SC_BLOCKS * 2 * TM;   // [block][half][row]

// rows of B a CTA holds per stage, stages, and shared memory
constexpr int b_rows(int bn, bool pair) { return pair ? bn / 2 : bn; }
constexpr int stages_of(int mode, int bn, bool pair) { return mode == DOWN ? 3 : (b_rows(bn, pair) == 256 ? 4 : 6); }
constexpr int OUT_BLOCK = 32 * 128;  // down: 32 rows x 32 columns of fp32, two a warp, on their way out
constexpr int ring_bytes(int mode, int bn, bool pair) {
  return stages_of(mode, bn, pair) * (A_STAGE + b_rows(bn, pair) * TK) + (mode == DOWN ? 2 * ADD_WARPS * OUT_BLOCK : 0);
}
constexpr int amax_bytes(int mode) { return mode == GATEUP ? 2 * 2 * TM * 4 : 0; }
constexpr int smem_bytes(int mode, int bn, bool pair) {
  return 1024 + ring_bytes(mode, bn, pair) + (2 * stages_of(mode, bn, pair) + 2 * (512 / bn) + 5) * 8 + 48 +
         amax_bytes(mode) + 2 * SC_FLOATS * 4;
}
constexpr int split_pitch(int bn) { return bn + 4; }  // floats; rows 16 bytes apart in the banks

// Loads into this CTA's shared memory; PAIR: the bytes are counted on a barrier of either CTA of the
// pair (bar: its shared::cluster address).
template <bool PAIR>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                         uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The shared::cluster address of rank's copy of a shared variable of this CTA.
__device__ __forceinline__ uint32_t cluster_address(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Arrivals that say "these TMEM columns have been read".  The reads are complete (tcgen05.wait::ld)
// and nothing in memory is passed on, so they are relaxed: a release would wait for the thread's
// outstanding loads of scales, 1700 cycles a block at cluster scope and 200 at CTA scope.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_here(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same instruction as tc_mma_f8 over a pair's two shared memories and TMEMs.
__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, {%5, %5, %5, %5, %5, %5, %5, %5}, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(0u)
      : "memory");
}

// Arrives on `bar` (PAIR: in both CTAs) once every MMA issued so far by this thread has completed.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    tc_commit(bar);
}

template <bool PAIR>
__device__ __forceinline__ void alloc_tmem(uint32_t* dst, uint32_t ncols) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, ncols);
    tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void free_tmem(uint32_t taddr, uint32_t ncols) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
  else
    tmem_dealloc(taddr, ncols);
}

// tcgen05.wait::ld that the registers of the load pass through, so that no use of them can be moved
// before it while other loads are in flight.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void store_32b(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Moves registers between the four-warp groups of a block (all four warps of a group call it).
template <int N>
__device__ __forceinline__ void reg_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

struct Tile {
  int e;     // matrix of B (expert)
  int row;   // first row of A
  int rows;  // rows of the tile that exist
  int n0;    // first column
};

// Tile t of the launch.  Dense: bands of 16 row tiles, column tiles outside rows in a band, so
// the CTAs that run together read few rows of both operands.  Grouped: the list's row tiles (an
// expert's are neighbours), column tiles inside.
template <bool PAIR>
__device__ __forceinline__ Tile tile_of(const TileParams& p, int t, int bn, bool grouped) {
  Tile w;
  if (grouped) {
    const int m = t / p.n_nt;
    const int4 q = __ldg(p.tiles + 1 + m);
    w.e = q.x, w.row = q.y, w.rows = q.z, w.n0 = (t - m * p.n_nt) * bn;
  } else {
    constexpr int BAND = PAIR ? 8 : 16;
    const int band = t / (BAND * p.n_nt), in = t - band * BAND * p.n_nt;
    const int high = min(BAND, p.n_mt - band * BAND);
    const int n = in / high;
    w.e = 0;
    constexpr int high_rows = PAIR ? 2 * TM : TM;
    w.row = (band * BAND + in - n * high) * high_rows;
    w.rows = min(high_rows, p.M - w.row);
    w.n0 = n * bn;
  }
  return w;
}

// The columns of a warp's half: two runs of 32 a step, BN / 2 apart in a gate/up tile (its gate and up columns).
template <int MODE, int BN>
__device__ __forceinline__ uint32_t tile_column(int half, int c) {
  constexpr int HALF = BN / 2;
  if constexpr (MODE == GATEUP) return uint32_t(c < HALF / 2 ? half * (HALF / 2) + c : TM + half * (HALF / 2) + c - HALF / 2);
  else return uint32_t(half * HALF + c);
}

// Adds n blocks' sums times one scale, then the other, read from memory again: what a batch of scales takes
// some of whose products are no ordinary numbers.  sa, sb: the first block's (sb_up further on the up's).
// Such a batch is held back at its barrier until every adding warp, waiting there, has seen its number, so
// that the loop that all others take has no choice to make: with one, its reads and additions did not run
// into one another as before (4096 x 5120 x 17408: 373 us without; a choice for every block 399 to 441, for
// every batch 381 to 389, with this in or out of line).
template <int MODE, int BN, bool PAIR>
__device__ __noinline__ bool add_with_both(float* sums, const float* sa, const float* sb, int64_t sb_up, int n, uint32_t it,
                                           uint32_t trow, int half, uint64_t* acc_full, uint64_t* acc_empty) {
  constexpr int HALF = BN / 2;
  constexpr uint32_t NACC = 512 / BN;
  for (int j = 0; j < n; ++j, ++it) {
    if (!mbar_wait_warp(&acc_full[it % NACC], (it / NACC) & 1)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < HALF; c += 32) {
      float first, second;
      fp8_factors(__ldg(sa + j), __ldg(sb + j + (c >= HALF / 2 ? sb_up : 0)), first, second);
      uint32_t v[32];
      tmem_ld_32x32b_x32(trow + (it % NACC) * BN + tile_column<MODE, BN>(half, c), v);
      tmem_ld_wait_for(v);
#pragma unroll
      for (int i = 0; i < 32; ++i) sums[c + i] = fmaf(__uint_as_float(v[i]) * first, second, sums[c + i]);
    }
    tc_fence_before();
    if ((threadIdx.x & 31) == 0) {
      if constexpr (PAIR) arrive_at(cluster_address(&acc_empty[it % NACC], 0));
      else arrive_here(&acc_empty[it % NACC]);
    }
  }
  return true;
}

template <int MODE, int BN, bool SPLIT, bool PAIR>
__global__ void __launch_bounds__(TTHREADS, 1)
fp8_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmD, const TileParams p) {
  constexpr int STAGES = stages_of(MODE, BN, PAIR);
  constexpr int B_ROWS = b_rows(BN, PAIR);
  constexpr int B_STAGE = B_ROWS * TK;
  static_assert(!PAIR || (MODE == DENSE && BN == 256 && !SPLIT), "a pair runs 256 x 256 tiles of a dense product, whole sums");
  constexpr int HALF = BN / 2;          // columns an adding warp holds
  constexpr uint32_t NACC = 512 / BN;   // accumulators: all of TMEM
  constexpr bool GROUPED = MODE != DENSE;
  static_assert(MODE != GATEUP || BN == 256, "a gate/up tile is one 128-column block of each");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_shared_1024(smem_raw);
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * A_STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + ring_bytes(MODE, BN, PAIR));
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;  // [NACC]
  uint64_t* acc_empty = acc_full + NACC;
  uint64_t* sc_full = acc_empty + NACC; // [2]
  uint64_t* sc_empty = sc_full + 2;     // [2]
  uint64_t* drain = sc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  // the rare batches of scales: their number + 1, from either scale warp, and from each adding warp once it knows
  volatile uint32_t* sc_rare = tmem_holder + 2;    // [2]
  volatile uint32_t* rare_seen = tmem_holder + 4;  // [ADD_WARPS]
  uint32_t* s_amax = reinterpret_cast<uint32_t*>(tmem_holder + 4 + ADD_WARPS);  // gate/up: [2][2][128]: tile parity, half, row
  float* s_scale = reinterpret_cast<float*>(s_amax + amax_bytes(MODE) / 4);  // [2][SC_BLOCKS][2][128]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < NACC; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], PAIR ? 2 * ADD_WARPS : ADD_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sc_full[b], 64);
      mbar_init(&sc_empty[b], ADD_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    for (int i = 0; i < 2; ++i) sc_rare[i] = 0u;
    for (int i = 0; i < ADD_WARPS; ++i) rare_seen[i] = 0u;
    mbar_fence_init();
  }
  if (warp == 1) alloc_tmem<PAIR>(tmem_holder, 512);
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
    if constexpr (MODE == DOWN) prefetch_tensormap(&tmD);
  }
  griddep_wait();  // the operands may come from the launch before
  tc_fence_before();
  __syncthreads();
  griddep_launch_dependents();  // TMEM is taken: a launch that starts now and allocates some cannot keep it from this one
  if constexpr (PAIR) cluster_barrier();  // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  auto abort_now = [&]() {
    *abort_flag = 1;
    atomicOr(p.status, kTimeout);
  };
  auto warp_aborted = [&]() { return __any_sync(0xffffffffu, *abort_flag) != 0; };  // one answer for a whole warp

  const int ranks = SPLIT ? p.split : 1;
  const int rank = SPLIT ? int(blockIdx.x) % ranks : 0;
  const int side = PAIR ? int(cluster_rank()) : 0;  // this CTA's half of the rows of A and of B
  const int kb0 = int(int64_t(p.nkb) * rank / ranks), kb1 = int(int64_t(p.nkb) * (rank + 1) / ranks);
  const int n_tiles = (GROUPED ? p.tiles[0].x : p.n_mt) * p.n_nt;
  constexpr int CTAS = PAIR ? 2 : 1;
  const int t_first = int(blockIdx.x) / (ranks * CTAS), t_step = int(gridDim.x) / (ranks * CTAS);
  // a grouped tile comes from the list in memory, so each role reads one tile ahead
  auto tile_at = [&](int t) { return t < n_tiles ? tile_of<PAIR>(p, t, BN, GROUPED) : Tile{0, 0, 1, 0}; };
  auto rows_of = [&](const Tile& w, int sd) { return max(0, min(TM, w.rows - sd * TM)); };

  if (warp < 4) {
    reg_give<40>();
    if (warp == 0 && elect_one()) {
      uint32_t it = 0;
      Tile next = tile_at(t_first);
      for (int t = t_first; t < n_tiles && !*abort_flag; t += t_step) {
        const Tile w = next;
        next = tile_at(t + t_step);
        const int boxes = (rows_of(w, side) + p.a_box - 1) / p.a_box;
        const int all_boxes = PAIR ? boxes + (rows_of(w, side ^ 1) + p.a_box - 1) / p.a_box : boxes;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&empty[s], ((it / STAGES) & 1) ^ 1)) {
            abort_now();
            break;
          }
          // a pair's bytes are counted by the first CTA, whose MMA reads both halves
          const uint32_t bar = PAIR ? cluster_address(&full[s], 0) : smem_u32(&full[s]);
          if (side == 0) mbar_arrive_expect_tx(&full[s], all_boxes * p.a_box * TK + CTAS * B_STAGE);
          for (int b = 0; b < boxes; ++b)
            load_box<PAIR>(sA + s * A_STAGE + b * p.a_box * TK, &tmA, kb * TK, w.row + side * TM + b * p.a_box, 0, bar);
          if constexpr (MODE == GATEUP) {
            load_box<PAIR>(sB + s * B_STAGE, &tmB, kb * TK, w.n0 / 2, 2 * w.e, bar);
            load_box<PAIR>(sB + s * B_STAGE + TM * TK, &tmB, kb * TK, w.n0 / 2, 2 * w.e + 1, bar);
          } else {
            load_box<PAIR>(sB + s * B_STAGE, &tmB, kb * TK, w.n0 + side * B_ROWS, w.e, bar);
          }
        }
      }
      // the copies land before the CTA leaves (a pair's are counted by its first CTA, and the second
      // waits for it at the end)
      if (*abort_flag && side == 0)
        for (uint32_t back = 0; back < STAGES && back < it; ++back) {
          const uint32_t j = it - 1 - back;
          mbar_wait(&full[j % STAGES], (j / STAGES) & 1, 1u << 16);
        }
    } else if (warp == 1 && side == 0 && elect_one()) {
      constexpr uint32_t idesc = idesc_f8(PAIR ? 2 * TM : TM, BN);
      uint32_t it = 0;
      bool ok = true;
      for (int t = t_first; t < n_tiles && ok && !*abort_flag; t += t_step) {
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ab = it % NACC;
          if (!mbar_wait(&acc_empty[ab], ((it / NACC) & 1) ^ 1) || !mbar_wait(&full[s], (it / STAGES) & 1)) {
            abort_now();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a_d = desc_kmajor_sw128(sA + s * A_STAGE);
          const uint64_t b_d = desc_kmajor_sw128(sB + s * B_STAGE);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // K = 32 per MMA: 32 bytes = 2 descriptor units
            if constexpr (PAIR) tc_mma_f8_pair(tmem + ab * BN, a_d + 2 * j, b_d + 2 * j, idesc, j != 0 ? 1u : 0u);
            else tc_mma_f8(tmem + ab * BN, a_d + 2 * j, b_d + 2 * j, idesc, j != 0 ? 1u : 0u);
          }
          commit<PAIR>(&empty[s]);
          commit<PAIR>(&acc_full[ab]);
        }
      }
      commit<PAIR>(drain);
      mbar_wait(drain, 0, 1u << 20);
    } else if (warp >= 2) {
      // the products of both scales for SC_BLOCKS blocks at a time: a lane takes rows l and l + 64
      const int l = (warp - 2) * 32 + lane;
      uint32_t batch = 0;
      Tile next = tile_at(t_first);
      // Whether some product of the batch's scales may be no ordinary number: by the smallest (zeros apart) and the
      // largest of both, so it says so of some batches without one too.
      auto rare = [&](const float (&a)[2][SC_BLOCKS], float b) {
        uint32_t lo = 0xFFFFFFFFu, hi = 0u;  // of the magnitudes' bits, lo less one: a zero counts as large
#pragma unroll
        for (int j = 0; j < SC_BLOCKS; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) lo = min(lo, abs_bits(a[i][j]) - 1u), hi = max(hi, abs_bits(a[i][j]));
        const uint32_t b_lo = __reduce_min_sync(0xffffffffu, abs_bits(b) - 1u), b_hi = __reduce_max_sync(0xffffffffu, abs_bits(b));
        return __any_sync(0xffffffffu, fp8_needs_both(__uint_as_float(lo + 1u), __uint_as_float(b_lo + 1u)) |
                                           fp8_needs_both(__uint_as_float(hi), __uint_as_float(b_hi))) != 0;
      };
      for (int t = t_first; t < n_tiles && !warp_aborted(); t += t_step) {
        const Tile w = next;
        next = tile_at(t + t_step);
        const float* sa[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          sa[i] = p.sa + int64_t(w.row + min(side * TM + l + 64 * i, w.rows - 1)) * p.lda_s;
        // lanes 0..7 read the first half's scale of B for blocks 0..7, lanes 8..15 the second's
        const int hb = (lane >> 3) & 1;
        const float* sb;
        if constexpr (MODE == GATEUP) sb = p.sb + (2 * w.e + hb) * p.sb_e + (w.n0 / 256) * p.ldb_s;
        else sb = p.sb + w.e * p.sb_e + min(w.n0 / TK + (BN == 256 ? hb : 0), p.nsb - 1) * p.ldb_s;
        for (int kb = kb0; kb < kb1; kb += SC_BLOCKS, ++batch) {
          const int last = kb1 - 1;
          float a[2][SC_BLOCKS];
#pragma unroll
          for (int j = 0; j < SC_BLOCKS; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) a[i][j] = __ldg(sa[i] + min(kb + j, last));
          const float b = __ldg(sb + min(kb + (lane & 7), last));
          if (!mbar_wait_warp(&sc_empty[batch & 1], ((batch >> 1) & 1) ^ 1)) {
            abort_now();
            break;
          }
          float* dst = s_scale + (batch & 1) * SC_FLOATS + l;
#pragma unroll
          for (int j = 0; j < SC_BLOCKS; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float bj = __shfl_sync(0xffffffffu, b, h * 8 + j);
#pragma unroll
              for (int i = 0; i < 2; ++i) dst[(j * 2 + h) * TM + 64 * i] = a[i][j] * bj;
            }
          if (rare(a, b)) {
            // the adding warps, held up at sc_full, see the number; when all have, the batch may go on
            if (lane == 0) sc_rare[warp - 2] = batch + 1;
            bool seen = false;
            for (uint32_t i = 0; i < (1u << 22) && !seen; ++i) {
              seen = __all_sync(0xffffffffu, int32_t(rare_seen[lane % ADD_WARPS] - (batch + 1)) >= 0);
              if (!seen) __nanosleep(64);
            }
            if (!seen) {
              abort_now();
              break;
            }
          }
          mbar_arrive(&sc_full[batch & 1]);
        }
      }
    }
  } else {
    reg_take<232>();
    const int q = warp & 3;               // the TMEM lane quarter this warp may read
    const int half = (warp - 4) >> 2;     // its half of the columns
    const uint32_t trow = tmem + (uint32_t(q * 32) << 16);
    const uint32_t release_bar = PAIR ? cluster_address(&acc_empty[0], 0) : 0u;
    uint32_t it = 0, batch = 0;
    int done = 0;
    for (int t = t_first; t < n_tiles && (MODE == GATEUP || !warp_aborted()); t += t_step, ++done) {
      const Tile pair_tile = tile_at(t);
      Tile w = pair_tile;  // this CTA's rows of it
      w.row += side * TM;
      w.rows = rows_of(pair_tile, side);
      const int r = q * 32 + lane;
      const bool live = q * 32 < w.rows;  // the same for the whole warp
      float acc[HALF];
#pragma unroll
      for (int i = 0; i < HALF; ++i) acc[i] = 0.0f;
      bool ok = true;
      auto sums_ready = [&](uint32_t i) { return mbar_try_wait(&acc_full[i % NACC], (i / NACC) & 1); };
      auto wait_sums = [&](uint32_t i) {
        if (!mbar_wait_warp(&acc_full[i % NACC], (i / NACC) & 1)) {
          abort_now();
          ok = false;
        }
      };
      auto is_rare = [&](uint32_t b) { return __any_sync(0xffffffffu, sc_rare[0] == b + 1 || sc_rare[1] == b + 1) != 0; };
      auto wait_scales = [&](uint32_t b) {
        for (uint32_t i = 0; i < (1u << 22); ++i) {
          if (__all_sync(0xffffffffu, mbar_try_wait(&sc_full[b & 1], (b >> 1) & 1))) return true;
          if (is_rare(b)) return false;
        }
        return false;
      };
      // The accumulator's columns have been read by this warp (tcgen05.wait::ld is the whole warp's).
      auto release_sums = [&](uint32_t i) {
        tc_fence_before();
        if (lane == 0) {
          if constexpr (PAIR) arrive_at(release_bar + 8 * (i % NACC));
          else arrive_here(&acc_empty[i % NACC]);
        }
      };
      // Chunks of 32 columns, each read and added before the next is read: the two warps of a
      // scheduler cover each other's reads.  A poll of the next block's barrier takes 250 cycles to
      // come back, so it is sent before the last chunk's additions.
      bool ready = false;
#pragma unroll 1
      for (int kb = kb0; kb < kb1 && ok; kb += SC_BLOCKS, ++batch) {
        int n = min(SC_BLOCKS, kb1 - kb);
        const float* sc = s_scale + (batch & 1) * SC_FLOATS + (MODE == GATEUP || BN == 128 ? 0 : half * TM) + r;
        if (!wait_scales(batch)) {
          // gave up, or a rare batch (add_with_both)
          ok = is_rare(batch);
          if (ok) {
            if (lane == 0) rare_seen[warp - 4] = batch + 1;
            const int nb = MODE == GATEUP ? w.n0 / 256 : min(w.n0 / TK + (BN == 256 ? half : 0), p.nsb - 1);
            const float* sa = p.sa + int64_t(MODE == DENSE ? min(w.row + r, p.M - 1) : w.row + min(r, w.rows - 1)) * p.lda_s + kb;
            const float* sb = p.sb + (MODE == GATEUP ? 2 * w.e : w.e) * p.sb_e + nb * p.ldb_s + kb;
            float sums[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) sums[i] = acc[i];
            ok = mbar_wait_warp(&sc_full[batch & 1], (batch >> 1) & 1) &&
                 add_with_both<MODE, BN, PAIR>(sums, sa, sb, MODE == GATEUP ? p.sb_e : 0, n, it, trow, half, acc_full, acc_empty);
#pragma unroll
            for (int i = 0; i < HALF; ++i) acc[i] = sums[i];
          }
          if (!ok) {
            abort_now();
            break;
          }
          it += n;
          n = 0;
          ready = false;
        }
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++it, sc += 2 * TM) {
          const float s0 = sc[0], s1 = MODE == GATEUP ? sc[TM] : s0;
          if (!__all_sync(0xffffffffu, ready)) {
            wait_sums(it);
            if (!ok) break;
          }
          tc_fence_after();
          if (live) {
#pragma unroll
            for (int c = 0; c < HALF; c += 32) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(trow + (it % NACC) * BN + tile_column<MODE, BN>(half, c), v);
              tmem_ld_wait_for(v);
              if (c + 32 == HALF) {
                release_sums(it);
                ready = kb + j + 1 < kb1 && sums_ready(it + 1);
              }
              const float x = c >= HALF / 2 ? s1 : s0;
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[c + i] = fmaf(__uint_as_float(v[i]), x, acc[c + i]);
            }
          } else {  // rows past the tile's last: the accumulators only pass through
            release_sums(it);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_empty[batch & 1]);
      }
      if (MODE != GATEUP && !ok) break;

      if constexpr (SPLIT) {
        // this rank's share, by row, over the idle ring (every stage of it has been consumed)
        if (live) {
          float* dst = reinterpret_cast<float*>(smem) + r * split_pitch(BN) + half * HALF;
#pragma unroll
          for (int i = 0; i < HALF / 2; i += 2) {
            float4 f;
            f.x = acc[2 * i], f.y = acc[2 * i + 1];
            f.z = acc[2 * i + 2], f.w = acc[2 * i + 3];
            *reinterpret_cast<float4*>(dst + 2 * i) = f;
          }
        }
      } else if constexpr (MODE == GATEUP) {
        // h = silu(g) * u, its row's maximum over the 128 columns, then its codes
        const int i0 = w.n0 / 2;
        float h[HALF / 2];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < HALF / 4; ++i) {
          float g[2], u[2];
          g[0] = acc[2 * i], g[1] = acc[2 * i + 1];
          u[0] = acc[HALF / 2 + 2 * i], u[1] = acc[HALF / 2 + 2 * i + 1];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            h[2 * i + j] = silu_times(g[j], u[j]);
            m = max(m, abs_bits(h[2 * i + j]));
          }
        }
        uint32_t* sm = s_amax + (done & 1) * 2 * TM;  // two tiles' worth: the barrier below orders reuse
        sm[half * TM + r] = m;
        if (add_barrier_any(!ok)) break;
        m = max(m, sm[(half ^ 1) * TM + r]);
        const Fp8Scale f = fp8_scale(m);
        if (r < w.rows) {
          const int64_t row = w.row + r;
          if (half == 0) p.h_scale[row * p.ldh_s + i0 / TK] = f.scale;
          uint8_t* dst = p.h_codes + row * p.ldh + i0 + half * (HALF / 2);
#pragma unroll
          for (int c = 0; c < HALF / 2; c += 16) {
            if (i0 + half * (HALF / 2) + c < p.I) {  // I is a multiple of 16
              uint4 o;
              o.x = fp8_encode4(h + c, f);
              o.y = fp8_encode4(h + c + 4, f);
              o.z = fp8_encode4(h + c + 8, f);
              o.w = fp8_encode4(h + c + 12, f);
              *reinterpret_cast<uint4*>(dst + c) = o;
            }
          }
        }
      } else if constexpr (MODE == DOWN) {
        const int n = w.n0 + half * HALF;
        if (live && n < p.N) {
          uint8_t* out = smem + STAGES * (A_STAGE + B_STAGE) + (warp - 4) * 2 * OUT_BLOCK;
          const bool whole = q * 32 + 32 <= w.rows;  // the rows after the last are another tile's
#pragma unroll
          for (int c = 0; c < HALF; c += 32) {
            if (whole) {
              // through shared memory and a tile store: 128 bytes of a row at a time (a lane storing its
              // own row takes a turn for every 32 bytes: 7000 cycles a tile)
              uint8_t* block = out + (c / 32 & 1) * OUT_BLOCK;
              bulk_wait_group_read<1>();
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float* v = acc + c + 4 * i;
                *reinterpret_cast<float4*>(block + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
              }
              fence_proxy_async_shared();
              __syncwarp();
              if (lane == 0) {
                if (n + c < p.N) tma_store_2d(&tmD, n + c, w.row + q * 32, block);
                bulk_commit_group();
              }
            } else if (r < w.rows) {
              float* d = static_cast<float*>(p.D) + int64_t(w.row + r) * p.ldd + n + c;
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                if (n + c + i < p.N) {  // N is a multiple of 16
                  uint32_t o[8];
#pragma unroll
                  for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(acc[c + i + j]);
                  store_32b(d + i, o);
                }
            }
          }
        }
      } else {
        const int n = w.n0 + half * HALF;
        if (!p.d_vec) {
          // Rows that do not start at multiples of 32 bytes: 32 x 32 blocks are transposed through
          // shuffles, and a store is 32 consecutive columns of one row.
          if (live) {
#pragma unroll
            for (int c = 0; c < HALF; c += 32) {
              float* v = acc + c;
#pragma unroll
              for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if ((i & o) == 0) {
                    const bool upper = (lane & o) != 0;
                    const float got = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + o], o);
                    if (upper) v[i] = got;
                    else v[i + o] = got;
                  }
              const int col = n + c + lane;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if (q * 32 + i < w.rows && col < p.N) {
                  const int64_t to = int64_t(w.row + q * 32 + i) * p.ldd + col;
                  if (p.d_f32) static_cast<float*>(p.D)[to] = v[i];
                  else static_cast<__nv_bfloat16*>(p.D)[to] = __float2bfloat16_rn(v[i]);
                }
              }
            }
          }
        } else if (r < w.rows) {
          const int64_t at = int64_t(w.row + r) * p.ldd + n;
          if (p.d_f32) {
            float* d = static_cast<float*>(p.D) + at;
#pragma unroll
            for (int c = 0; c < HALF; c += 8) {
              if (n + c + 8 <= p.N) {
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(acc[c + i]);
                store_32b(d + c, o);
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (n + c + i < p.N) d[c + i] = acc[c + i];
              }
            }
          } else {
            __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.D) + at;
#pragma unroll
            for (int c = 0; c < HALF; c += 16) {
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = bf16x2(acc[c + 2 * i], acc[c + 2 * i + 1]);
              if (n + c + 16 <= p.N) {
                store_32b(d + c, o);
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (n + c + i < p.N) d[c + i] = __ushort_as_bfloat16(static_cast<uint16_t>(o[i >> 1] >> (16 * (i & 1))));
              }
            }
          }
        }
      }
    }
  }

  if constexpr (MODE == DOWN)
    if (warp >= 4 && lane == 0) bulk_wait_group<0>();  // the last rows are out
  tc_fence_before();
  __syncthreads();
  // a pair leaves together: each CTA's shared memory and barriers are used by the other
  if constexpr (PAIR) cluster_barrier();
  tc_fence_after();
  if (warp == 1) free_tmem<PAIR>(tmem, 512);

  if constexpr (SPLIT) {
    // Every CTA of the cluster runs one tile (the grid is tiles * ranks), reaches both barriers on
    // every path, and sums its share of the tile's columns over the ranks in order.
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const Tile w = tile_of<PAIR>(p, t_first, BN, GROUPED);
    const int f0 = BN / 4 * rank / ranks, per_row = BN / 4 * (rank + 1) / ranks - f0;  // groups of four columns
    float* mine = reinterpret_cast<float*>(smem);
    for (int i = threadIdx.x; i < w.rows * per_row; i += TTHREADS) {
      const int r = i / per_row, c = (f0 + i - r * per_row) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < ranks; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(mine, k) + r * split_pitch(BN) + c);
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      const int n = w.n0 + c;
      const int64_t at = int64_t(w.row + r) * p.ldd + n;
      if (p.d_f32) {
        float* d = static_cast<float*>(p.D) + at;
        if (p.d_vec && n + 4 <= p.N) {
          *reinterpret_cast<float4*>(d) = v;
        } else {
          const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < p.N) d[j] = f[j];
        }
      } else {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.D) + at;
        const uint32_t o[2] = {bf16x2(v.x, v.y), bf16x2(v.z, v.w)};
        if (p.d_vec && n + 4 <= p.N) {
          *reinterpret_cast<uint2*>(d) = make_uint2(o[0], o[1]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < p.N) d[j] = __ushort_as_bfloat16(static_cast<uint16_t>(o[j >> 1] >> (16 * (j & 1))));
        }
      }
    }
    cluster.sync();  // no CTA leaves while another still reads its shared memory
  }
}

template <int MODE, int BN, bool SPLIT, bool PAIR>
cudaError_t launch_tiles(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& d, const TileParams& p, int grid,
                         cudaStream_t s) {
  constexpr auto kern = fp8_tile_kernel<MODE, BN, SPLIT, PAIR>;
  cudaError_t e = set_smem_limit_once<kern>(smem_bytes(MODE, BN, PAIR));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(TTHREADS);
  cfg.dynamicSmemBytes = smem_bytes(MODE, BN, PAIR);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (SPLIT || PAIR) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = PAIR ? 2 : p.split;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  // set-up runs under the end of the launch before, whichever that is; nothing is read or written first
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, a, b, d, p);
}

}  // namespace

// [mats][rows][K] bytes, rows `pitch` apart and matrices `mat_pitch`; box 128 bytes x box_rows,
// 128-byte swizzle.  Rows and bytes past the ends read as zero.
nvfp4moe_status make_fp8_map(CUtensorMap* map, const void* base, int64_t K, int64_t rows, int64_t mats, int64_t pitch,
                         int64_t mat_pitch, int box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return fail(NVFP4MOE_CUDA_ERROR, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[3] = {cuuint64_t(K), cuuint64_t(rows), cuuint64_t(mats)};
  const cuuint64_t strides[2] = {cuuint64_t(pitch), cuuint64_t(mat_pitch)};
  const cuuint32_t box[3] = {cuuint32_t(FP8_BLOCK), cuuint32_t(box_rows), 1u};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
                        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(NVFP4MOE_CUDA_ERROR, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return NVFP4MOE_OK;
}

namespace {

// Clusters of `split` CTAs that run at once, read once per device and variant.
template <int BN>
int resident_clusters(int split) {
  static std::atomic<int> known[64][kMaxSplit + 1];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64)
    if (const int v = known[dev][split].load(std::memory_order_relaxed)) return v;
  constexpr auto kern = fp8_tile_kernel<DENSE, BN, true, false>;
  int n = 0;
  if (set_smem_limit_once<kern>(smem_bytes(DENSE, BN, false)) == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(num_sms() / split * split));
    cfg.blockDim = dim3(TTHREADS);
    cfg.dynamicSmemBytes = smem_bytes(DENSE, BN, false);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
  }
  if (n < 1) {
    cudaGetLastError();  // the estimate below stands in
    n = num_sms() / (2 * split);
  }
  if (dev >= 0 && dev < 64) known[dev][split].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace

namespace {

// fp32 [rows][H], box 32 columns x 32 rows, 128-byte swizzle; stores past the last column are clipped.
nvfp4moe_status make_f32_rows_map(CUtensorMap* map, void* base, int64_t rows, int64_t H) {
  auto fn = tensor_map_encoder();
  if (!fn) return fail(NVFP4MOE_CUDA_ERROR, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[2] = {cuuint64_t(H), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(H * 4)};
  const cuuint32_t box[2] = {32u, 32u};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(NVFP4MOE_CUDA_ERROR, "cuTensorMapEncodeTiled (fp32 rows) failed (%d)", int(r));
  return NVFP4MOE_OK;
}

}  // namespace

// How a dense product is run: the width of a tile, the CTAs that split its K, and whether pairs of
// CTAs take 256 rows.  The estimate, in microseconds fitted to measurements on a B200: every round of
// resident tiles costs its blocks of K (a 128 x 128 tile's in 0.30, or 0.36 where more than half of the
// SMs are busy, a 128 x 256 tile's in 0.62, a pair's in 0.58) and 1.0 for its start and end; a split
// tile 2.0 + 0.8 a CTA instead, for the exchange.  E.g. 64 x 4096 x 4096: 11.5 measured with 128 columns split over 4, 16.1 unsplit, 27.7
// over 8 (clusters of 8 do not all fit at once); 2048 x 4096 x 4096: 42.6 in pairs, 46.3 unpaired.
DensePlan fp8_dense_plan(int64_t M, int64_t N, int64_t K) {
  const int sms = num_sms();
  const int nkb = int(fp8_blocks(K));
  auto rounds = [](int64_t tiles, int64_t at_once) { return double((tiles + at_once - 1) / at_once); };
  const int64_t pairs = ((M + 255) / 256) * ((N + 255) / 256);
  DensePlan best{256, 1, true};
  double least = M > TM ? rounds(pairs, sms / 2) * (nkb * 0.58 + 1.0) : 1e300;
  for (int bn : {256, 128}) {
    const int64_t tiles = ((M + TM - 1) / TM) * ((N + bn - 1) / bn);
    for (int split = 1; split <= kMaxSplit; ++split) {
      if (split > 1 && (split > nkb || tiles * split > sms)) break;
      const int64_t at_once = split == 1 ? sms : (bn == 256 ? resident_clusters<256>(split) : resident_clusters<128>(split));
      const double block = bn == 256 ? 0.62 : (tiles * split > sms / 2 ? 0.36 : 0.30);
      const double cost =
          rounds(tiles, at_once) * (((nkb + split - 1) / split) * block + (split > 1 ? 2.0 + 0.8 * split : 1.0));
      if (cost < least) {
        least = cost;
        best = DensePlan{bn, split, false};
      }
    }
  }
  return best;
}

nvfp4moe_status launch_fp8_dense(const uint8_t* A, int64_t lda, const float* A_scale, int64_t lda_s, const uint8_t* B,
                                 int64_t ldb, const float* B_scale, int64_t ldb_s, int64_t M, int64_t N, int64_t K,
                                 void* D, int64_t ldd, int d_f32, cudaStream_t s) {
  const DensePlan plan = fp8_dense_plan(M, N, K);
  TileParams p{};
  p.M = int(M), p.N = int(N), p.nkb = int(fp8_blocks(K)), p.nsb = int(fp8_blocks(N));
  const int high = plan.pair ? 2 * TM : TM;
  p.n_mt = int((M + high - 1) / high), p.n_nt = int((N + plan.bn - 1) / plan.bn);
  // Short products load only the 32-row groups of A that exist: 1 x 17408 x 5120 20.8 us, 26.0 with whole boxes.
  // With several groups there is no difference (33 to 128 rows of 4096 x 4096 and 17408 x 5120, within 1 %).
  p.a_box = M <= 96 ? 32 : TM;
  p.sa = A_scale, p.lda_s = lda_s, p.sb = B_scale, p.ldb_s = ldb_s, p.sb_e = 0;
  p.D = D, p.ldd = ldd, p.d_f32 = d_f32;
  const int64_t elt = d_f32 ? 4 : 2;
  p.d_vec = reinterpret_cast<uintptr_t>(D) % 32 == 0 && ldd * elt % 32 == 0;
  p.split = plan.split;
  p.status = device_status_ptr();
  if (!p.status) return fail(NVFP4MOE_CUDA_ERROR, "device status word unavailable");
  CUtensorMap am, bm;
  nvfp4moe_status st = make_fp8_map(&am, A, K, M, 1, lda, lda, p.a_box);
  if (st == NVFP4MOE_OK) st = make_fp8_map(&bm, B, K, N, 1, ldb, ldb, b_rows(plan.bn, plan.pair));
  if (st != NVFP4MOE_OK) return st;
  const int64_t tiles = int64_t(p.n_mt) * p.n_nt;
  const int ctas = plan.pair ? 2 : plan.split;  // of one tile
  const int resident = num_sms() / ctas;
  const int grid = plan.split > 1 ? int(tiles * ctas) : int(tiles < resident ? tiles : resident) * ctas;
  cudaError_t e;
  if (plan.pair)
    e = launch_tiles<DENSE, 256, false, true>(am, bm, bm, p, grid, s);
  else if (plan.bn == 256)
    e = plan.split > 1 ? launch_tiles<DENSE, 256, true, false>(am, bm, bm, p, grid, s)
                       : launch_tiles<DENSE, 256, false, false>(am, bm, bm, p, grid, s);
  else
    e = plan.split > 1 ? launch_tiles<DENSE, 128, true, false>(am, bm, bm, p, grid, s)
                       : launch_tiles<DENSE, 128, false, false>(am, bm, bm, p, grid, s);
  if (e != cudaSuccess) return fail(NVFP4MOE_CUDA_ERROR, "fp8_gemm: %s", cudaGetErrorString(e));
  return check_launch("fp8_gemm");
}

nvfp4moe_status launch_fp8_grouped(const GroupedArgs& g, cudaStream_t s) {
  uint32_t* status = device_status_ptr();
  if (!status) return fail(NVFP4MOE_CUDA_ERROR, "device status word unavailable");
  const int nI = int(fp8_blocks(g.I)), nH = int(fp8_blocks(g.H));
  CUtensorMap xm, w13, hm, w2, dm;
  nvfp4moe_status st = make_fp8_map(&xm, g.x_codes, g.H, g.rows, 1, g.H, g.H, 32);
  if (st == NVFP4MOE_OK)
    st = make_fp8_map(&w13, g.w13_codes, g.H, g.I, 2 * int64_t(g.E), g.H, int64_t(g.I) * g.H, TM);
  if (st == NVFP4MOE_OK) st = make_fp8_map(&hm, g.h_codes, g.I, g.rows, 1, g.I, g.I, 32);
  if (st == NVFP4MOE_OK) st = make_fp8_map(&w2, g.w2_codes, g.I, g.H, g.E, g.I, int64_t(g.I) * g.H, 256);
  if (st == NVFP4MOE_OK) st = make_f32_rows_map(&dm, g.slots, g.rows, g.H);
  if (st != NVFP4MOE_OK) return st;
  TileParams p{};
  p.a_box = 32;
  p.tiles = g.tiles;
  p.status = status;
  p.split = 1;
  p.I = g.I;
  // gate/up: column tile j covers columns [128 j, +128) of gate and of up
  p.nkb = nH, p.n_nt = nI, p.nsb = nI;
  p.sa = g.x_scale, p.lda_s = nH;
  p.sb = g.w13_scale, p.ldb_s = nH, p.sb_e = int64_t(nI) * nH;
  p.h_codes = g.h_codes, p.ldh = g.I, p.h_scale = g.h_scale, p.ldh_s = nI;
  const int64_t most = int64_t(g.max_row_tiles) * nI;
  const int grid1 = int(most < num_sms() ? most : num_sms());
  cudaError_t e = launch_tiles<GATEUP, 256, false, false>(xm, w13, w13, p, grid1, s);
  // down: fp32 rows in expert order
  p.nkb = nI, p.n_nt = int((g.H + 255) / 256), p.nsb = nH, p.N = g.H;
  p.sa = g.h_scale, p.lda_s = nI;
  p.sb = g.w2_scale, p.ldb_s = nI, p.sb_e = int64_t(nH) * nI;
  p.D = g.slots, p.ldd = g.H;
  const int64_t most2 = int64_t(g.max_row_tiles) * p.n_nt;
  const int grid2 = int(most2 < num_sms() ? most2 : num_sms());
  if (e == cudaSuccess) e = launch_tiles<DOWN, 256, false, false>(hm, w2, dm, p, grid2, s);
  if (e != cudaSuccess) return fail(NVFP4MOE_CUDA_ERROR, "fp8 grouped products: %s", cudaGetErrorString(e));
  return check_launch("fp8 grouped products");
}

}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" nvfp4moe_status fp8_gemm(const uint8_t* A, int64_t lda, const float* A_scale, int64_t lda_s,
                                    const uint8_t* B, int64_t ldb, const float* B_scale, int64_t ldb_s, int64_t M,
                                    int64_t N, int64_t K, void* D, int64_t ldd, int32_t d_dtype,
                                    nvfp4moe_stream_t stream) {
  const char* fn = "fp8_gemm";
  NVFP4_REQUIRE(d_dtype == NVFP4MOE_DTYPE_BF16 || d_dtype == NVFP4MOE_DTYPE_F32, NVFP4MOE_INVALID_ARG,
                "%s: d_dtype=%d", fn, d_dtype);
  NVFP4_REQUIRE(M >= 0 && N >= 0 && K >= 0, NVFP4MOE_INVALID_ARG, "%s: negative size", fn);
  if (M == 0 || N == 0) return NVFP4MOE_OK;
  NVFP4_REQUIRE(K >= 1, NVFP4MOE_UNSUPPORTED_SHAPE, "%s: K=0", fn);
  const int64_t most = int64_t(1) << 30;
  NVFP4_REQUIRE(M <= most && N <= most && K <= most && ((M + 127) / 128) * ((N + 127) / 128) <= (int64_t(1) << 27),
                NVFP4MOE_UNSUPPORTED_SHAPE, "%s: M=%lld N=%lld K=%lld", fn, (long long)M, (long long)N, (long long)K);
  NVFP4_REQUIRE(A && A_scale && B && B_scale && D, NVFP4MOE_INVALID_ARG, "%s: NULL pointer", fn);
  const int64_t nkb = fp8_blocks(K);
  NVFP4_REQUIRE(lda >= K && ldb >= K && ldd >= N && lda_s >= nkb && ldb_s >= nkb, NVFP4MOE_INVALID_ARG,
                "%s: a row pitch below the row's length", fn);
  NVFP4_REQUIRE(lda % 16 == 0 && ldb % 16 == 0 && aligned16(A) && aligned16(B), NVFP4MOE_UNSUPPORTED_SHAPE,
                "%s: rows of A and B must start at multiples of 16 bytes", fn);
  NVFP4_REQUIRE(lda < (int64_t(1) << 40) && ldb < (int64_t(1) << 40), NVFP4MOE_UNSUPPORTED_SHAPE,
                "%s: a row pitch of 2^40 bytes or more", fn);
  const int64_t elt = d_dtype == NVFP4MOE_DTYPE_F32 ? 4 : 2;
  NVFP4_REQUIRE(reinterpret_cast<uintptr_t>(D) % elt == 0, NVFP4MOE_INVALID_ARG, "%s: D is not aligned to its type",
                fn);
  return launch_fp8_dense(A, lda, A_scale, lda_s, B, ldb, B_scale, ldb_s, M, N, K, D, ldd,
                          d_dtype == NVFP4MOE_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream));
}
