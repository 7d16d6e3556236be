// fused_gemm.cuh -- block-scaled GEMMs with an activation, a gate and a residual in the epilogue, dense or grouped by
// expert:
//
//   y[m, n] = alpha[e] * row_scale[m] * sum_k A(m,k) sA(m,k/g) B[e](n,k) sB[e](n,k/g) + bias[e, n]
//   D[m, n] = act(y[m, n]) + residual[m, n]                        (gated: act(y[m, 2n]) * y[m, 2n + 1] + ...)
//
// for the rows offsets[e] <= m < offsets[e + 1] of each expert e (dense: one expert, every row).
//
// The product is computed transposed, D^T = B A^T: the weight is the MMA's 128-row operand (256 rows over a CTA pair)
// and the tokens are its N side.  An MMA's time falls with N (measured on one B200, clocks per 128 x N x 64 fp4 or
// 128 x N x 32 fp8 step: 128 at N = 256, 64 at N = 128, 48 at N = 64, a floor of 45 below; the same per CTA of a
// pair), so an expert's tokens are covered by tiles of just as many columns as it has rows (rounded up to 16, in
// pairs 32): a ragged expert costs what its rows cost, not what a whole 128- or 256-row tile would, and a decoding
// batch streams its weights past a narrow N.
//
// The rows of A are the experts' tokens one after another without padding.  An expert's first row is then anywhere
// inside a 128-row band of scale tiles: a tile's scale columns are shifted into place by the warps that copy them
// from shared to tensor memory (one select per word), so the activation is quantized as for any other GEMM.
//
// Roles, pipeline and bounded waits follow gemm.cu: warp 0 loads codes and warp 3 scales (TMA), warp 1 issues the MMAs,
// warp 2 of a pair's follower relays its arrivals to the leader, warps 4-7 copy scale factors into tensor memory, warps
// 8-15 are the epilogue.  Every CTA builds the table of the experts' tiles in shared memory from the offsets (a scan
// over the experts) and takes every gridDim-th tile: nothing is read back to the host.
//
// What bounds it, measured on one B200 (launches back to back on the same operands; a pass whose operands come from DRAM
// after others in brackets):
//  - large products: operand delivery and power.  A 256 x 256 tile of a pair takes 38 KB per SM and K step; the ring
//    runs at 548 clocks a step without MMAs (70 bytes a clock and SM from L2), 615 with them (an ideal of 514), at the
//    1.35 to 1.4 GHz that the 1000 W cap leaves: 32760 x 13824 x 5120 868 us in short bursts without a bias, 1033 over a
//    second with bias and relu [1077 with gelu_tanh].
//  - experts of a few hundred rows: per tile, the hand-over of the one 256-column accumulator (last MMA to first MMA of
//    the next tile, about 3000 clocks) beside 8 K steps of 520 to 600 clocks: 128 experts, 32768 rows, 1536 x 2048 gated
//    81 to 86 us [97].  Two 128-column accumulators instead (no hand-over, twice the weight traffic): 112 us.
//  - short K: the epilogue, about 900 clocks per warp for 32 tokens x 32 columns (200 of arithmetic, then one after
//    another the buffer's wait, the turn through shared memory, the fence and the store), plus 8 to 12 clocks of the
//    special-function unit for each activated value: 128 experts, 32768 x 2048 x 768 59 to 64 us, without it 43 [72];
//    32760 x 1536 x 1536 44 us with relu, 65 with gelu_tanh, 59 to 63 with silu, 80 with gelu, 74 with a residual.
//  - decoding batches: the weight stream; 512 rows over 117 of 128 experts of 1536 x 2048, 208 MB in 34 to 39 us [40].
//  - registers: with a residual, in fp32, or both, the epilogue spills where it has the accumulator in registers (-Xptxas
//    -v, bytes stored / loaded a thread: pairs 116 / 248 with a bf16 residual, 44 / 168 in fp32, 40 / 164 in fp32 with a
//    residual; single CTAs 20 / 72 at most).
// Not kept: an L2 prefetch of the next tile's weights (3 to 12% slower); the follower's warps arriving on the leader's
// barriers themselves (2 to 10% slower); experts dealt out in the order of their tiles' widths (1 to 2% slower); two
// boxes of D per fence and store, or a second staging buffer (the 16 KB cost a stage of the ring: 0 to 11% slower).
#pragma once

#include "activation.cuh"
#include "bsp_device.cuh"
#include "bsp_internal.h"
#include "tensor_maps.h"

namespace bsp {
namespace {

constexpr int kMaxExperts = BSP_MAX_EXPERTS;  // the tile table's two words per expert in shared memory
constexpr int kListed = 64;         // tiles of a CTA that it looks up before the roles start
constexpr int kMaxSplit = 4;        // CTAs of a cluster that share a tile's K range
constexpr int kMinSplitSteps = 16;  // K steps that each keeps at least

struct FusedParams {
  int M, N, E;
  int num_kb;     // 128-byte steps of K
  int panels;     // weight panels per expert
  int group_m;    // token tiles per rasterisation group
  int tn;         // most tokens per tile
  int stages, stage_bytes, x_bytes;  // CG = 1: the ring's layout, by tn
  int split;      // CG = 1: CTAs of a cluster sharing one tile's K range
  int act, gated;
  const int32_t* offsets;  // [E + 1], or NULL: one expert with every row
  const float* alpha;
  const float* row_scale;
  const uint16_t* bias;
  const void* residual;
  int64_t ld_res;
  void* D;
  int64_t ld_d;
  uint32_t* err;
};

// CG = 2: CTA pairs, 256 weight rows x up to 256 tokens.  CG = 1: 128 weight rows x up to 128 tokens, in a ring of as
// many stages as fit for the launch's token tile.
template <int KIND, int CG_>
struct FCfg {
  static constexpr int CG = CG_;
  static constexpr int TN = CG == 2 ? 256 : 128;         // most tokens per tile
  static constexpr int N_STEP = CG == 2 ? 32 : 16;       // granularity of the MMA's N
  static constexpr int X_ROWS = TN / CG;                 // token rows each CTA holds
  static constexpr int X_MAPS = X_ROWS / 32;             // sizes of the TMA box of tokens
  static constexpr int ATOMS = KIND == kNVF4 ? 4 : 1;    // 128x4 scale tiles per 128 rows per stage
  static constexpr int X_BANDS = CG == 2 ? 3 : 2;        // bands of scale tiles that TN rows at any offset touch
  static constexpr int X_WORDS = CG == 2 ? 8 : 4;        // scale columns per K-group tile
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int X_BYTES = X_ROWS * 128;
  static constexpr int BAND_BYTES = ATOMS * 512;
  static constexpr int STAGE_BYTES = (W_BYTES + X_BYTES + BAND_BYTES * (1 + X_BANDS) + 1023) / 1024 * 1024;
  static constexpr int SFW_COLS = ATOMS * 4;
  static constexpr int SFX_COLS = ATOMS * X_WORDS;
  static constexpr int SF_COLS = SFW_COLS + SFX_COLS;
  static constexpr int ACC_BUFS = CG == 2 ? 1 : 2;       // two 256-column accumulators leave no room for the scales
  static constexpr int ACC_COLS = TN * ACC_BUFS;
  static constexpr int TMEM_COLS = 512;
  static constexpr int SF_WARPS = 4;
  static constexpr int EPI_WARPS = 8;
  static constexpr int FIRST_SF_WARP = 4, FIRST_EPI_WARP = 8;
  static constexpr int THREADS = (8 + EPI_WARPS) * 32;
  static constexpr int STEPS = TN / 2 / 16;  // steps of 16 tokens per epilogue warp
  // Warpgroups 0 and 1 hand registers to the epilogue, which holds up to 128 accumulator columns a thread.  (With 40
  // for the first, as in gemm.cu, its loops spill: 7% of a large GEMM.)
  static constexpr int WG0_REGS = 72, SF_REGS = 88, EPI_REGS = 176;
  static_assert(128 * (WG0_REGS + SF_REGS + 2 * EPI_REGS) == THREADS * (65536 / THREADS), "register split");
  static constexpr int STG_BYTES = 2048;  // staging: per warp, a box of D for one TMA store
  static constexpr int SCALE_BYTES = 16 * STEPS * 4;  // and its tokens' scales
  static constexpr int TABLE_BYTES = (2 * (kMaxExperts + 1) * 4 + 15) / 16 * 16;
  static constexpr int LIST_BYTES = kListed * 16;
  static constexpr int BAR_BYTES = 512;
  static constexpr int FIXED_BYTES = EPI_WARPS * (STG_BYTES + SCALE_BYTES) + TABLE_BYTES + LIST_BYTES + BAR_BYTES + 1024;
  static constexpr int by_smem = (232448 - FIXED_BYTES) / STAGE_BYTES;
  static constexpr int by_tmem = (TMEM_COLS - ACC_COLS) / SF_COLS;
  static constexpr int MAX_STAGES = by_tmem < 8 ? by_tmem : 8;
  static constexpr int STAGES = by_smem < MAX_STAGES ? by_smem : MAX_STAGES;  // of the largest tile
  static constexpr int RING_BYTES = CG == 2 ? STAGES * STAGE_BYTES : (232448 - FIXED_BYTES) / 1024 * 1024;
  static constexpr int SMEM_BYTES = RING_BYTES + FIXED_BYTES;
  static_assert(STAGES >= 4 && SMEM_BYTES <= 232448 && ACC_COLS + MAX_STAGES * SF_COLS <= TMEM_COLS, "budget");
  static_assert((4 * MAX_STAGES + 8) * 8 <= BAR_BYTES, "barrier space");
  // split K: a CTA's partial tile, one word per epilogue thread and accumulator register, in its drained ring
  static_assert(CG == 2 || 16 * STEPS * EPI_WARPS * 32 * 4 <= RING_BYTES, "partial tile");
};

// TMA descriptors.  Tokens and their scales come in one box each per stage, of the smallest size that covers the
// tile: x[i] has 32 (i + 1) rows, sfx[i] has i + 1 bands.  (A loop over small boxes in the producer thread took 0.2 us
// per stage: 14.2 instead of 10.4 us at M = 16, N = 13824, K = 5120.)
struct FusedMaps {
  CUtensorMap w, sfw, x[4], sfx[3], d;
};

// Gated weights: accumulator row 16 b + j holds the gate of output column 8 b + j, row 16 b + 8 + j its up projection
// (j < 8), so that a thread of the epilogue has both.  The TMA load reorders the rows (a box of 8 rows two apart, both
// kinds, 8 blocks); this is the weight's row in accumulator row r.
__device__ __forceinline__ int gated_row(int r) { return (r & ~15) + 2 * (r & 7) + ((r >> 3) & 1); }

struct Tile {
  int e;      // expert
  int nb;     // weight panel
  int row0;   // first row of A
  int cnt;    // rows
  int nmma;   // rows rounded up to the MMA's granularity
};

// The experts' tiles: start[e] is the index of expert e's first tile, its rows are lo[e] <= m < lo[e + 1].
struct Table {
  int* start;
  int* lo;

  __device__ __forceinline__ void carve(void* mem) {
    start = static_cast<int*>(mem);
    lo = start + kMaxExperts + 1;
  }

  // Offsets are clamped to [0, M], and one below an earlier one counts as that one, so that the experts' rows never
  // overlap whatever the array holds.  Called by the whole CTA.
  __device__ __forceinline__ void build(const FusedParams& p) {
    const int TN = p.tn;
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) lo[e] = min(max(__ldg(p.offsets + e), 0), p.M);
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int top = lo[0];  // the rows before this expert
      int tiles = 0;
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        int h = e < p.E ? lo[e + 1] : 0;
        h = max(h, top);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, h, d);
          if (lane >= d) h = max(h, o);
        }
        int l = __shfl_up_sync(0xFFFFFFFFu, h, 1);
        if (lane == 0) l = top;
        int n = (h - l + TN - 1) / TN * p.panels;
        const int own = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, n, d);
          if (lane >= d) n += o;
        }
        if (e < p.E) {
          lo[e + 1] = h;
          start[e] = tiles + n - own;
        }
        top = __shfl_sync(0xFFFFFFFFu, h, 31);
        tiles += __shfl_sync(0xFFFFFFFFu, n, 31);
      }
      if (lane == 0) start[p.E] = tiles;
    }
    __syncthreads();
  }

  // Tile r of the expert e that has rows l .. l + rows - 1: token tiles within groups of group_m, fastest first, so
  // that the CTAs that run at once share weight panels and tokens in L2.  The rows are shared out evenly over the tiles.
  template <int N_STEP>
  static __device__ __forceinline__ Tile locate(int e, int l, int rows, int r, const FusedParams& p) {
    const int TN = p.tn;
    const int nt = rows <= TN ? 1 : (rows + TN - 1) / TN;
    int first = 0, size = nt, per = (rows + N_STEP - 1) / N_STEP * N_STEP;
    if (nt > 1) {  // (divisions are slow)
      per = ((rows + nt - 1) / nt + N_STEP - 1) / N_STEP * N_STEP;
      if (nt > p.group_m) {
        const int per_group = p.group_m * p.panels;
        const int g = r / per_group;
        first = g * p.group_m;
        size = min(p.group_m, nt - first);
        r -= g * per_group;
      }
    }
    const int nb = size > 1 ? r / size : r;
    Tile q;
    q.e = e;
    q.nb = nb;
    q.row0 = l + (first + r - nb * size) * per;
    q.cnt = min(per, l + rows - q.row0);
    q.nmma = (q.cnt + N_STEP - 1) / N_STEP * N_STEP;
    return q;
  }

  // Tile t: its expert by bisection.
  template <int N_STEP>
  __device__ __forceinline__ Tile get(int t, const FusedParams& p) const {
    if (p.offsets == nullptr) return locate<N_STEP>(0, 0, p.M, t, p);
    int a = 0, b = p.E;
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (start[mid] <= t) a = mid;
      else b = mid;
    }
    return locate<N_STEP>(a, lo[a], lo[a + 1] - lo[a], t - start[a], p);
  }
};

__device__ __forceinline__ void lds16(uint32_t* r, const uint8_t* p) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  r[0] = v.x;
  r[1] = v.y;
  r[2] = v.z;
  r[3] = v.w;
}

template <int ACT, bool GATED>
struct EpilogueVariant {
  static constexpr int kAct = ACT;
  static constexpr bool kGated = GATED;
};

template <int SHIFT, bool WIDE>
struct ScaleVariant {
  static constexpr int kShift = SHIFT;
  static constexpr bool kWide = WIDE;
};

// One lane's share of a stage's scale columns: the weight's tiles as they are, the tokens' shifted by SHIFT words (-1:
// the tile starts a band) plus one in the lanes with `carry`.  kWide: more than 128 tokens, two bands' words.
template <int KIND, int CG, int SHIFT, bool kWide>
__device__ __forceinline__ void copy_scales(uint32_t taddr, const uint8_t* sf, int w_line, int line, bool carry) {
  using C = FCfg<KIND, CG>;
  constexpr int kWords = kWide ? 8 : 4;
  constexpr int kBands = SHIFT < 0 ? (kWide ? 2 : 1) : (kWide ? 3 : 2);
  constexpr int kStep = C::ATOMS > 1 ? 2 : 1;  // K-group tiles whose loads are in flight at once
  uint32_t w[C::SFW_COLS];
#pragma unroll
  for (int a = 0; a < C::ATOMS; ++a) lds16(w + 4 * a, sf + 512 * a + w_line * 16);
  const uint8_t* sfx = sf + C::BAND_BYTES + line * 16;
#pragma unroll
  for (int a0 = 0; a0 < C::ATOMS; a0 += kStep) {
    uint32_t b[kStep][4 * kBands], x[kStep][kWords];
#pragma unroll
    for (int a = 0; a < kStep; ++a)
#pragma unroll
      for (int i = 0; i < kBands; ++i) lds16(b[a] + 4 * i, sfx + C::BAND_BYTES * i + 512 * (a0 + a));
    if (a0 == 0) {
      if constexpr (C::SFW_COLS == 16)
        tmem_st_16cols(taddr, w);
      else
        tmem_st_4cols(taddr, w);
    }
#pragma unroll
    for (int a = 0; a < kStep; ++a) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        if constexpr (SHIFT < 0) x[a][j] = b[a][j];
        else x[a][j] = carry ? b[a][SHIFT + j + 1] : b[a][SHIFT + j];
      }
    }
    const uint32_t tx = taddr + C::SFW_COLS + C::X_WORDS * a0;
    if constexpr (kStep * kWords == 16) {
      tmem_st_16cols(tx, x[0]);
    } else if constexpr (C::X_WORDS == kWords && kStep * kWords == 8) {
      tmem_st_8cols(tx, x[0]);
    } else {
#pragma unroll
      for (int a = 0; a < kStep; ++a) tmem_st_4cols(tx + C::X_WORDS * a, x[a]);
    }
  }
}

// kF32: D in fp32, else bf16.  kRes: with a residual.  (Template parameters: with the accumulator in registers, the
// epilogue has none to spare for what both sides of a branch would share.)
template <int KIND, int CG, bool kF32, bool kRes>
__global__ void __launch_bounds__(FCfg<KIND, CG>::THREADS, 1)
    fused_gemm_kernel(const __grid_constant__ FusedMaps maps, const FusedParams p) {
  using C = FCfg<KIND, CG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + C::RING_BYTES;
  uint8_t* table_mem = staging + C::EPI_WARPS * (C::STG_BYTES + C::SCALE_BYTES);
  int4* list = reinterpret_cast<int4*>(table_mem + C::TABLE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(table_mem + C::TABLE_BYTES + C::LIST_BYTES);
  uint64_t* empty = full + C::MAX_STAGES;
  uint64_t* sf_ready = empty + C::MAX_STAGES;
  uint64_t* sf_local = sf_ready + C::MAX_STAGES;  // pair follower: its scale warps, per stage
  uint64_t* acc_full = sf_local + C::MAX_STAGES;  // [ACC_BUFS]
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* acc_local = acc_empty + 2;  // pair follower: its epilogue warps
  uint64_t* drain = acc_local + 1;
  uint64_t* part_ready = drain + 1;  // split K: the partial tiles of every CTA of the cluster
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(part_ready + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  Table table;
  table.carve(table_mem);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  const uint32_t rank = C::CG == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0u;
  constexpr uint32_t kPeerArrivals = C::CG == 2 ? 1u : 0u;  // the follower's relayed arrival
  const int n_stages = C::CG == 2 ? C::STAGES : p.stages;
  const int stage_bytes = C::CG == 2 ? C::STAGE_BYTES : p.stage_bytes;
  const int x_bytes = C::CG == 2 ? C::X_BYTES : p.x_bytes;
  // split K: CTA k_rank of a cluster of k_split takes K steps kb0 .. kb1 of the cluster's one tile
  const int k_split = C::CG == 2 ? 1 : p.split;
  const int k_rank = k_split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int kb0 = k_split > 1 ? p.num_kb * k_rank / k_split : 0;
  const int kb1 = k_split > 1 ? p.num_kb * (k_rank + 1) / k_split : p.num_kb;

  if (warp == 0) {  // one lane a stage
    if (static_cast<int>(lane) < n_stages) {
      mbar_init(&full[lane], 1);
      mbar_init(&empty[lane], 1);
      mbar_init(&sf_ready[lane], C::SF_WARPS + kPeerArrivals);
      mbar_init(&sf_local[lane], C::SF_WARPS);
    } else if (lane >= 16u && lane < 18u) {
      mbar_init(&acc_full[lane - 16u], 1);
      mbar_init(&acc_empty[lane - 16u], C::EPI_WARPS + kPeerArrivals);
    } else if (lane == 18u) {
      mbar_init(acc_local, C::EPI_WARPS);
      mbar_init(drain, 1);
      mbar_init(part_ready, static_cast<uint32_t>(k_split * C::EPI_WARPS));
      *abort_flag = 0u;
    }
    fence_barrier_init();
  } else if (warp == 2) {
    const int i = static_cast<int>(lane);
    if (i == 0) prefetch_tensormap(&maps.w);
    else if (i == 1) prefetch_tensormap(&maps.sfw);
    else if (i == 2) prefetch_tensormap(&maps.d);
    else if (i >= 4 && i - 4 < p.tn / (32 * C::CG)) prefetch_tensormap(&maps.x[i - 4]);
    else if (i >= 8 && i - 8 < C::X_BANDS) prefetch_tensormap(&maps.sfx[i - 8]);
  }
  if (warp == 1) {
    if constexpr (C::CG == 2) {
      tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  __syncwarp();
  const int first_tile = static_cast<int>(blockIdx.x) / (C::CG * k_split);
  const int tile_step = static_cast<int>(gridDim.x) / (C::CG * k_split);
  // This CTA's first tiles are looked up once, side by side: a lookup takes 500 to 1000 clocks (a bisection and
  // divisions, between instructions that have to be fetched again), and one in front of every tile of every role cost
  // 2400 a tile in the epilogue (128 experts, 32768 x 2048 x 768: 72 us against 60).
  auto list_tiles = [&](int tiles) {
    const int i = static_cast<int>(threadIdx.x) - C::THREADS + kListed;  // the last warps: the first ones set up
    const int64_t t = first_tile + static_cast<int64_t>(i) * tile_step;
    if (i >= 0 && t < tiles) {
      const Tile q = table.get<C::N_STEP>(static_cast<int>(t), p);
      list[i] = make_int4(q.e, q.nb, q.row0, q.cnt);
    }
  };
  int num_tiles = 0;
  if (p.offsets == nullptr) {
    num_tiles = (p.M + p.tn - 1) / p.tn * p.panels;
    list_tiles(num_tiles);
  }
  tc_fence_before_sync();
  __syncwarp();
  if (C::CG == 2 || k_split > 1)
    cluster_sync();  // the peers' barriers are initialised before anything arrives on them
  else
    __syncthreads();
  // Set-up above overlaps the previous kernel under programmatic launch; every global access below comes after its
  // completion.
  grid_dependency_wait();
  // Every CTA is resident by now, so a dependent GEMM may take the SMs that finish early and set itself up; it waits for
  // this grid's completion as this one just did (1 us a launch back to back: N = 1536, K = 1536, M = 1, 6.0 -> 5.0 us).
  allow_dependent_launch();
  if (p.offsets != nullptr) {
    table.build(p);
    num_tiles = table.start[p.E];
    list_tiles(num_tiles);
    __syncthreads();
  }
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  auto tile_at = [&](int t, int it) {
    if (it >= kListed) return table.get<C::N_STEP>(t, p);
    const int4 v = list[it];
    return Tile{v.x, v.y, v.z, v.w, (v.w + C::N_STEP - 1) / C::N_STEP * C::N_STEP};
  };

  if (warp < C::FIRST_SF_WARP) {
    regs_dec<C::WG0_REGS>();
    if (warp == 0 || warp == 3) {
      // ------------------------------------------------------------ producers
      // Warp 0 loads the weights' and tokens' codes, warp 3 their scales: a thread takes about 40 clocks to issue a
      // TMA load, and a stage of a narrow tile has MMAs for 180 only.  Both wait for the same empty slot; warp 0's
      // arrival expects the bytes of all four loads.
      if (elect_one()) {
        int stage = 0;
        uint32_t phase = 0;
        uint32_t total = 0;  // stages issued
        bool ok = true;
        for (int t = first_tile, it = 0; t < num_tiles && ok; t += tile_step, ++it) {
          const Tile q = tile_at(t, it);
          const int band = q.nb * C::CG + static_cast<int>(rank);  // of 128 weight rows
          const int x_rows = q.nmma / C::CG;
          const int x_row = q.row0 + static_cast<int>(rank) * x_rows;
          const int x_box = (x_rows + 31) >> 5;
          const int x_bands = ((q.row0 & 127) + q.nmma + 127) >> 7;
          const CUtensorMap* mx = &maps.x[x_box - 1];
          const CUtensorMap* msfx = &maps.sfx[x_bands - 1];
          const uint32_t tx = static_cast<uint32_t>(C::W_BYTES + x_box * 4096 + C::BAND_BYTES * (1 + x_bands));
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            uint8_t* st = smem + stage * stage_bytes;
            if (warp == 0) {
              mbar_arrive_expect_tx(&full[stage], tx);
              if (p.gated)
                tma_load_5d(st, &maps.w, &full[stage], kb * 128, 0, 0, band * 8, q.e);
              else
                tma_load_3d(st, &maps.w, &full[stage], kb * 128, band * 128, q.e);
              tma_load_2d(st + C::W_BYTES, mx, &full[stage], kb * 128, x_row);
            } else {
              uint8_t* sf = st + C::W_BYTES + x_bytes;
              tma_load_4d(sf, &maps.sfw, &full[stage], 0, kb * C::ATOMS, band, q.e);
              tma_load_3d(sf + C::BAND_BYTES, msfx, &full[stage], 0, kb * C::ATOMS, q.row0 >> 7);
            }
            ++total;
            if (++stage == n_stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok) {
          *abort_flag = 1u;
          raise_error(p.err, kErrTimeout);
        }
        // Every issued copy must have landed before the CTA may exit.
        for (uint32_t s = 0; s < n_stages; ++s)
          if (total > s && !mbar_wait(&full[s], ((total - 1u - s) / n_stages) & 1u, nullptr))
            raise_error(p.err, kErrTimeout);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (leader && elect_one()) {
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        int it = 0;
        auto commit = [&](uint64_t* bar) {
          if constexpr (C::CG == 2)
            tc_commit_pair(bar, 0x3);
          else
            tc_commit(bar);
        };
        auto wait_shared = [&](uint64_t* bar, uint32_t par) {
          if constexpr (C::CG == 2)
            return mbar_wait_cluster(bar, par, abort_flag);
          else
            return mbar_wait(bar, par, abort_flag);
        };
        for (int t = first_tile; t < num_tiles && ok; t += tile_step, ++it) {
          const Tile q = tile_at(t, it);
          const int buf = it % C::ACC_BUFS;
          const uint32_t acc = tmem + static_cast<uint32_t>(buf * C::TN);
          if (!wait_shared(&acc_empty[buf], (static_cast<uint32_t>(it / C::ACC_BUFS) & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_shared(&sf_ready[stage], phase)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t sbase = smem_u32(smem + stage * stage_bytes);
            const uint32_t sfw_t = tmem + C::ACC_COLS + stage * C::SF_COLS;
            const uint32_t sfx_t = sfw_t + C::SFW_COLS;
            const uint64_t wdesc = desc_kmajor_sw128(sbase);
            const uint64_t xdesc = desc_kmajor_sw128(sbase + C::W_BYTES);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t accumulate = (kb > kb0 || kk > 0) ? 1u : 0u;
              if constexpr (KIND == kNVF4) {
                const uint32_t idesc = idesc_nvf4(128 * C::CG, q.nmma);
                const uint32_t sfx_k = sfx_t + static_cast<uint32_t>(C::X_WORDS * kk);
                if constexpr (C::CG == 2)
                  tc_mma_nvf4_pair(acc, wdesc + 2u * kk, xdesc + 2u * kk, idesc, sfw_t + 4u * kk, sfx_k, accumulate);
                else
                  tc_mma_nvf4(acc, wdesc + 2u * kk, xdesc + 2u * kk, idesc, sfw_t + 4u * kk, sfx_k, accumulate);
              } else {
                const uint32_t idesc = idesc_mxf8(128 * C::CG, q.nmma, static_cast<uint32_t>(kk));
                if constexpr (C::CG == 2)
                  tc_mma_mxf8_pair(acc, wdesc + 2u * kk, xdesc + 2u * kk, idesc, sfw_t, sfx_t, accumulate);
                else
                  tc_mma_mxf8(acc, wdesc + 2u * kk, xdesc + 2u * kk, idesc, sfw_t, sfx_t, accumulate);
              }
            }
            commit(&empty[stage]);
            if (++stage == n_stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          commit(&acc_full[buf]);
        }
        if (!ok) {
          *abort_flag = 1u;
          raise_error(p.err, kErrTimeout);
        }
        // No MMA may still be running when tensor memory is freed.
        commit(drain);
        if (!mbar_wait(drain, 0u, nullptr)) raise_error(p.err, kErrTimeout);
      } else if (!leader && lane == 0) {
        // pair follower: its MMAs are issued by the leader, whose last commit arrives here too
        if (!mbar_wait(drain, 0u, nullptr)) raise_error(p.err, kErrTimeout);
      }
    } else if (C::CG == 2 && !leader && lane == 0) {
      // pair follower, warp 2: relays to the leader each stage's scales and each released accumulator, whichever
      // comes (the scales run up to a ring ahead of the accumulators)
      const uint32_t peer_sf = mapa_shared(smem_u32(sf_ready), 0u), peer_acc = mapa_shared(smem_u32(acc_empty), 0u);
      int acc_left = first_tile < num_tiles ? (num_tiles - first_tile + tile_step - 1) / tile_step : 0;
      int64_t sf_left = static_cast<int64_t>(acc_left) * p.num_kb;
      int stage = 0;
      uint32_t sf_phase = 0, acc_phase = 0, idle = 0;
      uint64_t t0 = 0;
      while (sf_left > 0 || acc_left > 0) {
        bool got = false;
        if (sf_left > 0 && mbar_test_wait(smem_u32(&sf_local[stage]), sf_phase)) {
          mbar_arrive_remote_relaxed(peer_sf + 8u * stage);
          --sf_left;
          if (++stage == n_stages) {
            stage = 0;
            sf_phase ^= 1u;
          }
          got = true;
        }
        if (acc_left > 0 && mbar_test_wait(smem_u32(acc_local), acc_phase)) {
          mbar_arrive_remote_relaxed(peer_acc);
          --acc_left;
          acc_phase ^= 1u;
          got = true;
        }
        if (got) {
          idle = 0;
        } else if ((++idle & 63u) == 0u) {
          const uint64_t now = globaltimer_ns();
          if (idle == 64u) t0 = now;
          if (*abort_flag || now - t0 > kWaitLimitNs) {
            *abort_flag = 1u;
            raise_error(p.err, kErrTimeout);
            break;
          }
        }
      }
    }
  } else if (warp < C::FIRST_EPI_WARP) {
    // ------------------------------------------------------------ scale factors
    regs_dec<C::SF_REGS>();
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    uint64_t* sf_mine = leader ? sf_ready : sf_local;
    // gated: the accumulator's rows are the weight's in the order of the epilogue (gated_row)
    const int w_line = p.gated ? gated_row(static_cast<int>(lane)) : static_cast<int>(lane);
    for (int t = first_tile, it = 0; t < num_tiles && ok; t += tile_step, ++it) {
      const Tile q = tile_at(t, it);
      // Scale row i of the tile is row (row0 & 127) + i of the loaded bands.  Line `lane` of tensor memory takes the
      // words of rows lane + 32 j, which all sit in line (row0 + lane) & 31 of the tiles, at word `shift` + j (plus
      // one in the lanes where row0 + lane carries into the next 32 rows) of the bands' words one after another.
      const bool carry = (q.row0 & 31) + static_cast<int>(lane) >= 32;
      const int line = (q.row0 + static_cast<int>(lane)) & 31;
      // one loop over K for each variant: a choice inside it costs 3% of a large GEMM
      auto stages = [&](auto variant) {
        constexpr int kShift = decltype(variant)::kShift;
        constexpr bool kWide = decltype(variant)::kWide;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          copy_scales<KIND, CG, kShift, kWide>(tmem + lane_base + C::ACC_COLS + stage * C::SF_COLS,
                                               smem + stage * stage_bytes + C::W_BYTES + x_bytes, w_line, line,
                                               carry);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sf_mine[stage]);
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      };
      const int shift = (q.row0 & 127) == 0 ? -1 : (q.row0 & 127) >> 5;
      if (CG == 2 && q.nmma > 128) {
        if constexpr (CG == 2) {
          if (shift < 0) stages(ScaleVariant<-1, true>{});
          else if (shift == 0) stages(ScaleVariant<0, true>{});
          else if (shift == 1) stages(ScaleVariant<1, true>{});
          else if (shift == 2) stages(ScaleVariant<2, true>{});
          else stages(ScaleVariant<3, true>{});
        }
      } else {
        if (shift < 0) stages(ScaleVariant<-1, false>{});
        else if (shift == 0) stages(ScaleVariant<0, false>{});
        else if (shift == 1) stages(ScaleVariant<1, false>{});
        else if (shift == 2) stages(ScaleVariant<2, false>{});
        else stages(ScaleVariant<3, false>{});
      }
    }
    if (!ok) {
      *abort_flag = 1u;
      raise_error(p.err, kErrTimeout);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // A lane of tensor memory is a weight row, a column a token.  A warp reads its 32 rows x up to 16 STEPS tokens
    // into registers as 8 x 8 fragments (thread t: row t / 4, tokens 2 (t % 4) and the next), hands the accumulator
    // back, finishes the values in fp32, rounds them once and turns them over on the way to shared memory (stmatrix
    // with a transpose), 32 tokens x 32 columns of D at a time, from where they go out as one TMA store.  (16-byte
    // stores from the lanes took 25% longer over the whole GEMM; turning fp32 values over through shared memory and
    // storing 8 tokens at a time took twice as long as the MMAs at K = 1536.)  The box that holds an expert's last
    // rows is stored by the lanes, row by row: the rows after them belong to another expert.
    regs_inc<C::EPI_REGS>();
    const int ew = warp - C::FIRST_EPI_WARP;
    const int quarter = warp & 3;
    const int half = ew >> 2;
    const int fr = static_cast<int>(lane) >> 2, fc = 2 * (static_cast<int>(lane) & 3);  // fragment row, first token
    uint64_t* acc_mine = leader ? acc_empty : acc_local;
    const uint64_t evict_first = l2_policy_evict_first();
    float* scales = reinterpret_cast<float*>(staging + C::EPI_WARPS * C::STG_BYTES) + ew * 16 * C::STEPS;
    int it = 0;
    for (int t = first_tile; t < num_tiles; t += tile_step, ++it) {
      const Tile q = tile_at(t, it);
      const int buf = it % C::ACC_BUFS;
      const int width = (q.nmma / 2 + 31) & ~31;           // tokens per epilogue warp, whole boxes of D
      const int tok0 = half * width;                       // this warp's first token of the tile
      const int col0 = (q.nb * C::CG + static_cast<int>(rank)) * 128 + quarter * 32;  // first weight row
      const float alpha = p.alpha != nullptr ? __ldg(p.alpha + q.e) : 1.0f;
      float bias[4];  // of fragment rows fr + 8 i
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = col0 + (p.gated ? gated_row(fr + 8 * i) : fr + 8 * i);
        bias[i] = p.bias != nullptr && n < p.N ? bf16_bits_to_f32(__ldg(p.bias + static_cast<int64_t>(q.e) * p.N + n))
                                               : 0.0f;
      }
      // alpha x row scale of this warp's tokens
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16 * C::STEPS; j += 32) {
        const int tk = tok0 + j + static_cast<int>(lane);
        scales[j + lane] =
            (p.row_scale != nullptr && tk < q.cnt) ? __fmul_rn(alpha, __ldg(p.row_scale + q.row0 + tk)) : alpha;
      }
      __syncwarp();
      // A residual: this warp's rows on their way into L2 while the MMAs run, and the first box of them into registers
      // (16-byte chunks, as the boxes of D below are laid out); the next box is loaded while one is finished (in fp32 there
      // are no registers for that: a box is loaded when its sums are in shared memory).
      constexpr int kResRows = kF32 ? 16 : 32;
      uint4 res[4];
      const int res_row_chunks = (kF32 ? 8 : 4) >> p.gated;
      auto load_residual = [&](int tb) {
        const int row = static_cast<int>(lane) / res_row_chunks, step = 32 / res_row_chunks;
        const int col = (p.gated ? col0 >> 1 : col0) + static_cast<int>(lane) % res_row_chunks * (kF32 ? 4 : 8);
        const bool ok = col < (p.gated ? p.N >> 1 : p.N);
        const uint8_t* src = static_cast<const uint8_t*>(p.residual) +
                             ((q.row0 + tb + row) * p.ld_res + col) * (kF32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          res[i] = make_uint4(0u, 0u, 0u, 0u);
          if (ok && (i < 2 || !p.gated) && tb + row + i * step < q.cnt)
            res[i] = *reinterpret_cast<const uint4*>(src + i * step * (kF32 ? 4 : 2) * p.ld_res);
        }
      };
      if constexpr (kRes) {
        const int c0 = p.gated ? col0 >> 1 : col0;
        if (c0 < (p.gated ? p.N >> 1 : p.N)) {
#pragma unroll
          for (int j = kF32 ? 0 : kResRows; j < 16 * C::STEPS; j += 32) {
            const int tk = tok0 + j + static_cast<int>(lane);
            if (tk < q.cnt && j + static_cast<int>(lane) < width)
              prefetch_l2(static_cast<const uint8_t*>(p.residual) + ((q.row0 + tk) * p.ld_res + c0) * (kF32 ? 4 : 2));
          }
        }
        if constexpr (!kF32) load_residual(tok0);
      }
      const uint32_t par = static_cast<uint32_t>(it / C::ACC_BUFS) & 1u;
      const bool got = C::CG == 2 ? mbar_wait_cluster(&acc_full[buf], par, abort_flag)
                                  : mbar_wait(&acc_full[buf], par, abort_flag);
      if (!got) {
        *abort_flag = 1u;
        raise_error(p.err, kErrTimeout);
        break;
      }
      tc_fence_after_sync();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(buf * C::TN + tok0);
      // columns past `width` are read too, within the accumulator, and not used
      uint32_t r[2][C::STEPS / 4][32];  // [row half][64 tokens][4 x octet + 2 x row block + token]
#pragma unroll
      for (int c = 0; c < C::STEPS / 4; ++c) {
        tmem_ld_frag_64cols(taddr + 64u * c, r[0][c]);
        tmem_ld_frag_64cols(taddr + (16u << 16) + 64u * c, r[1][c]);
      }
      tmem_ld_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(C::CG == 2 ? acc_mine : &acc_empty[buf]);

      // the steps of this warp, one bit each
      const int lim = min(width, q.cnt - tok0);
      uint32_t steps = lim > 0 ? (1u << ((lim + 15) >> 4)) - 1u : 0u;
      if (C::CG == 1 && k_split > 1) {
        // Split K: every CTA leaves its partial tile in its own ring (all of its loads have been consumed: the cluster
        // has one tile), register by register, and finishes the steps that fall to it with the sum over the cluster in
        // rank order, whichever CTA came first.
        float* part = reinterpret_cast<float*>(smem) + ew * 32 + lane;
#pragma unroll
        for (int s = 0; s < C::STEPS; ++s) {
          if (steps >> s & 1u) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              part[(16 * s + i) * C::EPI_WARPS * 32] = __uint_as_float(r[i >> 3][s / 4][8 * (s & 3) + (i & 7)]);
          }
        }
        __syncwarp();
        if (static_cast<int>(lane) < k_split) mbar_arrive_remote(mapa_shared(smem_u32(part_ready), lane));
        if (!mbar_wait_cluster(part_ready, 0u, abort_flag)) {
          *abort_flag = 1u;
          raise_error(p.err, kErrTimeout);
          break;
        }
        uint32_t mine = 0;
#pragma unroll
        for (int s = 0; s < C::STEPS; ++s) {
          if ((steps >> s & 1u) && ((s >> 1) * 2 + half) % k_split == k_rank) {
            mine |= 1u << s;
            float sum[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[i] = 0.0f;
            for (int c = 0; c < k_split; ++c) {
              const uint32_t peer = mapa_shared(smem_u32(part), static_cast<uint32_t>(c));
#pragma unroll
              for (int i = 0; i < 16; ++i)
                sum[i] = __fadd_rn(sum[i], ld_shared_cluster_f1(peer + 4u * (16 * s + i) * C::EPI_WARPS * 32));
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i >> 3][s / 4][8 * (s & 3) + (i & 7)] = __float_as_uint(sum[i]);
          }
        }
        steps = mine;
      }

      // One straight line of code per activation and gate: the unrolled steps (the accumulator is in registers, so
      // they cannot be a loop) would otherwise carry every branch.
      auto finish = [&](auto kind) {
        constexpr int kAct = decltype(kind)::kAct;
        constexpr bool kGated = decltype(kind)::kGated;
        constexpr int kCols = kGated ? 16 : 32;  // columns of D per warp
        const int cols = kGated ? p.N >> 1 : p.N;
        const int d_col0 = kGated ? col0 >> 1 : col0;

        // A box of D in the staging buffer: kRows tokens, rows of kRow bytes in 16-byte chunks, swizzled as the TMA
        // store reads them.
        constexpr int kSize = kF32 ? 4 : 2;
        constexpr int kRow = kCols * kSize;
        constexpr int kRows = kF32 ? 16 : 32;
        constexpr int kChunks = kRows * (kRow / 16);
        static_assert(kRows * kRow <= C::STG_BYTES && kChunks % 32 == 0, "box");
        uint8_t* box = staging + ew * C::STG_BYTES;
        auto chunk = [](int row, int c) {
          return row * kRow + 16 * (c ^ (kRow == 128 ? row & 7 : kRow == 64 ? (row >> 1) & 3 : (row >> 2) & 1));
        };
        // this lane's chunks: column l_col of rows l_row + i kLaneRows
        constexpr int kLaneRows = 32 / (kRow / 16);
        const int l_chunk = static_cast<int>(lane) % (kRow / 16), l_row = static_cast<int>(lane) / (kRow / 16);
        const int l_col = d_col0 + l_chunk * (16 / kSize);
        const bool l_ok = l_col < cols;

        // z[o][n][u]: octet of tokens o, 8-column block n, token fc + u
        constexpr int kBlocks = kGated ? 2 : 4;
        auto values = [&](int s, float (&z)[2][kBlocks][2]) {
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const float2 sc2 = *reinterpret_cast<const float2*>(scales + 16 * s + 8 * o + fc);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float sc = u == 0 ? sc2.x : sc2.y;
              const int at = 4 * ((2 * s + o) & 7) + u;
              float y[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                y[i] = __fmaf_rn(__uint_as_float(r[i >> 1][s / 4][at + 2 * (i & 1)]), sc, bias[i]);
              if constexpr (kGated) {
                activate2<kAct>(y[0], y[2]);
                z[o][0][u] = y[0] * y[1];
                z[o][1][u] = y[2] * y[3];
              } else {
                activate2<kAct>(y[0], y[1]);
                activate2<kAct>(y[2], y[3]);
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) z[o][i][u] = y[i];
              }
            }
          }
        };
        // shared address of this lane's row of a group of four 8 x 8 matrices (lane l: row l % 8 of matrix l / 8):
        // the four blocks of octet `o` of the box, or gated both blocks of octets o and o + 1
        auto matrix_at = [&](int o) {
          const int m = static_cast<int>(lane) >> 3, l = static_cast<int>(lane) & 7;
          return smem_u32(box) + (kGated ? chunk(8 * (o + (m >> 1)) + l, m & 1) : chunk(8 * o + l, m));
        };

#pragma unroll
        for (int s0 = 0; s0 < C::STEPS; s0 += kRows / 16) {
          const int tb = tok0 + 16 * s0;  // first token of the box
          if (kRes && !kF32 && !(steps >> s0 & 1u) && (steps >> (s0 + kRows / 16) & 1u)) load_residual(tb + kRows);
          if (steps >> s0 & 1u) {         // warp-uniform
            constexpr int kSteps = kRows / 16;
            uint32_t w[kSteps][2][kBlocks];  // bf16 pairs of tokens
            if constexpr (!kRes && !kF32) {
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                float z[2][kBlocks][2];
                values(s0 + i, z);
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                  for (int n = 0; n < kBlocks; ++n) w[i][o][n] = pack_bf16x2(z[o][n][0], z[o][n][1]);
              }
            }
            if (elect_one()) bulk_wait_read_all();  // the store of the previous box has read the buffer
            __syncwarp();
            if constexpr (kRes && !kF32) {
#pragma unroll
              for (int i = 0; i < kChunks / 32; ++i)
                *reinterpret_cast<uint4*>(box + chunk(l_row + i * kLaneRows, l_chunk)) = res[i];
              if (steps >> (s0 + kRows / 16) & 1u) load_residual(tb + kRows);
              __syncwarp();
            }
            if constexpr (!kF32) {
              if constexpr (kRes) {
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                  float z[2][kBlocks][2];
                  values(s0 + i, z);
                  if constexpr (kGated) {
                    ldmatrix_x4_trans(matrix_at(2 * i), w[i][0][0], w[i][0][1], w[i][1][0], w[i][1][1]);
                  } else {
#pragma unroll
                    for (int o = 0; o < 2; ++o)
                      ldmatrix_x4_trans(matrix_at(2 * i + o), w[i][o][0], w[i][o][1], w[i][o][2 % kBlocks],
                                        w[i][o][3 % kBlocks]);
                  }
#pragma unroll
                  for (int o = 0; o < 2; ++o)
#pragma unroll
                    for (int n = 0; n < kBlocks; ++n)
                      w[i][o][n] = pack_bf16x2(z[o][n][0] + bf16_bits_to_f32(w[i][o][n] & 0xFFFFu),
                                               z[o][n][1] + bf16_bits_to_f32(w[i][o][n] >> 16));
                }
              }
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                if constexpr (kGated) {
                  stmatrix_x4_trans(matrix_at(2 * i), w[i][0][0], w[i][0][1], w[i][1][0], w[i][1][1]);
                } else {
#pragma unroll
                  for (int o = 0; o < 2; ++o)
                    stmatrix_x4_trans(matrix_at(2 * i + o), w[i][o][0], w[i][o][1], w[i][o][2 % kBlocks],
                                      w[i][o][3 % kBlocks]);
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                float z[2][kBlocks][2];
                values(s0 + i, z);
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                  for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                      // row 16 i + 8 o + fc + u, column 8 n + fr: n moves the chunk by an exclusive or with 2 n
                      float* at = reinterpret_cast<float*>(box + ((chunk(fc + u, fr >> 2) + 4 * (fr & 3)) ^ (32 * n)) +
                                                           (16 * i + 8 * o) * kRow);
                      *at = z[o][n][u];
                    }
              }
            }
            if constexpr (kRes && kF32) {
              // fp32 rows are whole 128-byte lines: the lanes add the residual and store them themselves (there are no
              // registers for a residual in the fragments' order beside the accumulator)
              float* dst = static_cast<float*>(p.D) + (q.row0 + tb + l_row) * p.ld_d + l_col;
              load_residual(tb);
              __syncwarp();
#pragma unroll
              for (int i = 0; i < kChunks / 32; ++i) {
                const float4 d = *reinterpret_cast<const float4*>(box + chunk(l_row + i * kLaneRows, l_chunk));
                if (l_ok && tb + l_row + i * kLaneRows < q.cnt)
                  __stcs(reinterpret_cast<float4*>(dst + i * kLaneRows * p.ld_d),
                         make_float4(d.x + __uint_as_float(res[i].x), d.y + __uint_as_float(res[i].y),
                                     d.z + __uint_as_float(res[i].z), d.w + __uint_as_float(res[i].w)));
              }
              __syncwarp();  // the box has been read
            } else if (tb + kRows <= q.cnt) {
              fence_proxy_async_smem();
              __syncwarp();
              if (elect_one()) {
                if (d_col0 < cols) tma_store_2d_hint(&maps.d, box, d_col0, q.row0 + tb, evict_first);
                bulk_commit_group();
              }
            } else {
              __syncwarp();
              uint8_t* dst = static_cast<uint8_t*>(p.D) + ((q.row0 + tb + l_row) * p.ld_d + l_col) * kSize;
#pragma unroll
              for (int i = 0; i < kChunks / 32; ++i)
                if (l_ok && tb + l_row + i * kLaneRows < q.cnt)
                  *reinterpret_cast<uint4*>(dst + i * (kLaneRows * kSize) * p.ld_d) =
                      *reinterpret_cast<const uint4*>(box + chunk(l_row + i * kLaneRows, l_chunk));
            }
          }
        }
      };
      if (p.gated) {
        switch (p.act) {
          case BSP_ACT_RELU: finish(EpilogueVariant<BSP_ACT_RELU, true>{}); break;
          case BSP_ACT_GELU: finish(EpilogueVariant<BSP_ACT_GELU, true>{}); break;
          case BSP_ACT_GELU_TANH: finish(EpilogueVariant<BSP_ACT_GELU_TANH, true>{}); break;
          case BSP_ACT_SILU: finish(EpilogueVariant<BSP_ACT_SILU, true>{}); break;
          default: finish(EpilogueVariant<BSP_ACT_NONE, true>{}); break;
        }
      } else {
        switch (p.act) {
          case BSP_ACT_RELU: finish(EpilogueVariant<BSP_ACT_RELU, false>{}); break;
          case BSP_ACT_GELU: finish(EpilogueVariant<BSP_ACT_GELU, false>{}); break;
          case BSP_ACT_GELU_TANH: finish(EpilogueVariant<BSP_ACT_GELU_TANH, false>{}); break;
          case BSP_ACT_SILU: finish(EpilogueVariant<BSP_ACT_SILU, false>{}); break;
          default: finish(EpilogueVariant<BSP_ACT_NONE, false>{}); break;
        }
      }
    }
    if (elect_one()) bulk_wait_read_all();
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncwarp();
  if (C::CG == 2 || k_split > 1)
    cluster_sync();  // no CTA leaves while another may still signal it or read its partial tile
  else
    __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    if constexpr (C::CG == 2)
      tmem_dealloc_pair(tmem, C::TMEM_COLS);
    else
      tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

struct FusedArgs {
  const uint8_t *A, *sfA, *B, *sfB;
  int64_t row_bytes, tiles_per_band;
};

// CTAs per tile: a split of K over a cluster when the tiles alone leave at least half of the SMs idle and every CTA
// keeps at least kMinSplitSteps 128-byte steps.  Measured (us, split / whole): N = 5120, K = 13824 (54 steps), M = 16:
// 14.6 / 18.3; N = 5120, K = 5120 (20 steps): two of 10 steps 11.5 / 10.9; N = 1536, K = 1536: 8.3 / 5.9.
int fused_split(int sm_count, int64_t tiles, int64_t num_kb) {
  int64_t s = sm_count / tiles;
  s = s < kMaxSplit ? s : kMaxSplit;
  s = s < num_kb / kMinSplitSteps ? s : num_kb / kMinSplitSteps;
  return s < 1 ? 1 : static_cast<int>(s);
}

template <int KIND, int CG, bool kF32, bool kRes>
int launch_variant(const DeviceInfo& dev, const FusedArgs& a, FusedParams p, cudaStream_t stream) {
  using C = FCfg<KIND, CG>;
  auto kernel = fused_gemm_kernel<KIND, CG, kF32, kRes>;
  static PerDevice attr_set;
  if (!attr_set.get(dev.id)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
      return launch_status();
    attr_set.set(dev.id, 1);
  }
  FusedMaps maps;
  int st;
  if ((st = p.gated ? encode_experts_gated(&maps.w, a.B, p.E, p.N, a.row_bytes)
                    : encode_experts(&maps.w, a.B, p.E, p.N, a.row_bytes, 128)) != BSP_OK)
    return st;
  if ((st = encode_expert_scales(&maps.sfw, a.sfB, p.E, ceil_div(p.N, 128), a.tiles_per_band, C::ATOMS)) != BSP_OK)
    return st;
  for (int i = 0; i < (p.tn / CG + 31) / 32; ++i)
    if ((st = encode_operand(&maps.x[i], a.A, p.M, a.row_bytes, 32 * (i + 1))) != BSP_OK) return st;
  for (int i = 0; i < C::X_BANDS; ++i)
    if ((st = encode_scales(&maps.sfx[i], a.sfA, ceil_div(p.M, 128), a.tiles_per_band, C::ATOMS, i + 1)) != BSP_OK)
      return st;
  if ((st = encode_rows(&maps.d, p.D, p.M, p.gated ? p.N / 2 : p.N, p.ld_d, kF32, kF32 ? 16 : 32,
                        p.gated ? 16 : 32)) != BSP_OK)
    return st;

  p.num_kb = static_cast<int>(ceil_div(a.row_bytes, 128));
  p.panels = static_cast<int>(ceil_div(p.N, 128 * CG));
  int64_t groups = dev.sm_count / CG / p.split;
  if constexpr (CG == 1) {
    p.x_bytes = static_cast<int>(round_up(p.tn, 32)) * 128;
    p.stage_bytes = static_cast<int>(round_up(C::W_BYTES + p.x_bytes + C::BAND_BYTES * (1 + C::X_BANDS), 1024));
    p.stages = C::RING_BYTES / p.stage_bytes;
    if (p.stages > C::MAX_STAGES) p.stages = C::MAX_STAGES;
  }
  const int64_t most = (ceil_div(p.M, p.tn) + (p.offsets == nullptr ? 0 : p.E < p.M ? p.E : p.M)) * p.panels;
  if (most > (1ll << 30)) return BSP_ERR_INVALID_ARG;  // tiles, at most
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  // programmatic launch: the kernel's set-up overlaps the previous kernel's tail
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int cluster = CG * p.split;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    static PerDevice resident[kMaxSplit + 1];  // clusters resident at once, by size
    int r = resident[cluster].get(dev.id);
    if (r == 0) {
      cfg.gridDim = dim3(static_cast<unsigned>(groups * cluster), 1, 1);
      if (cudaOccupancyMaxActiveClusters(&r, kernel, &cfg) != cudaSuccess) return launch_status();
      if (r < 1) return BSP_ERR_CUDA;  // a cluster does not fit: nothing launched
      resident[cluster].set(dev.id, r);
    }
    if (groups > r) groups = r;
    if (p.split > 1 && groups < most) {  // a split cluster takes one tile only
      p.split = 1;
      groups = dev.sm_count;
      cfg.numAttrs = 1;
    }
  }
  if (most < groups) groups = most;
  // Token tiles per rasterisation group, as in gemm.cu: weights well inside L2: just enough token tiles that the CTAs
  // running at once cover every panel; large weights: about 24 MiB of tokens per group.
  const int64_t b_bytes = static_cast<int64_t>(p.N) * a.row_bytes * 17 / 16;
  int64_t g = b_bytes < (32ll << 20) ? ceil_div(2 * groups, p.panels)
                                     : (24ll << 20) / (static_cast<int64_t>(p.tn) * a.row_bytes * 17 / 16);
  p.group_m = static_cast<int>(g < 8 ? 8 : g > (1 << 20) ? (1 << 20) : g);
  cfg.gridDim = dim3(static_cast<unsigned>(groups * CG * p.split), 1, 1);
  if (cudaLaunchKernelEx(&cfg, kernel, maps, p) != cudaSuccess) return launch_status();
  return launch_status();
}

template <int KIND, int CG>
int launch_fused(const DeviceInfo& dev, const FusedArgs& a, const FusedParams& p, bool f32, cudaStream_t stream) {
  if (f32)
    return p.residual ? launch_variant<KIND, CG, true, true>(dev, a, p, stream)
                      : launch_variant<KIND, CG, true, false>(dev, a, p, stream);
  return p.residual ? launch_variant<KIND, CG, false, true>(dev, a, p, stream)
                    : launch_variant<KIND, CG, false, false>(dev, a, p, stream);
}

// The form and the token tile, from the sizes and the experts' mean row count (their own are on the device; with a buffer
// taller than its live rows the mean is too high: 512 rows over 128 experts of 1536 x 2048 in a buffer of 32768 rows take
// pairs, 46.6 us against 41.5 in an exact one, 8192 rows 49.9 against 47.9).
//  - CTA pairs (256 x 256 tiles) once the 128 x 128 tiles of single CTAs no longer fit in one wave: the pair's operands
//    cost half the bandwidth (us, pairs / single: M = 4096, N = 13824, K = 5120: 121 / 162; M = 256, same weights:
//    18.2 / 20.5), but its epilogue and its larger tiles take longer where everything runs at once (M = 256, N = 5120,
//    K = 13824: 28.6 / 23.0).  Up to 8 K steps the single form's second accumulator, which overlaps the epilogue with
//    the next tile, is worth up to three waves (M = 4096, N = K = 1536: 16.4 / 14.2).
//    Experts: single up to a mean of 64 rows (with up to 4 K steps: 160), and above it while about 3.5 waves of single
//    tiles hold them all (us, pairs / single: 128 experts of 1536 x 2048 at 64 rows 48.1 / 48.0, at 128 56.5 / 62.4;
//    128 of 2048 x 768 at 128 rows 47.3 / 44.3; 16 of 2048 x 2048 at 128 rows, 2.6 waves, 20.1 / 16.5, at 256 20.9 /
//    22.7; 8 of 5120 x 5120 at 128 rows, 3.2 waves, 32.3 / 31.0, at 192 35.5 / 42.2).
//  - Single CTAs, token tile 32, 64 or 128: narrow tiles leave room for a deeper ring, but cost a pass over the weight
//    each.  Dense: the smallest that covers M; with up to 8 K steps, where a tile's time is its epilogue's, the
//    smallest whose tiles fit in one wave (M = 256, N = K = 1536: 6.9 against 7.4 at 128).  Experts: 32 up to a mean
//    of 8 rows, 64 up to 24 (128 experts of 1536 x 2048, tiles of 32 / 64 / 128: 39.9 / 40.6 / 41.4 at 8 rows, 41.8 /
//    39.7 / 40.9 at 16, 53.1 / 43.3 / 41.1 at 32).
struct FusedPlan {
  int ctas;   // 2: CTA pairs
  int tn;     // token tile
  int split;  // CTAs of a cluster sharing a tile's K range
};

FusedPlan plan_fused(int sm_count, bool grouped, int64_t E, int64_t M, int64_t N, int64_t num_kb) {
  const int64_t panels = ceil_div(N, 128), waves = num_kb <= 8 ? 3 : 1;
  if (!grouped) {
    if (ceil_div(M, 128) * panels > waves * sm_count) return {2, 256, 1};
    int tn = 32;
    for (; tn < 128; tn *= 2)
      if (M <= tn || (num_kb <= 8 && ceil_div(M, tn) * panels <= sm_count)) break;
    return {1, tn, fused_split(sm_count, ceil_div(M, tn) * panels, num_kb)};
  }
  const int64_t rows = ceil_div(M, E);
  const int64_t single = (2 * ceil_div(M, 128) + E) * panels;  // twice the single tiles, about
  if (rows > (num_kb <= 4 ? 160 : 64) && single > 7 * sm_count) return {2, 256, 1};
  return {1, rows <= 8 ? 32 : rows <= 24 ? 64 : 128, 1};
}

template <int KIND>
int run_fused(const bsp_fused_gemm_desc* d, cudaStream_t stream) {
  if (d == nullptr) return BSP_ERR_INVALID_ARG;
  const int64_t group = KIND == kNVF4 ? 16 : 32, E = d->E, M = d->M, N = d->N, K = d->K;
  if (E < 1 || E > (d->offsets ? kMaxExperts : 1) || M < 0 || N < 0 || K <= 0 || K % 32 != 0)
    return BSP_ERR_INVALID_ARG;
  if (d->d_dtype != BSP_OUT_BF16 && d->d_dtype != BSP_OUT_F32) return BSP_ERR_INVALID_ARG;
  if (d->activation < BSP_ACT_NONE || d->activation > BSP_ACT_SILU || (d->gated != 0 && d->gated != 1))
    return BSP_ERR_INVALID_ARG;
  if ((d->offsets && d->residual) || (KIND == kMXF8 && d->row_scale)) return BSP_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return BSP_OK;
  const int64_t cols = d->gated ? N / 2 : N;
  if (N % (d->gated ? 16 : 8) != 0 || d->ld_d < cols || (d->residual && d->ld_residual < cols))
    return BSP_ERR_INVALID_ARG;
  if (M > (1ll << 30) || N > (1ll << 30) || K > (1ll << 30)) return BSP_ERR_INVALID_ARG;
  if (!d->A || !d->B || !d->sfA || !d->sfB || !d->D) return BSP_ERR_INVALID_ARG;
  const int64_t esize = d->d_dtype == BSP_OUT_F32 ? 4 : 2;
  if (!aligned16(d->A) || !aligned16(d->B) || !aligned16(d->sfA) || !aligned16(d->sfB) || !aligned16(d->D) ||
      (d->bias && !aligned16(d->bias)) || (d->ld_d * esize) % 16 != 0 ||
      (d->residual && (!aligned16(d->residual) || (d->ld_residual * esize) % 16 != 0)) ||
      ((reinterpret_cast<uintptr_t>(d->row_scale) | reinterpret_cast<uintptr_t>(d->alpha) |
        reinterpret_cast<uintptr_t>(d->offsets)) & 3u))
    return BSP_ERR_ALIGNMENT;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != BSP_OK) return st;
  if (encode_tiled_fn() == nullptr) return BSP_ERR_CUDA;

  FusedArgs a;
  a.A = d->A, a.sfA = d->sfA, a.B = d->B, a.sfB = d->sfB;
  a.row_bytes = KIND == kNVF4 ? K / 2 : K;
  a.tiles_per_band = round_up(K / group, 4) / 4;
  FusedParams p = {};
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.E = static_cast<int>(E);
  p.act = static_cast<int>(d->activation);
  p.gated = static_cast<int>(d->gated);
  p.offsets = d->offsets;
  p.alpha = d->alpha;
  p.row_scale = d->row_scale;
  p.bias = d->bias;
  p.residual = d->residual;
  p.ld_res = d->ld_residual;
  p.D = d->D;
  p.ld_d = d->ld_d;
  p.err = dev.err_word;
  const bool f32 = d->d_dtype == BSP_OUT_F32;
  const FusedPlan plan = plan_fused(dev.sm_count, p.offsets != nullptr, E, M, N, ceil_div(a.row_bytes, 128));
  p.tn = plan.tn;
  p.split = plan.split;
  return plan.ctas == 2 ? launch_fused<KIND, 2>(dev, a, p, f32, stream) : launch_fused<KIND, 1>(dev, a, p, f32, stream);
}

}  // namespace
}  // namespace bsp
