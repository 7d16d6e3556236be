// fused_gemm.cu -- block-scaled GEMMs with an activation, a gate and a residual in the epilogue, dense or grouped by
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
// Roles, pipeline and bounded waits are those of gemm.cu: warp 0 TMA producer, warp 1 MMA issuer, warps 2 and 3 idle
// (relays of a pair's follower), warps 4-7 scale factors, warps 8 and up the epilogue.  Every CTA builds the table of
// the experts' tiles in shared memory from the offsets (a scan over the experts) and takes every gridDim-th tile:
// nothing is read back to the host.
#include "activation.cuh"
#include "bsp_device.cuh"
#include "bsp_internal.h"
#include "tensor_maps.h"

namespace bsp {
namespace {

constexpr int kMaxExperts = BSP_MAX_EXPERTS;  // the tile table's two words per expert in shared memory

struct FusedParams {
  int M, N, E;
  int num_kb;     // 128-byte steps of K
  int panels;     // weight panels per expert
  int group_m;    // token tiles per rasterisation group
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

// CG = 2: CTA pairs, 256 weight rows x up to 256 tokens.  CG = 1: 128 weight rows x up to 64 tokens.
template <int KIND, int CG_>
struct FCfg {
  static constexpr int CG = CG_;
  static constexpr int TN = CG == 2 ? 256 : 64;          // most tokens per tile
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
  static constexpr int EPI_WARPS = CG == 2 ? 8 : 4;
  static constexpr int FIRST_SF_WARP = 4, FIRST_EPI_WARP = 8;
  static constexpr int THREADS = (8 + EPI_WARPS) * 32;
  static constexpr int STEPS = TN / (EPI_WARPS / 4) / 16;  // steps of 16 tokens per epilogue warp
  // CTA pairs: warpgroups 0 and 1 hand registers to the epilogue, which holds 128 accumulator columns a thread.  (With
  // 40 for the first, as in gemm.cu, its loops spill: 7% of a large GEMM.)
  static constexpr int WG0_REGS = 72, SF_REGS = 88, EPI_REGS = 176;
  static_assert(CG == 1 || 128 * (WG0_REGS + SF_REGS + 2 * EPI_REGS) == THREADS * (65536 / THREADS), "register split");
  static constexpr int STG_BYTES = 1024;  // staging: two buffers per warp, each a box of D for one TMA store
  static constexpr int SCALE_BYTES = 16 * STEPS * 4;  // and its tokens' scales
  static constexpr int TABLE_BYTES = (2 * (kMaxExperts + 1) * 4 + 15) / 16 * 16;
  static constexpr int BAR_BYTES = 512;
  static constexpr int FIXED_BYTES = EPI_WARPS * (2 * STG_BYTES + SCALE_BYTES) + TABLE_BYTES + BAR_BYTES + 1024;
  static constexpr int by_smem = (232448 - FIXED_BYTES) / STAGE_BYTES;
  static constexpr int by_tmem = (TMEM_COLS - ACC_COLS) / SF_COLS;
  static constexpr int STAGES = by_smem < by_tmem ? (by_smem < 8 ? by_smem : 8) : (by_tmem < 8 ? by_tmem : 8);
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + FIXED_BYTES;
  static_assert(STAGES >= 4 && SMEM_BYTES <= 232448 && ACC_COLS + STAGES * SF_COLS <= TMEM_COLS, "budget");
  static_assert((4 * STAGES + 8) * 8 <= BAR_BYTES, "barrier space");
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
  template <int TN>
  __device__ __forceinline__ void build(const FusedParams& p) {
    if (p.offsets == nullptr) {
      if (threadIdx.x == 0) {
        lo[0] = 0;
        lo[1] = p.M;
        start[0] = 0;
        start[1] = (p.M + TN - 1) / TN * p.panels;
      }
      return;
    }
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
  }

  // Tile t: its expert by bisection, then token tiles within groups of group_m, fastest first, so that the CTAs that
  // run at once share weight panels and tokens in L2.  An expert's rows are shared out evenly over its tiles.
  template <int TN, int N_STEP>
  __device__ __forceinline__ Tile get(int t, const FusedParams& p) const {
    int a = 0, b = p.E;
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (start[mid] <= t) a = mid;
      else b = mid;
    }
    const int l = lo[a], rows = lo[a + 1] - l;
    const int nt = (rows + TN - 1) / TN;
    const int r = t - start[a];
    const int per_group = p.group_m * p.panels;
    const int g = r / per_group;
    const int first = g * p.group_m;
    const int size = min(p.group_m, nt - first);
    const int rr = r - g * per_group;
    const int nb = rr / size;
    const int mt = first + rr - nb * size;
    const int per = ((rows + nt - 1) / nt + N_STEP - 1) / N_STEP * N_STEP;
    Tile q;
    q.e = a;
    q.nb = nb;
    q.row0 = l + mt * per;
    q.cnt = min(per, l + rows - q.row0);
    q.nmma = (q.cnt + N_STEP - 1) / N_STEP * N_STEP;
    return q;
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
  uint8_t* staging = smem + C::STAGES * C::STAGE_BYTES;
  uint8_t* table_mem = staging + C::EPI_WARPS * (2 * C::STG_BYTES + C::SCALE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(table_mem + C::TABLE_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* sf_ready = empty + C::STAGES;
  uint64_t* sf_local = sf_ready + C::STAGES;  // pair follower: its scale warps, per stage
  uint64_t* acc_full = sf_local + C::STAGES;  // [ACC_BUFS]
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* acc_local = acc_empty + 2;  // pair follower: its epilogue warps
  uint64_t* drain = acc_local + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  Table table;
  table.carve(table_mem);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  const uint32_t rank = C::CG == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0u;
  constexpr uint32_t kPeerArrivals = C::CG == 2 ? 1u : 0u;  // the follower's relayed arrival

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sf_ready[s], C::SF_WARPS + kPeerArrivals);
      mbar_init(&sf_local[s], C::SF_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::EPI_WARPS + kPeerArrivals);
    }
    mbar_init(acc_local, C::EPI_WARPS);
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    prefetch_tensormap(&maps.w);
    prefetch_tensormap(&maps.sfw);
    for (int i = 0; i < C::X_MAPS; ++i) prefetch_tensormap(&maps.x[i]);
    for (int i = 0; i < C::X_BANDS; ++i) prefetch_tensormap(&maps.sfx[i]);
    prefetch_tensormap(&maps.d);
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
  // Set-up above overlaps the previous kernel under programmatic launch; every global access below comes after its
  // completion.
  grid_dependency_wait();
  table.build<C::TN>(p);
  tc_fence_before_sync();
  __syncwarp();
  if constexpr (C::CG == 2)
    cluster_sync();  // the peer's barriers are initialised before anything arrives on them
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int num_tiles = table.start[p.E];
  const int first_tile = static_cast<int>(blockIdx.x) / C::CG;
  const int tile_step = static_cast<int>(gridDim.x) / C::CG;

  if (warp < C::FIRST_SF_WARP) {
    if constexpr (C::CG == 2) regs_dec<C::WG0_REGS>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        uint32_t stage = 0, phase = 0;
        uint32_t total = 0;  // stages issued
        bool ok = true;
        for (int t = first_tile; t < num_tiles && ok; t += tile_step) {
          const Tile q = table.get<C::TN, C::N_STEP>(t, p);
          const int band = q.nb * C::CG + static_cast<int>(rank);  // of 128 weight rows
          const int x_rows = q.nmma / C::CG;
          const int x_row = q.row0 + static_cast<int>(rank) * x_rows;
          const int x_box = (x_rows + 31) >> 5;
          const int x_bands = ((q.row0 & 127) + q.nmma + 127) >> 7;
          const CUtensorMap* mx = &maps.x[x_box - 1];
          const CUtensorMap* msfx = &maps.sfx[x_bands - 1];
          const uint32_t tx = static_cast<uint32_t>(C::W_BYTES + x_box * 4096 + C::BAND_BYTES * (1 + x_bands));
          for (int kb = 0; kb < p.num_kb; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            uint8_t* st = smem + stage * C::STAGE_BYTES;
            uint8_t* sf = st + C::W_BYTES + C::X_BYTES;
            mbar_arrive_expect_tx(&full[stage], tx);
            if (p.gated)
              tma_load_5d(st, &maps.w, &full[stage], kb * 128, 0, 0, band * 8, q.e);
            else
              tma_load_3d(st, &maps.w, &full[stage], kb * 128, band * 128, q.e);
            tma_load_2d(st + C::W_BYTES, mx, &full[stage], kb * 128, x_row);
            tma_load_4d(sf, &maps.sfw, &full[stage], 0, kb * C::ATOMS, band, q.e);
            tma_load_3d(sf + C::BAND_BYTES, msfx, &full[stage], 0, kb * C::ATOMS, q.row0 >> 7);
            ++total;
            if (++stage == C::STAGES) {
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
        for (uint32_t s = 0; s < C::STAGES; ++s)
          if (total > s && !mbar_wait(&full[s], ((total - 1u - s) / C::STAGES) & 1u, nullptr))
            raise_error(p.err, kErrTimeout);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0 && leader) {
        uint32_t stage = 0, phase = 0;
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
          const Tile q = table.get<C::TN, C::N_STEP>(t, p);
          const int buf = it % C::ACC_BUFS;
          const uint32_t acc = tmem + static_cast<uint32_t>(buf * C::TN);
          if (!wait_shared(&acc_empty[buf], (static_cast<uint32_t>(it / C::ACC_BUFS) & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          for (int kb = 0; kb < p.num_kb; ++kb) {
            if (!wait_shared(&sf_ready[stage], phase)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t sbase = smem_u32(smem + stage * C::STAGE_BYTES);
            const uint32_t sfw_t = tmem + C::ACC_COLS + stage * C::SF_COLS;
            const uint32_t sfx_t = sfw_t + C::SFW_COLS;
            const uint64_t wdesc = desc_kmajor_sw128(sbase);
            const uint64_t xdesc = desc_kmajor_sw128(sbase + C::W_BYTES);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t accumulate = (kb > 0 || kk > 0) ? 1u : 0u;
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
            if (++stage == C::STAGES) {
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
      } else if (lane == 0) {
        // pair follower: its MMAs are issued by the leader, whose last commit arrives here too
        if (!mbar_wait(drain, 0u, nullptr)) raise_error(p.err, kErrTimeout);
      }
    } else if (C::CG == 2 && !leader && lane == 0) {
      // pair follower: warp 2 relays each stage's scales to the leader, warp 3 each released accumulator
      bool ok = true;
      if (warp == 2) {
        const uint32_t peer = mapa_shared(smem_u32(sf_ready), 0u);
        uint32_t stage = 0, phase = 0;
        for (int t = first_tile; t < num_tiles && ok; t += tile_step) {
          for (int kb = 0; kb < p.num_kb; ++kb) {
            if (!mbar_wait(&sf_local[stage], phase, abort_flag)) {
              ok = false;
              break;
            }
            mbar_arrive_remote_relaxed(peer + 8u * stage);
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      } else {
        const uint32_t peer = mapa_shared(smem_u32(acc_empty), 0u);
        int it = 0;
        for (int t = first_tile; t < num_tiles && ok; t += tile_step, ++it) {
          if (!mbar_wait(acc_local, static_cast<uint32_t>(it) & 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_remote_relaxed(peer);
        }
      }
      if (!ok) {
        *abort_flag = 1u;
        raise_error(p.err, kErrTimeout);
      }
    }
  } else if (warp < C::FIRST_EPI_WARP) {
    // ------------------------------------------------------------ scale factors
    if constexpr (C::CG == 2) regs_dec<C::SF_REGS>();
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    uint64_t* sf_mine = leader ? sf_ready : sf_local;
    // gated: the accumulator's rows are the weight's in the order of the epilogue (gated_row)
    const int w_line = p.gated ? gated_row(static_cast<int>(lane)) : static_cast<int>(lane);
    for (int t = first_tile; t < num_tiles && ok; t += tile_step) {
      const Tile q = table.get<C::TN, C::N_STEP>(t, p);
      // Scale row i of the tile is row (row0 & 127) + i of the loaded bands.  Line `lane` of tensor memory takes the
      // words of rows lane + 32 j, which all sit in line (row0 + lane) & 31 of the tiles, at word `shift` + j (plus
      // one in the lanes where row0 + lane carries into the next 32 rows) of the bands' words one after another.
      const bool carry = (q.row0 & 31) + static_cast<int>(lane) >= 32;
      const int line = (q.row0 + static_cast<int>(lane)) & 31;
      // one loop over K for each variant: a choice inside it costs 3% of a large GEMM
      auto stages = [&](auto variant) {
        constexpr int kShift = decltype(variant)::kShift;
        constexpr bool kWide = decltype(variant)::kWide;
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          copy_scales<KIND, CG, kShift, kWide>(tmem + lane_base + C::ACC_COLS + stage * C::SF_COLS,
                                               smem + stage * C::STAGE_BYTES + C::W_BYTES + C::X_BYTES, w_line, line,
                                               carry);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sf_mine[stage]);
          if (++stage == C::STAGES) {
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
    // with a transpose), 16 tokens x 32 columns of D at a time, from where they go out as one TMA store.  (16-byte
    // stores from the lanes took 25% longer over the whole GEMM; turning fp32 values over through shared memory and
    // storing 8 tokens at a time took twice as long as the MMAs at K = 1536.)  The box that holds an expert's last
    // rows is stored by the lanes, row by row: the rows after them belong to another expert.
    if constexpr (C::CG == 2) regs_inc<C::EPI_REGS>();
    const int ew = warp - C::FIRST_EPI_WARP;
    const int quarter = warp & 3;
    const int half = ew >> 2;
    const int fr = static_cast<int>(lane) >> 2, fc = 2 * (static_cast<int>(lane) & 3);  // fragment row, first token
    uint64_t* acc_mine = leader ? acc_empty : acc_local;
    const uint64_t evict_first = l2_policy_evict_first();
    float* scales = reinterpret_cast<float*>(staging + C::EPI_WARPS * 2 * C::STG_BYTES) + ew * 16 * C::STEPS;
    uint32_t seq = 0;  // boxes of this warp (picks the staging buffer)
    int it = 0;
    for (int t = first_tile; t < num_tiles; t += tile_step, ++it) {
      const Tile q = table.get<C::TN, C::N_STEP>(t, p);
      const int buf = it % C::ACC_BUFS;
      const int width = C::CG == 2 ? q.nmma / 2 : q.nmma;  // tokens per epilogue warp
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

      // One straight line of code per activation and gate: the unrolled steps (the accumulator is in registers, so
      // they cannot be a loop) would otherwise carry every branch.
      const int lim = min(width, q.cnt - tok0);
      auto finish = [&](auto kind) {
        constexpr int kAct = decltype(kind)::kAct;
        constexpr bool kGated = decltype(kind)::kGated;
        constexpr int kCols = kGated ? 16 : 32;  // columns of D per warp
        const int cols = kGated ? p.N >> 1 : p.N;
        const int d_col0 = kGated ? col0 >> 1 : col0;

        // A box of D in a staging buffer: rows of kRow bytes, 16-byte chunks swizzled as the TMA store reads them.
        auto chunk = [](int row, int c, int row_bytes) {
          return row * row_bytes + 16 * (c ^ (row_bytes == 128 ? row & 7 : row_bytes == 64 ? (row >> 1) & 3 : (row >> 2) & 1));
        };
        auto open_box = [&]() {
          if (lane == 0) bulk_wait_read_allow<1>();  // the store from this buffer, two boxes back, has read it
          __syncwarp();
          return staging + (ew * 2 + (seq++ & 1)) * C::STG_BYTES;
        };
        // the residual's box, one 16-byte chunk per lane and turn, into the buffer
        auto fill_box = [&](uint8_t* box, int tb, int rows, int row_bytes, int esize) {
          const int per_row = row_bytes >> 4;
#pragma unroll 1
          for (int c = static_cast<int>(lane); c < rows * per_row; c += 32) {
            const int row = c / per_row, cc = c - row * per_row;
            const int col = d_col0 + cc * (16 / esize);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (tb + row < q.cnt && col < cols)
              v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.residual) +
                                                  ((q.row0 + tb + row) * p.ld_res + col) * esize);
            *reinterpret_cast<uint4*>(box + chunk(row, cc, row_bytes)) = v;
          }
          __syncwarp();
        };
        auto close_box = [&](uint8_t* box, int tb, int rows, int row_bytes, int esize) {
          if (tb + rows <= q.cnt) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && d_col0 < cols) tma_store_2d_hint(&maps.d, box, d_col0, q.row0 + tb, evict_first);
          } else {
            __syncwarp();
            const int per_row = row_bytes >> 4;
#pragma unroll 1
            for (int c = static_cast<int>(lane); c < rows * per_row; c += 32) {
              const int row = c / per_row, cc = c - row * per_row;
              const int col = d_col0 + cc * (16 / esize);
              if (tb + row < q.cnt && col < cols)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.D) + ((q.row0 + tb + row) * p.ld_d + col) * esize) =
                    *reinterpret_cast<const uint4*>(box + chunk(row, cc, row_bytes));
            }
          }
          if (lane == 0) bulk_commit_group();  // one group per box, empty or not: open_box counts boxes
        };

#pragma unroll
        for (int s = 0; s < C::STEPS; ++s) {
          const int tb = tok0 + 16 * s;  // first token of the step
          if (16 * s < lim) {  // warp-uniform
            // z[o][n][u]: octet of tokens o, 8-column block n, token fc + u
            constexpr int kBlocks = kGated ? 2 : 4;
            float z[2][kBlocks][2];
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
#pragma unroll
                for (int i = 0; i < kBlocks; ++i)
                  z[o][i][u] = kGated ? activate<kAct>(y[2 * i & 3]) * y[(2 * i + 1) & 3] : activate<kAct>(y[i]);
              }
            }
            if constexpr (!kF32) {
              constexpr int kRow = 2 * kCols;
              uint8_t* box = open_box();
              // lane l addresses row l % 8 of matrix l / 8 of a group of four
              const int m = static_cast<int>(lane) >> 3;
              uint32_t at[kGated ? 1 : 2];
              if constexpr (kGated) {
                at[0] = smem_u32(box) + chunk(8 * (m >> 1) + (lane & 7), m & 1, kRow);  // (octet, block)
              } else {
                at[0] = smem_u32(box) + chunk(lane & 7, m, kRow);
                at[1] = smem_u32(box) + chunk(8 + (lane & 7), m, kRow);
              }
              uint32_t w[2][kBlocks];
              if constexpr (kRes) {
                fill_box(box, tb, 16, kRow, 2);
                if constexpr (kGated) {
                  ldmatrix_x4_trans(at[0], w[0][0], w[0][1], w[1][0], w[1][1]);
                } else {
                  ldmatrix_x4_trans(at[0], w[0][0], w[0][1], w[0][2 % kBlocks], w[0][3 % kBlocks]);
                  ldmatrix_x4_trans(at[1], w[1][0], w[1][1], w[1][2 % kBlocks], w[1][3 % kBlocks]);
                }
                __syncwarp();  // every lane has read before the result takes the residual's place
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                  for (int i = 0; i < kBlocks; ++i) {
                    z[o][i][0] += bf16_bits_to_f32(w[o][i] & 0xFFFFu);
                    z[o][i][1] += bf16_bits_to_f32(w[o][i] >> 16);
                  }
              }
#pragma unroll
              for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) w[o][i] = pack_bf16x2(z[o][i][0], z[o][i][1]);
              if constexpr (kGated) {
                stmatrix_x4_trans(at[0], w[0][0], w[0][1], w[1][0], w[1][1]);
              } else {
                stmatrix_x4_trans(at[0], w[0][0], w[0][1], w[0][2 % kBlocks], w[0][3 % kBlocks]);
                stmatrix_x4_trans(at[1], w[1][0], w[1][1], w[1][2 % kBlocks], w[1][3 % kBlocks]);
              }
              close_box(box, tb, 16, kRow, 2);
            } else {
              constexpr int kRow = 4 * kCols;
              constexpr int kRows = kGated ? 16 : 8;  // a box is 1 KB
#pragma unroll
              for (int o0 = 0; o0 < 2; o0 += kRows / 8) {
                if (tb + 8 * o0 < q.cnt) {  // warp-uniform
                  uint8_t* box = open_box();
                  if constexpr (kRes) fill_box(box, tb + 8 * o0, kRows, kRow, 4);
#pragma unroll
                  for (int o = o0; o < o0 + kRows / 8; ++o)
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                      for (int u = 0; u < 2; ++u) {
                        const int row = 8 * (o - o0) + fc + u, n = 8 * i + fr;
                        float* at = reinterpret_cast<float*>(box + chunk(row, n >> 2, kRow)) + (n & 3);
                        *at = kRes ? z[o][i][u] + *at : z[o][i][u];
                      }
                  close_box(box, tb + 8 * o0, kRows, kRow, 4);
                }
              }
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
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncwarp();
  if constexpr (C::CG == 2)
    cluster_sync();  // no CTA of the pair leaves while the other may still signal it
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

template <int KIND, int CG, bool kF32, bool kRes>
int launch_variant(const DeviceInfo& dev, const FusedArgs& a, FusedParams p, cudaStream_t stream) {
  using C = FCfg<KIND, CG>;
  auto kernel = fused_gemm_kernel<KIND, CG, kF32, kRes>;
  static bool attr_set[64] = {};
  if (!attr_set[dev.id]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
      return launch_status();
    attr_set[dev.id] = true;
  }
  FusedMaps maps;
  int st;
  if ((st = p.gated ? encode_experts_gated(&maps.w, a.B, p.E, p.N, a.row_bytes)
                    : encode_experts(&maps.w, a.B, p.E, p.N, a.row_bytes, 128)) != BSP_OK)
    return st;
  if ((st = encode_expert_scales(&maps.sfw, a.sfB, p.E, ceil_div(p.N, 128), a.tiles_per_band, C::ATOMS)) != BSP_OK)
    return st;
  for (int i = 0; i < C::X_MAPS; ++i)
    if ((st = encode_operand(&maps.x[i], a.A, p.M, a.row_bytes, 32 * (i + 1))) != BSP_OK) return st;
  for (int i = 0; i < C::X_BANDS; ++i)
    if ((st = encode_scales(&maps.sfx[i], a.sfA, ceil_div(p.M, 128), a.tiles_per_band, C::ATOMS, i + 1)) != BSP_OK)
      return st;
  if ((st = encode_rows(&maps.d, p.D, p.M, p.gated ? p.N / 2 : p.N, p.ld_d, kF32, kF32 && !p.gated ? 8 : 16,
                        p.gated ? 16 : 32)) != BSP_OK)
    return st;

  p.num_kb = static_cast<int>(ceil_div(a.row_bytes, 128));
  p.panels = static_cast<int>(ceil_div(p.N, 128 * CG));
  const int64_t most = (ceil_div(p.M, C::TN) + (p.E < p.M ? p.E : p.M)) * p.panels;  // tiles, at most
  if (most > (1ll << 30)) return BSP_ERR_INVALID_ARG;
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
  int64_t groups = dev.sm_count / CG;
  if constexpr (CG == 2) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    static int resident[64] = {};  // pairs resident at once, per device
    if (resident[dev.id] == 0) {
      cfg.gridDim = dim3(static_cast<unsigned>(groups * 2), 1, 1);
      int r = 0;
      if (cudaOccupancyMaxActiveClusters(&r, kernel, &cfg) != cudaSuccess) return launch_status();
      if (r < 1) return BSP_ERR_CUDA;  // a pair does not fit: nothing launched
      resident[dev.id] = r;
    }
    if (groups > resident[dev.id]) groups = resident[dev.id];
  }
  if (most < groups) groups = most;
  // Token tiles per rasterisation group, as in gemm.cu: weights well inside L2: just enough token tiles that the CTAs
  // running at once cover every panel; large weights: about 24 MiB of tokens per group.
  const int64_t b_bytes = static_cast<int64_t>(p.N) * a.row_bytes * 17 / 16;
  int64_t g = b_bytes < (32ll << 20) ? ceil_div(2 * groups, p.panels)
                                     : (24ll << 20) / (static_cast<int64_t>(C::TN) * a.row_bytes * 17 / 16);
  p.group_m = static_cast<int>(g < 8 ? 8 : g > (1 << 20) ? (1 << 20) : g);
  cfg.gridDim = dim3(static_cast<unsigned>(groups * CG), 1, 1);
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

template <int KIND>
int run_fused(const uint8_t* A, const uint8_t* sfA, const uint8_t* B, const uint8_t* sfB, const int32_t* offsets,
              int64_t E, int64_t M, int64_t N, int64_t K, const float* alpha, const float* row_scale,
              const uint16_t* bias, int act, int gated, const void* residual, int64_t ld_res, void* D, int d_dtype,
              int64_t ld_d, cudaStream_t stream) {
  const int64_t group = KIND == kNVF4 ? 16 : 32;
  if (E < 1 || E > kMaxExperts || M < 0 || N < 0 || K <= 0 || K % 32 != 0) return BSP_ERR_INVALID_ARG;
  if (d_dtype != BSP_OUT_BF16 && d_dtype != BSP_OUT_F32) return BSP_ERR_INVALID_ARG;
  if (act < BSP_ACT_NONE || act > BSP_ACT_SILU || (gated != 0 && gated != 1)) return BSP_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return BSP_OK;
  const int64_t cols = gated ? N / 2 : N;
  if (N % (gated ? 16 : 8) != 0 || ld_d < cols || (residual && ld_res < cols)) return BSP_ERR_INVALID_ARG;
  if (M > (1ll << 30) || N > (1ll << 30) || K > (1ll << 30)) return BSP_ERR_INVALID_ARG;
  if (!A || !B || !sfA || !sfB || !D) return BSP_ERR_INVALID_ARG;
  const int64_t esize = d_dtype == BSP_OUT_F32 ? 4 : 2;
  if (!aligned16(A) || !aligned16(B) || !aligned16(sfA) || !aligned16(sfB) || !aligned16(D) ||
      (bias && !aligned16(bias)) || (ld_d * esize) % 16 != 0 ||
      (residual && (!aligned16(residual) || (ld_res * esize) % 16 != 0)) ||
      ((reinterpret_cast<uintptr_t>(row_scale) | reinterpret_cast<uintptr_t>(alpha) |
        reinterpret_cast<uintptr_t>(offsets)) & 3u))
    return BSP_ERR_ALIGNMENT;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != BSP_OK) return st;
  if (encode_tiled_fn() == nullptr) return BSP_ERR_CUDA;

  FusedArgs a;
  a.A = A, a.sfA = sfA, a.B = B, a.sfB = sfB;
  a.row_bytes = KIND == kNVF4 ? K / 2 : K;
  a.tiles_per_band = round_up(K / group, 4) / 4;
  FusedParams p = {};
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.E = static_cast<int>(E);
  p.act = act;
  p.gated = gated;
  p.offsets = offsets;
  p.alpha = alpha;
  p.row_scale = row_scale;
  p.bias = bias;
  p.residual = residual;
  p.ld_res = ld_res;
  p.D = D;
  p.ld_d = ld_d;
  p.err = dev.err_word;
  // CTA pairs for experts of more than 64 rows on average
  if (ceil_div(M, E) > 64) return launch_fused<KIND, 2>(dev, a, p, d_dtype == BSP_OUT_F32, stream);
  return launch_fused<KIND, 1>(dev, a, p, d_dtype == BSP_OUT_F32, stream);
}

}  // namespace
}  // namespace bsp

extern "C" {

int nvfp4_gemm_fused(const uint8_t* A, const uint8_t* sfA, const uint8_t* B, const uint8_t* sfB, int64_t M, int64_t N,
                     int64_t K, const float* alpha, const float* row_scale, const uint16_t* bias, int activation,
                     int gated, const void* residual, int64_t ld_residual, void* D, int d_dtype, int64_t ld_d,
                     bsp_stream_t stream) {
  return bsp::run_fused<bsp::kNVF4>(A, sfA, B, sfB, nullptr, 1, M, N, K, alpha, row_scale, bias, activation, gated,
                                    residual, ld_residual, D, d_dtype, ld_d, stream);
}

int mxfp8_gemm_fused(const uint8_t* A, const uint8_t* sfA, const uint8_t* B, const uint8_t* sfB, int64_t M, int64_t N,
                     int64_t K, const float* alpha, const uint16_t* bias, int activation, int gated,
                     const void* residual, int64_t ld_residual, void* D, int d_dtype, int64_t ld_d,
                     bsp_stream_t stream) {
  return bsp::run_fused<bsp::kMXF8>(A, sfA, B, sfB, nullptr, 1, M, N, K, alpha, nullptr, bias, activation, gated,
                                    residual, ld_residual, D, d_dtype, ld_d, stream);
}

int nvfp4_grouped_gemm(const uint8_t* A, const uint8_t* sfA, const uint8_t* B, const uint8_t* sfB,
                       const int32_t* offsets, int64_t E, int64_t M, int64_t N, int64_t K, const float* alpha,
                       const float* row_scale, const uint16_t* bias, int activation, int gated, void* D, int d_dtype,
                       int64_t ld_d, bsp_stream_t stream) {
  if (offsets == nullptr && M > 0 && N > 0) return BSP_ERR_INVALID_ARG;
  return bsp::run_fused<bsp::kNVF4>(A, sfA, B, sfB, offsets, E, M, N, K, alpha, row_scale, bias, activation, gated,
                                    nullptr, 0, D, d_dtype, ld_d, stream);
}

int mxfp8_grouped_gemm(const uint8_t* A, const uint8_t* sfA, const uint8_t* B, const uint8_t* sfB,
                       const int32_t* offsets, int64_t E, int64_t M, int64_t N, int64_t K, const float* alpha,
                       const uint16_t* bias, int activation, int gated, void* D, int d_dtype, int64_t ld_d,
                       bsp_stream_t stream) {
  if (offsets == nullptr && M > 0 && N > 0) return BSP_ERR_INVALID_ARG;
  return bsp::run_fused<bsp::kMXF8>(A, sfA, B, sfB, offsets, E, M, N, K, alpha, nullptr, bias, activation, gated,
                                    nullptr, 0, D, d_dtype, ld_d, stream);
}

}  // extern "C"
