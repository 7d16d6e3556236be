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

constexpr int kMaxExperts = BSP_MAX_EXPERTS;  // the tile table's three words per expert in shared memory

struct FusedParams {
  int M, N, E;
  int num_kb;     // 128-byte steps of K
  int panels;     // weight panels per expert
  int group_m;    // token tiles per rasterisation group
  int act, gated, out_f32;
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
  static constexpr int X_BOX = 32;                       // rows per TMA box of tokens
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
  static constexpr int CHUNKS = TN / (EPI_WARPS / 4) / 16;  // 16-token chunks per epilogue warp
  // CTA pairs: warpgroups 0 and 1 hand registers to the epilogue, which holds 128 accumulator columns a thread
  static constexpr int WG0_REGS = 40, SF_REGS = 88, EPI_REGS = 192;
  static_assert(CG == 1 || 128 * (WG0_REGS + SF_REGS + 2 * EPI_REGS) == THREADS * (65536 / THREADS), "register split");
  // staging: 16 tokens x 32 weight rows of fp32 per warp, rows padded to 36 words so that 16-byte reads of 8 lanes
  // (two tokens x four 8-column segments) touch every bank once
  static constexpr int STG_LD = 36;
  static constexpr int STG_BYTES = 16 * STG_LD * 4;
  static constexpr int TABLE_BYTES = ((3 * kMaxExperts + 1) * 4 + 15) / 16 * 16;
  static constexpr int BAR_BYTES = 512;
  static constexpr int FIXED_BYTES = EPI_WARPS * STG_BYTES + TABLE_BYTES + BAR_BYTES + 1024;
  static constexpr int by_smem = (232448 - FIXED_BYTES) / STAGE_BYTES;
  static constexpr int by_tmem = (TMEM_COLS - ACC_COLS) / SF_COLS;
  static constexpr int STAGES = by_smem < by_tmem ? (by_smem < 8 ? by_smem : 8) : (by_tmem < 8 ? by_tmem : 8);
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + FIXED_BYTES;
  static_assert(STAGES >= 4 && SMEM_BYTES <= 232448 && ACC_COLS + STAGES * SF_COLS <= TMEM_COLS, "budget");
  static_assert((4 * STAGES + 8) * 8 <= BAR_BYTES, "barrier space");
};

struct Tile {
  int e;      // expert
  int nb;     // weight panel
  int row0;   // first row of A
  int cnt;    // rows
  int nmma;   // rows rounded up to the MMA's granularity
};

// The experts' tiles: start[e] is the index of expert e's first tile, rows lo[e] <= m < hi[e].
struct Table {
  int* start;
  int* lo;
  int* hi;

  __device__ __forceinline__ void carve(void* mem) {
    start = static_cast<int*>(mem);
    lo = start + kMaxExperts + 1;
    hi = lo + kMaxExperts;
  }

  // Offsets are clamped to [0, M], and one below an earlier one counts as that one, so that the experts' rows never
  // overlap whatever the array holds.  Called by the whole CTA.
  template <int TN>
  __device__ __forceinline__ void build(const FusedParams& p) {
    if (p.offsets == nullptr) {
      if (threadIdx.x == 0) {
        lo[0] = 0;
        hi[0] = p.M;
        start[0] = 0;
        start[1] = (p.M + TN - 1) / TN * p.panels;
      }
      return;
    }
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) hi[e] = min(max(__ldg(p.offsets + e + 1), 0), p.M);
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int top = min(max(__ldg(p.offsets), 0), p.M);  // the rows before this expert
      int tiles = 0;
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        int h = e < p.E ? hi[e] : 0;
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
          lo[e] = l;
          hi[e] = h;
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
    const int l = lo[a], rows = hi[a] - l;
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
    q.cnt = min(per, hi[a] - q.row0);
    q.nmma = (q.cnt + N_STEP - 1) / N_STEP * N_STEP;
    return q;
  }
};

template <int KIND, int CG>
__global__ void __launch_bounds__(FCfg<KIND, CG>::THREADS, 1)
    fused_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ CUtensorMap tmXfull, const __grid_constant__ CUtensorMap tmSFW,
                      const __grid_constant__ CUtensorMap tmSFX, const FusedParams p) {
  using C = FCfg<KIND, CG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + C::STAGES * C::STAGE_BYTES;
  uint8_t* table_mem = staging + C::EPI_WARPS * C::STG_BYTES;
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
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmXfull);
    prefetch_tensormap(&tmSFW);
    prefetch_tensormap(&tmSFX);
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
        uint32_t issued[C::STAGES];
        for (int s = 0; s < C::STAGES; ++s) issued[s] = 0;
        bool ok = true;
        for (int t = first_tile; t < num_tiles && ok; t += tile_step) {
          const Tile q = table.get<C::TN, C::N_STEP>(t, p);
          const int band = q.nb * C::CG + static_cast<int>(rank);  // of 128 weight rows
          const int x_rows = q.nmma / C::CG;
          const int x_row = q.row0 + static_cast<int>(rank) * x_rows;
          const int boxes = (x_rows + C::X_BOX - 1) / C::X_BOX;
          const int x_band = q.row0 >> 7;
          const int x_bands = ((q.row0 & 127) + q.nmma + 127) >> 7;
          const uint32_t tx = static_cast<uint32_t>(C::W_BYTES + boxes * C::X_BOX * 128 + C::BAND_BYTES * (1 + x_bands));
          for (int kb = 0; kb < p.num_kb; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            uint8_t* st = smem + stage * C::STAGE_BYTES;
            mbar_arrive_expect_tx(&full[stage], tx);
            tma_load_3d(st, &tmW, &full[stage], kb * 128, band * 128, q.e);
            if (boxes == C::X_ROWS / C::X_BOX) {
              tma_load_2d(st + C::W_BYTES, &tmXfull, &full[stage], kb * 128, x_row);
            } else {
              for (int b = 0; b < boxes; ++b)
                tma_load_2d(st + C::W_BYTES + b * C::X_BOX * 128, &tmX, &full[stage], kb * 128, x_row + b * C::X_BOX);
            }
            uint8_t* sf = st + C::W_BYTES + C::X_BYTES;
            tma_load_4d(sf, &tmSFW, &full[stage], 0, kb * C::ATOMS, band, q.e);
            for (int b = 0; b < x_bands; ++b)
              tma_load_3d(sf + C::BAND_BYTES * (1 + b), &tmSFX, &full[stage], 0, kb * C::ATOMS, x_band + b);
            ++issued[stage];
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
        for (int s = 0; s < C::STAGES; ++s)
          if (issued[s] && !mbar_wait(&full[s], (issued[s] - 1u) & 1u, nullptr)) raise_error(p.err, kErrTimeout);
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
    for (int t = first_tile; t < num_tiles && ok; t += tile_step) {
      const Tile q = table.get<C::TN, C::N_STEP>(t, p);
      // Scale row i of the tile is row (row0 & 127) + i of the loaded bands.  Line `lane` of tensor memory takes the
      // words of rows lane + 32 j, which all sit in line (row0 + lane) & 31 of the tiles, at word `shift` + j (plus
      // one in the lanes where row0 + lane carries into the next 32 rows) of the bands' words one after another.
      const int shift = (q.row0 & 127) >> 5;
      const bool carry = (q.row0 & 31) + static_cast<int>(lane) >= 32;
      const int line = (q.row0 + static_cast<int>(lane)) & 31;
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!mbar_wait(&full[stage], phase, abort_flag)) {
          ok = false;
          break;
        }
        const uint8_t* sfw_s = smem + stage * C::STAGE_BYTES + C::W_BYTES + C::X_BYTES;
        const uint8_t* sfx_s = sfw_s + C::BAND_BYTES;
        const uint32_t taddr = tmem + lane_base + C::ACC_COLS + stage * C::SF_COLS;
        uint32_t w[C::SFW_COLS];
#pragma unroll
        for (int a = 0; a < C::ATOMS; ++a) {
          const uint4 v = *reinterpret_cast<const uint4*>(sfw_s + 512 * a + lane * 16);
          w[4 * a + 0] = v.x;
          w[4 * a + 1] = v.y;
          w[4 * a + 2] = v.z;
          w[4 * a + 3] = v.w;
        }
        if constexpr (C::SFW_COLS == 16)
          tmem_st_16cols(taddr, w);
        else
          tmem_st_4cols(taddr, w);
#pragma unroll
        for (int a = 0; a < C::ATOMS; ++a) {
          uint32_t b[4 * C::X_BANDS], x[C::X_WORDS];
#pragma unroll
          for (int i = 0; i < C::X_BANDS; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(sfx_s + C::BAND_BYTES * i + 512 * a + line * 16);
            b[4 * i + 0] = v.x;
            b[4 * i + 1] = v.y;
            b[4 * i + 2] = v.z;
            b[4 * i + 3] = v.w;
          }
          switch (shift) {
            case 0:
#pragma unroll
              for (int j = 0; j < C::X_WORDS; ++j) x[j] = carry ? b[j + 1] : b[j];
              break;
            case 1:
#pragma unroll
              for (int j = 0; j < C::X_WORDS; ++j) x[j] = carry ? b[j + 2] : b[j + 1];
              break;
            case 2:
#pragma unroll
              for (int j = 0; j < C::X_WORDS; ++j) x[j] = carry ? b[j + 3] : b[j + 2];
              break;
            default:
#pragma unroll
              for (int j = 0; j < C::X_WORDS; ++j) x[j] = carry ? b[j + 4] : b[j + 3];
              break;
          }
          if constexpr (C::X_WORDS == 8)
            tmem_st_8cols(taddr + C::SFW_COLS + 8 * a, x);
          else
            tmem_st_4cols(taddr + C::SFW_COLS + 4 * a, x);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_mine[stage]);
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
  } else {
    // ------------------------------------------------------------ epilogue
    // A lane of tensor memory is a weight row, a column a token.  A warp reads its 32 rows x up to 16 CHUNKS tokens
    // into registers, hands the accumulator back, and turns them over through shared memory 16 tokens at a time:
    // then lane (token, segment) holds 8 consecutive columns of one token's row of D, which are finished in fp32 and
    // written with one 16-byte store (bf16), 64 bytes of a row per four lanes.
    if constexpr (C::CG == 2) regs_inc<C::EPI_REGS>();
    const int ew = warp - C::FIRST_EPI_WARP;
    const int quarter = warp & 3;
    const int half = ew >> 2;
    float* stg = reinterpret_cast<float*>(staging + ew * C::STG_BYTES);
    const int seg = static_cast<int>(lane) & 3, sub = static_cast<int>(lane) >> 2;
    uint64_t* acc_mine = leader ? acc_empty : acc_local;
    int it = 0;
    for (int t = first_tile; t < num_tiles; t += tile_step, ++it) {
      const Tile q = table.get<C::TN, C::N_STEP>(t, p);
      const int buf = it % C::ACC_BUFS;
      const int width = C::CG == 2 ? q.nmma / 2 : q.nmma;  // tokens per epilogue warp
      const int tok0 = half * width;                       // this warp's first token of the tile
      const int n0 = (q.nb * C::CG + static_cast<int>(rank)) * 128 + quarter * 32 + seg * 8;
      const bool n_ok = n0 < p.N;
      const float alpha = p.alpha != nullptr ? __ldg(p.alpha + q.e) : 1.0f;
      uint4 bias = make_uint4(0u, 0u, 0u, 0u);  // of this lane's 8 columns
      if (p.bias != nullptr && n_ok)
        bias = __ldg(reinterpret_cast<const uint4*>(p.bias + static_cast<int64_t>(q.e) * p.N + n0));
      // alpha x row scale of this warp's tokens, one per lane, handed out by shuffles
      float scale[(C::CHUNKS + 1) / 2];
#pragma unroll
      for (int j = 0; j < (C::CHUNKS + 1) / 2; ++j) {
        const int tk = tok0 + 32 * j + static_cast<int>(lane);
        scale[j] = (p.row_scale != nullptr && tk < q.cnt) ? __fmul_rn(alpha, __ldg(p.row_scale + q.row0 + tk)) : alpha;
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
      uint32_t r[C::CHUNKS][16];  // columns past `width` are read too, within the accumulator, and not used
#pragma unroll
      for (int c = 0; c < C::CHUNKS; ++c) tmem_ld_16cols(taddr + 16u * c, r[c]);
      tmem_ld_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(C::CG == 2 ? acc_mine : &acc_empty[buf]);

#pragma unroll
      for (int c = 0; c < C::CHUNKS; ++c) {
        if (16 * c < width && tok0 + 16 * c < q.cnt) {  // warp-uniform
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 16; ++i) stg[i * C::STG_LD + lane] = __uint_as_float(r[c][i]);
          __syncwarp();
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int i = 8 * h + sub;  // token of the chunk
            const float sc = __shfl_sync(0xFFFFFFFFu, scale[c / 2], (16 * c + i) & 31);
            const int tk = tok0 + 16 * c + i;
            const int64_t m = q.row0 + tk;
            const float4 lo4 = *reinterpret_cast<const float4*>(stg + i * C::STG_LD + 8 * seg);
            const float4 hi4 = *reinterpret_cast<const float4*>(stg + i * C::STG_LD + 8 * seg + 4);
            float y[8] = {lo4.x, lo4.y, lo4.z, lo4.w, hi4.x, hi4.y, hi4.z, hi4.w};
            const uint32_t bw[4] = {bias.x, bias.y, bias.z, bias.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[2 * j] = __fmaf_rn(y[2 * j], sc, bf16_bits_to_f32(bw[j] & 0xFFFFu));
              y[2 * j + 1] = __fmaf_rn(y[2 * j + 1], sc, bf16_bits_to_f32(bw[j] >> 16));
            }
            const bool store = n_ok && tk < q.cnt;
            if (!p.gated) {
              activate<8, 1>(y, p.act);
              if (store) {
                if (p.out_f32) {
                  if (p.residual != nullptr) {
                    const float4* rp =
                        reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) + m * p.ld_res + n0);
                    const float4 u = rp[0], v = rp[1];
                    y[0] += u.x, y[1] += u.y, y[2] += u.z, y[3] += u.w;
                    y[4] += v.x, y[5] += v.y, y[6] += v.z, y[7] += v.w;
                  }
                  float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.D) + m * p.ld_d + n0);
                  __stcs(d, make_float4(y[0], y[1], y[2], y[3]));
                  __stcs(d + 1, make_float4(y[4], y[5], y[6], y[7]));
                } else {
                  if (p.residual != nullptr) {
                    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.residual) +
                                                                    m * p.ld_res + n0);
                    const uint32_t rw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                      y[2 * j] += bf16_bits_to_f32(rw[j] & 0xFFFFu);
                      y[2 * j + 1] += bf16_bits_to_f32(rw[j] >> 16);
                    }
                  }
                  __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.D) + m * p.ld_d + n0),
                         make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                    pack_bf16x2(y[6], y[7])));
                }
              }
            } else {
              activate<8, 2>(y, p.act);
              float z[4] = {y[0] * y[1], y[2] * y[3], y[4] * y[5], y[6] * y[7]};
              const int nh = n0 >> 1;
              if (store) {
                if (p.out_f32) {
                  if (p.residual != nullptr) {
                    const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) +
                                                                      m * p.ld_res + nh);
                    z[0] += u.x, z[1] += u.y, z[2] += u.z, z[3] += u.w;
                  }
                  __stcs(reinterpret_cast<float4*>(static_cast<float*>(p.D) + m * p.ld_d + nh),
                         make_float4(z[0], z[1], z[2], z[3]));
                } else {
                  if (p.residual != nullptr) {
                    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.residual) +
                                                                    m * p.ld_res + nh);
                    z[0] += bf16_bits_to_f32(v.x & 0xFFFFu), z[1] += bf16_bits_to_f32(v.x >> 16);
                    z[2] += bf16_bits_to_f32(v.y & 0xFFFFu), z[3] += bf16_bits_to_f32(v.y >> 16);
                  }
                  __stcs(reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.D) + m * p.ld_d + nh),
                         make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3])));
                }
              }
            }
          }
        }
      }
    }
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

template <int KIND, int CG>
int launch_fused(const DeviceInfo& dev, const FusedArgs& a, FusedParams p, cudaStream_t stream) {
  using C = FCfg<KIND, CG>;
  auto kernel = fused_gemm_kernel<KIND, CG>;
  static bool attr_set[64] = {};
  if (!attr_set[dev.id]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
      return launch_status();
    attr_set[dev.id] = true;
  }
  CUtensorMap tmW, tmX, tmXfull, tmSFW, tmSFX;
  int st;
  if ((st = encode_experts(&tmW, a.B, p.E, p.N, a.row_bytes, 128)) != BSP_OK) return st;
  if ((st = encode_operand(&tmX, a.A, p.M, a.row_bytes, C::X_BOX)) != BSP_OK) return st;
  if ((st = encode_operand(&tmXfull, a.A, p.M, a.row_bytes, C::X_ROWS)) != BSP_OK) return st;
  if ((st = encode_expert_scales(&tmSFW, a.sfB, p.E, ceil_div(p.N, 128), a.tiles_per_band, C::ATOMS)) != BSP_OK)
    return st;
  if ((st = encode_scales(&tmSFX, a.sfA, ceil_div(p.M, 128), a.tiles_per_band, C::ATOMS, 1)) != BSP_OK) return st;

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
  if (cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, tmXfull, tmSFW, tmSFX, p) != cudaSuccess) return launch_status();
  return launch_status();
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
  p.out_f32 = d_dtype == BSP_OUT_F32;
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
  if (ceil_div(M, E) > 64) return launch_fused<KIND, 2>(dev, a, p, stream);
  return launch_fused<KIND, 1>(dev, a, p, stream);
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
