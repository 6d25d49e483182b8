// linear_pair.cu -- the linear layer's products with enough output tiles to
// fill the GPU: 2-CTA (cta_group::2) tcgen05.mma, 256 x 256 (or 256 x 128)
// tiles, fp32 accumulators in TMEM, operands by TMA.
//
//   forward  y[t][n]  = act(sum_k x[t][k] W[k][n] + b_n) + res[t][n], and z before act
//   dx       dx[t][k] = sum_n dz[t][n] W[k][n]
//   dW       dW[k][n] = sum_t x[t][k] dz[t][n]
// In LinearArgs' terms, out[c][l]: the rows c are the MMA's M (A operand =
// LinearArgs::b), the columns l its N (B operand = LinearArgs::a); each operand
// is read as it lies (reduction-major or not) through the descriptor's major
// bit, and ragged ends read as zero by TMA and are clipped by its stores.
//
// What bounds it: the tensor pipe, fed at 32 KB of operands per CTA for 64
// reduction steps of a 256 x 256 tile -- half the traffic of two single-CTA
// 128 x 256 tiles, which the L2 could not carry (linear_split.cu on 16384 x 4096 x
// 14336: 598 TFLOP/s).
//
// Measured: 8192^3 703-710 us for either gradient (1.55 PFLOP/s; the tensor pipe is
// active in 98 % of the SMs' cycles, and the power cap sets the clock, 1.42 GHz),
// forward 713; 16384 x 4096 x 14336 1230 us bare, 1300 with bias and z.  An operand that
// lies along the M or N side comes in one 3-D copy a stage: as two copies it cost
// dW 4 %.  Short reductions are bound by the epilogue: 8192 x 512 x 4096 31 us
// bare (floor 21), 35 with bias, 60 with bias, residual and z.
//
// A pair of CTAs owns a tile: each loads its own 128 rows of A and half of the
// columns of B; the leader issues the MMAs for both.  Persistent pairs stride
// through the tiles, two accumulators, so a tile's epilogue overlaps the next
// tile's products.  Warps: 0 = TMA, 1 = MMA (leader) and TMEM, then the
// epilogue: 4 warps with a ring of 6 stages for the gradients, whose epilogue
// only rounds; 8 warps with 5 stages for the forward, two per TMEM lane
// quarter on half of the columns each, so that bias, activation and residual
// stay hidden behind shorter reductions too.  (Sixteen warps in two groups on
// alternate tiles gained 10-25 % at reductions up to 256 and lost 3-7 % from 1024
// on, with the residual most: not kept.)
//
// Epilogue rows leave as 32 x 32 boxes through shared memory by TMA (a
// lane writes its own row, conflict-free under the 64-byte swizzle); the
// residual's boxes come in the same way, up to three chunks ahead (while the
// tile's products still run), into the box that the chunk's y then overwrites.
#include "linear.cuh"
#include "pair_pipe.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int BM = 256;
constexpr int BM_CTA = 128;
constexpr int BK = 64;
constexpr int kABytes = BM_CTA * BK * 2;
constexpr int kBBytes = BK * 128 * 2;        // this CTA's half of BN <= 256
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kAtomBytes = BK * 64 * 2;
constexpr int kTmemCols = 512;
constexpr int kAccCols = 256;
constexpr int kBoxBytes = 32 * 32 * 2;
constexpr int kWarpBytes = 4 * kBoxBytes;    // an epilogue warp's boxes: four chunks of y, or two of (y, z)
constexpr long long kL2GroupBudget = 48ll << 20;

template <bool FULL>  // FULL: the forward's epilogue; else only a rounding
struct Cfg {
  static constexpr int kStages = FULL ? 5 : 6;
  static constexpr int kEpi = FULL ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpi;
};

template <int STAGES, int EPI>
struct __align__(8) PairShared {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint64_t rbar[EPI][4];  // an epilogue warp's residual box landed, per slot
  PairDrain pd;
  uint32_t tmem_base;
  int abort_flag;
};

struct Maps {
  CUtensorMap a, b, y, z, res;
};

// Tiles in blocks of gm x gn (M x N), M fastest inside a block (as the grouped
// GEMM's raster): all of M when its panels fit the L2 budget, else about a
// square wave.
struct Raster {
  int mt, nt, gm, gn;
  __device__ __forceinline__ void decode(int tile, int& m, int& n) const {
    const int bm = tile / (gm * nt), rem = tile - bm * gm * nt;
    const int gmb = min(gm, mt - bm * gm);
    const int bn = rem / (gmb * gn), rem2 = rem - bn * gmb * gn;
    n = bn * gn + rem2 / gmb;
    m = bm * gm + rem2 % gmb;
  }
};

__device__ __forceinline__ uint32_t sw64(int row, int unit) {
  return static_cast<uint32_t>(row * 64 + ((unit ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ void box_put(uint8_t* box, int lane, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(box + sw64(lane, j)) =
        make_uint4(pack2(v[8 * j], v[8 * j + 1]), pack2(v[8 * j + 2], v[8 * j + 3]),
                   pack2(v[8 * j + 4], v[8 * j + 5]), pack2(v[8 * j + 6], v[8 * j + 7]));
}

__device__ __forceinline__ void box_add(const uint8_t* box, int lane, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float r[8];
    unpack8(*reinterpret_cast<const uint4*>(box + sw64(lane, j)), r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * j + i] += r[i];
  }
}

// This CTA's half of one stage: 128 rows of the M side and half of the N side.
template <bool AMN, bool BMN>
__device__ __forceinline__ void load_operands(const CUtensorMap& ma, const CUtensorMap& mb, uint8_t* sA, uint8_t* sB,
                                              uint32_t bar, int m0, int n0, int k, int half_bn, const LinearArgs& a) {
  if (AMN && a.b_3d) {
    tma_load_3d_pair(sA, &ma, bar, 0, k, m0 >> 6);
  } else if (AMN) {
    tma_load_2d_pair(sA, &ma, bar, m0, k);
    tma_load_2d_pair(sA + kAtomBytes, &ma, bar, m0 + 64, k);
  } else {
    tma_load_2d_pair(sA, &ma, bar, k, m0);
  }
  if (BMN && a.a_3d) {
    tma_load_3d_pair(sB, &mb, bar, 0, k, n0 >> 6);
  } else if (BMN) {
    for (int j = 0; j < half_bn / 64; ++j) tma_load_2d_pair(sB + j * kAtomBytes, &mb, bar, n0 + j * 64, k);
  } else {
    tma_load_2d_pair(sB, &mb, bar, k, n0);
  }
}

template <bool AMN, bool BMN>
__device__ __forceinline__ void mma_stage(uint32_t d_tmem, uint32_t aA, uint32_t idesc, bool accumulate) {
  const uint32_t aB = aA + kABytes;
#pragma unroll
  for (int kk = 0; kk < BK / 16; ++kk)
    umma_bf16_pair(d_tmem,
                   AMN ? smem_desc_sw128(aA + kk * 2048, kAtomBytes, 1024) : smem_desc_sw128(aA + kk * 32, 16, 1024),
                   BMN ? smem_desc_sw128(aB + kk * 2048, kAtomBytes, 1024) : smem_desc_sw128(aB + kk * 32, 16, 1024),
                   idesc, accumulate || kk != 0 ? 1u : 0u);
}

// AMN / BMN: the M side's (N side's) index runs along its rows in memory.
template <bool AMN, bool BMN, bool FULL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<FULL>::kThreads, 1)
    linear_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ LinearArgs a) {
  constexpr int STAGES = Cfg<FULL>::kStages, EPI = Cfg<FULL>::kEpi;
  using Shared = PairShared<STAGES, EPI>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* boxes = smem + STAGES * kStageBytes;
  Shared& sh = *reinterpret_cast<Shared*>(boxes + EPI * kWarpBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int bn = a.bn, half_bn = bn / 2;
  const int kblocks = (a.red + BK - 1) / BK;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.tfull[b], 1);
      mbar_init(&sh.tempty[b], 2 * EPI);
    }
    mbar_init(&sh.drain, 1);
    for (int w = 0; w < EPI; ++w) {
      for (int i = 0; i < 4; ++i) mbar_init(&sh.rbar[w][i], 1);
    }
    pair_drain_init(sh.pd);
    sh.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&maps.a);
    tma_prefetch_map(&maps.b);
    tma_prefetch_map(&maps.y);
  }
  if (warp == 1) {
    tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem_base = sh.tmem_base;
  volatile int* abort_flag = &sh.abort_flag;
  const uint64_t wait_ns = wait_limit_ns(a.wait_ctl);
  const uint32_t peer_abort = map_to_cta(smem_addr(&sh.abort_flag), rank ^ 1u);

  Raster ra;
  ra.mt = (a.C + BM - 1) / BM;
  ra.nt = (a.L + bn - 1) / bn;
  ra.gm = ra.mt;
  ra.gn = ra.nt;
  if (static_cast<long long>(ra.mt) * BM * a.red * 2 > kL2GroupBudget) {
    const int gm = static_cast<int>(sqrtf(static_cast<float>(npairs) * bn / BM));
    ra.gm = max(1, min(gm, ra.mt));
    ra.gn = max(1, min(npairs / ra.gm, ra.nt));
  }
  const int total = ra.mt * ra.nt;

  if (warp == 0) {
    // ================= TMA
    if (lane == 0) {
      const uint32_t full_leader0 = map_to_cta(smem_addr(&sh.full[0]), 0);
      const uint32_t tx_pair = 2u * (kABytes + static_cast<uint32_t>(half_bn) * BK * 2u);
      uint32_t it = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < total; tile += npairs) {
        int m, n;
        ra.decode(tile, m, n);
        const int m0 = m * BM + static_cast<int>(rank) * BM_CTA, n0 = n * bn + static_cast<int>(rank) * half_bn;
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&sh.empty[s], ((it / STAGES) & 1u) ^ 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns, false,
                         peer_abort)) {
            ok = false;
            break;
          }
          uint8_t* sA = smem + s * kStageBytes;
          uint8_t* sB = sA + kABytes;
          const uint32_t bar = full_leader0 + static_cast<uint32_t>(s) * 8u;
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], tx_pair);
          load_operands<AMN, BMN>(maps.a, maps.b, sA, sB, bar, m0, n0, kb * BK, half_bn, a);
        }
      }
      // no copy into either CTA is in flight when it exits, whatever stopped the loop
      pair_producer_drain<STAGES>(sh.pd, sh.full, it, rank, tx_pair / 2u, a.err);
    }
  } else if (warp == 1) {
    // ================= MMA (leader)
    if (rank == 0) {
      const bool issuer = elect_one();
      const uint32_t idesc = umma_idesc_bf16(BM, bn, BMN ? 1u : 0u, AMN ? 1u : 0u);
      uint32_t it = 0, tcount = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < total; tile += npairs, ++tcount) {
        const uint32_t buf = tcount & 1u;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sh.tempty[buf], ((tcount >> 1) & 1u) ^ 1u, abort_flag, a.err,
                                               MOE_DEVERR_TIMEOUT, wait_ns, true, peer_abort)))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * kAccCols;
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sh.full[s], (it / STAGES) & 1u, abort_flag, a.err,
                                                 MOE_DEVERR_TIMEOUT, wait_ns, false, peer_abort))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (issuer) {
            mma_stage<AMN, BMN>(d_tmem, smem_addr(smem + s * kStageBytes), idesc, kb != 0);
            umma_commit_pair_mc(&sh.empty[s], 0x3);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (issuer) umma_commit_pair_mc(&sh.tfull[buf], 0x3);
        __syncwarp();
      }
      if (issuer) umma_commit_pair(&sh.drain);
      volatile int no_abort = 0;
      mbar_wait(&sh.drain, 0, &no_abort, a.err, MOE_DEVERR_TIMEOUT, kWaitTimeoutNs);
    }
  } else {
    // ================= epilogue
    const int q = warp & 3, w = warp - 2;
    uint8_t* my = boxes + w * kWarpBytes;
    const int span = EPI == 8 ? half_bn : bn, c_lo = EPI == 8 ? (w >> 2) * half_bn : 0;
    const uint32_t tempty_leader0 = map_to_cta(smem_addr(&sh.tempty[0]), 0);
    const bool has_bias = FULL && a.bias != nullptr, bias_wide = (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0;
    const bool has_res = FULL && a.residual != nullptr, has_z = FULL && a.z != nullptr;
    // chunk n of this warp uses slot n % slots; a residual is loaded `slots` - 1 chunks ahead of its use
    const uint32_t slots = has_z ? 2u : 4u, slot_bytes = kWarpBytes / slots;
    uint32_t tcount = 0, n = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < total; tile += npairs, ++tcount) {
      int tm, tn;
      ra.decode(tile, tm, tn);
      const uint32_t buf = tcount & 1u;
      const int row0 = tm * BM + static_cast<int>(rank) * BM_CTA + q * 32;
      const int col0 = tn * bn + c_lo;
      // chunks with anything to write; the others are outside the matrix
      const int chunks = row0 < a.C && col0 < a.L ? (min(span, a.L - col0) + 31) / 32 : 0;
      int issued = 0;  // residual boxes of this tile under way or landed
      auto load_res = [&](int upto) {
        for (; issued < min(upto, chunks); ++issued) {
          const uint32_t slot = (n + issued) % slots;
          if (lane == 0) {
            bulk_wait_group_read0();  // the slot's previous store has read it
            mbar_arrive_expect_tx(&sh.rbar[w][slot], kBoxBytes);
            tma_load_2d(my + slot * slot_bytes, &maps.res, &sh.rbar[w][slot], col0 + issued * 32, row0);
          }
        }
      };
      const uint32_t n0 = n;
      auto res_wait = [&](int i, volatile int* stop, uint64_t limit) {  // lane 0
        return mbar_wait(&sh.rbar[w][(n0 + i) % slots], ((n0 + i) / slots) & 1u, stop, a.err, MOE_DEVERR_TIMEOUT, limit,
                         false, peer_abort);
      };
      if (has_res) load_res(static_cast<int>(slots) - 1);
      // the next chunk's bias, loaded a chunk ahead from addresses that all lanes share
      float bias[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) bias[j] = 0.f;
      auto load_bias = [&](int col) {
        if (bias_wide) {  // whole groups of 8 columns lie inside or outside the matrix
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            uint4 b = make_uint4(0u, 0u, 0u, 0u);
            if (col + j < a.L) b = ld_global16(a.bias + col + j);
            bias[j] = __uint_as_float(b.x);
            bias[j + 1] = __uint_as_float(b.y);
            bias[j + 2] = __uint_as_float(b.z);
            bias[j + 3] = __uint_as_float(b.w);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) bias[j] = col + j < a.L ? ld_global(a.bias + col + j) : 0.f;
        }
      };
      if (has_bias && chunks > 0) load_bias(col0);
      bool got = true;
      if (lane == 0)
        got = mbar_wait(&sh.tfull[buf], (tcount >> 1) & 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns, false,
                        peer_abort);
      ok = warp_take(got);
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kAccCols + c_lo;
      int i = 0;
      uint32_t u[32];  // the next chunk's sums, on their way while this one is worked on
      if (ok && chunks > 0) tmem_ld_32x32b_x32(taddr, u);
#pragma unroll 1
      for (; ok && i < chunks; ++i) {
        const int col = col0 + i * 32;
        uint8_t* box = my + (n0 + i) % slots * slot_bytes;
        if (has_res) {
          got = true;
          if (lane == 0) got = res_wait(i, abort_flag, wait_ns);
          ok = warp_take(got);
        } else {
          // the store that used this slot last has read it
          if (lane == 0) bulk_wait_group_read_allow(static_cast<int>(slots) - 1);
          __syncwarp();
        }
        tmem_ld_wait();
        if (!ok) break;
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
        if (FULL) {
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            halves(add2(pair_of(v[j], v[j + 1]), pair_of(bias[j], bias[j + 1])), v[j], v[j + 1]);
        }
        if (i + 1 < chunks) {
          tmem_ld_32x32b_x32(taddr + (i + 1) * 32, u);
          if (has_bias) load_bias(col + 32);
        }
        if (has_z) box_put(box + kBoxBytes, lane, v);
        if (FULL) act_apply(v, a.act);
        if (has_res) box_add(box, lane, v);
        box_put(box, lane, v);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&maps.y, box, col, row0);
          if (has_z) tma_store_2d(&maps.z, box + kBoxBytes, col, row0);
          bulk_commit_group();
        }
        if (has_res) load_res(i + static_cast<int>(slots));
      }
      if (!ok && has_res && lane == 0) {  // let the residual boxes in flight land (default limit)
        volatile int no_abort = 0;
        for (; i < issued; ++i) res_wait(i, &no_abort, kWaitTimeoutNs);
      }
      n += chunks;
      tc_fence_before();
      __syncwarp();
      if (!ok) break;
      if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader0 + buf * 8u);
    }
    // the stores have completed before the CTA's shared memory goes away
    if (lane == 0) bulk_wait_group0();
  }

  griddep_launch_dependents();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

// ---- few tiles, long reductions: a tile's reduction split over the S pairs of a
// cluster of 2 S CTAs, one tile a cluster.  Each CTA leaves its 128 rows of fp32
// sums in its idle ring (row by row, 16 bytes of padding against bank
// conflicts); pair p then reads all pairs' columns [p per, (p + 1) per) of its
// CTAs' rows through distributed shared memory, adds them in pair order and
// finishes them.
constexpr int kSplitStages = 6;
constexpr int kSplitThreads = 320;   // TMA, MMA, 8 warps that read TMEM; all of them finish

struct __align__(8) SplitPairShared {
  uint64_t full[kSplitStages], empty[kSplitStages];
  uint64_t tfull, drain;
  PairDrain pd;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t kSplitSmem = 1024 + kSplitStages * kStageBytes + sizeof(SplitPairShared);
static_assert(128 * (256 + 4) * 4 <= kSplitStages * kStageBytes, "the sums exceed the idle ring");

template <bool AMN, bool BMN>
__global__ void __launch_bounds__(kSplitThreads, 1)
    linear_pair_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                             const __grid_constant__ LinearArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  SplitPairShared& sh = *reinterpret_cast<SplitPairShared*>(smem + kSplitStages * kStageBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = a.pair_split;
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, base = crank & ~1u;
  const int p = static_cast<int>(crank >> 1);
  const int tile = blockIdx.x / (2 * S), mt = (a.C + BM - 1) / BM;
  const int bn = a.bn, half_bn = bn / 2;
  const int m0 = tile % mt * BM + static_cast<int>(rank) * BM_CTA, t0 = tile / mt * bn;
  const int kb = (a.red + BK - 1) / BK, k_lo = kb * p / S, k_hi = kb * (p + 1) / S;

  if (tid == 0) {
    for (int s = 0; s < kSplitStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.tfull, 1);
    mbar_init(&sh.drain, 1);
    pair_drain_init(sh.pd);
    sh.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == 1) {
    tmem_alloc_pair(&sh.tmem_base, 256);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem_base = sh.tmem_base;
  volatile int* abort_flag = &sh.abort_flag;
  const uint64_t wait_ns = wait_limit_ns(a.wait_ctl);
  const uint32_t peer_abort = map_to_cta(smem_addr(&sh.abort_flag), crank ^ 1u);
  griddep_launch_dependents();  // all CTAs are running by the time it takes effect

  const uint32_t tx_pair = 2u * (kABytes + static_cast<uint32_t>(half_bn) * BK * 2u);
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full_leader0 = map_to_cta(smem_addr(&sh.full[0]), base);
      const int n0 = t0 + static_cast<int>(rank) * half_bn;
      uint32_t it = 0;
      for (int k = k_lo; k < k_hi; ++k, ++it) {
        const int s = it % kSplitStages;
        if (!mbar_wait(&sh.empty[s], ((it / kSplitStages) & 1u) ^ 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns,
                       false, peer_abort))
          break;
        uint8_t* sA = smem + s * kStageBytes;
        uint8_t* sB = sA + kABytes;
        const uint32_t bar = full_leader0 + static_cast<uint32_t>(s) * 8u;
        if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], tx_pair);
        load_operands<AMN, BMN>(map_a, map_b, sA, sB, bar, m0, n0, k * BK, half_bn, a);
      }
      pair_producer_drain<kSplitStages>(sh.pd, sh.full, it, rank, tx_pair / 2u, a.err, base);
    }
  } else if (warp == 1 && rank == 0) {
    const bool issuer = elect_one();
    const uint32_t idesc = umma_idesc_bf16(BM, bn, BMN ? 1u : 0u, AMN ? 1u : 0u);
    const uint16_t both = static_cast<uint16_t>(0x3u << base);
    uint32_t it = 0;
    for (int k = k_lo; k < k_hi; ++k, ++it) {
      const int s = it % kSplitStages;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sh.full[s], (it / kSplitStages) & 1u, abort_flag, a.err,
                                             MOE_DEVERR_TIMEOUT, wait_ns, false, peer_abort)))
        break;
      tc_fence_after();
      if (issuer) {
        mma_stage<AMN, BMN>(tmem_base, smem_addr(smem + s * kStageBytes), idesc, it > 0);
        umma_commit_pair_mc(&sh.empty[s], both);
      }
      __syncwarp();
    }
    // also after a wait that gave up: the accumulator's readers go on (to undefined sums)
    if (issuer) {
      umma_commit_pair_mc(&sh.tfull, both);
      umma_commit_pair(&sh.drain);
    }
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait(&sh.drain, 0, &no_abort, a.err, MOE_DEVERR_TIMEOUT, kWaitTimeoutNs);
  }
  __syncwarp();
  const int pitch = (bn + 4) * 4;  // bytes of a row of sums
  const uint32_t mine = smem_addr(smem);
  volatile int no_abort = 0;
  if (lane == 0) mbar_wait(&sh.tfull, 0, &no_abort, a.err, MOE_DEVERR_TIMEOUT, kWaitTimeoutNs);
  __syncthreads();  // the loads have landed (warp 0) and the products are done
  tc_fence_after();
  if (warp >= 2) {
    const int q = warp & 3, row = q * 32 + lane, col0 = (warp - 2) / 4 * half_bn;
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + col0;
    uint8_t* dst = smem + row * pitch + col0 * 4;
    for (int j0 = 0; j0 < half_bn; j0 += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(taddr + j0, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(dst + (j0 + 4 * j) * 4) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    tc_fence_before();
  }
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 256);
  }
  const int per = (bn / 4 + S - 1) / S, first = p * per, nv = min(per, bn / 4 - first);  // groups of 4 columns
  const int items = nv > 0 ? BM_CTA * nv : 0;
  constexpr int U = 4;
  for (int i = tid; i < items; i += U * kSplitThreads) {
    int c[U], l[U];
    bool in[U];
    uint32_t from[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int iu = i + u * kSplitThreads, row = iu / nv, vec = first + iu - row * nv;
      c[u] = m0 + row;
      l[u] = t0 + vec * 4;
      in[u] = iu < items && c[u] < a.C && l[u] < a.L;
      from[u] = mine + static_cast<uint32_t>(row * pitch + vec * 16);
    }
    finish_groups<U>(a, c, l, in, from, S, rank, 2u);
  }
  cluster_sync();  // nobody leaves while its sums are being read
}

template <bool FULL>
constexpr size_t smem_of() {
  return 1024 + static_cast<size_t>(Cfg<FULL>::kStages) * kStageBytes + Cfg<FULL>::kEpi * kWarpBytes +
         sizeof(PairShared<Cfg<FULL>::kStages, Cfg<FULL>::kEpi>);
}
static_assert(smem_of<true>() <= 232448 && smem_of<false>() <= 232448, "shared memory above the per-block opt-in limit");

template <bool AMN, bool BMN, bool FULL>
cudaError_t prepare_t() {
  return cudaFuncSetAttribute(linear_pair_kernel<AMN, BMN, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(smem_of<FULL>()));
}

template <bool AMN, bool BMN, bool FULL>
cudaError_t launch_t(const Maps& m, const LinearArgs& a, int grid, cudaStream_t s) {
  return launch_pdl(linear_pair_kernel<AMN, BMN, FULL>, dim3(grid), dim3(Cfg<FULL>::kThreads), smem_of<FULL>(), s, m, a);
}

template <bool AMN, bool BMN>
cudaError_t launch_split_t(const CUtensorMap& mma, const CUtensorMap& mmb, const LinearArgs& a, int tiles, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * 2 * a.pair_split));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = kSplitSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(2 * a.pair_split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_pair_split_kernel<AMN, BMN>, mma, mmb, a);
}

template <bool AMN, bool BMN>
cudaError_t prepare_split_t() {
  return cudaFuncSetAttribute(linear_pair_split_kernel<AMN, BMN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kSplitSmem));
}

}  // namespace

cudaError_t prepare_linear_pair() {
  cudaError_t e = prepare_t<false, true, true>();
  if (e == cudaSuccess) e = prepare_t<false, false, false>();
  if (e == cudaSuccess) e = prepare_t<true, true, false>();
  if (e == cudaSuccess) e = prepare_split_t<false, true>();
  if (e == cudaSuccess) e = prepare_split_t<false, false>();
  if (e == cudaSuccess) e = prepare_split_t<true, true>();
  return e;
}

cudaError_t linear_pair_slots(LinearSlots* slots) {
  for (int S = 1; S <= 4; ++S) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * S));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = kSplitSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(2 * S);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&slots->pairs[S], linear_pair_split_kernel<false, true>, &cfg);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Tile width and split of a product, and how long it should take (us), fitted to
// 935 timings over the 261 products of linear_split.cu's model (11 % rms off near
// the best).  64 reduction steps of a tile take 0.374 us 256 wide and 0.284 us 128
// wide (a step's barriers and commit bound the narrow tile, so it pays only where
// the wide one leaves SMs idle); a persistent tile 1.9 or 1.1 us more than its
// reduction; a wave of split tiles 7.8 us to fill, exchange and finish, 3.4 more
// for 100 pairs at it, and 1 for each pair beyond two that shares a wide tile;
// nothing is faster than its bytes.
double plan_linear_pair(LinearArgs& a, const LinearSlots& slots) {
  const int kb = (a.red + BK - 1) / BK;
  const double out = static_cast<double>(a.L) * a.C * (1 + (a.z != nullptr) + (a.residual != nullptr));
  const double mb = 2e-6 * (static_cast<double>(a.red) * (static_cast<double>(a.L) + a.C) + out);
  double best = 0.0;
  a.pair_bn = 0;
  for (int bn = 128; bn <= 256; bn *= 2) {
    const long long tiles = static_cast<long long>((a.C + BM - 1) / BM) * ((a.L + bn - 1) / bn);
    const double step = bn == 256 ? 0.374 : 0.284;
    for (int S = 1; S <= 4 && S <= kb; ++S) {
      if (slots.pairs[S] == 0 || (S > 1 && tiles > 4 * slots.pairs[S])) continue;
      const double waves = static_cast<double>((tiles + slots.pairs[S] - 1) / slots.pairs[S]);
      const double reduction = (kb + S - 1) / S * step;
      const double pairs = static_cast<double>(tiles < slots.pairs[S] ? tiles : slots.pairs[S]) * S;
      double t = S == 1 ? 4.2 + waves * (reduction + (bn == 256 ? 1.88 : 1.08))
                        : waves * (7.8 + (bn == 256 ? 1.03 * (S - 2) : 0.0) + 0.034 * pairs + reduction);
      t = fmax(t, mb / 6.5 + 4.9);
      if (a.pair_bn == 0 || t < best) {
        best = t;
        a.pair_bn = bn;
        a.pair_split = S;
      }
    }
  }
  return best;
}

cudaError_t launch_linear_pair(const LinearArgs& a, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& my,
                               const CUtensorMap& mz, const CUtensorMap& mr, int grid, cudaStream_t s) {
  const long long tiles = static_cast<long long>((a.C + BM - 1) / BM) * ((a.L + a.bn - 1) / a.bn);
  if (a.pair_split > 1) {
    const int n = static_cast<int>(tiles);
    if (!a.b_mn && a.a_mn) return launch_split_t<false, true>(mb, ma, a, n, s);
    if (!a.b_mn) return launch_split_t<false, false>(mb, ma, a, n, s);
    return launch_split_t<true, true>(mb, ma, a, n, s);
  }
  const Maps m{mb, ma, my, mz, mr};
  if (2 * tiles < grid) grid = static_cast<int>(2 * tiles);
  if (!a.b_mn && a.a_mn) return launch_t<false, true, true>(m, a, grid, s);
  if (!a.b_mn) return launch_t<false, false, false>(m, a, grid, s);
  return launch_t<true, true, false>(m, a, grid, s);
}

}  // namespace moe
