// linear_split.cu -- the linear layer's products when they have too few output
// tiles to fill the GPU with 256 x 256 pair tiles: a decode step's rows, small
// batches, gradients of narrow layers.
//
//   forward  y[t][n]  = sum_k x[t][k] W[k][n]       lanes n, columns t
//   dx       dx[t][k] = sum_n dz[t][n] W[k][n]      lanes k, columns t
//   dW       dW[k][n] = sum_t x[t][k] dz[t][n]      lanes n, columns k
//
// All three are out[c][l] = sum_r A(l, r) B(c, r) with `lanes` l contiguous in
// memory: l is the M side of the tcgen05.mma (128 TMEM lanes) and c its N side,
// so a few rows of x cost a few MMA columns and not a padded 128-row tile.  A
// and B are read as they lie: reduction-major or the other way, by the
// descriptors' major bit.
//
// What bounds it: at few columns the bytes of W, otherwise the loads of both
// operands.  A tile has 128 lanes x BN <= 256 columns; when tiles are fewer
// than SMs, the reduction of a tile is split over the S CTAs of a cluster.  Each
// CTA runs its part of the reduction through its own TMA ring and TMEM
// accumulator and leaves its fp32 sums in its shared memory; CTA q then reads
// every CTA's columns [BN q/S, BN (q+1)/S) through distributed shared memory,
// adds them in rank order, applies the epilogue and stores.  No workspace, no
// counters, and a fixed order of every sum.
//
// Measured (device time in a graph, by the GPU and its clock): one row of 4096 x 4096
// 8.3-10.2 us (33.6 MB of W: 5.1 us at a copy's rate; the rest is launch, first loads
// and exchange), 61 rows of 1000 x 2056 6.7-7.9 us, 700 rows of 4096 x 1024 14.0-16.5 us
// (360-420 TFLOP/s).
//
// Warps: 0 = TMA, 1 = MMA issue and TMEM, 2-5 = TMEM to shared memory, then all
// of them the epilogue, 4 lanes (8 bytes of output) a thread.
#include <cmath>
#include <type_traits>

#include "linear.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kLanes = 128;
constexpr int kABytes = kLanes * 64 * 2;  // 16 KB: 128 lanes x 64 reduction
constexpr int kAtom = 64 * 64 * 2;
constexpr int kMaxStages = 12;
constexpr int kThreads = 192;

struct __align__(8) SplitShared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// A_MN: A's lanes are contiguous in memory (else its reduction); B_MN likewise
// for B's columns.
template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kThreads)
    linear_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                        const __grid_constant__ LinearArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kABytes + a.bn * 128;
  SplitShared& sh = *reinterpret_cast<SplitShared*>(ring + a.ring_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = a.split;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile = blockIdx.x / S;
  const int l0 = tile % a.tiles_l * kLanes, c0 = tile / a.tiles_l * a.bn;  // neighbours share B's tile
  const int kb = (a.red + 63) / 64;
  const int k_lo = static_cast<int>(static_cast<long long>(kb) * rank / S);
  const int k_hi = static_cast<int>(static_cast<long long>(kb) * (rank + 1) / S);
  volatile int* abort_flag = &sh.abort_flag;

  if (tid == 0) {
    sh.abort_flag = 0;
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.done, 1);
    fence_mbar_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem_base, a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem_base = sh.tmem_base;
  const uint64_t wait_ns = wait_limit_ns(a.wait_ctl);
  griddep_launch_dependents();  // all CTAs are running by the time it takes effect

  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      for (int k = k_lo; k < k_hi; ++k, ++it) {
        const int s = it % a.stages;
        if (!mbar_wait(&sh.empty[s], ((it / a.stages) & 1u) ^ 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns))
          break;
        uint8_t* sA = ring + s * stage_bytes;
        uint8_t* sB = sA + kABytes;
        mbar_arrive_expect_tx(&sh.full[s], stage_bytes);
        if (A_MN && a.a_3d) {
          tma_load_3d(sA, &map_a, &sh.full[s], 0, k * 64, l0 >> 6);
        } else if (A_MN) {
          tma_load_2d(sA, &map_a, &sh.full[s], l0, k * 64);
          tma_load_2d(sA + kAtom, &map_a, &sh.full[s], l0 + 64, k * 64);
        } else {
          tma_load_2d(sA, &map_a, &sh.full[s], k * 64, l0);
        }
        if (B_MN && a.b_3d) {
          tma_load_3d(sB, &map_b, &sh.full[s], 0, k * 64, c0 >> 6);
        } else if (B_MN) {
          for (int j = 0; j < a.bn / 64; ++j) tma_load_2d(sB + j * kAtom, &map_b, &sh.full[s], c0 + j * 64, k * 64);
        } else {
          tma_load_2d(sB, &map_b, &sh.full[s], k * 64, c0);
        }
      }
      // the copies in flight land before the ring is used again (default limit)
      volatile int no_abort = 0;
      for (uint32_t j = it > static_cast<uint32_t>(a.stages) ? it - a.stages : 0; j < it; ++j)
        mbar_wait(&sh.full[j % a.stages], (j / a.stages) & 1u, &no_abort, a.err, MOE_DEVERR_TIMEOUT, kWaitTimeoutNs);
    }
  } else if (warp == 1) {
    {
      const bool issuer = elect_one();
      const uint32_t idesc = umma_idesc_bf16(kLanes, a.bn, B_MN ? 1u : 0u, A_MN ? 1u : 0u);
      uint32_t it = 0;
      for (int k = k_lo; k < k_hi; ++k, ++it) {
        const int s = it % a.stages;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sh.full[s], (it / a.stages) & 1u, abort_flag, a.err,
                                               MOE_DEVERR_TIMEOUT, wait_ns)))
          break;
        tc_fence_after();
        const uint32_t aA = smem_addr(ring + s * stage_bytes), aB = aA + kABytes;
        if (issuer) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem_base,
                      A_MN ? smem_desc_sw128(aA + kk * 2048, kAtom, 1024) : smem_desc_sw128(aA + kk * 32, 16, 1024),
                      B_MN ? smem_desc_sw128(aB + kk * 2048, kAtom, 1024) : smem_desc_sw128(aB + kk * 32, 16, 1024),
                      idesc, it > 0 || kk > 0 ? 1u : 0u);
          umma_commit(&sh.empty[s]);
        }
        __syncwarp();
      }
      if (issuer) umma_commit(&sh.done);
      __syncwarp();
    }
  }
  // every thread: the MMAs issued are done (also after a wait that gave up; default limit)
  volatile int no_abort = 0;
  if (lane == 0) ok = mbar_wait(&sh.done, 0, &no_abort, a.err, MOE_DEVERR_TIMEOUT, kWaitTimeoutNs);
  ok = __syncthreads_and(ok && !*abort_flag) != 0;
  tc_fence_after();

  // ---- this CTA's partial sums, [column][lane] fp32, into its idle ring
  const uint32_t mine = smem_addr(ring);
  if (warp >= 2) {
    const int q = warp & 3, col = q * 32 + lane;
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    for (int j0 = 0; j0 < a.bn; j0 += 16) {
      uint32_t v[16];
      tmem_ld16(taddr + j0, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j)
        *reinterpret_cast<uint32_t*>(ring + ((j0 + j) * kLanes + col) * 4) = v[j];
    }
    tc_fence_before();
  }
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, a.tmem_cols);
  }

  // ---- epilogue of this rank's columns: a warp a column, 4 lanes a thread, the
  // ranks' sums added in rank order
  const int first = rank * a.per, items = ok ? min(a.per, a.bn - first) * (kLanes / 4) : 0;
  auto finish = [&](auto groups) {  // groups a thread at a time
    constexpr int U = decltype(groups)::value;
    for (int i = tid; i < items; i += U * kThreads) {
      int c[U], l[U];
      bool in[U];
      uint32_t from[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int iu = i + u * kThreads, at = first + iu / (kLanes / 4), lv = (iu % (kLanes / 4)) * 4;
        c[u] = c0 + at;
        l[u] = l0 + lv;
        in[u] = iu < items && c[u] < a.C && l[u] < a.L;
        from[u] = mine + static_cast<uint32_t>((at * kLanes + lv) * 4);
      }
      finish_groups<U>(a, c, l, in, from, S, 0u, 1u);
    }
  };
  // with few groups the code to fetch is what counts, with many the loads under way: one against two
  // groups a thread 8.3 and 8.8 us for one row of 4096 x 4096 (2 columns a rank), 10.1 and 10.8 for dx of
  // 157 x 1056 x 2328 (10 columns), 12.2 and 12.6 at 16 columns (128 x 4096 x 4096); but 14.4 and 14.0 at 22
  // (700 x 4096 x 1024), 7.6 and 7.1 at 27 (303 x 464 x 1288), 15.0 and 13.4 at 59 (523 x 1912 x 1704).
  // (Four a thread: 10.3 us for the one row.)
  if (items <= 2 * kThreads)
    finish(std::integral_constant<int, 1>{});
  else
    finish(std::integral_constant<int, 2>{});
  cluster_sync();  // nobody leaves while its sums are being read
}

template <bool A_MN, bool B_MN>
cudaError_t launch_t(const LinearArgs& a, const CUtensorMap& ma, const CUtensorMap& mb, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.tiles_l * a.tiles_c * a.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_split_kernel<A_MN, B_MN>, ma, mb, a);
}

__global__ void __launch_bounds__(kThreads) occupancy_stand_in() {}

constexpr int kSmemMax = 232448;
constexpr int kHalfSmem = 110 * 1024;  // two CTAs a SM

}  // namespace

template <bool A_MN, bool B_MN>
static cudaError_t prepare_t() {
  cudaError_t e = cudaFuncSetAttribute(linear_split_kernel<A_MN, B_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemMax);
  // the whole SM's memory as shared memory, so that two CTAs with half of it fit
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(linear_split_kernel<A_MN, B_MN>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  return e;
}

cudaError_t prepare_linear_split() {
  cudaError_t e = prepare_t<true, false>();
  if (e == cudaSuccess) e = prepare_t<false, false>();
  if (e == cudaSuccess) e = prepare_t<true, true>();
  return e;
}

// Tile and split of a product, and how long it should take (us).  The model is
// fitted to 1427 timings of column tile and split over 261 products (9.5 % rms off
// near the best; with linear_pair.cu's, the choice is on average 1.3 % slower
// than the best one measured).  A wave of CTAs takes 4.8 us to start and finish,
// 1.8 for 100 columns of epilogue, nearly as much again where SMs hold two CTAs,
// and 0.11 for the exchange of 100 columns with each further rank; its reduction, a
// CTA's own loads (79 GB/s with half an SM's shared memory, 72 beside another CTA, 94 with all) and its
// share of the HBM's rate together, or the L2's rate (16.4 TB/s).
double plan_linear_split(LinearArgs& a, const LinearSlots& slots) {
  const int kb = (a.red + 63) / 64;
  const int granule = a.b_mn ? 64 : 16;
  a.tiles_l = (a.L + kLanes - 1) / kLanes;
  const double unique = 2.0 * a.red * (static_cast<double>(a.L) + a.C) * 1e-6;  // MB
  double best = 0.0;
  a.split = 0;
  for (int nt = (a.C + 255) / 256; nt <= (a.C + 255) / 256 * 4; nt *= 2) {
    const int bn = ((a.C + nt - 1) / nt + granule - 1) / granule * granule;
    const int tiles_c = (a.C + bn - 1) / bn;
    const long long tiles = static_cast<long long>(a.tiles_l) * tiles_c;
    const bool half = bn <= 128;
    for (int S = 1; S <= 8 && S <= kb; S += S == 4 ? 4 : 1) {  // 5 to 7 never paid
      const long long ctas = tiles * S, room = static_cast<long long>(half ? slots.half[S] : slots.whole[S]) * S;
      if (room == 0) continue;
      const double cta_mb = static_cast<double>((kb + S - 1) / S) * (kABytes + bn * 128) * 1e-6;
      auto wave = [&](double n) {
        const bool shared = n > slots.whole[1];  // SMs that hold two CTAs
        const double own = cta_mb * 1e3 / (!half ? 93.5 : (shared ? 72.0 : 78.8));
        const double hbm = unique * n / static_cast<double>(ctas) / 6.5;
        return 4.77 + bn * (0.0178 + 0.00108 * (S - 1) + (shared ? 0.0166 : 0.0)) +
               fmax(sqrt(own * own + hbm * hbm), cta_mb * n / 16.4);
      };
      const long long left = ctas % room;
      const double t = (left > 0 ? wave(static_cast<double>(left)) : 0.0) +
                       (ctas >= room ? static_cast<double>(ctas / room) * wave(static_cast<double>(room)) : 0.0);
      if (a.split == 0 || t < best) {
        best = t;
        a.split = S;
        a.bn = bn;
        a.tiles_c = tiles_c;
      }
    }
    if (bn <= granule) break;
  }
  a.per = (a.bn + a.split - 1) / a.split;
  const int stage = kABytes + a.bn * 128;
  const int room = (a.bn <= 128 ? kHalfSmem : kSmemMax) - 1024 - static_cast<int>(sizeof(SplitShared));
  a.stages = room / stage;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const int exchange = a.bn * kLanes * 4;
  a.ring_bytes = a.stages * stage > exchange ? a.stages * stage : exchange;
  a.tmem_cols = 32;
  while (a.tmem_cols < static_cast<uint32_t>(a.bn)) a.tmem_cols <<= 1;
  return best;
}

// Clusters of S CTAs that fit the device at once, with half an SM's shared
// memory each and with all of it.  The occupancy query counts a kernel that
// allocates tensor memory as one CTA an SM whatever it allocates; two CTAs with
// half the shared memory and at most 128 TMEM columns each do run side by side
// (224 measured active at once), so the query is made of a stand-in of the same
// launch shape.
cudaError_t linear_split_slots(LinearSlots* slots) {
  cudaError_t e = cudaFuncSetAttribute(occupancy_stand_in, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  for (int S = 1; S <= 8 && e == cudaSuccess; ++S)
    for (int half = 0; half < 2 && e == cudaSuccess; ++half) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(S));
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = half ? kHalfSmem : kSmemMax;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(S);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(half ? &slots->half[S] : &slots->whole[S], occupancy_stand_in, &cfg);
    }
  return e;
}

cudaError_t launch_linear_split(const LinearArgs& a, const CUtensorMap& ma, const CUtensorMap& mb, cudaStream_t s) {
  const size_t smem = 1024 + static_cast<size_t>(a.ring_bytes) + sizeof(SplitShared);
  if (smem > static_cast<size_t>(kSmemMax) || a.stages < 2) return cudaErrorInvalidValue;
  if (a.a_mn && a.b_mn) return launch_t<true, true>(a, ma, mb, smem, s);
  if (a.a_mn) return launch_t<true, false>(a, ma, mb, smem, s);
  return launch_t<false, false>(a, ma, mb, smem, s);
}

}  // namespace moe
