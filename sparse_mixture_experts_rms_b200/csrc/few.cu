// few.cu -- the whole MoE layer for a few tokens (a decode step) as one
// cooperative kernel.
//
// CODA sparse-MoE thread (digg.com): RMS statistic r, router logits scaled by
// r after the product; MoE glossary (inferensys.com): top-k gates, capacity,
// "Fused MoE kernels" combining routing, permutation and expert matmuls.
//   r_t = 1/sqrt(mean x_t^2 + eps)      l_te = r_t sum_i x_ti gamma_i Wr_ie + b_e
//   h = silu(r_t xg_t W1_e) * (r_t xg_t W3_e)      out_t = res_t + sum_j gate_tj h W2_e
//
// What bounds it: the chosen experts' weights, 6 d f_e bytes each, read once
// from HBM; a handful of tokens makes the products themselves nearly free.  So
// the kernel is a weight stream: it keeps one CTA per SM, gives every CTA an
// equal, contiguous share of the weight bytes of each phase, and nothing ever
// stops the loads but a full ring.
//
// Phases:
//   0  route: CTAs do slices of the tokens (xg = x * gamma as a bf16 pair, r,
//      logits, top-k, gates); every CTA waits for all tokens and builds the
//      index tables.
//   1  up:   tiles of 128 columns of an expert's W1 and the same of W3.
//   2  down: tiles of 256 columns of an expert's W2.
//      grid-wide wait
//   3  combine: out = residual + gate-weighted sums of the partial products.
//
// The products run on the tensor cores with the WEIGHTS as the M operand
// (tcgen05.mma, M = 128 weight columns, MN-major as they lie in memory) and
// the tokens as N, so a tile's MMAs cost the same for 1 token and for 8, and
// no row of a 128-row tile is padding.  Activations enter as bf16 pairs
// hi + lo (16 significant bits), two groups of N columns whose products are
// added in the epilogue: the tensor pipe has room to spare, and the
// activations lose nothing that the formula's fp32 would keep visible in the
// bf16 output.
//
// Measured (device time of a call in a graph, by the GPU; floor = the chosen experts'
// bytes at the 6.55 TB/s of a copy): 8 experts of 4096 x 14336, top-2, one token
// (705 MB) 122-126 us against 107, 64 tokens (2.8 GB) 447-460 against 430; 7 tokens of 64
// experts of 2048 x 512, top-8, 55-58 us against 37, where the chain of dependent steps
// shows: routing 3.5 us, choice and tables 3.3, first tile 3, from the last up
// tile to the first down stage about 8, combine and its wait 3.  DRAM reads are
// the weights' bytes to 0.1 %.
//
// Shares: the stages (64 reduction rows of a tile, 32 KB of weights) of the
// tiles of a phase form a line, and CTA c takes stages [c S/G, (c+1) S/G).  A
// tile whose reduction is cut by a share boundary has its pieces summed in
// share order by whichever CTA finishes last (up) or by the combine (down):
// the order of the sum depends on the shares alone, so a call's result is
// always the same bits.
//
// Warps (320 threads, all for the routing): 0 = weight loads by TMA, 1 = MMA issue
// and TMEM, 2-5 = epilogue (one per TMEM lane quarter), 6 = activation loads
// (four-row TMA gathers of the tokens' rows, boxes of H).  Up and down use one
// ring: while the activation loads wait for another CTA's H, the next weight
// stages are already in flight.
#include "few.cuh"

namespace moe {
namespace {

constexpr int kWTile = 128 * 64 * 2;     // 128 weight columns x 64 reduction rows
constexpr int kWAtom = 64 * 64 * 2;      // 64 columns x 64 rows: one TMA box
constexpr int kWStage = 2 * kWTile;

struct __align__(16) FewShared {
  uint64_t full_w[kFewMaxStages];   // the stage's weights landed
  uint64_t full_b[kFewMaxStages];   // the stage's activations landed
  uint64_t empty[kFewMaxStages];    // the MMAs that read the stage are done
  uint64_t tfull[2], tempty[2];     // accumulator buffers
  uint64_t drain;
  FewLine line[kFewLines];          // up A, up B, down A, down B
  uint32_t tmem_base;
  int abort_flag;
  int last;                         // epilogue: this CTA finishes the tile
  float r[MOE_FEW_MAX_TOKENS];
  FewTables tab;
};

// A share's piece of one tile: reduction stages [k0, k1) of kb.
struct Piece {
  int e, m, k0, k1, kb;
};

// A line's share boundaries, and the share that a stage belongs to (in stages).
__device__ __forceinline__ int share_begin(const FewLine& l, int c) {
  return static_cast<int>(static_cast<uint32_t>(l.total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(l.shares)) *
         l.unit;
}
__device__ __forceinline__ int share_owner(const FewLine& l, int stage) {
  const uint32_t u = static_cast<uint32_t>(stage) / static_cast<uint32_t>(l.unit);
  return static_cast<int>(((u + 1) * static_cast<uint32_t>(l.shares) - 1u) / static_cast<uint32_t>(l.total));
}

// Walks a CTA's share piece by piece.
struct Walk {
  int s, s1, e;
  __device__ __forceinline__ void begin(const FewLine& l) {
    s = s1 = e = 0;
    if (static_cast<int>(blockIdx.x) < l.shares) {
      s = share_begin(l, blockIdx.x);
      s1 = share_begin(l, blockIdx.x + 1);
    }
  }
  __device__ __forceinline__ bool next(const FewArgs& a, const FewTables& tab, const FewLine& l, bool down, Piece& p) {
    if (s >= s1) return false;
    while (s >= l.start[e + 1] * l.unit) ++e;
    p.e = e;
    p.kb = down ? (tab.off[e + 1] - tab.off[e]) / 64 : a.d / 64;
    const int local = s - l.start[e] * l.unit;
    p.m = local / p.kb;
    p.k0 = local - p.m * p.kb;
    p.k1 = min(p.kb, p.k0 + s1 - s);
    s += p.k1 - p.k0;
    return true;
  }
};

__device__ __forceinline__ int rows_of(const FewTables& t, int e) { return t.rows[e + 1] - t.rows[e]; }

// Generic-proxy accesses that this thread has observed come before its later
// async-proxy (TMA) accesses.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Rows r0..r3 of a map whose box is one row high, columns from c0, to four
// consecutive 128-byte rows at dst (swizzled by their shared-memory address).
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t r0,
                                            int32_t r1, int32_t r2, int32_t r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
      : "memory");
}

// 32 lanes x 2 consecutive 32-bit TMEM columns.
__device__ __forceinline__ void tmem_ld_x2(uint32_t taddr, uint32_t (&v)[2]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(taddr));
}

// Floats from upart to the piece of a cut up tile that CTA c left: slot 1 if
// the tile starts in its share (a share's last piece), slot 0 otherwise (its
// first).
__device__ __forceinline__ size_t few_slot(const FewArgs& a, int li, int c, bool starts) {
  return ((static_cast<size_t>(li) * kFewMaxGrid + c) * 2 + (starts ? 1 : 0)) * 2 * a.T * 128;
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same barrier, and whether `v` holds in all four warps: they go on or give
// up together.
__device__ __forceinline__ bool epi_all(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Sums of tokens j0 and j0 + 1 of both accumulators for this thread's column: the
// products with the high parts plus those with the low parts.  (Eight tokens at a
// time is four times the code, and the epilogue runs a handful of times: its
// instructions, fetched while the weights stream, took 3.5 us.)
__device__ __forceinline__ void acc_read(uint32_t taddr, int n8, int j0, float (&s0)[2], float (&s1)[2]) {
  uint32_t h[2], l[2], h1[2], l1[2];
  tmem_ld_x2(taddr + j0, h);
  tmem_ld_x2(taddr + n8 + j0, l);
  tmem_ld_x2(taddr + 128 + j0, h1);
  tmem_ld_x2(taddr + 128 + n8 + j0, l1);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    s0[j] = __uint_as_float(h[j]) + __uint_as_float(l[j]);
    s1[j] = __uint_as_float(h1[j]) + __uint_as_float(l1[j]);
  }
}

__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map3,
               const __grid_constant__ CUtensorMap map2, const __grid_constant__ CUtensorMap map_x,
               const __grid_constant__ CUtensorMap map_h, const __grid_constant__ FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kWStage + a.b_bytes;
  FewShared& sh = *reinterpret_cast<FewShared*>(ring + a.stages * stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = a.stages;
  const uint64_t wait_ns = wait_limit_ns(a.wait_ctl);
  volatile int* abort_flag = &sh.abort_flag;

  if (tid == 0) {
    sh.abort_flag = 0;
    few_tables_at(sh.tab, reinterpret_cast<uint8_t*>(&sh + 1), a.T * a.k);
    for (int s = 0; s < S; ++s) {
      mbar_init(&sh.full_w[s], 1);
      mbar_init(&sh.full_b[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.tfull[b], 1);
      mbar_init(&sh.tempty[b], 4);
    }
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
    tma_prefetch_map(&map1);
    tma_prefetch_map(&map3);
    tma_prefetch_map(&map2);
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_h);
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }

  // ---- phase 0
  few_clear(a);
  few_route(a, ring);
  if (tid <= a.E) sh.tab.off[tid] = a.ffn.off[tid];
  if (tid < kMaxExperts) sh.tab.bias[tid] = a.bias != nullptr && tid < a.E ? a.bias[tid] : 0.f;
  __syncthreads();
  // the ring as scratch: counts per group of 32 assignments, logits per warp
  uint8_t* cnt = ring;
  for (int i = tid; i < (a.T * a.k + 31) / 32 * kMaxExperts / 4; i += kFewThreads)
    reinterpret_cast<uint32_t*>(cnt)[i] = 0;
  bool ok = few_cta_wait(a.bar_a, a.T * few_slices(a), abort_flag, a.err, wait_ns);
  if (ok) {
    few_pick(a, sh.tab, sh.r, ring + 8 * 1024);
    few_tables(a, sh.tab, sh.line, cnt);
  }
  fence_proxy_async_smem();  // the ring was scratch: its plain accesses come before the copies into it
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = sh.tmem_base;

  if (ok) {
    if (warp == 0) {
      // ================= weight loads
      if (lane == 0) {
        uint32_t it = 0;
        bool go = true;
        for (int li = 0; li < kFewLines && go; ++li) {
          const bool down = li >= 2;
          Walk w;
          Piece p;
          w.begin(sh.line[li]);
          while (go && w.next(a, sh.tab, sh.line[li], down, p)) {
            const int o = sh.tab.off[p.e];
            const bool two = !down || p.m * 256 + 128 < a.d;
            for (int k = p.k0; k < p.k1; ++k, ++it) {
              const int s = it % S;
              if (!mbar_wait(&sh.empty[s], ((it / S) & 1u) ^ 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns)) {
                go = false;
                break;
              }
              uint8_t* dst = ring + s * stage_bytes;
              mbar_arrive_expect_tx(&sh.full_w[s], two ? kWStage : kWTile);
              if (!down) {
                tma_load_2d(dst, &map1, &sh.full_w[s], o + p.m * 128, k * 64);
                tma_load_2d(dst + kWAtom, &map1, &sh.full_w[s], o + p.m * 128 + 64, k * 64);
                tma_load_2d(dst + kWTile, &map3, &sh.full_w[s], o + p.m * 128, k * 64);
                tma_load_2d(dst + kWTile + kWAtom, &map3, &sh.full_w[s], o + p.m * 128 + 64, k * 64);
              } else {
                for (int j = 0; j < (two ? 4 : 2); ++j)
                  tma_load_2d(dst + j * kWAtom, &map2, &sh.full_w[s], p.m * 256 + j * 64, o + k * 64);
              }
            }
          }
        }
        // the copies in flight land before the CTA goes on (default limit)
        volatile int no_abort = 0;
        for (uint32_t j = it > static_cast<uint32_t>(S) ? it - S : 0; j < it; ++j)
          mbar_wait(&sh.full_w[j % S], (j / S) & 1u, &no_abort, a.err, MOE_DEVERR_TIMEOUT, kWaitTimeoutNs);
      }
    } else if (warp == 1) {
      // ================= MMA issue
      if (lane == 0) {
        uint32_t it = 0, n = 0;
        bool go = true;
        for (int li = 0; li < kFewLines && go; ++li) {
          const bool down = li >= 2;
          Walk w;
          Piece p;
          w.begin(sh.line[li]);
          for (; go && w.next(a, sh.tab, sh.line[li], down, p); ++n) {
            const int n8 = (rows_of(sh.tab, p.e) + 7) & ~7;
            const uint32_t idesc = umma_idesc_bf16(128, 2 * n8, 0u, 1u);
            const bool two = !down || p.m * 256 + 128 < a.d;
            const uint32_t buf = n & 1u, d_tmem = tmem_base + buf * 256;
            if (!mbar_wait(&sh.tempty[buf], ((n >> 1) & 1u) ^ 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns)) {
              go = false;
              break;
            }
            tc_fence_after();
            for (int k = p.k0; k < p.k1; ++k, ++it) {
              const int s = it % S;
              if (!mbar_wait(&sh.full_w[s], (it / S) & 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns) ||
                  !mbar_wait(&sh.full_b[s], (it / S) & 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns)) {
                go = false;
                break;
              }
              tc_fence_after();
              const uint32_t aW = smem_addr(ring + s * stage_bytes), aB = aW + kWStage;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint64_t bd = smem_desc_sw128(aB + kk * 32, 16, 1024);
                const uint32_t acc = k > p.k0 || kk > 0 ? 1u : 0u;
                umma_bf16(d_tmem, smem_desc_sw128(aW + kk * 2048, kWAtom, 1024), bd, idesc, acc);
                if (two)
                  umma_bf16(d_tmem + 128, smem_desc_sw128(aW + kWTile + kk * 2048, kWAtom, 1024), bd, idesc, acc);
              }
              umma_commit(&sh.empty[s]);
            }
            if (go) umma_commit(&sh.tfull[buf]);
          }
        }
        umma_commit(&sh.drain);
        volatile int no_abort = 0;
        mbar_wait(&sh.drain, 0, &no_abort, a.err, MOE_DEVERR_TIMEOUT, kWaitTimeoutNs);
      }
    } else if (warp < 6) {
      // ================= epilogue: thread = one weight column of the tile
      const int q = warp & 3, col = q * 32 + lane;
      uint32_t n = 0;
      bool go = true;
      for (int li = 0; li < kFewLines && go; ++li) {
        const bool down = li >= 2;
        const FewLine& line = sh.line[li];
        Walk w;
        Piece p;
        w.begin(line);
        for (; w.next(a, sh.tab, line, down, p); ++n) {
          const uint32_t buf = n & 1u;
          bool got = true;
          if (lane == 0)
            got = mbar_wait(&sh.tfull[buf], (n >> 1) & 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns);
          __syncwarp();
          if (!epi_all(got)) {
            go = false;
            break;
          }
          tc_fence_after();
          const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * 256;
          const int row0 = sh.tab.rows[p.e], ne = rows_of(sh.tab, p.e), n8 = (ne + 7) & ~7;
          const bool whole = p.k0 == 0 && p.k1 == p.kb;
          const bool two = !down || p.m * 256 + 128 < a.d;
          // Where the sums go: H (a whole up tile), or as they are to dst + token * ld and, for the
          // second accumulator, `second` further on.  Down: the first piece of a tile to y, a later one to the
          // CTA's own rows.  Up, cut tile: the CTA's slot, [2][T][128].
          bool to_h = !down && whole, from_parts = false;
          float* dst;
          int ld = 128, second = a.T * 128, c0 = 0, c1 = 0;
          if (down) {
            dst = p.k0 == 0 ? a.y + static_cast<size_t>(row0) * a.d + p.m * 256
                            : a.ypart + (static_cast<size_t>(li - 2) * kFewMaxGrid + blockIdx.x) * a.T * 256;
            ld = p.k0 == 0 ? a.d : 256;
            second = 128;
          } else {
            dst = a.upart + few_slot(a, li, blockIdx.x, p.k0 == 0);
          }
          dst += col;
          for (;;) {
#pragma unroll 1
            for (int j0 = 0; j0 < ne; j0 += 2) {
              float s0[2], s1[2];
              if (!from_parts) {
                acc_read(taddr, n8, j0, s0, s1);
              } else {
                // pieces in share order: the CTA that starts the tile left it in slot 1, the others in slot 0
                s0[0] = s0[1] = s1[0] = s1[1] = 0.f;
#pragma unroll 2
                for (int c = c0; c <= c1; ++c) {
                  // token j0 + 1 may be absent: what lies there is not used
                  const float* part = a.upart + few_slot(a, li, c, c == c0) + j0 * 128 + col;
                  s0[0] += __ldcg(part);
                  s0[1] += __ldcg(part + 128);
                  s1[0] += __ldcg(part + a.T * 128);
                  s1[1] += __ldcg(part + a.T * 128 + 128);
                }
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if (j0 + j >= ne) break;
                if (to_h) {
                  const float r = sh.r[sh.tab.token[row0 + j0 + j]];
                  few_store_h(a, row0 + j0 + j, p.m * 128 + col, few_silu(r * s0[j]) * (r * s1[j]));
                } else {
                  dst[static_cast<size_t>(j0 + j) * ld] = s0[j];
                  if (two) dst[static_cast<size_t>(j0 + j) * ld + second] = s1[j];
                }
              }
            }
            if (!from_parts) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh.tempty[buf]);
            }
            if (down) break;
            epi_sync();
            if (to_h) {  // these columns of H are complete: count the tile
              if (warp == 2 && lane == 0) red_add_release(&a.done[li], 1u);
              break;
            }
            // a cut tile: the CTA that counts the last piece goes round again for the sums of all
            const int t0 = line.start[p.e] * line.unit + p.m * p.kb;  // the tile's first stage
            c0 = share_owner(line, t0);
            c1 = share_owner(line, t0 + p.kb - 1);
            if (warp == 2 && lane == 0)
              sh.last = atom_add_acq_rel(&a.tile_cnt[li * kFewMaxGrid + c0], 1u) == static_cast<uint32_t>(c1 - c0);
            epi_sync();
            if (!sh.last) break;
            to_h = from_parts = true;
          }
        }
      }
    } else if (warp == 6) {
      // ================= activation loads: rows of the expert's tokens, 64
      // elements a stage, the high parts from row 0 of the tile, the low parts from
      // row n8.  Up: gathers of four tokens' rows, a lane a gather (lanes 16 on: the
      // low parts), the last token again where fewer are left.  Down: boxes of eight
      // rows of H; what a box reads past the expert's rows lands in columns nobody
      // uses.
      const int part = lane & 15, low = lane >> 4;
      uint32_t it = 0;
      bool go = true;
      fence_proxy_async_all();  // xg: written plainly by other CTAs, read here by TMA
      for (int li = 0; li < kFewLines && go; ++li) {
        const bool down = li >= 2;
        Walk w;
        Piece p;
        w.begin(sh.line[li]);
        bool ready = !down;
        while (go && w.next(a, sh.tab, sh.line[li], down, p)) {
          const int row0 = sh.tab.rows[p.e], ne = rows_of(sh.tab, p.e), n8 = (ne + 7) & ~7;
          if (!ready) {
            // H of the line's experts is complete when all tiles of their up line are
            bool got = true;
            if (lane == 0) got = few_wait_word(&a.done[li - 2], sh.line[li - 2].tiles, abort_flag, a.err, wait_ns);
            if (!warp_take(got)) {
              go = false;
              break;
            }
            fence_proxy_async_all();
            ready = true;
          }
          const int copies = down ? n8 / 8 : (ne + 3) / 4;  // per half
          const uint32_t tx = 2u * 128u * static_cast<uint32_t>(down ? n8 : copies * 4);
          const uint32_t off = static_cast<uint32_t>((low ? n8 : 0) + part * (down ? 8 : 4)) * 128u;
          int r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (down)
              r[j] = (low ? a.T * a.k : 0) + row0 + part * 8;
            else
              r[j] = (low ? a.T : 0) + sh.tab.token[row0 + min(part * 4 + j, ne - 1)];
          }
          for (int k = p.k0; k < p.k1; ++k, ++it) {
            const int s = it % S;
            bool got = true;
            if (lane == 0) {
              got = mbar_wait(&sh.empty[s], ((it / S) & 1u) ^ 1u, abort_flag, a.err, MOE_DEVERR_TIMEOUT, wait_ns);
              if (got) mbar_arrive_expect_tx(&sh.full_b[s], tx);
            }
            if (!warp_take(got)) {
              go = false;
              break;
            }
            if (part < copies) {
              uint8_t* dst = ring + s * stage_bytes + kWStage + off;
              if (down)
                tma_load_2d(dst, &map_h, &sh.full_b[s], k * 64, r[0]);
              else
                tma_gather4(dst, &map_x, &sh.full_b[s], k * 64, r[0], r[1], r[2], r[3]);
            }
          }
        }
      }
      if (lane == 0) {  // the copies in flight land before the CTA goes on (default limit)
        volatile int no_abort = 0;
        for (uint32_t j = it > static_cast<uint32_t>(S) ? it - S : 0; j < it; ++j)
          mbar_wait(&sh.full_b[j % S], (j / S) & 1u, &no_abort, a.err, MOE_DEVERR_TIMEOUT, kWaitTimeoutNs);
      }
    }
  }

  ok = __syncthreads_and(ok && !*abort_flag) != 0;
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  // ---- phase 3: a warp sums 32 columns of one token, 4 at a lane; lanes
  // 8g .. 8g + 7 take slots g, g + 4, ..., and the four sums meet at the end
  if (ok) ok = few_grid_wait(a.bar_b, gridDim.x, abort_flag, a.err, wait_ns);
  if (ok) {
    const int per_token = a.d / 32;
    for (int i = blockIdx.x + gridDim.x * warp; i < a.T * per_token; i += gridDim.x * (kFewThreads / 32)) {
      const int t = i / per_token, c = (i - t * per_token) * 32 + (lane & 7) * 4, m = c >> 8;
      const size_t o = static_cast<size_t>(t) * a.d + c;
      uint2 res = make_uint2(0u, 0u);
      if (a.residual != nullptr && lane < 8) res = *reinterpret_cast<const uint2*>(a.residual + o);
      float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int j = lane >> 3; j < a.k; j += 4) {
        const int row = sh.tab.pos[t * a.k + j];
        if (row < 0) continue;
        const int e = sh.tab.expert[t * a.k + j];
        const int li = sh.line[2].start[e] < sh.line[2].start[e + 1] ? 2 : 3;
        const FewLine& line = sh.line[li];
        const int kb = (sh.tab.off[e + 1] - sh.tab.off[e]) / 64, t0 = line.start[e] + m * kb;
        const int c0 = share_owner(line, t0), c1 = share_owner(line, t0 + kb - 1);
        float4 y = __ldcg(reinterpret_cast<const float4*>(a.y + static_cast<size_t>(row) * a.d + c));
        const float* part = a.ypart + (static_cast<size_t>(li - 2) * kFewMaxGrid * a.T + row - sh.tab.rows[e]) * 256 +
                            (c & 255);
#pragma unroll 4
        for (int ct = c0 + 1; ct <= c1; ++ct) {
          const float4 z = __ldcg(reinterpret_cast<const float4*>(part + static_cast<size_t>(ct) * a.T * 256));
          y.x += z.x;
          y.y += z.y;
          y.z += z.z;
          y.w += z.w;
        }
        const float g = sh.tab.gate[t * a.k + j];
        out.x = fmaf(g, y.x, out.x);
        out.y = fmaf(g, y.y, out.y);
        out.z = fmaf(g, y.z, out.z);
        out.w = fmaf(g, y.w, out.w);
      }
      __syncwarp();
#pragma unroll
      for (int q = 8; q <= 16; q <<= 1) {
        out.x += __shfl_xor_sync(0xFFFFFFFFu, out.x, q);
        out.y += __shfl_xor_sync(0xFFFFFFFFu, out.y, q);
        out.z += __shfl_xor_sync(0xFFFFFFFFu, out.z, q);
        out.w += __shfl_xor_sync(0xFFFFFFFFu, out.w, q);
      }
      if (lane < 8) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(out.x + __uint_as_float(res.x << 16),
                                                        out.y + __uint_as_float(res.x & 0xFFFF0000u));
        const __nv_bfloat162 hi = __floats2bfloat162_rn(out.z + __uint_as_float(res.y << 16),
                                                        out.w + __uint_as_float(res.y & 0xFFFF0000u));
        *reinterpret_cast<uint2*>(a.out + o) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
  }
  few_exit(a);
}

constexpr size_t kSmemMax = 232448;

}  // namespace

cudaError_t prepare_few() {
  return cudaFuncSetAttribute(few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemMax));
}

cudaError_t launch_few(FewArgs& a, const CUtensorMap& map1, const CUtensorMap& map3, const CUtensorMap& map2,
                       const CUtensorMap& map_x, const CUtensorMap& map_h, int sms, cudaStream_t s) {
  // as many stages as fit beside the tables: 6 for up to 8 tokens, 4 for 64
  a.b_bytes = 2 * ((a.T + 7) & ~7) * 128;
  const size_t fixed = 1024 + sizeof(FewShared) + few_table_bytes(a.T * a.k);
  const int stage = kWStage + a.b_bytes;
  a.stages = static_cast<int>((kSmemMax - fixed) / stage);
  if (a.stages > kFewMaxStages) a.stages = kFewMaxStages;
  if (a.stages < 2 || a.stages * stage < static_cast<int>(kFewScratchBytes)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms < kFewMaxGrid ? sms : kFewMaxGrid));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = fixed + static_cast<size_t>(a.stages) * stage;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel, map1, map3, map2, map_x, map_h, static_cast<const FewArgs&>(a));
}

}  // namespace moe
