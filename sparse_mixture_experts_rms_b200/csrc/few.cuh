// few.cuh -- routing, index tables and grid-wide waits of the few-token layer
// (few.cu).
#pragma once

#include "moe_internal.h"
#include "ptx.cuh"

namespace moe {

// One line of stages (64 reduction rows of a tile): the up or the down tiles of
// a group of experts, cut into `shares` equal shares, one per CTA.  With
// `unit` above 1 a share is a whole number of tiles of that many stages.
struct FewLine {
  int start[kMaxExperts + 1];  // first unit of each expert
  int total;                   // units
  int unit;                    // stages per unit
  int shares;                  // at most one per CTA, never an empty one
  int tiles;                   // up lines: tiles in all
};
constexpr int kFewLines = 4;   // up A, up B, down A, down B

// Index tables of a call, built by every CTA from the routing; the arrays lie
// behind the struct in shared memory.
struct FewTables {
  int rows[kMaxExperts + 1];   // first row (kept assignment) of each expert
  int off[kMaxExperts + 1];    // cumulative expert widths: indexed by lane, which the parameter bank would serialise
  float bias[kMaxExperts];     // router bias
  float* gate;                 // [T*k]
  int16_t* token;              // [kept] token of each row
  int16_t* pos;                // [T*k] row of each assignment, -1 if dropped
  uint8_t* expert;             // [T*k]
};
__host__ __device__ constexpr int few_table_bytes(int tk) { return (tk * 9 + 15) & ~15; }
__device__ __forceinline__ void few_tables_at(FewTables& t, uint8_t* p, int tk) {
  t.gate = reinterpret_cast<float*>(p);
  t.token = reinterpret_cast<int16_t*>(p + 4 * tk);
  t.pos = t.token + tk;
  t.expert = reinterpret_cast<uint8_t*>(t.pos + tk);
}

// ---- grid-wide waits
__device__ __forceinline__ uint32_t ld_acquire_u32(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t atom_add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}
// Counts one arrival: what this CTA wrote before (and joined by a barrier) is
// visible to whoever acquires the count.
__device__ __forceinline__ void red_add_release(uint32_t* p, uint32_t v) {
  asm volatile("red.add.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Wait until *p >= target, giving up like mbar_wait (the same limit, flag and
// error bit).  One thread.
__device__ __forceinline__ bool few_wait_word(const uint32_t* p, uint32_t target, volatile int* abort,
                                              uint32_t* err, uint64_t timeout_ns) {
  if (ld_acquire_u32(p) >= target) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (ld_acquire_u32(p) >= target) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > timeout_ns) {
      *abort = 1;
      atomicOr(err, MOE_DEVERR_TIMEOUT);
      return false;
    }
  }
}

// Every thread calls it; what was written before the counted arrivals is
// visible after it.
__device__ __forceinline__ bool few_cta_wait(const uint32_t* bar, uint32_t n, volatile int* abort, uint32_t* err,
                                             uint64_t timeout_ns) {
  bool ok = true;
  if (threadIdx.x == 0) ok = few_wait_word(bar, n, abort, err, timeout_ns);
  return __syncthreads_and(ok) != 0;
}

// All CTAs of the grid.
__device__ __forceinline__ bool few_grid_wait(uint32_t* bar, uint32_t n, volatile int* abort, uint32_t* err,
                                              uint64_t timeout_ns) {
  __syncthreads();
  if (threadIdx.x == 0) red_add_release(bar, 1u);
  return few_cta_wait(bar, n, abort, err, timeout_ns);
}

// The words that must be zero once the routing is known (CTA 0 has a slice of
// token 0, so its writes come before its arrival); the header words bar_a and
// bar_x are zero between calls.
__device__ __forceinline__ void few_clear(const FewArgs& a) {
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kFewSyncWords; i += kFewThreads) a.sync[i] = 0;
}

// The last CTA to leave zeroes the two words of the header for the next call.
__device__ __forceinline__ void few_exit(const FewArgs& a) {
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(a.bar_x, 1u) == gridDim.x - 1) {
    *a.bar_a = 0;
    *a.bar_x = 0;
    __threadfence();
  }
}

// z sigmoid(z) by the fast exponential (2 + 1.17 |z| ulp) and division (2 ulp): within
// 2^-18 of itself down to z = -20, where it is 4e-8, and looser only below that.  H
// keeps 16 bits of its product with v.  Below z = -87.3 the division gives 0 (its
// divisor is above 2^126; the value is smaller than 1e-36).
__device__ __forceinline__ float few_silu(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

// v as hi + lo, two bf16 (16 significant bits; lo = 0 where hi is not finite,
// so that an infinity stays one).
__device__ __forceinline__ void bf16_split(float v, __nv_bfloat16& hi, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  const float h = __bfloat162float(hi);
  lo = __float2bfloat16_rn(fabsf(h) <= 3.4e38f ? v - h : 0.f);
}

__device__ __forceinline__ void few_store_h(const FewArgs& a, int row, int f, float h) {
  __nv_bfloat16 hi, lo;
  bf16_split(h, hi, lo);
  const size_t o = static_cast<size_t>(row) * a.ldh + f;
  a.H[o] = hi;
  a.H[a.h_lo + o] = lo;
}

// ---- phase 0: routing.  Token t's elements are cut into `nsl` slices, a CTA a
// slice, which leaves the slice's logit sums and sum of squares in lpart and
// arrives at bar_a; then every CTA adds up every token's slices in slice order
// and picks the experts for itself, a warp a token: that costs each CTA less
// than waiting for one CTA's choice to come back through L2.
//
// Each product x*gamma*Wr of three bf16 has 24 significant bits, so fp32 holds
// it exactly; a thread adds at most 16 of them in fp32 before its sum moves to
// fp64, and everything after that -- across threads and slices, the scaling by
// r, the bias -- is fp64, rounded once to the fp32 logit.  A thread takes `vec`
// (8 when E allows 16-byte loads, else 1) neighbouring experts of every
// (kFewThreads * vec / E)-th row of Wr.
//
// One CTA a token (no slices) took 13 us of the 140 us of a Mixtral-shaped
// token and 36 us with 64 experts of d = 2048: one SM's loads of Wr.
constexpr int kFewSlices = 16;
__device__ __forceinline__ int few_slices(const FewArgs& a) {
  int n = static_cast<int>(gridDim.x) / a.T;
  n = n < kFewSlices ? n : kFewSlices;
  n = n < a.d / 128 ? n : a.d / 128;
  return n > 1 ? n : 1;
}

__device__ __forceinline__ void few_route(const FewArgs& a, uint8_t* smem) {
  const int nsl = few_slices(a);
  const int t = blockIdx.x / nsl, sl = blockIdx.x - t * nsl;
  if (t >= a.T) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kFewThreads / 32;
  double* wpart = reinterpret_cast<double*>(smem);  // [kWarps][64]
  double* ssum = wpart + kWarps * kMaxExperts;      // [kWarps]
  const int E = a.E, d = a.d;
  const int begin = d / 128 * sl / nsl * 128, end = d / 128 * (sl + 1) / nsl * 128;
  const bool wide = (E & 7) == 0 && (reinterpret_cast<uintptr_t>(a.Wr) & 15) == 0;
  const int vec = wide ? 8 : 1;
  const int nv = E / vec;                           // threads that share a row of Wr
  int nvp = 1;                                      // ... rounded up to a power of two
  while (nvp < nv) nvp <<= 1;
  const int nrow = kFewThreads / nvp;               // rows of Wr per step
  const int row0 = tid / nvp, v = tid & (nvp - 1);
  const __nv_bfloat16* x = a.x + static_cast<size_t>(t) * d;
  // this thread's first 8 elements for the pair and the sum of squares, under way during the logits
  uint4 xv = make_uint4(0u, 0u, 0u, 0u), gv = xv;
  if (begin + tid * 8 < end) {
    xv = *reinterpret_cast<const uint4*>(x + begin + tid * 8);
    gv = __ldg(reinterpret_cast<const uint4*>(a.gamma + begin + tid * 8));
  }
  wpart[warp * kMaxExperts + lane] = wpart[warp * kMaxExperts + 32 + lane] = 0.0;
  double acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0;
  if (v < nv) {
    const __nv_bfloat16* w = a.Wr + v * vec;
    for (int i0 = begin + row0; i0 < end; i0 += nrow * 16) {
      float run[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) run[j] = 0.f;
#pragma unroll 1
      for (int s0 = 0; s0 < 16 && i0 + s0 * nrow < end; s0 += 4) {
        uint4 wv[4];
        float xg[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // 4 rows' loads in flight; rows past the slice count as zero
          const int i = i0 + (s0 + u) * nrow;
          const bool in = i < end;
          wv[u] = make_uint4(0u, 0u, 0u, 0u);
          if (in && wide) wv[u] = __ldg(reinterpret_cast<const uint4*>(w + static_cast<size_t>(i) * E));
          if (in && !wide) wv[u].x = *reinterpret_cast<const uint16_t*>(w + static_cast<size_t>(i) * E);
          xg[u] = in ? __bfloat162float(x[i]) * __bfloat162float(a.gamma[i]) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t ww[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            run[2 * j] += xg[u] * __uint_as_float(ww[j] << 16);
            run[2 * j + 1] += xg[u] * __uint_as_float(ww[j] & 0xFFFF0000u);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += static_cast<double>(run[j]);
    }
  }
  // the lanes of a warp that hold the same experts, then the warps
  for (int q = 16; q >= nvp; q >>= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], q);
  __syncwarp();
  if (lane < nvp && v < nv) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < vec) wpart[warp * kMaxExperts + v * vec + j] = acc[j];
  }
  double ss = 0.0;
  for (int i = begin + tid * 8; i < end; i += kFewThreads * 8) {
    if (i != begin + tid * 8) {
      xv = *reinterpret_cast<const uint4*>(x + i);
      gv = __ldg(reinterpret_cast<const uint4*>(a.gamma + i));
    }
    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w}, gw[4] = {gv.x, gv.y, gv.z, gv.w};
    __align__(16) __nv_bfloat16 hi[8], lo[8];
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float xf = __uint_as_float((j & 1) ? (xw[j / 2] & 0xFFFF0000u) : (xw[j / 2] << 16));
      const float gf = __uint_as_float((j & 1) ? (gw[j / 2] & 0xFFFF0000u) : (gw[j / 2] << 16));
      bf16_split(xf * gf, hi[j], lo[j]);
      sq = fmaf(xf, xf, sq);
    }
    ss += static_cast<double>(sq);
    *reinterpret_cast<uint4*>(a.xg + static_cast<size_t>(t) * d + i) = *reinterpret_cast<const uint4*>(hi);
    *reinterpret_cast<uint4*>(a.xg + static_cast<size_t>(a.T + t) * d + i) = *reinterpret_cast<const uint4*>(lo);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, s);
  if (lane == 0) ssum[warp] = ss;
  __syncthreads();
  double* slice = a.lpart + (static_cast<size_t>(t) * kFewSlices + sl) * (kMaxExperts + 1);
  if (tid <= E) {
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += tid < E ? wpart[w * kMaxExperts + tid] : ssum[w];
    slice[tid < E ? tid : kMaxExperts] = s;
  }
  __syncthreads();
  if (tid == 0) red_add_release(a.bar_a, 1u);
}

// Adds up the slices, a thread a (token, expert) pair (and the sums of squares
// as one expert more), 16 loads in flight a thread: the slices of one pair, or
// of 2^sh pairs where slices are few.
__device__ __forceinline__ void few_add_slices(const FewArgs& a, double* sums, double* rs, int nsl) {
  const int E1 = a.E + 1, npair = a.T * E1;
  const int sh = nsl <= 4 ? 2 : 0, per = kFewSlices >> sh;
  const float inv = 1.0f / static_cast<float>(E1);  // i / E1 for i < 64 * 65: (i + 1/2) inv is never near an integer
  for (int i0 = threadIdx.x; i0 < npair; i0 += kFewThreads << sh) {
    double v[kFewSlices], s = 0.0;
#pragma unroll
    for (int q = 0; q < kFewSlices; ++q) {
      const int i = i0 + q / per * kFewThreads, sl = q & (per - 1);
      const int t = static_cast<int>((static_cast<float>(i) + 0.5f) * inv), e = i - t * E1;
      v[q] = i < npair && sl < nsl ? __ldcg(a.lpart + (t * kFewSlices + sl) * (kMaxExperts + 1) + (e < a.E ? e : kMaxExperts))
                                   : 0.0;
    }
#pragma unroll
    for (int q = 0; q < kFewSlices; ++q) {
      s += v[q];
      const int i = i0 + q / per * kFewThreads;
      if ((q & (per - 1)) != per - 1 || i >= npair) continue;
      const int t = static_cast<int>((static_cast<float>(i) + 0.5f) * inv), e = i - t * E1;
      if (e < a.E)
        sums[t * a.E + e] = s;
      else
        rs[t] = rsqrt(s * a.inv_d + static_cast<double>(a.eps));
      s = 0.0;
    }
  }
}

// Logits, softmax and top-k of every token into the tables (and, by CTA 0,
// into the caller's copies).  An expert's slot is the number of experts that
// come before it -- a larger logit, or an equal one and a lower index -- so the k
// slots are found at once.  A NaN compares with nothing: a token with one takes
// the router's own k scans, in which it wins only as the first expert still free.
__device__ __forceinline__ void few_pick(const FewArgs& a, FewTables& tab, float* r_s, uint8_t* smem) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nsl = few_slices(a), E = a.E;
  constexpr int kWarps = kFewThreads / 32;
  double* sums = reinterpret_cast<double*>(smem);                                    // [T][E]
  double* rs = sums + static_cast<size_t>(a.T) * E;                                  // [T]
  float* lg = reinterpret_cast<float*>(rs + a.T) + warp * kMaxExperts;               // [warps][64]
  few_add_slices(a, sums, rs, nsl);
  __syncthreads();
  // 8, 16 or 32 lanes a token, each with expert `el` and, above 32, el + 32
  const int lanes = E <= 8 ? 8 : (E <= 16 ? 16 : 32), el = lane & (lanes - 1);
  const int nt = 32 / lanes;
  lg += (lane / lanes) * lanes;
  for (int t0 = warp * nt; t0 < a.T; t0 += kWarps * nt) {
    const int t = t0 + lane / lanes;
    const bool live = t < a.T;
    const double rv = rs[live ? t : 0];
    float l[2], ex[2], m = -INFINITY;
    int before[2] = {0, 0};
    float sum = 0.f, gsum = 0.f;
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = el + 32 * h;
      l[h] = e < E && live ? static_cast<float>(fma(rv, sums[t * E + e], static_cast<double>(tab.bias[e]))) : -INFINITY;
      if (h == 0 || E > 32) lg[e] = l[h];
      m = fmaxf(m, l[h]);
    }
    for (int q = lanes >> 1; q > 0; q >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, q));
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ex[h] = el + 32 * h < E ? expf(l[h] - m) : 0.f;
      sum += ex[h];
    }
#pragma unroll 4
    for (int e = 0; e < E; ++e) {
      const float o = lg[e];
      before[0] += o > l[0] || (o == l[0] && e < el);
      before[1] += o > l[1] || (o == l[1] && e < el + 32);
    }
    if (__any_sync(0xFFFFFFFFu, l[0] != l[0] || l[1] != l[1])) {
      uint64_t used = 0;
      before[0] = before[1] = a.k;
      for (int j = 0; j < a.k; ++j) {
        int best = -1;
        for (int e = 0; e < E; ++e)
          if (!((used >> e) & 1u) && (best < 0 || lg[e] > lg[best])) best = e;
        used |= uint64_t(1) << best;
        if (best == el) before[0] = j;
        if (best == el + 32) before[1] = j;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (el + 32 * h < E && before[h] < a.k) gsum += ex[h];
    for (int q = lanes >> 1; q > 0; q >>= 1) {
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, q);
      gsum += __shfl_xor_sync(0xFFFFFFFFu, gsum, q);
    }
    if (!live) continue;
    // a NaN among the logits makes every gate one, renormalised or not: 0 * sum
    const float inv = 1.0f / (a.renormalize ? gsum + 0.f * sum : sum);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = el + 32 * h;
      if (e >= E || before[h] >= a.k) continue;
      const int i = t * a.k + before[h];
      tab.expert[i] = static_cast<uint8_t>(e);
      tab.gate[i] = ex[h] * inv;
      if (blockIdx.x == 0) {
        if (a.idx_out != nullptr) a.idx_out[i] = e;
        if (a.gate_out != nullptr) a.gate_out[i] = ex[h] * inv;
      }
    }
    if (el == 0) {
      r_s[t] = static_cast<float>(rv);
      if (blockIdx.x == 0 && a.r_out != nullptr) a.r_out[t] = static_cast<float>(rv);
    }
  }
}

// Sum over the lanes below of a value.
__device__ __forceinline__ int warp_excl_sum(int v, int lane) {
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += u;
  }
  return s - v;
}

// How a line is shared.  A cut tile costs a round trip of its pieces through
// L2 and a second turn of the epilogue, about as long as 8 stages stream: so
// whole tiles where the most loaded CTA then has at most 8 stages more than an
// equal share (13 tokens of 768 x (2048 + 7 x 1024) 30.0 us, 32.6 when it was 4 and
// the tiles were cut; 8 tokens of 896 x 4 x 6144 42.1 against 47.6; above 14 the
// idle CTAs begin to cost, 61 -> 69 us at 16 tokens of 1664 x 64 x 384), and no
// share below `least` stages: 4 up; down, where the pieces meet in the combine, 2
// to 4, an eighth of the widest expert's tile.  (A tiny layer, 8 stages in all, measured
// 5 us more with one stage per CTA; 18 tokens of 256 x 32 x 640 26.2 us with 2 down
// and 28.0 with 4, 13 tokens of 768 x (2048 + 7 x 1024) 31.0 and 30.0.)
__device__ __forceinline__ void few_line(FewLine& l, int stages, int kb_all, int grid, int least) {
  const int tiles = kb_all > 0 ? stages / kb_all : 0;
  if (kb_all > 0 && (tiles + grid - 1) / grid * kb_all <= stages / grid + 8) {
    l.unit = kb_all;
    l.total = tiles;
    l.shares = tiles < grid ? tiles : grid;
  } else {
    l.unit = 1;
    l.total = stages;
    const int most = max(1, stages / least);
    l.shares = most < grid ? most : grid;
  }
}

// ---- index tables: stable ranks inside each expert in assignment order
// a = t*k + j, the first `capacity` kept.  A warp takes 32 assignments at a
// time: the lanes that chose the same expert find one another by a match, and
// the counts per group of 32 are then summed over the groups before it.
// Warp w < 4 also lays out line w: the experts are split into groups A and
// B of about equal weight, and the order up A, up B, down A, down B puts a
// group's whole up line between the other's up and its down, so that no CTA
// waits for H while the last up tiles finish.  That pays when the lines are long:
// one token of 8 experts of 4096 x 14336, 97 up stages a CTA, takes 121.7 us against
// 126.8 with every expert in group A; 7 tokens of 64 of 2048 x 512, 35 stages, 65.5
// against 58.2, since each line cuts tiles and ends with a CTA's wait.  So group A
// holds every expert below 60.  In between (30 layers, four shapes of d, E, k and T by
// width, two groups against one): +10 to +1 % of the time at 34-38 stages, +0.5 to -2 %
// at 45-49, +1 to -9 % at 55-62, -3 to -7 % from 65 to 97, -1 % at 138.
__device__ __forceinline__ void few_tables(const FewArgs& a, FewTables& tab, FewLine* line, uint8_t* cnt) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.T * a.k, groups = (n + 31) / 32;  // cnt: [groups][64], zeroed
  __syncthreads();
  for (int g = warp; g < groups; g += kFewThreads / 32) {
    const int i = g * 32 + lane;
    const int e = i < n ? tab.expert[i] : kMaxExperts + lane;  // absent: no two alike
    const unsigned peers = __match_any_sync(0xFFFFFFFFu, e);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    if (i < n) {
      tab.pos[i] = static_cast<int16_t>(rank);
      if (rank == 0) cnt[g * kMaxExperts + e] = static_cast<uint8_t>(__popc(peers));
    }
  }
  __syncthreads();
  if (warp < kFewLines) {
    int c[2] = {0, 0}, kept[2], up[2], mine[2];
    const int kb = a.d / 64, mt = (a.d + 255) / 256;
    for (int g = 0; g < groups; ++g) {
      const uint32_t w = *reinterpret_cast<const uint16_t*>(cnt + g * kMaxExperts + 2 * lane);
      c[0] += w & 0xFF;
      c[1] += w >> 8;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = 2 * lane + h;
      kept[h] = a.capacity >= 0 && c[h] > a.capacity ? a.capacity : c[h];
      const int f = e < a.E && kept[h] > 0 ? tab.off[e + 1] - tab.off[e] : 0;
      up[h] = f / 128 * kb;
      mine[h] = warp < 2 ? up[h] : f / 64 * mt;
    }
    const int u0 = warp_excl_sum(up[0] + up[1], lane);
    const int total = __shfl_sync(0xFFFFFFFFu, u0 + up[0] + up[1], 31);
    const bool split = total >= 60 * static_cast<int>(gridDim.x);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in_a = !split || 2 * (u0 + (h ? up[0] : 0)) < total;
      if (in_a != ((warp & 1) == 0)) mine[h] = 0;
    }
    const int s0 = warp_excl_sum(mine[0] + mine[1], lane);
    const int all = __shfl_sync(0xFFFFFFFFu, s0 + mine[0] + mine[1], 31);
    FewLine& l = line[warp];
    FewLine how;
    few_line(how, all, warp < 2 ? kb : 0, gridDim.x, warp < 2 ? 4 : min(max(a.ldh / 512, 2), 4));
    l.start[2 * lane] = s0 / how.unit;
    l.start[2 * lane + 1] = (s0 + mine[0]) / how.unit;
    if (lane == 0) {
      l.start[kMaxExperts] = l.total = how.total;
      l.unit = how.unit;
      l.shares = how.shares;
      l.tiles = all / kb;
    }
    if (warp == 0) {
      const int r0 = warp_excl_sum(kept[0] + kept[1], lane);
      tab.rows[2 * lane] = r0;
      tab.rows[2 * lane + 1] = r0 + kept[0];
      if (lane == 31) tab.rows[kMaxExperts] = r0 + kept[0] + kept[1];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (2 * lane + h < a.E && a.counts_out != nullptr && blockIdx.x == 0) a.counts_out[2 * lane + h] = c[h];
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += kFewThreads) {
    const int e = tab.expert[i];
    int rank = tab.pos[i];
    for (int g = 0; g < i >> 5; ++g) rank += cnt[g * kMaxExperts + e];
    const int p = a.capacity >= 0 && rank >= a.capacity ? -1 : tab.rows[e] + rank;
    tab.pos[i] = static_cast<int16_t>(p);
    if (p >= 0) tab.token[p] = static_cast<int16_t>(i / a.k);
  }
  __syncthreads();
}

}  // namespace moe
