// linear.cu -- the elementwise part of the linear layer's backward:
//   dz = dy * act'(z),  db = sum_t dz
// (the products dx = dz W^T and dW = x^T dz, like the forward's, are in
// linear_split.cu and linear_pair.cu).
//
// dz is rounded to bf16 for those products: the tensor cores take operands of 16
// bits, and two halves (as the few-token layer's activations have) would double the
// products' time, nearly all of the backward.  What it costs: dx and dW are off from
// the formula by 2.35e-3 normwise instead of the 1.66e-3 that their own rounding to
// bf16 alone gives (1001 x 1024 x 4096 GELU and 16384 x 4096 x 14336 SiLU).  dbias is
// summed from unrounded dz.
#include "linear.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

// dz and the column sums of a chunk of rows: one pass over dy and z, bound by
// their bytes.  A thread has 8 neighbouring columns (16-byte loads), 32 threads
// a row of 256 columns, 8 rows at a time, the loads of the next two rows of
// both (or four rows of dy alone) in flight: 64 KB an SM with four CTAs on it.  A
// thread's fp32 run is at most 16 terms, then fp64, kept in shared memory: in
// registers the sums made the fourth CTA's 64 registers spill (287 us against
// 247, 16384 x 14336 of SiLU with dz written: 5.7 TB/s of 6.55; GELU 258, sums
// alone 164).  With a single chunk the sums are dbias.
template <bool HAS_Z>
__global__ void __launch_bounds__(256, 4) linear_dz_kernel(const LinearDzArgs a) {
  constexpr int AHEAD = HAS_Z ? 2 : 4;
  __shared__ double sums[8][256];
  const int tid = threadIdx.x, cv = tid & 31, rl = tid >> 5;
  const int col = blockIdx.x * 256 + cv * 8;
  const int row_end = min(a.T, (static_cast<int>(blockIdx.y) + 1) * a.chunk_rows);
  griddep_wait();
  double* acc = &sums[rl][cv];  // column j of this thread: acc[32 * j]
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[32 * j] = 0.0;
  if (col < a.N) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int row_first = static_cast<int>(blockIdx.y) * a.chunk_rows + rl;
    float run[8] = {};
    int terms = 0;
    uint4 g[AHEAD], z[HAS_Z ? AHEAD : 1];
    auto load = [&](int r, int s) {
      g[s] = r < row_end ? ld_global16(a.dy + r * a.lddy + col) : zero;
      if (HAS_Z) z[s] = r < row_end ? ld_global16(a.z + r * a.ldz + col) : zero;
    };
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) load(row_first + 8 * s, s);
    for (int r0 = row_first; r0 < row_end; r0 += 8 * AHEAD) {
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        const int r = r0 + 8 * s;
        float v[8], zz[8];
        unpack8(g[s], v);
        if (HAS_Z) unpack8(z[s], zz);
        load(r + 8 * AHEAD, s);
        if (HAS_Z) act_grad_apply(v, zz, a.act);
        if (a.dz != nullptr && r < row_end)
          *reinterpret_cast<uint4*>(a.dz + static_cast<long long>(r) * a.N + col) = pack8(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) run[j] += v[j];  // rows past the end add zero
      }
      if ((terms += AHEAD) == 16) {
        terms = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[32 * j] += static_cast<double>(run[j]);
          run[j] = 0.f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[32 * j] += static_cast<double>(run[j]);
  }
  griddep_launch_dependents();
  if (a.dbias == nullptr) return;
  __syncthreads();
  const int c = blockIdx.x * 256 + tid;
  if (c >= a.N) return;
  double s = 0.0;
  for (int i = 0; i < 8; ++i) s += sums[i][tid % 8 * 32 + tid / 8];
  if (a.chunks == 1)
    a.dbias[c] = static_cast<float>(s);
  else
    a.part[static_cast<size_t>(blockIdx.y) * a.N + c] = s;
}

// dbias_n: the chunks' sums.  32 columns a CTA; warp w takes chunks w, w + 8, ...,
// and the eight sums are added in warp order.
// AFTER: a product was launched between this kernel and linear_dz_kernel.  This one
// starts once all CTAs of the product let it, which they do after their own wait for
// what came before them, so the partial sums are complete and in L2 by then, and it
// works beside the product.  Its own wait, which would make them visible to every
// kind of load, comes after it reads them: so it reads them from L2 (__ldcg), past an
// L1 that may hold lines of an earlier call's sums at the same addresses.  It waits
// for the product before it ends, since whoever comes next waits for this kernel only.
template <bool AFTER>
__global__ void __launch_bounds__(256) linear_dbias_kernel(const double* part, float* dbias, int N, int chunks) {
  __shared__ double sums[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, n = blockIdx.x * 32 + lane;
  if (!AFTER) griddep_wait();
  griddep_launch_dependents();
  double s = 0.0;
  if (n < N) {
#pragma unroll 8
    for (int c = w; c < chunks; c += 8) s += __ldcg(part + static_cast<size_t>(c) * N + n);
  }
  sums[w][lane] = s;
  __syncthreads();
  if (w == 0 && n < N) {
    for (int i = 1; i < 8; ++i) s += sums[i][lane];
    dbias[n] = static_cast<float>(s);
  }
  if (AFTER) griddep_wait();
}

}  // namespace

cudaError_t launch_linear_dz(const LinearDzArgs& a, cudaStream_t s) {
  return launch_pdl(a.act != MOE_ACT_NONE ? linear_dz_kernel<true> : linear_dz_kernel<false>,
                             dim3((a.N + 255) / 256, a.chunks), dim3(256), 0, s, a);
}

cudaError_t launch_linear_dbias(const LinearDzArgs& a, bool after_product, cudaStream_t s) {
  if (a.dbias == nullptr || a.chunks == 1) return cudaSuccess;
  return launch_pdl(after_product ? linear_dbias_kernel<true> : linear_dbias_kernel<false>, dim3((a.N + 31) / 32),
                    dim3(256), 0, s, static_cast<const double*>(a.part), a.dbias, a.N, a.chunks);
}

}  // namespace moe
