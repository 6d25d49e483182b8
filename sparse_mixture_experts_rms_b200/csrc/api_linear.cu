// api_linear.cu -- the C ABI of the dense linear layer: argument checks,
// workspace layout and launch sequencing.
#include <algorithm>
#include <initializer_list>

#include "api_detail.h"

namespace moe {
namespace api {
namespace {

constexpr int64_t kMaxLd = int64_t(1) << 38;  // a TMA row distance is below 2^40 bytes
constexpr int32_t kMaxExtent = 1 << 30;       // tile arithmetic is 32-bit
constexpr size_t kFwdBytes = 4096;            // the forward's workspace: the header, and room for more like it

struct LinearLayout {
  size_t part, dz, total;
  int chunks, chunk_rows;
};

int64_t ld_of(int64_t ld, int width) { return ld != 0 ? ld : width; }

moe_status_t linear_validate(const moe_linear_t* l) {
  if (l == nullptr) return MOE_ERR_INVALID_ARG;
  if (l->T < 0 || l->K <= 0 || l->N <= 0 || l->K % 8 != 0 || l->N % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (l->activation < MOE_ACT_NONE || l->activation > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  if (l->T > kMaxExtent || l->K > kMaxExtent || l->N > kMaxExtent) return MOE_ERR_UNSUPPORTED;
  const int64_t lds[8] = {l->ldx, l->ldw, l->ldr, l->ldy, l->ldz, l->lddy, l->lddx, l->lddw};
  const int width[8] = {l->K, l->N, l->N, l->N, l->N, l->N, l->K, l->N};
  for (int i = 0; i < 8; ++i) {
    if (lds[i] != 0 && (lds[i] < width[i] || lds[i] % 8 != 0)) return MOE_ERR_INVALID_ARG;
    if (lds[i] > kMaxLd) return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

LinearLayout linear_layout(const moe_linear_t& l) {
  LinearLayout L{};
  size_t off = kHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align_up(bytes > 0 ? bytes : 1, 1024);
    return o;
  };
  // column sums: chunks of at least 32 rows (a thread's four loads in flight), four CTAs per SM
  // over the 256-column blocks; two or three times as many, shorter ones where whole chunks would
  // leave more than 3 % of the slots empty (16384 x 14336: 253 us with 10 chunks of 56 blocks in
  // 592 slots, 247 with 21 in 1184; but 8192 x 8192: 65 with 18 of 32, 66 with 37)
  const int nb = (l.N + 255) / 256;
  const int most = (l.T + 31) / 32;
  int waves = 1;
  while (waves < 3 && 592 * waves / nb * nb * 100 < 97 * 592 * waves) ++waves;
  L.chunks = std::max(1, std::min(most, 592 * waves / nb));
  L.chunk_rows = (l.T + L.chunks - 1) / L.chunks;
  L.part = take(static_cast<size_t>(L.chunks) * l.N * 8);
  L.dz = take(static_cast<size_t>(l.T) * l.N * 2);
  L.total = std::max(off, kFwdBytes);
  return L;
}

moe_status_t linear_ws(void* ws, size_t ws_bytes, size_t needed) {
  if (ws == nullptr || ws_bytes < needed) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// An output that starts where another argument does.
bool same(const void* out, std::initializer_list<const void*> others) {
  return out != nullptr && std::find(others.begin(), others.end(), out) != others.end();
}

const __nv_bfloat16* bf(const moe_bf16_t* p) { return reinterpret_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* bf(moe_bf16_t* p) { return reinterpret_cast<__nv_bfloat16*>(p); }

// The map of an operand: `mn` lanes or columns by `red`; a stage takes `box` x 64 of it.
bool operand_map(CUtensorMap* m, const void* p, bool by_mn, bool* three_d, uint64_t mn, uint64_t red, int64_t ld,
                 int box) {
  *three_d = by_mn && mn % 64 == 0;
  if (*three_d) return make_map_atoms(m, p, mn, red, ld, box / 64);
  return by_mn ? make_map(m, p, mn, red, ld, 64, 64) : make_map(m, p, red, mn, ld, 64, box);
}

// Shape of a product: its operands' majors, lanes, columns and reduction.
LinearArgs product_of(const moe_linear_t& l, int product) {
  LinearArgs a{};
  if (product == MOE_LINEAR_FWD) {  // [T, N]: lanes n, columns t, reduction k
    a.a_mn = true;
    a.L = l.N;
    a.C = l.T;
    a.red = l.K;
  } else if (product == MOE_LINEAR_DX) {  // [T, K]: lanes k, columns t, reduction n
    a.L = l.K;
    a.C = l.T;
    a.red = l.N;
  } else {  // [K, N]: lanes n, columns k, reduction t
    a.a_mn = a.b_mn = true;
    a.L = l.N;
    a.C = l.K;
    a.red = l.T;
  }
  return a;
}

// Plans a product on the current device; whether it is linear_pair.cu's, the
// kernel whose plan is the shorter.
bool plan_product(LinearArgs& a) {
  const LinearSlots slots = linear_slots_of_current_device();
  const double split = plan_linear_split(a, slots), pair = plan_linear_pair(a, slots);
  if (pair < split) a.bn = a.pair_bn;
  return pair < split;
}

moe_status_t run_product(LinearArgs& a, void* ws, cudaStream_t s) {
  a.err = at<uint32_t>(ws, 0);
  a.wait_ctl = at<uint32_t>(ws, kWaitCtlOffset);
  const uint64_t L = static_cast<uint64_t>(a.L), C = static_cast<uint64_t>(a.C), R = static_cast<uint64_t>(a.red);
  CUtensorMap ma, mb, my, mz, mr;
  if (plan_product(a)) {
    if (!operand_map(&ma, a.a, a.a_mn, &a.a_3d, L, R, a.lda, a.bn / 2) ||
        !operand_map(&mb, a.b, a.b_mn, &a.b_3d, C, R, a.ldb, 128) ||
        !make_map(&my, a.out, L, C, a.ldo, 32, 32, true))
      return MOE_ERR_CUDA;
    mz = mr = my;  // unused ones repeat another
    if ((a.z != nullptr && !make_map(&mz, a.z, L, C, a.ldz, 32, 32, true)) ||
        (a.residual != nullptr && !make_map(&mr, a.residual, L, C, a.ldr, 32, 32, true)))
      return MOE_ERR_CUDA;
    return cuda_status(launch_linear_pair(a, ma, mb, my, mz, mr, gemm_grid_of_current_device(), s));
  }
  if (!operand_map(&ma, a.a, a.a_mn, &a.a_3d, L, R, a.lda, 128) ||
      !operand_map(&mb, a.b, a.b_mn, &a.b_3d, C, R, a.ldb, a.bn))
    return MOE_ERR_CUDA;
  return cuda_status(launch_linear_split(a, ma, mb, s));
}

}  // namespace
}  // namespace api
}  // namespace moe

using namespace moe;
using namespace moe::api;

extern "C" {

size_t moe_linear_workspace_size(const moe_linear_t* lin) {
  if (linear_validate(lin) != MOE_OK) return 0;
  return linear_layout(*lin).total;
}

size_t moe_linear_fwd_workspace_size(const moe_linear_t* lin) {
  return linear_validate(lin) == MOE_OK ? kFwdBytes : 0;
}

moe_status_t moe_linear_plan(const moe_linear_t* lin, int32_t product, int32_t has_residual, int32_t has_z,
                             moe_linear_plan_t* plan) {
  moe_status_t st = linear_validate(lin);
  if (st != MOE_OK) return st;
  if (plan == nullptr || lin->T == 0 || product < MOE_LINEAR_FWD || product > MOE_LINEAR_DW) return MOE_ERR_INVALID_ARG;
  int sms;
  if ((st = device_ready(&sms)) != MOE_OK) return st;
  LinearArgs a = product_of(*lin, product);
  // the plan asks whether these are there, not where
  if (product == MOE_LINEAR_FWD && has_residual) a.residual = reinterpret_cast<const __nv_bfloat16*>(plan);
  if (product == MOE_LINEAR_FWD && has_z) a.z = reinterpret_cast<__nv_bfloat16*>(plan);
  const bool pair = plan_product(a);
  plan->kernel = !pair ? MOE_LINEAR_SPLIT : (a.pair_split > 1 ? MOE_LINEAR_PAIR_SPLIT : MOE_LINEAR_PAIR);
  plan->tile = a.bn;
  plan->split = pair ? a.pair_split : a.split;
  return MOE_OK;
}

moe_status_t moe_linear_fwd(const moe_linear_t* lin, const moe_bf16_t* x, const moe_bf16_t* W, const float* bias,
                            const moe_bf16_t* residual, moe_bf16_t* y, moe_bf16_t* z, void* ws, size_t ws_bytes,
                            void* stream) {
  moe_status_t st = linear_validate(lin);
  if (st != MOE_OK) return st;
  const moe_linear_t& l = *lin;
  if (l.T == 0) return MOE_OK;
  if (!x || !W || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(bias, 4) || !aligned(residual, 16) || !aligned(y, 16) ||
      !aligned(z, 16))
    return MOE_ERR_ALIGNMENT;
  if (same(y, {x, W, z}) || same(z, {x, W, residual})) return MOE_ERR_INVALID_ARG;
  if (residual == y && l.T > 1 && ld_of(l.ldr, l.N) != ld_of(l.ldy, l.N)) return MOE_ERR_INVALID_ARG;
  if ((st = linear_ws(ws, ws_bytes, kFwdBytes)) != MOE_OK) return st;
  int sms;
  if ((st = device_ready(&sms)) != MOE_OK) return st;
  LinearArgs a = product_of(l, MOE_LINEAR_FWD);
  a.a = bf(W);
  a.lda = ld_of(l.ldw, l.N);
  a.b = bf(x);
  a.ldb = ld_of(l.ldx, l.K);
  a.bias = bias;
  a.residual = bf(residual);
  a.ldr = ld_of(l.ldr, l.N);
  a.out = bf(y);
  a.ldo = ld_of(l.ldy, l.N);
  a.z = bf(z);
  a.ldz = ld_of(l.ldz, l.N);
  a.act = l.activation;
  return run_product(a, ws, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_linear_bwd(const moe_linear_t* lin, const moe_bf16_t* x, const moe_bf16_t* W, const moe_bf16_t* z,
                            const moe_bf16_t* dy, moe_bf16_t* dx, moe_bf16_t* dW, float* dbias, void* ws,
                            size_t ws_bytes, void* stream) {
  moe_status_t st = linear_validate(lin);
  if (st != MOE_OK) return st;
  const moe_linear_t& l = *lin;
  if (!dx && !dW && !dbias) return MOE_OK;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(z, 16) || !aligned(dy, 16) || !aligned(dx, 16) ||
      !aligned(dW, 16) || !aligned(dbias, 4))
    return MOE_ERR_ALIGNMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms;
  if (l.T == 0) {  // sums over no rows
    if (!dW && !dbias) return MOE_OK;
    if ((st = device_ready(&sms)) != MOE_OK) return st;
    if (dW && (st = cuda_status(cudaMemset2DAsync(dW, ld_of(l.lddw, l.N) * 2, 0, static_cast<size_t>(l.N) * 2,
                                                  l.K, s))) != MOE_OK)
      return st;
    if (dbias) return cuda_status(cudaMemsetAsync(dbias, 0, static_cast<size_t>(l.N) * 4, s));
    return MOE_OK;
  }
  const bool has_act = l.activation != MOE_ACT_NONE;
  if (!dy || (has_act && !z) || (dx && !W) || (dW && !x)) return MOE_ERR_INVALID_ARG;
  if (same(dx, {x, W, z, dy, dW}) || same(dW, {x, W, z, dy}) || same(dbias, {x, W, z, dy, dx, dW}))
    return MOE_ERR_INVALID_ARG;
  const LinearLayout L = linear_layout(l);
  if ((st = linear_ws(ws, ws_bytes, L.total)) != MOE_OK) return st;
  if ((st = device_ready(&sms)) != MOE_OK) return st;
  const __nv_bfloat16* dz = bf(dy);
  int64_t lddz = ld_of(l.lddy, l.N);
  const bool make_dz = has_act && (dx || dW);
  LinearDzArgs a{};
  if (make_dz || dbias) {
    a.dy = bf(dy);
    a.lddy = ld_of(l.lddy, l.N);
    a.z = bf(z);
    a.ldz = ld_of(l.ldz, l.N);
    a.dz = make_dz ? at<__nv_bfloat16>(ws, L.dz) : nullptr;
    a.part = at<double>(ws, L.part);
    a.dbias = dbias;
    a.T = l.T;
    a.N = l.N;
    a.chunks = L.chunks;
    a.chunk_rows = L.chunk_rows;
    a.act = l.activation;
    if ((st = cuda_status(launch_linear_dz(a, s))) != MOE_OK) return st;
    if (make_dz) {
      dz = a.dz;
      lddz = l.N;
    }
  }
  if (dx) {
    LinearArgs p = product_of(l, MOE_LINEAR_DX);
    p.a = bf(W);
    p.lda = ld_of(l.ldw, l.N);
    p.b = dz;
    p.ldb = lddz;
    p.out = bf(dx);
    p.ldo = ld_of(l.lddx, l.K);
    if ((st = run_product(p, ws, s)) != MOE_OK) return st;
  }
  if (dW) {
    LinearArgs p = product_of(l, MOE_LINEAR_DW);
    p.a = dz;
    p.lda = lddz;
    p.b = bf(x);
    p.ldb = ld_of(l.ldx, l.K);
    p.out = bf(dW);
    p.ldo = ld_of(l.lddw, l.N);
    if ((st = run_product(p, ws, s)) != MOE_OK) return st;
  }
  return cuda_status(launch_linear_dbias(a, dx || dW, s));
}

}  // extern "C"
