// api_few.cu -- the C ABI of the few-token layer: workspace layout, argument
// checks and the launch.
#include "api_detail.h"

namespace moe {
namespace api {
namespace {

constexpr size_t kFewBarA = 32, kFewBarX = 36;  // header words that are zero between calls

struct FewLayout {
  size_t sync, xg, lpart, H, upart, y, ypart, total;
  int ldh;
};

moe_status_t few_validate(const moe_config_t* c) {
  const moe_status_t st = validate(c);
  if (st != MOE_OK) return st;
  if (c->T > MOE_FEW_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
  // the kernel's 32-bit share arithmetic: stages (64 x 128 weights of W1 and W3) times CTAs
  const int64_t stages = static_cast<int64_t>(c->ffn_offsets[c->E]) / 64 * ((c->d_model + 127) / 128);
  return stages * kFewMaxGrid >= (int64_t(1) << 31) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

FewLayout few_layout(const moe_config_t& c) {
  FewLayout L{};
  size_t off = kHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align_up(bytes > 0 ? bytes : 1, 256);
    return o;
  };
  const size_t T = static_cast<size_t>(c.T), tk = T * c.k, d = static_cast<size_t>(c.d_model);
  for (int e = 0; e < c.E; ++e) {
    const int w = c.ffn_offsets[e + 1] - c.ffn_offsets[e];
    L.ldh = w > L.ldh ? w : L.ldh;
  }
  L.sync = take(kFewSyncWords * 4);
  L.xg = take(2 * T * d * 2);
  L.H = take(2 * tk * static_cast<size_t>(L.ldh) * 2);
  L.lpart = take(T * 16 * (kMaxExperts + 1) * 8);
  L.upart = take(2 * static_cast<size_t>(kFewMaxGrid) * 2 * 2 * T * 128 * 4);
  L.y = take(tk * d * 4);
  L.ypart = take(2 * static_cast<size_t>(kFewMaxGrid) * T * 256 * 4);
  L.total = off;
  return L;
}

}  // namespace
}  // namespace api
}  // namespace moe

using namespace moe;
using namespace moe::api;

extern "C" {

size_t moe_few_workspace_size(const moe_config_t* cfg) {
  if (few_validate(cfg) != MOE_OK) return 0;
  return few_layout(*cfg).total;
}

moe_status_t moe_layer_fwd_few(const moe_config_t* cfg, const moe_bf16_t* x, const moe_bf16_t* gamma,
                               const moe_bf16_t* Wr, const float* bias, const moe_bf16_t* W1,
                               const moe_bf16_t* W3, const moe_bf16_t* W2, const moe_bf16_t* residual,
                               moe_bf16_t* out, int32_t* expert_idx, float* gate, float* r, int32_t* counts,
                               void* ws, size_t ws_bytes, void* stream) {
  moe_status_t st = few_validate(cfg);
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms;
  if (cfg->T == 0) {  // no tokens: only the optional counts are written (zeros)
    if (counts == nullptr) return MOE_OK;
    if (!aligned(counts, 4)) return MOE_ERR_ALIGNMENT;
    if ((st = device_ready(&sms)) != MOE_OK) return st;
    return cuda_status(cudaMemsetAsync(counts, 0, cfg->E * sizeof(int32_t), s));
  }
  if (!x || !gamma || !Wr || !W1 || !W3 || !W2 || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(gamma, 16) || !aligned(Wr, 2) || !aligned(bias, 4) || !aligned(W1, 16) ||
      !aligned(W3, 16) || !aligned(W2, 16) || !aligned(residual, 16) || !aligned(out, 16) ||
      !aligned(expert_idx, 4) || !aligned(gate, 4) || !aligned(r, 4) || !aligned(counts, 4))
    return MOE_ERR_ALIGNMENT;
  const FewLayout L = few_layout(*cfg);
  if (ws == nullptr || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return MOE_ERR_ALIGNMENT;
  if ((st = device_ready(&sms)) != MOE_OK) return st;
  const moe_config_t& c = *cfg;
  if (sms < c.T) return MOE_ERR_UNSUPPORTED;  // few_route: a CTA takes one token's slice
  FewArgs a{};
  a.x = reinterpret_cast<const __nv_bfloat16*>(x);
  a.gamma = reinterpret_cast<const __nv_bfloat16*>(gamma);
  a.Wr = reinterpret_cast<const __nv_bfloat16*>(Wr);
  a.W1 = reinterpret_cast<const __nv_bfloat16*>(W1);
  a.W3 = reinterpret_cast<const __nv_bfloat16*>(W3);
  a.W2 = reinterpret_cast<const __nv_bfloat16*>(W2);
  a.bias = bias;
  a.residual = reinterpret_cast<const __nv_bfloat16*>(residual);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.idx_out = expert_idx;
  a.gate_out = gate;
  a.r_out = r;
  a.counts_out = counts;
  a.xg = at<__nv_bfloat16>(ws, L.xg);
  a.H = at<__nv_bfloat16>(ws, L.H);
  a.h_lo = static_cast<size_t>(c.T) * c.k * L.ldh;
  a.bar_a = at<uint32_t>(ws, kFewBarA);
  a.bar_x = at<uint32_t>(ws, kFewBarX);
  a.lpart = at<double>(ws, L.lpart);
  a.sync = at<uint32_t>(ws, L.sync);
  a.bar_b = a.sync;
  a.done = a.sync + 32;
  a.tile_cnt = a.sync + 64;
  a.upart = at<float>(ws, L.upart);
  a.y = at<float>(ws, L.y);
  a.ypart = at<float>(ws, L.ypart);
  a.err = at<uint32_t>(ws, 0);
  a.wait_ctl = at<uint32_t>(ws, kWaitCtlOffset);
  a.T = c.T;
  a.d = c.d_model;
  a.E = c.E;
  a.k = c.k;
  a.F = c.ffn_offsets[c.E];
  a.ldh = L.ldh;
  a.capacity = static_cast<int>(capacity_of(c));
  a.inv_d = 1.0 / c.d_model;
  a.eps = c.eps;
  a.renormalize = c.renormalize ? 1 : 0;
  for (int e = 0; e <= c.E; ++e) a.ffn.off[e] = c.ffn_offsets[e];
  CUtensorMap m1, m3, m2, mx, mh;
  const uint64_t d = static_cast<uint64_t>(c.d_model), F = static_cast<uint64_t>(a.F);
  const uint64_t T2 = 2 * static_cast<uint64_t>(c.T), ldh = static_cast<uint64_t>(a.ldh);
  if (!make_map(&m1, W1, F, d, F, 64, 64) || !make_map(&m3, W3, F, d, F, 64, 64) ||
      !make_map(&m2, W2, d, F, d, 64, 64) || !make_map(&mx, a.xg, d, T2, d, 64, 1) ||
      !make_map(&mh, a.H, ldh, T2 * c.k, ldh, 64, 8))
    return MOE_ERR_CUDA;
  return cuda_status(launch_few(a, m1, m3, m2, mx, mh, sms, s));
}

}  // extern "C"
