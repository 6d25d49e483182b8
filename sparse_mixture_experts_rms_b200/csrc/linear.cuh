// linear.cuh -- the linear layer's activations, their derivatives and bf16
// packing.
#pragma once

#include "moe_internal.h"
#include "ptx.cuh"

namespace moe {

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Loads of what the kernel before may have written while this one was already
// starting: `ld.global.nc` (__ldg) is for memory that nobody writes while the kernel
// runs.  As asm they keep its freedom to move past the kernel's own stores, though
// not past griddep_wait; plain loads made linear_dz_kernel spill (16384 x 14336 of
// SiLU 181 -> 193 us).
__device__ __forceinline__ uint4 ld_global16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_global(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// Two fp32 in a register pair: one instruction adds, multiplies or
// multiply-adds both.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair_of(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pair_of(a, a); }
__device__ __forceinline__ void halves(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ f32x2 ex2_pair(f32x2 v) {
  float a, b;
  halves(v, a, b);
  return pair_of(ex2_approx(a), ex2_approx(b));
}
__device__ __forceinline__ f32x2 rcp_pair(f32x2 v) {
  float a, b;
  halves(v, a, b);
  return pair_of(rcp_approx(a), rcp_approx(b));
}
// 1 / (1 + 2^w)
__device__ __forceinline__ f32x2 logistic2(f32x2 w) { return rcp_pair(add2(ex2_pair(w), both(1.0f))); }

// e^(-z^2/2)
__device__ __forceinline__ f32x2 bell2(f32x2 z) { return ex2_pair(mul2(mul2(z, z), both(-0.72134752044448171f))); }
// |z|, at most 1e30: a zero factor beside it stays one where z is infinite
__device__ __forceinline__ f32x2 magnitude2(f32x2 z) {
  float a, b;
  halves(z, a, b);
  return pair_of(fminf(fabsf(a), 1e30f), fminf(fabsf(b), 1e30f));
}
// Phi(-|z|) / e^(-z^2/2) = erfcx(|z| / sqrt 2) / 2 for the normal distribution's
// Phi: a polynomial without constant term in t = 1 / (1 + 0.35 |z|), fitted to
// a small largest relative error over 0 <= |z| <= 14 (beyond, e^(-z^2/2) is zero in
// fp32): 6.0e-8 with these coefficients in exact arithmetic, reached at both
// ends; the evaluation in fp32 adds a few roundings of that size.
__device__ __forceinline__ f32x2 phi_ratio2(f32x2 az) {
  const f32x2 t = rcp_pair(fma2(both(0.35f), az, both(1.0f)));
  f32x2 p = both(-0.02914595790207386f);
  p = fma2(p, t, both(0.14397183060646057f));
  p = fma2(p, t, both(-0.2557145357131958f));
  p = fma2(p, t, both(0.15917445719242096f));
  p = fma2(p, t, both(-0.02311003766953945f));
  p = fma2(p, t, both(0.10550808906555176f));
  p = fma2(p, t, both(0.1198328509926796f));
  p = fma2(p, t, both(0.13986186683177948f));
  p = fma2(p, t, both(0.13962140679359436f));
  return mul2(p, t);
}
// GELU_TANH's -2u log2(e), u = sqrt(2/pi) (z + 0.044715 z^3)
__device__ __forceinline__ f32x2 tanh_arg2(f32x2 z) {
  return mul2(z, fma2(mul2(z, z), both(-0.10294324f), both(-2.3022082f)));
}

// act(z) and act'(z) of two values, fp32, each form chosen to keep its relative
// accuracy for z far below zero, where 1 + erf and 1 + tanh would cancel.
//  SILU       z s, s = sigmoid(z);  derivative s (1 + z (1 - s))
//  GELU       z Phi(z) = max(z, 0) - |z| Phi(-|z|);
//             derivative Phi(z) + z phi(z), phi(z) = e^(-z^2/2) / sqrt(2 pi)
//  GELU_TANH  with u as above: (1 + tanh u) / 2 = sigmoid(2u) = s, value z s,
//             derivative s + z s (1 - s) 2 u'
// 1 - s cancels for large z: an error of two half steps of 1 there, |z| or
// |2 z u'| times that in a derivative that is about 1.
// They take the hardware's exponential and reciprocal as they are (2^-22 and
// 2^-23 relative, and 2^-23 of the exponential's argument for the argument's
// rounding, which matters only where e^-|z| has made the result small; results
// below 1e-36 may be flushed to zero), and two values an instruction otherwise.
template <int ACT>
__device__ __forceinline__ f32x2 act_value2(f32x2 z) {
  if (ACT == MOE_ACT_SILU) return mul2(z, logistic2(mul2(z, both(-1.4426950408889634f))));
  if (ACT == MOE_ACT_GELU_TANH) return mul2(z, logistic2(tanh_arg2(z)));
  float a, b;
  halves(z, a, b);
  if (ACT == MOE_ACT_GELU) {
    const f32x2 az = magnitude2(z), half = mul2(phi_ratio2(az), bell2(z));
    return fma2(mul2(az, both(-1.0f)), half, pair_of(fmaxf(a, 0.f), fmaxf(b, 0.f)));
  }
  return pair_of(a > 0.f || a != a ? a : 0.f, b > 0.f || b != b ? b : 0.f);  // RELU
}

template <int ACT>
__device__ __forceinline__ f32x2 act_grad2(f32x2 z) {
  const f32x2 one = both(1.0f);
  if (ACT == MOE_ACT_SILU) {
    const f32x2 s = logistic2(mul2(z, both(-1.4426950408889634f)));
    return mul2(s, fma2(z, fma2(s, both(-1.0f), one), one));
  }
  if (ACT == MOE_ACT_GELU_TANH) {
    const f32x2 s = logistic2(tanh_arg2(z));
    // 2 u' kept finite: 1 - s or z s is 0 long before, and 0 times infinity is not
    float a, b;
    halves(fma2(mul2(z, z), both(0.21406444881780073f), both(1.5957691216057308f)), a, b);
    const f32x2 du2 = pair_of(fminf(a, 1e30f), fminf(b, 1e30f));
    return fma2(mul2(z, s), mul2(fma2(s, both(-1.0f), one), du2), s);
  }
  float a, b;
  halves(z, a, b);
  if (ACT == MOE_ACT_GELU) {
    const f32x2 e = bell2(z), half = mul2(phi_ratio2(magnitude2(z)), e), rest = fma2(half, both(-1.0f), one);
    float h0, h1, r0, r1;
    halves(half, h0, h1);
    halves(rest, r0, r1);
    return fma2(mul2(z, both(0.39894228040143268f)), e, pair_of(a > 0.f ? r0 : h0, b > 0.f ? r1 : h1));
  }
  return pair_of(a > 0.f ? 1.f : (a != a ? a : 0.f), b > 0.f ? 1.f : (b != b ? b : 0.f));  // RELU
}

template <int ACT, int N>
__device__ __forceinline__ void act_all(float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 2) halves(act_value2<ACT>(pair_of(v[j], v[j + 1])), v[j], v[j + 1]);
}
template <int ACT, int N>
__device__ __forceinline__ void act_grad_all(float (&v)[N], const float (&z)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 2)
    halves(mul2(pair_of(v[j], v[j + 1]), act_grad2<ACT>(pair_of(z[j], z[j + 1]))), v[j], v[j + 1]);
}

// act over a register array, the activation's branch outside the loop.
template <int N>
__device__ __forceinline__ void act_apply(float (&v)[N], int act) {
  switch (act) {
    case MOE_ACT_RELU: act_all<MOE_ACT_RELU>(v); break;
    case MOE_ACT_SILU: act_all<MOE_ACT_SILU>(v); break;
    case MOE_ACT_GELU: act_all<MOE_ACT_GELU>(v); break;
    case MOE_ACT_GELU_TANH: act_all<MOE_ACT_GELU_TANH>(v); break;
    default: break;
  }
}

// v *= act'(z), the branch outside the loop.
template <int N>
__device__ __forceinline__ void act_grad_apply(float (&v)[N], const float (&z)[N], int act) {
  switch (act) {
    case MOE_ACT_RELU: act_grad_all<MOE_ACT_RELU>(v, z); break;
    case MOE_ACT_SILU: act_grad_all<MOE_ACT_SILU>(v, z); break;
    case MOE_ACT_GELU: act_grad_all<MOE_ACT_GELU>(v, z); break;
    case MOE_ACT_GELU_TANH: act_grad_all<MOE_ACT_GELU_TANH>(v, z); break;
    default: break;
  }
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// 4 floats from a shared::cluster address (16-byte aligned).
__device__ __forceinline__ void ld_cluster_f32x4(uint32_t addr, float& a, float& b, float& c, float& d) {
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a), "=f"(b), "=f"(c), "=f"(d) : "r"(addr));
}

// Finishes U groups of 4 lanes, (c[u], l[u]) where in[u]: adds up the S ranks'
// sums at from[u] (rank s of the cluster: first + s * step) in rank order, then
// bias, z, activation, residual and y.  The residuals' and the sums' loads of
// all groups are under way together.  Groups of 4, so that the neighbouring
// threads' 16-byte loads from another CTA's shared memory lie side by side.
template <int U>
__device__ __forceinline__ void finish_groups(const LinearArgs& a, const int (&c)[U], const int (&l)[U],
                                              const bool (&in)[U], const uint32_t (&from)[U], int S, uint32_t first,
                                              uint32_t step) {
  uint2 res[U];
  float v[4 * U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    res[u] = in[u] && a.residual != nullptr ? *reinterpret_cast<const uint2*>(a.residual + c[u] * a.ldr + l[u])
                                            : make_uint2(0u, 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * u + j] = in[u] && a.bias != nullptr ? ld_global(a.bias + l[u] + j) : 0.f;
  }
  float sum[4 * U];
#pragma unroll
  for (int j = 0; j < 4 * U; ++j) sum[j] = 0.f;
#pragma unroll 2
  for (int s = 0; s < S; ++s) {
    float x[4 * U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (in[u])
        ld_cluster_f32x4(map_to_cta(from[u], first + s * step), x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (in[u]) sum[4 * u + j] += x[4 * u + j];
  }
#pragma unroll
  for (int j = 0; j < 4 * U; ++j) v[j] += sum[j];
  if (a.z != nullptr) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (in[u])
        *reinterpret_cast<uint2*>(a.z + c[u] * a.ldz + l[u]) =
            make_uint2(pack2(v[4 * u], v[4 * u + 1]), pack2(v[4 * u + 2], v[4 * u + 3]));
  }
  act_apply(v, a.act);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!in[u]) continue;
    if (a.residual != nullptr) {
      v[4 * u] += __uint_as_float(res[u].x << 16);
      v[4 * u + 1] += __uint_as_float(res[u].x & 0xFFFF0000u);
      v[4 * u + 2] += __uint_as_float(res[u].y << 16);
      v[4 * u + 3] += __uint_as_float(res[u].y & 0xFFFF0000u);
    }
    *reinterpret_cast<uint2*>(a.out + c[u] * a.ldo + l[u]) =
        make_uint2(pack2(v[4 * u], v[4 * u + 1]), pack2(v[4 * u + 2], v[4 * u + 3]));
  }
}

}  // namespace moe
