// The gated products' activations, a(g) = g sig(p(g)) with sig(x) = 1 / (1 + exp(-x)):
//   SP_ACT_SILU       p(g) = g
//   SP_ACT_GELU_TANH  p(g) = 2 sqrt(2 / pi) (g + 0.044715 g^3), as 0.5 (1 + tanh(p / 2)) = sig(p)
// In fp32, with fused steps written out: a value does not depend on the tile that holds it.
#pragma once

#include <hip/hip_runtime.h>

#include "spmm_csr_spmv.h"

namespace spx {

constexpr float kGelu = 1.5957691216057308f;            // 2 sqrt(2 / pi)
constexpr float kGelu3 = 1.5957691216057308f * 0.044715f;

// Where exp(-p) overflows sig is 0, and so is a of a finite g (its limit), not NaN.
__device__ __forceinline__ float gate_sig(float g, int act) {
#pragma clang fp contract(off)
    const float p = act == SP_ACT_SILU ? g : g * fmaf(kGelu3, g * g, kGelu);
    return 1.0f / (1.0f + expf(-p));
}

// a(g) u
__device__ __forceinline__ float gated(float g, float u, int act) {
#pragma clang fp contract(off)
    return g * gate_sig(g, act) * u;
}

// The gradients of a(g) u, given its own: dg = dh u a'(g) with a' = sig + g sig (1 - sig) p', and du = dh a(g).
// Where sig is 0 so are a and a', where it is 1 so is a': g p' may be beyond fp32's range there, and g and u Infs (sums
// that the operands' type cannot hold), which would make NaN of a limit.
__device__ __forceinline__ void gated_backward(float dh, float g, float u, int act, float& dg, float& du) {
#pragma clang fp contract(off)
    const float s = gate_sig(g, act);
    const float dp = act == SP_ACT_SILU ? 1.0f : fmaf(3.0f * kGelu3, g * g, kGelu);
    const auto held = [](float v) { return fabsf(v) == __builtin_inff() ? 0.0f : v; };
    du = dh * (s == 0.0f ? s * held(g) : g * s);
    dg = s == 0.0f ? dh * s * held(u) : dh * u * (s == 1.0f ? s : s * fmaf(g * dp, 1.0f - s, 1.0f));
}

}  // namespace spx
