// The gate activations of a gated MLP block and their slopes.  Both are x
// times the logistic function of z(x):
//   SiLU          z = x
//   GeLU (tanh)   z = 2 sqrt(2/pi) (x + 0.044715 x^3)   (Hendrycks & Gimpel 2016)
// act(x) = x s, act'(x) = s + x s (1 - s) z'(x) with s = 1 / (1 + e^-z).  Two
// MUFU operations per value (the exponential, two units in the last place, and
// the reciprocal, one): these kernels wait for memory or for the tensor cores,
// and the reciprocal on the FMA pipe that a GeLU epilogue without a gate uses
// costs eight instructions more.
#pragma once

#include "gelu.cuh"
#include "shmm.h"

__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

template <int ACT>
__device__ __forceinline__ float gate_z2(float x) {  // z(x) log2(e)
    if (ACT == SHMM_SILU) return x * 1.4426950408889634f;
    const float k0 = 2.0f * 0.7978845608028654f * 1.4426950408889634f;
    return x * fmaf(x * x, k0 * 0.044715f, k0);
}

// e^-z may overflow: its reciprocal is then 0, as s is.
template <int ACT>
__device__ __forceinline__ float gate_act(float x) {
    return x * rcp_approx(1.0f + ex2_approx(-gate_z2<ACT>(x)));
}

// act(x) and act'(x).  The exponential is taken of -|z|, so s and 1 - s both
// keep their relative precision: with e = e^-|z|, y = 1 / (1 + e), s is y for z
// >= 0 and e y for z < 0, and 1 - s the other one.  Where either has vanished
// the product with z' is left out: z' may be infinite there.
template <int ACT>
__device__ __forceinline__ float gate_act_slope(float x, float *slope) {
    const float z2 = gate_z2<ACT>(x);
    const float e = ex2_approx(-fabsf(z2)), y = rcp_approx(1.0f + e), ey = e * y;
    const float s = z2 >= 0.0f ? y : ey;
    float dz = 1.0f;
    if (ACT == SHMM_GELU_TANH) {
        const float k0 = 2.0f * 0.7978845608028654f;
        dz = fmaf(x * x, k0 * 3.0f * 0.044715f, k0);
    }
    const float st = y * ey;
    *slope = st == 0.0f ? s : fmaf(x * st, dz, s);
    return x * s;
}
