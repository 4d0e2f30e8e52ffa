// The gate activations of a gated MLP block and their slopes.  Both are x
// times the logistic function of z(x):
//   SiLU          z = x
//   GeLU (tanh)   z = 2 sqrt(2/pi) (x + 0.044715 x^3)   (Hendrycks & Gimpel 2016)
// act(x) = x s, act'(x) = s + x s (1 - s) z'(x) with s = 1 / (1 + e^-z).  The
// exponential is taken of -|z|, so nothing overflows and both s and 1 - s keep
// their relative precision: with e = e^-|z|, y = 1 / (1 + e), s is y for
// z >= 0 and e y for z < 0, and 1 - s the other one.
#pragma once

#include "gelu.cuh"
#include "shmm.h"

// s and 1 - s at z = z2 / log2(e).
__device__ __forceinline__ void logistic_pair(float z2, float *s, float *t) {
    const float e = ex2_approx(-fabsf(z2));
    const float y = recip_1_2(1.0f + e), ey = e * y;
    *s = z2 >= 0.0f ? y : ey;
    *t = z2 >= 0.0f ? ey : y;
}

template <int ACT>
__device__ __forceinline__ float gate_z2(float x) {  // z(x) log2(e)
    if (ACT == SHMM_SILU) return x * 1.4426950408889634f;
    const float k0 = 2.0f * 0.7978845608028654f * 1.4426950408889634f;
    return x * fmaf(x * x, k0 * 0.044715f, k0);
}

template <int ACT>
__device__ __forceinline__ float gate_act(float x) {
    const float z2 = gate_z2<ACT>(x);
    const float e = ex2_approx(-fabsf(z2));
    const float y = recip_1_2(1.0f + e);
    return x * (z2 >= 0.0f ? y : e * y);
}

// act(x) and act'(x).  Where s or 1 - s has vanished the product with z' is
// left out: z' may be infinite there.
template <int ACT>
__device__ __forceinline__ float gate_act_slope(float x, float *slope) {
    float s, t;
    logistic_pair(gate_z2<ACT>(x), &s, &t);
    float dz = 1.0f;
    if (ACT == SHMM_GELU_TANH) {
        const float k0 = 2.0f * 0.7978845608028654f;
        dz = fmaf(x * x, k0 * 3.0f * 0.044715f, k0);
    }
    const float st = s * t;
    *slope = st == 0.0f ? s : fmaf(x * st, dz, s);
    return x * s;
}
