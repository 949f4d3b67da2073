// Launchers of the gated linear recurrence (internal to the library; the C ABI in api.cpp
// validates arguments and then calls these) and the arithmetic its kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "common.h"

namespace ssm {

constexpr int kGlrStateSteps = 128;  // SSM_GLR_STATE_STEPS

struct GlrIn {
    int B, L, D;
    bool bf16;
    int form;  // 0 decay, 1 convex
    const void* x;
    const void* r;
    const void* i;
    const float* A;
    const void* z;
    int ldx, ldr, ldi, ldz;  // elements from a row to the next
    const int* seqlens;
};

struct GlrArgs {
    GlrIn in;
    const float* h0;
    void* y;
    float* h_final;
    float* states;
    void* ws;
};

struct GlrBwdArgs {
    GlrIn in;
    const float* states;
    const void* dy;
    const float* dh_final;
    void* dx;
    void* dr;
    void* di;
    float* dA;
    void* dz;
    float* dh0;
    void* ws;
};

struct GlrStepArgs {
    GlrIn in;  // L = 1, no seqlens
    float* state;
    void* y;
};

size_t glr_workspace_bytes(int B, int L, int D);
size_t glr_bwd_workspace_bytes(int B, int L, int D);
hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t stream);
hipError_t launch_glr_bwd(const GlrBwdArgs& a, hipStream_t stream);
hipError_t launch_glr_step(const GlrStepArgs& a, hipStream_t stream);

// ------------------------------------------------------------------ arithmetic
constexpr float kTiny = 1.17549435e-38f;  // smallest normal fp32

// sigmoid(v) and 1 - sigmoid(v), the second to its own relative precision (e s, where
// 1 - s would cancel); e is held below infinity, where s is 0 (as it is from e = 2^126 on).
struct Sigmoid {
    float s, om;
    __device__ __forceinline__ explicit Sigmoid(float v) {
        const float e = exp2_fast(-v * kLog2e);
        s = rcp_fast(1.0f + e);
        om = __builtin_fminf(e, __FLT_MAX__) * s;
    }
};

// 1 - a^2 for a = exp(t), t <= 0. Close to 0 the difference would cancel: there the series of
// -expm1(2 t), whose next term is (2 t)^5 / 720 of the first (4e-8 relative at t = -1/16). Beyond,
// what the roundings of a leave is 1e-6 relative at most, where 1 - a^2 is still small.
__device__ __forceinline__ float one_minus_square(float t, float a) {
    float q = __builtin_fmaf(t, 4.0f / 15.0f, 2.0f / 3.0f);
    q = __builtin_fmaf(t, q, 4.0f / 3.0f);
    q = __builtin_fmaf(t, q, 2.0f);
    q = __builtin_fmaf(t, q, 2.0f);
    const float series = -t * q, difference = __builtin_fmaf(-a, a, 1.0f);
    return t > -0.0625f ? series : difference;
}

// a and u of one element; FORM 0: A2 = A log2(e).
template <int FORM>
__device__ __forceinline__ void glr_coefficients(float x, float r, float i, float A2, float A, float* a, float* u) {
    if constexpr (FORM == 0) {
        const float sr = rcp_fast(1.0f + exp2_fast(-r * kLog2e)), si = rcp_fast(1.0f + exp2_fast(-i * kLog2e));
        *a = exp2_fast(A2 * sr);
        *u = __builtin_amdgcn_sqrtf(one_minus_square(A * sr, *a)) * si * x;
    } else {
        // 1 - k cancels where k is close to 1: e k there
        const float e = exp2_fast(-r * kLog2e), k = rcp_fast(1.0f + e);
        *a = r > 0.0f ? e * k : 1.0f - k;
        *u = k * x;
    }
}

// The gradient of one element from g, the state before it and its inputs; dl: what dA adds.
// k: sigma(r), q: sigma(i).
template <int FORM>
__device__ __forceinline__ void glr_gradient(float g, float before, float a, float x, const Sigmoid& k, const Sigmoid& q,
                                             float A, float* dx, float* dr, float* di, float* dl) {
    if constexpr (FORM == 0) {
        const float t = A * k.s, m2 = one_minus_square(t, a);
        // 1 / m; 0 where m is 0 (the limit of dr as the gate closes)
        const float rs = __builtin_amdgcn_rsqf(m2), rm = m2 > kTiny ? rs : 0.0f, gq = g * q.s, m = m2 * rm;
        *dx = gq * m;
        *di = *dx * x * q.om;
        const float w = a * (g * before - a * rm * gq * x);  // d / d(A s)
        *dl = w * k.s;
        // in this order what is too small for fp32 stays so: where |t| > 104, w is 0
        *dr = w * k.om * t;
    } else {
        *dx = g * k.s;
        *dr = *dx * (x - before) * k.om;
        *di = *dl = 0.0f;
    }
}

__device__ __forceinline__ int glr_length(const int* seqlens, int b, int L) {
    return seqlens ? max(0, min(seqlens[b], L)) : L;
}

}  // namespace ssm
