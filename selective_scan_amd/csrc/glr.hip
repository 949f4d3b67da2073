// Gated linear recurrence over whole sequences on gfx950, and its gradient:
//   h_t = a_t h_{t-1} + u_t,   y = h [silu(z)],   g_t = dy_t [silu(z_t)] + a_{t+1} g_{t+1}
// First form: a lane per (batch, channel), one step after the other.
#include "glr.h"
#include "launch.h"

#include <algorithm>

namespace ssm {
namespace {

constexpr int kT = 64;

template <bool BF16>
__device__ __forceinline__ float ld(const void* p, size_t i) {
    if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void st(void* p, size_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
    else static_cast<float*>(p)[i] = v;
}

template <bool BF16, int FORM>
__global__ void __launch_bounds__(kT) glr_fwd_serial(GlrArgs a) {
    const int d = blockIdx.x * kT + threadIdx.x, b = blockIdx.y;
    const GlrIn& in = a.in;
    if (d >= in.D) return;
    const int n = glr_length(in.seqlens, b, in.L), blocks = (in.L + kGlrStateSteps - 1) / kGlrStateSteps;
    const float A = FORM == 0 ? in.A[d] : 0.0f;
    float h = a.h0 ? a.h0[(size_t)b * in.D + d] : 0.0f;
    for (int t = 0; t < in.L; ++t) {
        const size_t row = (size_t)b * in.L + t;
        if (a.states && t % kGlrStateSteps == 0)
            a.states[((size_t)b * blocks + t / kGlrStateSteps) * in.D + d] = h;
        float y = 0.0f;
        if (t < n) {
            float c, u;
            glr_coefficients<FORM>(ld<BF16>(in.x, row * in.ldx + d), ld<BF16>(in.r, row * in.ldr + d),
                                   FORM == 0 ? ld<BF16>(in.i, row * in.ldi + d) : 0.0f, A * kLog2e, 2.0f * A, &c, &u);
            h = __builtin_fmaf(c, h, u);
            y = in.z ? h * silu(ld<BF16>(in.z, row * in.ldz + d)) : h;
        }
        st<BF16>(a.y, row * in.D + d, y);
    }
    if (a.h_final) a.h_final[(size_t)b * in.D + d] = h;
}

template <bool BF16, int FORM>
__global__ void __launch_bounds__(kT) glr_bwd_serial(GlrBwdArgs a, float* hs, float* part) {
    const int d = blockIdx.x * kT + threadIdx.x, b = blockIdx.y;
    const GlrIn& in = a.in;
    if (d >= in.D) return;
    const int n = glr_length(in.seqlens, b, in.L), blocks = (in.L + kGlrStateSteps - 1) / kGlrStateSteps;
    const float A = FORM == 0 ? in.A[d] : 0.0f, A2 = A * kLog2e, At = 2.0f * A;
    float h = 0.0f;
    for (int t = 0; t < n; ++t) {
        const size_t row = (size_t)b * in.L + t;
        if (t % kGlrStateSteps == 0) h = a.states[((size_t)b * blocks + t / kGlrStateSteps) * in.D + d];
        hs[row * in.D + d] = h;  // before the step
        float c, u;
        glr_coefficients<FORM>(ld<BF16>(in.x, row * in.ldx + d), ld<BF16>(in.r, row * in.ldr + d),
                               FORM == 0 ? ld<BF16>(in.i, row * in.ldi + d) : 0.0f, A2, At, &c, &u);
        h = __builtin_fmaf(c, h, u);
    }
    float g = a.dh_final ? a.dh_final[(size_t)b * in.D + d] : 0.0f, dA = 0.0f;
    for (int t = in.L - 1; t >= 0; --t) {
        const size_t row = (size_t)b * in.L + t, o = row * in.D + d;
        float dx = 0.0f, dr = 0.0f, di = 0.0f, dz = 0.0f;
        if (t < n) {
            const float x = ld<BF16>(in.x, row * in.ldx + d), r = ld<BF16>(in.r, row * in.ldr + d);
            const float i = FORM == 0 ? ld<BF16>(in.i, row * in.ldi + d) : 0.0f;
            float c, u, dl, e = ld<BF16>(a.dy, o);
            glr_coefficients<FORM>(x, r, i, A2, At, &c, &u);
            if (in.z) {
                const float z = ld<BF16>(in.z, row * in.ldz + d);
                const Sigmoid s(z);
                dz = e * __builtin_fmaf(c, hs[o], u) * s.s * __builtin_fmaf(z, s.om, 1.0f);
                e *= z * s.s;
            }
            g += e;
            glr_gradient<FORM>(g, hs[o], x, r, i, A, A2, At, &dx, &dr, &di, &dl);
            dA += dl;
            g *= c;
        }
        st<BF16>(a.dx, o, dx);
        st<BF16>(a.dr, o, dr);
        if constexpr (FORM == 0) st<BF16>(a.di, o, di);
        if (in.z) st<BF16>(a.dz, o, dz);
    }
    if (a.dh0) a.dh0[(size_t)b * in.D + d] = g;
    if constexpr (FORM == 0) part[(size_t)b * in.D + d] = dA;
}

__global__ void __launch_bounds__(kT) glr_sum_parts(const float* part, int n, int D, float* dA) {
    const int d = blockIdx.x * kT + threadIdx.x;
    if (d >= D) return;
    float s = 0.0f;
    for (int k = 0; k < n; ++k) s += part[(size_t)k * D + d];
    dA[d] = s;
}

}  // namespace

size_t glr_workspace_bytes(int, int, int) { return 0; }

size_t glr_bwd_workspace_bytes(int B, int L, int D) { return ((size_t)B * L * D + (size_t)B * D) * 4; }

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.in.D + kT - 1) / kT), (unsigned)a.in.B);
    if (a.in.bf16 && a.in.form == 0) launch((glr_fwd_serial<true, 0>), grid, dim3(kT), 0, s, a);
    else if (a.in.bf16) launch((glr_fwd_serial<true, 1>), grid, dim3(kT), 0, s, a);
    else if (a.in.form == 0) launch((glr_fwd_serial<false, 0>), grid, dim3(kT), 0, s, a);
    else launch((glr_fwd_serial<false, 1>), grid, dim3(kT), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_glr_bwd(const GlrBwdArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.in.D + kT - 1) / kT), (unsigned)a.in.B);
    float* hs = static_cast<float*>(a.ws);
    float* part = hs + (size_t)a.in.B * a.in.L * a.in.D;
    if (a.in.bf16 && a.in.form == 0) launch((glr_bwd_serial<true, 0>), grid, dim3(kT), 0, s, a, hs, part);
    else if (a.in.bf16) launch((glr_bwd_serial<true, 1>), grid, dim3(kT), 0, s, a, hs, part);
    else if (a.in.form == 0) launch((glr_bwd_serial<false, 0>), grid, dim3(kT), 0, s, a, hs, part);
    else launch((glr_bwd_serial<false, 1>), grid, dim3(kT), 0, s, a, hs, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.in.form != 0) return e;
    launch(glr_sum_parts, dim3((unsigned)((a.in.D + kT - 1) / kT)), dim3(kT), 0, s, part, a.in.B, a.in.D, a.dA);
    return hipGetLastError();
}

}  // namespace ssm
