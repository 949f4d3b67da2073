// One-token step of the gated linear recurrence on gfx950, state updated in place:
//   h = a h + u,  y = h [silu(z)]
// A handful of bytes an element (19 in bf16 with gate, 8 of them the state's) and no sums:
// latency for one user's token, the bytes for a batch's. Every lane takes two neighbouring
// channels where rows hold whole pairs, one otherwise.
#include "glr.h"
#include "launch.h"

namespace ssm {
namespace {

constexpr int kT = 256;

template <bool BF16>
__device__ __forceinline__ float ld(const void* p, size_t i) {
    if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}

template <bool BF16, int FORM>
__global__ void __launch_bounds__(kT) glr_step_kernel(GlrStepArgs a, long long n) {
    const long long q = (long long)blockIdx.x * kT + threadIdx.x;
    if (q >= n) return;
    const GlrIn& in = a.in;
    const int b = (int)(q / in.D), d = (int)(q % in.D);
    const float x = ld<BF16>(in.x, (size_t)b * in.ldx + d), r = ld<BF16>(in.r, (size_t)b * in.ldr + d);
    const float i = FORM == 0 ? ld<BF16>(in.i, (size_t)b * in.ldi + d) : 0.0f, A = FORM == 0 ? in.A[d] : 0.0f;
    const float z = in.z ? ld<BF16>(in.z, (size_t)b * in.ldz + d) : 0.0f;
    float c, u;
    glr_coefficients<FORM>(x, r, i, A * kLog2e, 2.0f * A, &c, &u);
    const float h = __builtin_fmaf(c, a.state[q], u), y = in.z ? h * silu(z) : h;
    a.state[q] = h;
    if constexpr (BF16) static_cast<uint16_t*>(a.y)[q] = f32_to_bf16(y);
    else static_cast<float*>(a.y)[q] = y;
}

}  // namespace

hipError_t launch_glr_step(const GlrStepArgs& a, hipStream_t s) {
    const long long n = (long long)a.in.B * a.in.D;
    const dim3 grid((unsigned)((n + kT - 1) / kT));
    if (a.in.bf16 && a.in.form == 0) launch((glr_step_kernel<true, 0>), grid, dim3(kT), 0, s, a, n);
    else if (a.in.bf16) launch((glr_step_kernel<true, 1>), grid, dim3(kT), 0, s, a, n);
    else if (a.in.form == 0) launch((glr_step_kernel<false, 0>), grid, dim3(kT), 0, s, a, n);
    else launch((glr_step_kernel<false, 1>), grid, dim3(kT), 0, s, a, n);
    return hipGetLastError();
}

}  // namespace ssm
