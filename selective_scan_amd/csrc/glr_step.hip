// One-token step of the gated linear recurrence on gfx950, state updated in place:
//   h = a h + u,  y = h [silu(z)]
// A handful of bytes an element (19 in bf16 with gate, 8 of them the state's) and no sums:
// latency for one user's token, the bytes for a batch's. A lane takes four neighbouring channels
// where rows hold whole fours, one otherwise. Measured: B256 D2560 bf16 with gate 3.9 us, B1 D1536
// 2.2 us (latency; the call's host side takes 8).
#include "glr.h"
#include "launch.h"

namespace ssm {
namespace {

constexpr int kT = 256;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <bool BF16, int V>
__device__ __forceinline__ void ld(const void* p, size_t i, float (&v)[V]) {
    if constexpr (V == 1) {
        if constexpr (BF16) v[0] = bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
        else v[0] = static_cast<const float*>(p)[i];
    } else if constexpr (BF16) {
        const u32x2 q = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = k & 1 ? bf16_hi(q[k / 2]) : bf16_lo(q[k / 2]);
    } else {
        const f32x4 q = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = q[k];
    }
}

template <bool BF16, int V>
__device__ __forceinline__ void st(void* p, size_t i, const float (&v)[V]) {
    if constexpr (V == 1) {
        if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(v[0]);
        else static_cast<float*>(p)[i] = v[0];
    } else if constexpr (BF16) {
        u32x2 q;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            q[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * k], v[2 * k + 1]}, bf16x2));
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + i) = q;
    } else {
        *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i) = f32x4{v[0], v[1], v[2], v[3]};
    }
}

template <bool BF16, int V, int FORM>
__global__ void __launch_bounds__(kT) glr_step_kernel(GlrStepArgs a, unsigned n, unsigned per) {
    const unsigned q = blockIdx.x * kT + threadIdx.x;
    if (q >= n) return;
    const GlrIn& in = a.in;
    const unsigned b = q / per, d = (q - b * per) * V;
    const size_t at = (size_t)q * V;
    float x[V], r[V], i[V], A[V], z[V], h[V];
    ld<BF16>(in.x, (size_t)b * in.ldx + d, x);
    ld<BF16>(in.r, (size_t)b * in.ldr + d, r);
    if constexpr (FORM == 0) {
        ld<BF16>(in.i, (size_t)b * in.ldi + d, i);
        ld<false>(in.A, d, A);
    }
    if (in.z) ld<BF16>(in.z, (size_t)b * in.ldz + d, z);
    ld<false>(a.state, at, h);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float c, u;
        glr_coefficients<FORM>(x[v], r[v], FORM == 0 ? i[v] : 0.0f, FORM == 0 ? A[v] * kLog2e : 0.0f,
                               FORM == 0 ? A[v] : 0.0f, &c, &u);
        h[v] = __builtin_fmaf(c, h[v], u);
    }
    st<false>(a.state, at, h);
    if (in.z)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] *= silu(z[v]);
    st<BF16>(a.y, at, h);
}

// Whether every row starts on four elements and holds whole fours.
bool fours(const GlrIn& in) {
    const void* p[] = {in.x, in.r, in.i, in.z};
    const int stride[] = {in.ldx, in.ldr, in.ldi, in.ldz};
    if (in.D % 4 != 0) return false;
    for (int k = 0; k < 4; ++k)
        if (p[k] && (reinterpret_cast<uintptr_t>(p[k]) % (in.bf16 ? 8 : 16) != 0 || stride[k] % 4 != 0)) return false;
    return true;
}

template <bool BF16, int V>
hipError_t run(const GlrStepArgs& a, hipStream_t s) {
    const unsigned per = (unsigned)a.in.D / V, n = (unsigned)a.in.B * per;  // B * D <= 2^30
    const dim3 grid((n + kT - 1) / kT);
    if (a.in.form == 0) launch((glr_step_kernel<BF16, V, 0>), grid, dim3(kT), 0, s, a, n, per);
    else launch((glr_step_kernel<BF16, V, 1>), grid, dim3(kT), 0, s, a, n, per);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_glr_step(const GlrStepArgs& a, hipStream_t s) {
    if (fours(a.in)) return a.in.bf16 ? run<true, 4>(a, s) : run<false, 4>(a, s);
    return a.in.bf16 ? run<true, 1>(a, s) : run<false, 1>(a, s);
}

}  // namespace ssm
