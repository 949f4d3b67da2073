// One-token decode step of linear attention with a decay per head on gfx950, state
// updated in place, with the group norm and gate of the output fused in:
//   S = lam S + k (x) v,   o = scale q . S,   [o = ((o - mean) rstd w + b) silu(z)]
//
// Bandwidth-bound: the fp32 state is read and written once. One workgroup of 256
// lanes per (batch, head) holds the whole state of that head in registers, every
// load issued before the first store; a wave's load covers whole rows of V values.
// o is summed over the row groups through LDS, so the workgroup has a head's V values
// and the norm needs no other launch.
// Measured: B64 H24 K128 V64 bf16 with norm and gate 17.3 us a call (101 MB, 5.9 TB/s, the
// state partly in the memory-side cache; a copy of that size reaches 5.5), B1 H16
// K = V = 128 4.4 us (latency; the call's host side takes 9).
#include "common.h"
#include "launch.h"
#include "linattn.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float ld1(const void* p, size_t i) {
    if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void st1(void* p, size_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
    else static_cast<float*>(p)[i] = v;
}

template <int K, int V, bool BF16>
__global__ void __launch_bounds__(kThreads) linattn_step_kernel(LinattnStepArgs a) {
    constexpr int CQ = V / 4;            // float4 columns
    constexpr int RG = kThreads / CQ;    // rows in flight at once
    constexpr int R = K / RG;            // rows per lane
    __shared__ float4 part[RG][CQ];
    __shared__ float red[2][kThreads / 64];
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const int tid = threadIdx.x, cq = tid % CQ, rg = tid / CQ;
    float4* S = reinterpret_cast<float4*>(a.state + (size_t)bh * K * V) + cq;
    float4 s[R];
    float kn[R], qn[R];
#pragma unroll
    for (int u = 0; u < R; ++u) s[u] = S[(rg + RG * u) * CQ];
    const size_t gk = ((size_t)b * a.G + g) * K;
#pragma unroll
    for (int u = 0; u < R; ++u) {
        kn[u] = ld1<BF16>(a.k, gk + rg + RG * u);
        qn[u] = ld1<BF16>(a.q, gk + rg + RG * u);
    }
    float4 v;
    const size_t hv = (size_t)bh * V;
    v.x = ld1<BF16>(a.v, hv + 4 * cq);
    v.y = ld1<BF16>(a.v, hv + 4 * cq + 1);
    v.z = ld1<BF16>(a.v, hv + 4 * cq + 2);
    v.w = ld1<BF16>(a.v, hv + 4 * cq + 3);
    const Decay decay(a.log_decay[h]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < R; ++u) {
        float4 w;
        w.x = __builtin_fmaf(kn[u], v.x, decay(s[u].x));
        w.y = __builtin_fmaf(kn[u], v.y, decay(s[u].y));
        w.z = __builtin_fmaf(kn[u], v.z, decay(s[u].z));
        w.w = __builtin_fmaf(kn[u], v.w, decay(s[u].w));
        S[(rg + RG * u) * CQ] = w;
        y.x = __builtin_fmaf(qn[u], w.x, y.x);
        y.y = __builtin_fmaf(qn[u], w.y, y.y);
        y.z = __builtin_fmaf(qn[u], w.z, y.z);
        y.w = __builtin_fmaf(qn[u], w.w, y.w);
    }
    part[rg][cq] = y;
    __syncthreads();
    float o = 0.0f;
    const int j = tid;
    if (j < V) {
#pragma unroll
        for (int u = 0; u < RG; ++u) o += reinterpret_cast<const float*>(part[u])[j];
        o *= a.scale;
    }
    if (a.norm.on) {
        // two passes over the V values: their mean, then the squared distances to it
        float m = o;
#pragma unroll
        for (int f = 1; f < 64; f <<= 1) m += __shfl_xor(m, f);
        if ((tid & 63) == 0) red[0][tid >> 6] = m;
        __syncthreads();
        m = red[0][0];
        if constexpr (V > 64) m += red[0][1];
        m *= 1.0f / V;
        const float d = j < V ? o - m : 0.0f;
        float q = d * d;
#pragma unroll
        for (int f = 1; f < 64; f <<= 1) q += __shfl_xor(q, f);
        if ((tid & 63) == 0) red[1][tid >> 6] = q;
        __syncthreads();
        q = red[1][0];
        if constexpr (V > 64) q += red[1][1];
        if (j < V) {
            const int c = h * V + j;
            o = d * (1.0f / sqrtf(q * (1.0f / V) + a.norm.eps));
            if (a.norm.weight) o *= a.norm.weight[c];
            if (a.norm.bias) o += a.norm.bias[c];
            if (a.norm.z) o *= silu(ld1<BF16>(a.norm.z, hv + j));
        }
    }
    if (j < V) st1<BF16>(a.o, hv + j, o);
}

template <int K, int V>
hipError_t run(const LinattnStepArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)a.B * a.H);
    if (a.bf16) launch((linattn_step_kernel<K, V, true>), grid, dim3(kThreads), 0, st, a);
    else launch((linattn_step_kernel<K, V, false>), grid, dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linattn_step(const LinattnStepArgs& a, hipStream_t st) {
    if (a.K == 64) return a.V == 64 ? run<64, 64>(a, st) : run<64, 128>(a, st);
    return a.V == 64 ? run<128, 64>(a, st) : run<128, 128>(a, st);
}

}  // namespace ssm
