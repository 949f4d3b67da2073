// Group norm over channels-last data on gfx950, with activation and / or gate, and its
// gradient. Per sample m and group g, over its S * C/G values:
//   xhat = (x - mean) rstd,  u = xhat w + b,  y = act(u) [silu(z)]
//   du = dy [silu(z)] act'(u),  dz = dy act(u) silu'(z),  dw = sum du xhat,  db = sum du
//   dn = du w,  dx = rstd (dn - mean(dn) - xhat mean(dn xhat))
// Statistics, sums and every intermediate value are fp32.
#include "common.h"
#include "group_norm.h"
#include "launch.h"

namespace ssm {
namespace {

constexpr int kT = 256;

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

// Sum over the workgroup's lanes, the same value in every lane (a fixed order).
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int f = 1; f < 64; f <<= 1) v += __shfl_xor(v, f);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) s += red[w];
    return s;
}

__device__ __forceinline__ float sigmoid(float x) { return rcp_fast(1.0f + exp2_fast(-x * kLog2e)); }

// One workgroup per (sample, group): mean, squared distances to it, output.
template <bool BF16>
__global__ void __launch_bounds__(kT) gn_fwd(GroupNormArgs a) {
    __shared__ float red[kT / 64];
    const int g = blockIdx.x % a.G, m = blockIdx.x / a.G, cg = a.C / a.G;
    const long long n = (long long)a.S * cg;
    const size_t base = (size_t)m * a.S * a.C + (size_t)g * cg;
    float s = 0.0f;
    for (long long e = threadIdx.x; e < n; e += kT) s += ld1<BF16>(a.x, base + (e / cg) * a.C + e % cg);
    const float mean = block_sum(s, red) / (float)n;
    float q = 0.0f;
    for (long long e = threadIdx.x; e < n; e += kT) {
        const float d = ld1<BF16>(a.x, base + (e / cg) * a.C + e % cg) - mean;
        q = __builtin_fmaf(d, d, q);
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, red) / (float)n + a.eps);
    if (threadIdx.x == 0 && a.mean) {
        a.mean[(size_t)m * a.G + g] = mean;
        a.rstd[(size_t)m * a.G + g] = rstd;
    }
    for (long long e = threadIdx.x; e < n; e += kT) {
        const int c = g * cg + (int)(e % cg);
        const size_t at = base + (e / cg) * a.C + e % cg;
        float u = (ld1<BF16>(a.x, at) - mean) * rstd;
        if (a.weight) u *= a.weight[c];
        if (a.bias) u += a.bias[c];
        if (a.act) u *= sigmoid(u);
        if (a.z) u *= silu(ld1<BF16>(a.z, at));
        st1<BF16>(a.y, at, u);
    }
}

// du and (with a gate) dz of one value.
template <bool BF16>
__device__ __forceinline__ float du_of(const GroupNormBwdArgs& a, size_t at, int c, float xhat, float* dz) {
    float u = xhat;
    if (a.weight) u *= a.weight[c];
    if (a.bias) u += a.bias[c];
    const float su = sigmoid(u);
    float d = ld1<BF16>(a.dy, at);
    if (a.z) {
        const float z = ld1<BF16>(a.z, at), sz = sigmoid(z);
        *dz = d * (a.act ? u * su : u) * (sz * (1.0f + z * (1.0f - sz)));
        d *= z * sz;
    }
    return a.act ? d * (su * (1.0f + u * (1.0f - su))) : d;
}

// One workgroup per (sample, group): the two means of the group, then dx and dz.
template <bool BF16>
__global__ void __launch_bounds__(kT) gn_bwd(GroupNormBwdArgs a) {
    __shared__ float red[kT / 64];
    const int g = blockIdx.x % a.G, m = blockIdx.x / a.G, cg = a.C / a.G;
    const long long n = (long long)a.S * cg;
    const size_t base = (size_t)m * a.S * a.C + (size_t)g * cg;
    const float mean = a.mean[(size_t)m * a.G + g], rstd = a.rstd[(size_t)m * a.G + g];
    float s0 = 0.0f, s1 = 0.0f, dz = 0.0f;
    for (long long e = threadIdx.x; e < n; e += kT) {
        const int c = g * cg + (int)(e % cg);
        const size_t at = base + (e / cg) * a.C + e % cg;
        const float xhat = (ld1<BF16>(a.x, at) - mean) * rstd;
        float dn = du_of<BF16>(a, at, c, xhat, &dz);
        if (a.weight) dn *= a.weight[c];
        s0 += dn;
        s1 = __builtin_fmaf(dn, xhat, s1);
    }
    s0 = block_sum(s0, red) / (float)n;
    s1 = block_sum(s1, red) / (float)n;
    for (long long e = threadIdx.x; e < n; e += kT) {
        const int c = g * cg + (int)(e % cg);
        const size_t at = base + (e / cg) * a.C + e % cg;
        const float xhat = (ld1<BF16>(a.x, at) - mean) * rstd;
        float dn = du_of<BF16>(a, at, c, xhat, &dz);
        if (a.weight) dn *= a.weight[c];
        st1<BF16>(a.dx, at, rstd * (dn - s0 - xhat * s1));
        if (a.z) st1<BF16>(a.dz, at, dz);
    }
}

// One workgroup per channel: dw and db over every sample and position.
template <bool BF16>
__global__ void __launch_bounds__(kT) gn_bwd_affine(GroupNormBwdArgs a) {
    __shared__ float red[kT / 64];
    const int c = blockIdx.x, g = c / (a.C / a.G);
    float dw = 0.0f, db = 0.0f, dz;
    const long long rows = (long long)a.M * a.S;
    for (long long i = threadIdx.x; i < rows; i += kT) {
        const size_t mg = (size_t)(i / a.S) * a.G + g, at = (size_t)i * a.C + c;
        const float xhat = (ld1<BF16>(a.x, at) - a.mean[mg]) * a.rstd[mg];
        const float du = du_of<BF16>(a, at, c, xhat, &dz);
        dw = __builtin_fmaf(du, xhat, dw);
        db += du;
    }
    dw = block_sum(dw, red);
    db = block_sum(db, red);
    if (threadIdx.x == 0) {
        if (a.dweight) a.dweight[c] = dw;
        if (a.dbias) a.dbias[c] = db;
    }
}

}  // namespace

size_t group_norm_workspace_bytes(int, int, int, int, bool) { return 0; }
size_t group_norm_bwd_workspace_bytes(int, int, int, int, bool) { return 0; }

hipError_t launch_group_norm_fwd(const GroupNormArgs& a, hipStream_t st) {
    if (a.M == 0) return hipSuccess;
    const dim3 grid((unsigned)((size_t)a.M * a.G));
    if (a.bf16) launch(gn_fwd<true>, grid, dim3(kT), 0, st, a);
    else launch(gn_fwd<false>, grid, dim3(kT), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_group_norm_bwd(const GroupNormBwdArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((size_t)a.M * a.G)), gc((unsigned)a.C);
    if (a.M > 0) {
        if (a.bf16) launch(gn_bwd<true>, grid, dim3(kT), 0, st, a);
        else launch(gn_bwd<false>, grid, dim3(kT), 0, st, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dweight || a.dbias) {
        if (a.bf16) launch(gn_bwd_affine<true>, gc, dim3(kT), 0, st, a);
        else launch(gn_bwd_affine<false>, gc, dim3(kT), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace ssm
