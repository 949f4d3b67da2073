// Residual add with dropout and layer norm or RMS norm on gfx950, its gradient, and dropout alone:
//   s = residual + dropout(x),  y = (s - mean) rstd w + b   (rms: s rstd w + b)
//   ds = rstd (dn - mean(dn) - xhat mean(dn xhat)) + dsum,  dn = dy w   (rms: no mean(dn))
//   dresidual = ds,  dx = dropout(ds),  dw = sum dy xhat,  db = sum dy
// First form: a wave per row, the row passed over as often as its sums ask.
#include "add_norm.h"
#include "common.h"
#include "launch.h"

#include <algorithm>

namespace ssm {
namespace {

constexpr int kT = 64;
constexpr int kParts = 256;

__device__ __forceinline__ float ld(const void* p, size_t i, bool bf16) {
    return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void st(void* p, size_t i, float v, bool bf16) {
    if (bf16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
    else static_cast<float*>(p)[i] = v;
}

__device__ __forceinline__ float sum_wave(float v) {
#pragma unroll
    for (int f = 1; f < 64; f <<= 1) v += __shfl_xor(v, f);
    return v;
}

__device__ __forceinline__ float dropped(float v, const Dropout& d, int m, int c, int C) {
    if (d.least == 0) return v;
    const Philox p(d.rng[0], d.rng[1] + (unsigned long long)m * ((C + 7) / 8) + c / 8);
    return p.bits(c % 8) >= d.least ? v * d.scale : 0.0f;
}

__global__ void __launch_bounds__(kT) add_norm_fwd_simple(AddNormArgs a) {
    const int m = blockIdx.x, l = threadIdx.x;
    const size_t base = (size_t)m * a.C;
    auto value = [&](int c) {
        float v = dropped(ld(a.x, base + c, a.bf16), a.drop, m, c, a.C);
        return a.residual ? v + ld(a.residual, base + c, a.res_bf16) : v;
    };
    float s = 0.0f;
    for (int c = l; c < a.C; c += kT) s += value(c);
    const float mean = a.rms ? 0.0f : sum_wave(s) / (float)a.C;
    s = 0.0f;
    for (int c = l; c < a.C; c += kT) {
        const float d = value(c) - mean;
        s = __builtin_fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(sum_wave(s) / (float)a.C + a.eps);
    if (l == 0) {
        if (a.mean) a.mean[m] = mean;
        if (a.rstd) a.rstd[m] = rstd;
    }
    for (int c = l; c < a.C; c += kT) {
        const float v = value(c);
        if (a.sum) st(a.sum, base + c, v, a.res_bf16);
        st(a.y, base + c, __builtin_fmaf((v - mean) * rstd, a.weight ? a.weight[c] : 1.0f, a.bias ? a.bias[c] : 0.0f),
           a.bf16);
    }
}

__global__ void __launch_bounds__(kT) add_norm_bwd_simple(AddNormBwdArgs a) {
    const int m = blockIdx.x, l = threadIdx.x;
    const size_t base = (size_t)m * a.C;
    const float mean = a.rms ? 0.0f : a.mean[m], rstd = a.rstd[m];
    float s0 = 0.0f, s1 = 0.0f;
    for (int c = l; c < a.C; c += kT) {
        const float xhat = (ld(a.sum, base + c, a.res_bf16) - mean) * rstd;
        const float dn = ld(a.dy, base + c, a.bf16) * (a.weight ? a.weight[c] : 1.0f);
        s0 += dn;
        s1 = __builtin_fmaf(dn, xhat, s1);
    }
    s0 = a.rms ? 0.0f : sum_wave(s0) / (float)a.C;
    s1 = sum_wave(s1) / (float)a.C;
    for (int c = l; c < a.C; c += kT) {
        const float xhat = (ld(a.sum, base + c, a.res_bf16) - mean) * rstd;
        const float dn = ld(a.dy, base + c, a.bf16) * (a.weight ? a.weight[c] : 1.0f);
        float ds = rstd * (dn - s0 - xhat * s1);
        if (a.dsum) ds += ld(a.dsum, base + c, a.res_bf16);
        if (a.dresidual) st(a.dresidual, base + c, ds, a.res_bf16);
        if (a.dx) st(a.dx, base + c, dropped(ds, a.drop, m, c, a.C), a.bf16);
    }
}

__global__ void __launch_bounds__(kT) add_norm_affine(AddNormBwdArgs a, float* part) {
    const int c = blockIdx.x * kT + threadIdx.x;
    if (c >= a.C) return;
    float dw = 0.0f, db = 0.0f;
    for (int m = blockIdx.y; m < a.M; m += gridDim.y) {
        const size_t at = (size_t)m * a.C + c;
        const float dy = ld(a.dy, at, a.bf16), mean = a.rms ? 0.0f : a.mean[m];
        dw = __builtin_fmaf(dy, (ld(a.sum, at, a.res_bf16) - mean) * a.rstd[m], dw);
        db += dy;
    }
    part[(size_t)blockIdx.y * 2 * a.C + c] = dw;
    part[(size_t)blockIdx.y * 2 * a.C + a.C + c] = db;
}

__global__ void __launch_bounds__(kT) add_norm_sum(const float* part, int n, int C, float* dweight, float* dbias) {
    const int c = blockIdx.x * kT + threadIdx.x;
    if (c >= C) return;
    float dw = 0.0f, db = 0.0f;
    for (int k = 0; k < n; ++k) {
        dw += part[(size_t)k * 2 * C + c];
        db += part[(size_t)k * 2 * C + C + c];
    }
    if (dweight) dweight[c] = dw;
    if (dbias) dbias[c] = db;
}

__global__ void __launch_bounds__(kT) dropout_simple(DropoutArgs a) {
    const int m = blockIdx.x;
    for (int c = threadIdx.x; c < a.C; c += kT) {
        const size_t at = (size_t)m * a.C + c;
        st(a.y, at, dropped(ld(a.x, at, a.bf16), a.drop, m, c, a.C), a.bf16);
    }
}

int parts(int M) { return std::min(kParts, M); }

}  // namespace

size_t add_norm_bwd_workspace_bytes(int M, int C, bool, bool) { return (size_t)parts(M) * 2 * C * 4; }

hipError_t launch_add_norm_fwd(const AddNormArgs& a, hipStream_t s) {
    if (a.M == 0) return hipSuccess;
    launch(add_norm_fwd_simple, dim3((unsigned)a.M), dim3(kT), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t s) {
    const int n = parts(a.M);
    float* part = static_cast<float*>(a.ws);
    const unsigned cols = (unsigned)((a.C + kT - 1) / kT);
    hipError_t e = hipSuccess;
    if (a.M > 0) {
        launch(add_norm_bwd_simple, dim3((unsigned)a.M), dim3(kT), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!a.dweight && !a.dbias) return e;
    if (a.M > 0) {
        launch(add_norm_affine, dim3(cols, (unsigned)n), dim3(kT), 0, s, a, part);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    launch(add_norm_sum, dim3(cols), dim3(kT), 0, s, part, n, a.C, a.dweight, a.dbias);
    return hipGetLastError();
}

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s) {
    if (a.M == 0) return hipSuccess;
    launch(dropout_simple, dim3((unsigned)a.M), dim3(kT), 0, s, a);
    return hipGetLastError();
}

}  // namespace ssm
