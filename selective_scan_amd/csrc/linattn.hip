// Linear attention with a decay per head on gfx950: whole sequences and their gradient.
//
// Forward, per (batch, head) with lam = exp(log_decay[h]):
//   S_t = lam S_{t-1} + x2_t (x) x3_t,   out_t = x1_t . S_t      (x1, x2, x3) = (q, k, v)
// The gradient is three runs of the same operator (the exact chain rule; T is the
// gradient of the final state, R_t the state of the run backwards in time):
//   dq: forwards  on (dout, v, k), from h0 transposed
//   dk: backwards on (v, dout, q), from T transposed
//   dv: backwards on (k, q, dout), from T; what leaves at the front is dh0
// Backwards in time the decay follows the read-out instead of preceding the update
// (R_t = P_{t+1} + x2_t (x) x3_t, out_t = x1_t . R_t, P_t = lam R_t, P_n = T).
#include "common.h"
#include "launch.h"
#include "linattn.h"

namespace ssm {
namespace {

// One run of the operator: x1, x2 [B, L, ., KD], x3 [B, L, ., VD], out [B, L, H, VD].
struct Mix {
    int B, L, H, r;       // r heads share a group of queries and keys
    const void* x1;
    const void* x2;
    const void* x3;
    int g1, g2, g3;       // nonzero: held per group ([B, L, H / r, .])
    const float* log_decay;
    const int* seqlens;
    float out_scale;      // factor of every output
    float kv_scale;       // factor of x2 (x) x3
    const float* init;    // [B, H, KD, VD], transposed ([B, H, VD, KD]) if init_t; or NULL
    int init_t;
    void* out;            // io dtype, or fp32 if out_f32
    int out_f32;
    float* final_state;   // [B, H, KD, VD] or NULL
};

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

__device__ __forceinline__ int seq_len(const int* seqlens, int b, int L) {
    return seqlens ? max(0, min(seqlens[b], L)) : L;
}

// One workgroup per (batch, head), one lane per column of the state, the recurrence
// step by step; rows of x1 and x2 pass through LDS kT steps at a time.
template <int KD, int VD, bool BF16, bool REV>
__global__ void __launch_bounds__(VD) mix_kernel(Mix a) {
    constexpr int kT = 16;
    __shared__ float s1[kT][KD], s2[kT][KD];
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, j = threadIdx.x;
    const int G = a.H / a.r;
    const int h1 = a.g1 ? h / a.r : h, n1 = a.g1 ? G : a.H;
    const int h2 = a.g2 ? h / a.r : h, n2 = a.g2 ? G : a.H;
    const int h3 = a.g3 ? h / a.r : h, n3 = a.g3 ? G : a.H;
    const int len = seq_len(a.seqlens, b, a.L);
    const Decay decay(a.log_decay[h]);
    float S[KD];
#pragma unroll
    for (int i = 0; i < KD; ++i)
        S[i] = !a.init ? 0.0f
               : a.init_t ? a.init[((size_t)bh * VD + j) * KD + i] : a.init[((size_t)bh * KD + i) * VD + j];
    for (int c0 = 0; c0 < a.L; c0 += kT) {
        const int n = min(kT, a.L - c0);
        __syncthreads();
        for (int e = j; e < n * KD; e += VD) {
            const int u = e / KD, i = e % KD, t = REV ? a.L - 1 - (c0 + u) : c0 + u;
            const size_t row = (size_t)b * a.L + t;
            s1[u][i] = t < len ? ld1<BF16>(a.x1, (row * n1 + h1) * KD + i) : 0.0f;
            s2[u][i] = t < len ? ld1<BF16>(a.x2, (row * n2 + h2) * KD + i) * a.kv_scale : 0.0f;
        }
        __syncthreads();
        for (int u = 0; u < n; ++u) {
            const int t = REV ? a.L - 1 - (c0 + u) : c0 + u;
            const size_t row = (size_t)b * a.L + t;
            float y = 0.0f;
            if (t < len) {
                const float w = ld1<BF16>(a.x3, (row * n3 + h3) * VD + j);
#pragma unroll
                for (int i = 0; i < KD; ++i) {
                    if constexpr (!REV) S[i] = decay(S[i]);
                    S[i] = __builtin_fmaf(s2[u][i], w, S[i]);
                    y = __builtin_fmaf(s1[u][i], S[i], y);
                    if constexpr (REV) S[i] = decay(S[i]);
                }
            }
            const size_t at = (row * a.H + h) * VD + j;
            if (a.out_f32) static_cast<float*>(a.out)[at] = y * a.out_scale;
            else st1<BF16>(a.out, at, y * a.out_scale);
        }
    }
    if (a.final_state)
#pragma unroll
        for (int i = 0; i < KD; ++i) a.final_state[((size_t)bh * KD + i) * VD + j] = S[i];
}

// Sum over the r heads of each group of an fp32 [rows, G, r, D] tensor, in head order,
// rounded once to [rows, G, D].
template <bool BF16>
__global__ void __launch_bounds__(256) sum_heads(const float* __restrict__ p, void* out, size_t n, int r, int D) {
    const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= n) return;
    const float* q = p + (e / D) * r * D + e % D;
    float s = 0.0f;
    for (int k = 0; k < r; ++k) s += q[(size_t)k * D];
    st1<BF16>(out, e, s);
}

template <int KD, int VD, bool BF16>
hipError_t run_mix_t(const Mix& m, bool rev, hipStream_t st) {
    const dim3 grid((unsigned)m.B * m.H);
    if (rev) launch((mix_kernel<KD, VD, BF16, true>), grid, dim3(VD), 0, st, m);
    else launch((mix_kernel<KD, VD, BF16, false>), grid, dim3(VD), 0, st, m);
    return hipGetLastError();
}

hipError_t run_mix(const Mix& m, int KD, int VD, bool bf16, bool rev, hipStream_t st) {
    if (KD == 64 && VD == 64) return bf16 ? run_mix_t<64, 64, true>(m, rev, st) : run_mix_t<64, 64, false>(m, rev, st);
    if (KD == 64) return bf16 ? run_mix_t<64, 128, true>(m, rev, st) : run_mix_t<64, 128, false>(m, rev, st);
    if (VD == 64) return bf16 ? run_mix_t<128, 64, true>(m, rev, st) : run_mix_t<128, 64, false>(m, rev, st);
    return bf16 ? run_mix_t<128, 128, true>(m, rev, st) : run_mix_t<128, 128, false>(m, rev, st);
}

hipError_t run_sum_heads(const float* p, void* out, size_t n, int r, int D, bool bf16, hipStream_t st) {
    const dim3 grid((unsigned)((n + 255) / 256));
    if (bf16) launch(sum_heads<true>, grid, dim3(256), 0, st, p, out, n, r, D);
    else launch(sum_heads<false>, grid, dim3(256), 0, st, p, out, n, r, D);
    return hipGetLastError();
}

}  // namespace

bool linattn_supported_dim(int d) { return d == 64 || d == 128; }

size_t linattn_workspace_bytes(int, int, int, int, int, int, bool) { return 0; }

// fp32 dq or dk per head, where heads share a group
size_t linattn_bwd_workspace_bytes(int B, int L, int H, int G, int K, int, bool) {
    return H == G ? 0 : (size_t)B * L * H * K * 4;
}

hipError_t launch_linattn_fwd(const LinattnArgs& a, hipStream_t st) {
    const Mix m{a.B, a.L, a.H, a.H / a.G, a.q, a.k, a.v, 1, 1, 0, a.log_decay, a.seqlens,
                a.scale, 1.0f, a.h0, 0, a.o, 0, a.h_final};
    return run_mix(m, a.K, a.V, a.bf16, false, st);
}

hipError_t launch_linattn_bwd(const LinattnBwdArgs& a, hipStream_t st) {
    const int r = a.H / a.G;
    const bool shared = r > 1;
    const size_t ng = (size_t)a.B * a.L * a.G * a.K;
    hipError_t e;
    const Mix mq{a.B, a.L, a.H, r, a.dout, a.v, a.k, 0, 0, 1, a.log_decay, a.seqlens,
                 a.scale, 1.0f, a.h0, 1, shared ? a.ws : a.dq, shared, nullptr};
    if ((e = run_mix(mq, a.V, a.K, a.bf16, false, st)) != hipSuccess) return e;
    if (shared && ng > 0)
        if ((e = run_sum_heads(static_cast<float*>(a.ws), a.dq, ng, r, a.K, a.bf16, st)) != hipSuccess) return e;
    const Mix mk{a.B, a.L, a.H, r, a.v, a.dout, a.q, 0, 0, 1, a.log_decay, a.seqlens,
                 1.0f, a.scale, a.dh_final, 1, shared ? a.ws : a.dk, shared, nullptr};
    if ((e = run_mix(mk, a.V, a.K, a.bf16, true, st)) != hipSuccess) return e;
    if (shared && ng > 0)
        if ((e = run_sum_heads(static_cast<float*>(a.ws), a.dk, ng, r, a.K, a.bf16, st)) != hipSuccess) return e;
    const Mix mv{a.B, a.L, a.H, r, a.k, a.q, a.dout, 1, 1, 0, a.log_decay, a.seqlens,
                 1.0f, a.scale, a.dh_final, 0, a.dv, 0, a.dh0};
    return run_mix(mv, a.K, a.V, a.bf16, true, st);
}

}  // namespace ssm
