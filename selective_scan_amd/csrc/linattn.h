// Launchers of linear attention with a decay per head (internal to the library;
// the C ABI in api.cpp validates arguments and then calls these).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace ssm {

// A state's decay by lam = exp(a). Above one half it is applied as S + S (lam - 1), with
// lam - 1 = expm1(a): the rounding of lam itself (up to 2^-25) would act in the same
// direction on every application to a slowly decaying state. Below, S lam keeps the
// relative precision of what is left.
// Both are one fma with the state masked to itself or to 0 as the addend: no branch.
struct Decay {
    float m;
    unsigned keep;
    __device__ __forceinline__ explicit Decay(float a) {
        const bool slow = a > -0.69f;
        m = slow ? expm1f(a) : expf(a);
        keep = slow ? 0xffffffffu : 0u;
    }
    __device__ __forceinline__ float operator()(float s) const {
        return __builtin_fmaf(s, m, __uint_as_float(__float_as_uint(s) & keep));
    }
};

// Group norm and gate after the attention (per token and head, over V values).
struct LinattnNorm {
    bool on;
    const float* weight;
    const float* bias;
    const void* z;
    float eps;
};

struct LinattnArgs {
    int B, L, H, G, K, V;
    bool bf16;
    const void* q;
    const void* k;
    const void* v;
    const float* log_decay;
    float scale;
    const int* seqlens;
    const float* h0;
    void* o;
    float* h_final;
    void* ws;
};

struct LinattnBwdArgs {
    int B, L, H, G, K, V;
    bool bf16;
    const void* q;
    const void* k;
    const void* v;
    const float* log_decay;
    float scale;
    const int* seqlens;
    const float* h0;
    const void* dout;
    const float* dh_final;
    void* dq;
    void* dk;
    void* dv;
    float* dh0;
    void* ws;
};

struct LinattnStepArgs {
    int B, H, G, K, V;
    bool bf16;
    float* state;
    const void* q;
    const void* k;
    const void* v;
    const float* log_decay;
    float scale;
    LinattnNorm norm;
    void* o;
};

bool linattn_supported_dim(int d);
// chunks, super-chunks, chunks of one, pieces, chunks of one, heads that share a workgroup
void linattn_plan(int B, int L, int H, int G, int K, int V, bool bf16, bool bwd, int plan[6]);
size_t linattn_workspace_bytes(int B, int L, int H, int G, int K, int V, bool bf16);
size_t linattn_bwd_workspace_bytes(int B, int L, int H, int G, int K, int V, bool bf16);
hipError_t launch_linattn_fwd(const LinattnArgs& a, hipStream_t stream);
hipError_t launch_linattn_bwd(const LinattnBwdArgs& a, hipStream_t stream);
hipError_t launch_linattn_step(const LinattnStepArgs& a, hipStream_t stream);

}  // namespace ssm
