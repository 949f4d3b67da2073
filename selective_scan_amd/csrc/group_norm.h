// Launchers of the channels-last group norm (internal to the library; the C ABI in
// api.cpp validates arguments and then calls these).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace ssm {

struct GroupNormArgs {
    int M, S, C, G;
    bool bf16;
    int act;  // 0 none, 1 SiLU
    const void* x;
    const float* weight;
    const float* bias;
    const void* z;
    float eps;
    void* y;
    float* mean;
    float* rstd;
    void* ws;
};

struct GroupNormBwdArgs {
    int M, S, C, G;
    bool bf16;
    int act;
    const void* x;
    const float* weight;
    const float* bias;
    const void* z;
    const float* mean;
    const float* rstd;
    const void* dy;
    void* dx;
    float* dweight;
    float* dbias;
    void* dz;
    void* ws;
};

size_t group_norm_workspace_bytes(int M, int S, int C, int G, bool bf16);
size_t group_norm_bwd_workspace_bytes(int M, int S, int C, int G, bool bf16);
hipError_t launch_group_norm_fwd(const GroupNormArgs& a, hipStream_t stream);
hipError_t launch_group_norm_bwd(const GroupNormBwdArgs& a, hipStream_t stream);

}  // namespace ssm
