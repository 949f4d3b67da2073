// Launchers of the residual add with norm and dropout, and of dropout alone (internal to the
// library; the C ABI in api.cpp validates arguments and then calls these), and the counter
// that dropout draws from.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

struct Dropout {
    unsigned least;                 // an element is kept if its 16 bits are at least this (0: no dropout)
    float scale;                    // 65536 / (65536 - least)
    const unsigned long long* rng;  // seed, offset
};

struct AddNormArgs {
    int M, C;
    bool bf16, res_bf16, rms;
    const void* x;
    const void* residual;
    const float* weight;
    const float* bias;
    float eps;
    Dropout drop;
    void* y;
    void* sum;
    float* mean;
    float* rstd;
};

struct AddNormBwdArgs {
    int M, C;
    bool bf16, res_bf16, rms;
    const void* sum;
    const float* weight;
    const float* mean;
    const float* rstd;
    const void* dy;
    const void* dsum;
    Dropout drop;
    void* dx;
    void* dresidual;
    float* dweight;
    float* dbias;
    void* ws;
};

struct DropoutArgs {
    int M, C;
    bool bf16;
    const void* x;
    Dropout drop;
    void* y;
};

size_t add_norm_bwd_workspace_bytes(int M, int C, bool bf16, bool res_bf16);
hipError_t launch_add_norm_fwd(const AddNormArgs& a, hipStream_t stream);
hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t stream);
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t stream);

// Philox-4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3;
// 2011): the four words of a block number under a seed. Eight channels of a row share a
// block, 16 bits each: the keep probability is then a multiple of 2^-16, which the scale
// takes exactly, and a value costs half of a word-sized draw's multiplications.
struct Philox {
    uint32_t w[4];
    __device__ __forceinline__ Philox(unsigned long long seed, unsigned long long block) {
        uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = 0, c3 = 0;
        uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
            c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
            c1 = (uint32_t)p1;
            c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
            c3 = (uint32_t)p0;
            k0 += 0x9E3779B9u;
            k1 += 0xBB67AE85u;
        }
        w[0] = c0;
        w[1] = c1;
        w[2] = c2;
        w[3] = c3;
    }
    // the 16 bits of the block's channel j
    __device__ __forceinline__ uint32_t bits(int j) const { return j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu; }
};

}  // namespace ssm
