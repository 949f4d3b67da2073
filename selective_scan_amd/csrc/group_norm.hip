// Group norm over channels-last data on gfx950, with activation and / or gate, and its
// gradient. Per sample m and group g, over its S * C/G values:
//   xhat = (x - mean) rstd,  u = xhat w + b,  y = act(u) [silu(z)]
//   du = dy [silu(z)] act'(u),  dz = dy act(u) silu'(z),  dw = sum du xhat,  db = sum du
//   dn = du w,  dx = rstd (dn - mean(dn) - xhat mean(dn xhat))
// Statistics, sums and every intermediate value are fp32 (a running mean 64 bits). Variances come
// from squared distances to a mean, that of a batch of rows where the data is passed over once
// (merged by count, mean and sum of squares), never from a difference of large sums.
//
// Bandwidth-bound throughout. Three shapes of the work:
//   rows    S = 1: a group is Cg = C / G consecutive values. T lanes of a wave (a power of
//           two) hold it in registers, 16 bytes a lane and up to 8 of those: one read, sums
//           by lane exchange, one write.
//   block   a sample's group fits a workgroup's registers (16 x 16 bytes a lane).
//   tiles   otherwise: a workgroup passes over a range of positions of a tile of channels,
//           every lane on channels of its own, and leaves its part of the statistics;
//           a second launch merges the parts of each group and writes the result. The data
//           is read twice, the second time largely from the cache behind the L2s.
// Rows whose channels are not whole 16-byte pieces are taken value by value.
// Measured: 64 x 2048 bf16 in 16 groups with gate 3.5 us (rows; latency); 16 samples of
// 64 x 64 x 512 bf16 in 32 groups with SiLU 50-55 us (tiles: 20 + 31; 134 MB that have to
// move, 27 us at a copy's rate, 201 MB moved); gradient of 32768 x 1536 bf16 in 24 groups
// with gate 112 us a call (rows: 503 MB, 4.5 TB/s), of 8 x 1025 x 320 fp32 in 32 groups
// 20 us (tiles, two launches of little work each: latency).
#include "common.h"
#include "group_norm.h"
#include "launch.h"

#include <algorithm>

namespace ssm {
namespace {

constexpr int kT = 256;
constexpr int kBlockPieces = 16;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// V consecutive values starting at element i: a 16-byte piece, or one value (V = 1).
template <bool BF16, int V>
__device__ __forceinline__ void load(const void* p, size_t i, float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (BF16) x[0] = bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
        else x[0] = static_cast<const float*>(p)[i];
    } else if constexpr (BF16) {
        const u32x4 q = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = bf16_lo(q[k]);
            x[2 * k + 1] = bf16_hi(q[k]);
        }
    } else {
        const u32x4 q = *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(q[k]);
    }
}

// f(i, U) for i, i + U step, ... below end with U = N while N rows are left, then one by one:
// f loads its U rows before it stores any (the compiler moves no load above a store to an
// output that might be an input).
template <int N, typename F>
__device__ __forceinline__ void in_batches(int i, int end, int step, F f) {
    for (; i + (N - 1) * step < end; i += N * step) f(i, std::integral_constant<int, N>{});
    for (; i < end; i += step) f(i, std::integral_constant<int, 1>{});
}

template <bool BF16, int V>
__device__ __forceinline__ void store(void* p, size_t i, const float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(x[0]);
        else static_cast<float*>(p)[i] = x[0];
    } else if constexpr (BF16) {
        u32x4 q;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            q[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2 * k], x[2 * k + 1]}, bf16x2));
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = q;
    } else {
        u32x4 q;
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = __float_as_uint(x[k]);
        *reinterpret_cast<u32x4*>(static_cast<float*>(p) + i) = q;
    }
}

// A channel's parameter (NULL: a constant).
template <int V>
__device__ __forceinline__ void params(const float* p, int c, float missing, float (&x)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = p ? p[c + v] : missing;
}

__device__ __forceinline__ float sigmoid(float x) { return rcp_fast(1.0f + exp2_fast(-x * kLog2e)); }

// Sum over aligned groups of T lanes of a wave, in every lane.
template <int T>
__device__ __forceinline__ float sum_lanes(float v) {
    auto add = [&](auto ctrl) {
        v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    if constexpr (T >= 2) add(std::integral_constant<int, 0xb1>{});    // lanes 1, 0, 3, 2
    if constexpr (T >= 4) add(std::integral_constant<int, 0x4e>{});    // lanes 2, 3, 0, 1
    if constexpr (T >= 8) add(std::integral_constant<int, 0x141>{});   // 8 lanes mirrored
    if constexpr (T >= 16) add(std::integral_constant<int, 0x140>{});  // 16 lanes mirrored
    if constexpr (T >= 32) v += __shfl_xor(v, 16);
    if constexpr (T >= 64) v += __shfl_xor(v, 32);
    return v;
}

// Sum over the workgroup, in every lane (a fixed order).
__device__ __forceinline__ float sum_block(float v, float* red) {
    v = sum_lanes<64>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int w = 1; w < kT / 64; ++w) s += red[w];
    return s;
}

// y of V values whose mean, rstd and parameters are known.
template <int V>
__device__ __forceinline__ void finish(float (&x)[V], float mean, float rstd, const float (&w)[V], const float (&b)[V],
                                       int act) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = __builtin_fmaf((x[v] - mean) * rstd, w[v], b[v]);
    if (act)
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] *= sigmoid(x[v]);
}

// du (in d, which holds dy) and dz of one value.
template <bool GATE>
__device__ __forceinline__ float gate_du(float d, float u, float z, int act, float* dz) {
    const float su = act ? sigmoid(u) : 1.0f;
    if constexpr (GATE) {
        const float sz = sigmoid(z);
        *dz = d * (u * su) * (sz * (1.0f + z * (1.0f - sz)));
        d *= z * sz;
    }
    return act ? d * (su * (1.0f + u * (1.0f - su))) : d;
}

// Workgroups beyond kFold of grid.x go on in grid.z: a grid's dimension holds 2^32 lanes.
constexpr long long kFold = 1 << 22;
__device__ __forceinline__ unsigned folded() { return blockIdx.z * gridDim.x + blockIdx.x; }
dim3 fold(long long n, int y = 1) {
    return dim3((unsigned)std::min(n, kFold), (unsigned)y, (unsigned)((n + kFold - 1) / kFold));
}

// ------------------------------------------------------------------ rows
// T lanes per (sample, group), R pieces a lane; consecutive groups are consecutive in memory.
template <bool BF16, int V, int T, int R>
__global__ void __launch_bounds__(kT) gn_rows_fwd(GroupNormArgs a, long long groups, int cg) {
    const long long q = (long long)folded() * (kT / T) + threadIdx.x / T;
    if (q >= groups) return;
    const int l = threadIdx.x % T, g = (int)(q % a.G);
    float x[R][V], s = 0.0f;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (l + k * T) * V;
        if (c < cg) load<BF16, V>(a.x, q * cg + c, x[k]);
        else
#pragma unroll
            for (int v = 0; v < V; ++v) x[k][v] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) s += x[k][v];
    }
    const float mean = sum_lanes<T>(s) / (float)cg;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < R; ++k)
        if ((l + k * T) * V < cg)
#pragma unroll
            for (int v = 0; v < V; ++v) s = __builtin_fmaf(x[k][v] - mean, x[k][v] - mean, s);
    const float rstd = 1.0f / sqrtf(sum_lanes<T>(s) / (float)cg + a.eps);
    if (l == 0 && a.mean) {
        a.mean[q] = mean;
        a.rstd[q] = rstd;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (l + k * T) * V;
        if (c >= cg) continue;
        float w[V], b[V], z[V];
        params<V>(a.weight, g * cg + c, 1.0f, w);
        params<V>(a.bias, g * cg + c, 0.0f, b);
        if (a.z) load<BF16, V>(a.z, q * cg + c, z);
        finish<V>(x[k], mean, rstd, w, b, a.act);
        if (a.z)
#pragma unroll
            for (int v = 0; v < V; ++v) x[k][v] *= silu(z[v]);
        store<BF16, V>(a.y, q * cg + c, x[k]);
    }
}

// The gradient: a workgroup keeps to kT / T groups of channels and passes over samples
// blockIdx.y, + gridDim.y, ..., so that every lane sums dw and db of channels of its own;
// they are left in part [gridDim.y][2][C].
template <bool BF16, int V, int T, int R, bool GATE>
__global__ void __launch_bounds__(kT) gn_rows_bwd(GroupNormBwdArgs a, int cg, float* part) {
    const int g = blockIdx.x * (kT / T) + threadIdx.x / T, l = threadIdx.x % T;
    if (g >= a.G) return;
    float w[R][V], b[R][V], dw[R][V], db[R][V];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (l + k * T) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) dw[k][v] = db[k][v] = w[k][v] = b[k][v] = 0.0f;
        if (c < cg) {
            params<V>(a.weight, g * cg + c, 1.0f, w[k]);
            params<V>(a.bias, g * cg + c, 0.0f, b[k]);
        }
    }
    const float inv = 1.0f / (float)cg;
    for (int m = blockIdx.y; m < a.M; m += gridDim.y) {
        const size_t q = (size_t)m * a.G + g;
        float x[R][V], d[R][V], z[R][V];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (l + k * T) * V;
#pragma unroll
            for (int v = 0; v < V; ++v) x[k][v] = d[k][v] = z[k][v] = 0.0f;
            if (c < cg) {
                load<BF16, V>(a.x, q * cg + c, x[k]);
                load<BF16, V>(a.dy, q * cg + c, d[k]);
                if constexpr (GATE) load<BF16, V>(a.z, q * cg + c, z[k]);
            }
        }
        const float mean = a.mean[q], rstd = a.rstd[q];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const bool in = (l + k * T) * V < cg;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float xhat = in ? (x[k][v] - mean) * rstd : 0.0f, u = __builtin_fmaf(xhat, w[k][v], b[k][v]);
                float du = gate_du<GATE>(d[k][v], u, z[k][v], a.act, &z[k][v]);
                db[k][v] += du;
                dw[k][v] = __builtin_fmaf(du, xhat, dw[k][v]);
                du *= w[k][v];
                s0 += du;
                s1 = __builtin_fmaf(du, xhat, s1);
                x[k][v] = xhat;
                d[k][v] = du;
            }
        }
        s0 = sum_lanes<T>(s0) * inv;
        s1 = sum_lanes<T>(s1) * inv;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (l + k * T) * V;
            if (c >= cg) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) d[k][v] = rstd * (d[k][v] - s0 - x[k][v] * s1);
            store<BF16, V>(a.dx, q * cg + c, d[k]);
            if constexpr (GATE) store<BF16, V>(a.dz, q * cg + c, z[k]);
        }
    }
    if (!part) return;
    float* p = part + (size_t)blockIdx.y * 2 * a.C + (size_t)g * cg;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (l + k * T) * V;
        if (c < cg)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[c + v] = dw[k][v];
                p[a.C + c + v] = db[k][v];
            }
    }
}

// ------------------------------------------------------------------ block
// One workgroup per (sample, group), piece tid + k kT of its S * cg / V pieces in registers.
template <bool BF16, int V, int R>
__global__ void __launch_bounds__(kT) gn_block_fwd(GroupNormArgs a, int cg) {
    __shared__ float red[kT / 64];
    const unsigned wg = folded(), sample = wg / a.G;
    if (sample >= (unsigned)a.M) return;
    const int g = wg % a.G, m = sample, per = cg / V, n = a.S * per;
    const size_t base = (size_t)m * a.S * a.C + (size_t)g * cg;
    float x[R][V], s = 0.0f;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = threadIdx.x + k * kT;
        if (i < n) load<BF16, V>(a.x, base + (size_t)(i / per) * a.C + (i % per) * V, x[k]);
        else
#pragma unroll
            for (int v = 0; v < V; ++v) x[k][v] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) s += x[k][v];
    const float inv = 1.0f / ((float)a.S * (float)cg), mean = sum_block(s, red) * inv;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < R; ++k)
        if (threadIdx.x + k * kT < n)
#pragma unroll
            for (int v = 0; v < V; ++v) s = __builtin_fmaf(x[k][v] - mean, x[k][v] - mean, s);
    const float rstd = 1.0f / sqrtf(sum_block(s, red) * inv + a.eps);
    if (threadIdx.x == 0 && a.mean) {
        a.mean[(size_t)m * a.G + g] = mean;
        a.rstd[(size_t)m * a.G + g] = rstd;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = threadIdx.x + k * kT;
        if (i >= n) continue;
        const size_t at = base + (size_t)(i / per) * a.C + (i % per) * V;
        float w[V], b[V], z[V];
        params<V>(a.weight, g * cg + (i % per) * V, 1.0f, w);
        params<V>(a.bias, g * cg + (i % per) * V, 0.0f, b);
        if (a.z) load<BF16, V>(a.z, at, z);
        finish<V>(x[k], mean, rstd, w, b, a.act);
        if (a.z)
#pragma unroll
            for (int v = 0; v < V; ++v) x[k][v] *= silu(z[v]);
        store<BF16, V>(a.y, at, x[k]);
    }
}

// ------------------------------------------------------------------ tiles
// A workgroup's tile: gt whole groups, or one of tpg tiles of a group; every lane has V
// channels of its own (lr lanes span the tile) and one of rl rows in turn.
struct Tiles {
    int cg;      // channels per group
    int gt;      // groups per tile (1 where a group is cut)
    int tpg;     // tiles per group (1 where groups are whole)
    int width;   // channels per tile, but for the last
    int tiles;   // tiles of a sample
    int splits;  // ranges of positions of a sample
    int rows;    // positions per range
};

template <int V>
struct Place {
    int g0, ng;        // first group, groups
    int c0, width;     // first channel, channels
    int lr, rl;        // lanes per row, rows at once
    int col, row;      // this lane's first channel in the tile, first row
    int s0, s1;        // positions
    int part, parts;   // which part of its groups' statistics this workgroup is
    bool on;
    __device__ __forceinline__ Place(const Tiles& t, int S, int C, int tile, int split) {
        if (t.tpg == 1) {
            g0 = tile * t.gt;
            ng = min(t.gt, C / t.cg - g0);
            c0 = g0 * t.cg;
            width = ng * t.cg;
        } else {
            g0 = tile / t.tpg;
            ng = 1;
            c0 = g0 * t.cg + (tile % t.tpg) * t.width;
            width = min(t.width, t.cg - (tile % t.tpg) * t.width);
        }
        lr = width / V;
        rl = kT / lr;
        col = (int)(threadIdx.x % lr) * V;
        row = threadIdx.x / lr;
        on = row < rl;
        s0 = split * t.rows;
        s1 = min(S, s0 + t.rows);
        part = t.tpg == 1 ? split : (tile % t.tpg) * t.splits + split;
        parts = t.splits * t.tpg;
    }
    // values of a group in part p
    static __device__ __forceinline__ float count(const Tiles& t, int S, int p) {
        const int split = p % t.splits, tile = p / t.splits;
        const int w = t.tpg == 1 ? t.cg : min(t.width, t.cg - tile * t.width);
        return (float)w * (float)(min(S, (split + 1) * t.rows) - split * t.rows);
    }
};

// Parts of the statistics: stat[(m G + g) parts + part] = mean, sum of squared distances to it.
// A lane takes its rows in batches that it holds in registers: a batch's mean from the distances
// to its first row, then the squared distances to that mean, merged by count. Distances to any one
// row of the data would lose digits for all rows far from that row (a border of zeros, one large
// position). The running mean is kept in 64 bits, 3 of some 40 operations a batch: 2000 merges
// rounded to 32 leave it 4e-6 of the spread off and the variance 5e-7, 64 bits 4e-8 and 2e-7
// (16384 x 33 fp32, a zero row before 300 +- 1). 16 x 4096 x 512 bf16: 19.6 us, where the
// distances to one row alone take 18.7.
template <bool BF16, int V>
__global__ void __launch_bounds__(kT) gn_stats(GroupNormArgs a, Tiles t, float2* stat) {
    __shared__ float sm[kT * V], sq[kT * V];
    const unsigned wg = folded(), sample = wg / t.tiles;
    if (sample >= (unsigned)a.M) return;
    const int tile = wg % t.tiles, m = sample, split = blockIdx.y;
    const Place<V> p(t, a.S, a.C, tile, split);
    const size_t base = (size_t)m * a.S * a.C + p.c0 + p.col;
    if (p.on) {
        double mean[V];
        float q[V];
#pragma unroll
        for (int v = 0; v < V; ++v) mean[v] = q[v] = 0.0f;
        int n = 0;
        in_batches<8>(p.s0 + p.row, p.s1, p.rl, [&](int i, auto rows) {
            constexpr int U = decltype(rows)::value;
            float x[U][V];
#pragma unroll
            for (int k = 0; k < U; ++k) load<BF16, V>(a.x, base + (size_t)(i + k * p.rl) * a.C, x[k]);
            const float share = (float)U / (float)(n + U), between = (float)n * share;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float s = 0.0f, d2 = 0.0f;
#pragma unroll
                for (int k = 1; k < U; ++k) s += x[k][v] - x[0][v];
                const float mb = __builtin_fmaf(s, 1.0f / (float)U, x[0][v]);
#pragma unroll
                for (int k = 0; k < U; ++k) d2 = __builtin_fmaf(x[k][v] - mb, x[k][v] - mb, d2);
                const float d = (float)((double)mb - mean[v]);
                mean[v] = __builtin_fma((double)d, (double)share, mean[v]);
                q[v] += __builtin_fmaf(d * d, between, d2);
            }
            n += U;
        });
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sm[p.row * p.width + p.col + v] = (float)mean[v];
            sq[p.row * p.width + p.col + v] = q[v];
        }
    }
    __syncthreads();
    // a channel's rows: lane r of a channel saw (rows - r + rl - 1) / rl of them
    const int rows = p.s1 - p.s0;
    const float inv_rows = 1.0f / (float)rows;
    for (int c = threadIdx.x; c < p.width; c += kT) {
        float mean = 0.0f, m2 = 0.0f;
        for (int r = 0; r < p.rl; ++r) {
            const int cnt = max(0, (rows - r + p.rl - 1) / p.rl);
            mean = __builtin_fmaf((float)cnt * inv_rows, sm[r * p.width + c] - sm[c], mean);
        }
        mean += sm[c];
        for (int r = 0; r < p.rl; ++r) {
            const int cnt = max(0, (rows - r + p.rl - 1) / p.rl);
            const float d = sm[r * p.width + c] - mean;
            if (cnt > 0) m2 += sq[r * p.width + c] + (float)cnt * d * d;
        }
        sm[c] = mean;
        sq[c] = m2;
    }
    __syncthreads();
    // a group's channels: one wave each
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, w = p.width / p.ng;
    for (int g = wave; g < p.ng; g += kT / 64) {
        const float ref = sm[g * w];
        float s1 = 0.0f;
        for (int c = lane; c < w; c += 64) s1 += sm[g * w + c] - ref;
        const float mean = ref + sum_lanes<64>(s1) / (float)w;
        float s2 = 0.0f;
        for (int c = lane; c < w; c += 64) {
            const float d = sm[g * w + c] - mean;
            s2 += sq[g * w + c] + (float)rows * d * d;
        }
        s2 = sum_lanes<64>(s2);
        if (lane == 0) stat[((size_t)m * a.G + p.g0 + g) * p.parts + p.part] = make_float2(mean, s2);
    }
}

// The parts of the tile's groups merged (one wave each), then the output.
template <bool BF16, int V>
__global__ void __launch_bounds__(kT) gn_apply(GroupNormArgs a, Tiles t, const float2* stat) {
    extern __shared__ float2 gs[];  // [groups of the tile]: mean, rstd
    const unsigned wg = folded(), sample = wg / t.tiles;
    if (sample >= (unsigned)a.M) return;
    const int tile = wg % t.tiles, m = sample, split = blockIdx.y;
    const Place<V> p(t, a.S, a.C, tile, split);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const float inv = 1.0f / ((float)a.S * (float)t.cg);
    for (int g = wave; g < p.ng; g += kT / 64) {
        const float2* st = stat + ((size_t)m * a.G + p.g0 + g) * p.parts;
        const float ref = st[0].x;
        float s = 0.0f;
        for (int k = lane; k < p.parts; k += 64) s = __builtin_fmaf(Place<V>::count(t, a.S, k), st[k].x - ref, s);
        const float mean = __builtin_fmaf(sum_lanes<64>(s), inv, ref);
        float m2 = 0.0f;
        for (int k = lane; k < p.parts; k += 64) {
            const float d = st[k].x - mean;
            m2 += st[k].y + Place<V>::count(t, a.S, k) * d * d;
        }
        const float rstd = 1.0f / sqrtf(sum_lanes<64>(m2) * inv + a.eps);
        if (lane == 0) {
            gs[g] = make_float2(mean, rstd);
            if (p.part == 0 && a.mean) {
                a.mean[(size_t)m * a.G + p.g0 + g] = mean;
                a.rstd[(size_t)m * a.G + p.g0 + g] = rstd;
            }
        }
    }
    __syncthreads();
    if (!p.on) return;
    float mean[V], rstd[V], w[V], b[V];
    params<V>(a.weight, p.c0 + p.col, 1.0f, w);
    params<V>(a.bias, p.c0 + p.col, 0.0f, b);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float2 s = gs[t.tpg == 1 ? (p.col + v) / t.cg : 0];
        mean[v] = s.x;
        rstd[v] = s.y;
    }
    const size_t base = (size_t)m * a.S * a.C + p.c0 + p.col;
#pragma unroll 8
    for (int i = p.s0 + p.row; i < p.s1; i += p.rl) {
        float x[V], z[V];
        load<BF16, V>(a.x, base + (size_t)i * a.C, x);
        if (a.z) load<BF16, V>(a.z, base + (size_t)i * a.C, z);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float u = __builtin_fmaf((x[v] - mean[v]) * rstd[v], w[v], b[v]);
            if (a.act) u *= sigmoid(u);
            if (a.z) u *= silu(z[v]);
            x[v] = u;
        }
        store<BF16, V>(a.y, base + (size_t)i * a.C, x);
    }
}

// What a lane of the gradient's kernels knows of its channels.
template <int V>
struct Chan {
    float mean[V], rstd[V], w[V], b[V];
    __device__ __forceinline__ Chan(const GroupNormBwdArgs& a, const Tiles& t, const Place<V>& p, int m) {
        params<V>(a.weight, p.c0 + p.col, 1.0f, w);
        params<V>(a.bias, p.c0 + p.col, 0.0f, b);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const size_t q = (size_t)m * a.G + p.g0 + (t.tpg == 1 ? (p.col + v) / t.cg : 0);
            mean[v] = a.mean[q];
            rstd[v] = a.rstd[q];
        }
    }
};

// Sums over a range of positions: of du and du xhat per channel, left in part [m splits +
// split][2][C] (dw's first) if there is one, and, times w, per group in stat.
template <bool BF16, int V, bool GATE>
__global__ void __launch_bounds__(kT) gn_bwd_sums(GroupNormBwdArgs a, Tiles t, float2* stat, float* part) {
    __shared__ float sa[kT * V], sb[kT * V];
    const unsigned wg = folded(), sample = wg / t.tiles;
    if (sample >= (unsigned)a.M) return;
    const int tile = wg % t.tiles, m = sample, split = blockIdx.y;
    const Place<V> p(t, a.S, a.C, tile, split);
    float s0[V], s1[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s0[v] = s1[v] = 0.0f;
    if (p.on) {
        const Chan<V> c(a, t, p, m);
        const size_t base = (size_t)m * a.S * a.C + p.c0 + p.col;
#pragma unroll 4
        for (int i = p.s0 + p.row; i < p.s1; i += p.rl) {
            float x[V], d[V], z[V], dz;
            load<BF16, V>(a.x, base + (size_t)i * a.C, x);
            load<BF16, V>(a.dy, base + (size_t)i * a.C, d);
            if constexpr (GATE) load<BF16, V>(a.z, base + (size_t)i * a.C, z);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float xhat = (x[v] - c.mean[v]) * c.rstd[v];
                const float du = gate_du<GATE>(d[v], __builtin_fmaf(xhat, c.w[v], c.b[v]), GATE ? z[v] : 0.0f, a.act, &dz);
                s0[v] += du;
                s1[v] = __builtin_fmaf(du, xhat, s1[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sa[p.row * p.width + p.col + v] = s0[v];
            sb[p.row * p.width + p.col + v] = s1[v];
        }
    }
    __syncthreads();
    float* out = part ? part + ((size_t)m * t.splits + split) * 2 * a.C + p.c0 : nullptr;
    for (int c = threadIdx.x; c < p.width; c += kT) {
        float u = 0.0f, v = 0.0f;
        for (int r = 0; r < p.rl; ++r) {
            u += sa[r * p.width + c];
            v += sb[r * p.width + c];
        }
        if (out) {
            out[c] = v;
            out[a.C + c] = u;
        }
        const float w = a.weight ? a.weight[p.c0 + c] : 1.0f;
        sa[c] = u * w;
        sb[c] = v * w;
    }
    __syncthreads();
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, w = p.width / p.ng;
    for (int g = wave; g < p.ng; g += kT / 64) {
        float u = 0.0f, v = 0.0f;
        for (int c = lane; c < w; c += 64) {
            u += sa[g * w + c];
            v += sb[g * w + c];
        }
        u = sum_lanes<64>(u);
        v = sum_lanes<64>(v);
        if (lane == 0) stat[((size_t)m * a.G + p.g0 + g) * p.parts + p.part] = make_float2(u, v);
    }
}

// dweight and dbias from n parts [n][2][C]: 16 of the 2 C sums per workgroup (a 64-byte line
// of a part), sixteen lanes each.
__device__ __forceinline__ void sum_parts(const float* __restrict__ part, int n, int C, unsigned wg, float* dweight,
                                          float* dbias) {
    __shared__ float s[16][17];
    const int i = threadIdx.x & 15, r = threadIdx.x >> 4, e = wg * 16 + i;
    float v = 0.0f;
    if (e < 2 * C)
#pragma unroll 8
        for (int k = r; k < n; k += 16) v += part[(size_t)k * 2 * C + e];
    s[r][i] = v;
    __syncthreads();
    if (r != 0 || e >= 2 * C) return;
    for (int k = 1; k < 16; ++k) v += s[k][i];
    if (e < C) {
        if (dweight) dweight[e] = v;
    } else if (dbias) {
        dbias[e - C] = v;
    }
}

// dx and dz; the workgroups behind the last sample's sum the n parts of dw and db (n = 0: none),
// which saves a launch: 8 x 1025 x 320 fp32 takes 24 us on the GPU and not 27.
template <bool BF16, int V, bool GATE>
__global__ void __launch_bounds__(kT) gn_bwd_apply(GroupNormBwdArgs a, Tiles t, const float2* stat,
                                                   const float* part, int n) {
    extern __shared__ float2 gs[];  // [groups of the tile]: mean of dn, mean of dn xhat
    const unsigned wg = folded(), sample = wg / t.tiles;
    if (sample >= (unsigned)a.M) {
        const unsigned at = (wg - t.tiles * (unsigned)a.M) * gridDim.y + blockIdx.y;
        if (n > 0 && at * 16 < 2 * (unsigned)a.C) sum_parts(part, n, a.C, at, a.dweight, a.dbias);
        return;
    }
    const int tile = wg % t.tiles, m = sample, split = blockIdx.y;
    const Place<V> p(t, a.S, a.C, tile, split);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const float inv = 1.0f / ((float)a.S * (float)t.cg);
    for (int g = wave; g < p.ng; g += kT / 64) {
        const float2* st = stat + ((size_t)m * a.G + p.g0 + g) * p.parts;
        float u = 0.0f, v = 0.0f;
        for (int k = lane; k < p.parts; k += 64) {
            u += st[k].x;
            v += st[k].y;
        }
        u = sum_lanes<64>(u);
        v = sum_lanes<64>(v);
        if (lane == 0) gs[g] = make_float2(u * inv, v * inv);
    }
    __syncthreads();
    if (!p.on) return;
    const Chan<V> c(a, t, p, m);
    float m0[V], m1[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float2 s = gs[t.tpg == 1 ? (p.col + v) / t.cg : 0];
        m0[v] = s.x;
        m1[v] = s.y;
    }
    const size_t base = (size_t)m * a.S * a.C + p.c0 + p.col;
    in_batches<4>(p.s0 + p.row, p.s1, p.rl, [&](int i, auto n) {
        constexpr int U = decltype(n)::value;
        float x[U][V], d[U][V], z[U][V];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const size_t e = base + (size_t)(i + k * p.rl) * a.C;
            load<BF16, V>(a.x, e, x[k]);
            load<BF16, V>(a.dy, e, d[k]);
            if constexpr (GATE) load<BF16, V>(a.z, e, z[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const size_t e = base + (size_t)(i + k * p.rl) * a.C;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float xhat = (x[k][v] - c.mean[v]) * c.rstd[v];
                const float u = __builtin_fmaf(xhat, c.w[v], c.b[v]);
                const float dn = gate_du<GATE>(d[k][v], u, GATE ? z[k][v] : 0.0f, a.act, &z[k][v]) * c.w[v];
                x[k][v] = c.rstd[v] * (dn - m0[v] - xhat * m1[v]);
            }
            store<BF16, V>(a.dx, e, x[k]);
            if constexpr (GATE) store<BF16, V>(a.dz, e, z[k]);
        }
    });
}

// dw and db of a range of rows (sample and position), every lane on channels of its own;
// left in part [gridDim.y][2][C].
template <bool BF16, int V, bool GATE>
__global__ void __launch_bounds__(kT) gn_bwd_affine(GroupNormBwdArgs a, long long rows, int cg, float* part) {
    const int c = (blockIdx.x * kT + threadIdx.x) * V;
    if (c >= a.C) return;
    float w[V], b[V], dw[V], db[V];
    params<V>(a.weight, c, 1.0f, w);
    params<V>(a.bias, c, 0.0f, b);
#pragma unroll
    for (int v = 0; v < V; ++v) dw[v] = db[v] = 0.0f;
#pragma unroll 2
    for (long long i = blockIdx.y; i < rows; i += gridDim.y) {
        const size_t mg = (size_t)(i / a.S) * a.G;
        float x[V], d[V], z[V], dz;
        load<BF16, V>(a.x, (size_t)i * a.C + c, x);
        load<BF16, V>(a.dy, (size_t)i * a.C + c, d);
        if constexpr (GATE) load<BF16, V>(a.z, (size_t)i * a.C + c, z);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = (c + v) / cg;
            const float xhat = (x[v] - a.mean[mg + g]) * a.rstd[mg + g];
            const float du = gate_du<GATE>(d[v], __builtin_fmaf(xhat, w[v], b[v]), GATE ? z[v] : 0.0f, a.act, &dz);
            db[v] += du;
            dw[v] = __builtin_fmaf(du, xhat, dw[v]);
        }
    }
    float* p = part + (size_t)blockIdx.y * 2 * a.C + c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p[v] = dw[v];
        p[a.C + v] = db[v];
    }
}

__global__ void __launch_bounds__(kT) gn_sum_parts(const float* __restrict__ part, int n, int C, float* dweight,
                                                   float* dbias) {
    sum_parts(part, n, C, blockIdx.x, dweight, dbias);
}

// ------------------------------------------------------------------ choices
// Parts of dw and db that gn_rows_bwd and gn_bwd_affine leave, at most: 32768 x 1536 bf16 takes
// 163 us with 512, 123 with 1024, 131 with 2048 (whose parts cost 4 us more to sum).
constexpr int kParts = 1024;

bool pieces(int C, int cg, int V) { return C % V == 0 && cg % V == 0; }

int vec(int C, bool bf16) {
    const int V = bf16 ? 8 : 4;
    return C % V == 0 ? V : 1;
}

// Lanes and pieces per lane of the rows kernels; false if a group does not fit.
bool rows_shape(int cg, int V, int max_r, int* T, int* R) {
    const int n = (cg + V - 1) / V;
    *T = 1;
    while (*T < n && *T < 64) *T *= 2;
    *R = (n + *T - 1) / *T;
    *R = *R <= 1 ? 1 : *R <= 2 ? 2 : *R <= 4 ? 4 : *R <= 8 ? 8 : 16;
    return *R <= max_r;
}

int gcd(int x, int y) { return y ? gcd(y, x % y) : x; }

// The tiles of a sample, and V: pieces where whole ones make up every tile.
Tiles tiles_of(int M, int S, int C, int G, bool bf16, int* V) {
    Tiles t;
    t.cg = C / G;
    *V = vec(C, bf16);
    for (;;) {
        const int most = kT * *V, unit = *V / gcd(t.cg, *V);  // groups whose channels are whole pieces
        if (t.cg <= most) {
            t.gt = most / t.cg / unit * unit;
            if (t.gt > 0) {
                t.gt = std::min(t.gt, G);
                t.tpg = 1;
                t.width = t.gt * t.cg;
                t.tiles = (G + t.gt - 1) / t.gt;
                break;
            }
        } else if (t.cg % *V == 0) {
            t.gt = 1;
            t.tpg = (t.cg + most - 1) / most;
            t.width = most;
            t.tiles = G * t.tpg;
            break;
        }
        *V = 1;
    }
    // three workgroups a CU, but at least eight rows a lane (16 samples of 64 x 64 x 512 bf16:
    // 52 us with 512 workgroups, 49.5 with 768, 52 with 1024, 64 with 2048)
    const int rl = std::max(1, kT / (t.width / *V));
    const long want = std::max<long>(1, 768 / std::max<long>(1, (long)M * t.tiles));
    const long most = std::max<long>(1, (S + 8L * rl - 1) / (8L * rl));
    t.splits = (int)std::min(std::min(want, most), 256L);
    t.rows = (S + t.splits - 1) / t.splits;
    t.splits = (S + t.rows - 1) / t.rows;
    return t;
}

size_t stat_bytes(int M, int G, const Tiles& t) { return ((size_t)M * G * t.splits * t.tpg * 8 + 15) / 16 * 16; }

enum Path { kRows, kBlock, kTiles };

Path fwd_path(int S, int C, int G, bool bf16) {
    const int cg = C / G, W = bf16 ? 8 : 4, V = pieces(C, cg, W) ? W : 1;
    int T, R;
    if (S == 1 && rows_shape(cg, V, 8, &T, &R)) return kRows;
    // whole 64-byte lines of a row per group, or rows that follow each other
    const bool lines = V > 1 && (S == 1 || cg * (bf16 ? 2 : 4) % 64 == 0);
    if (lines && (long long)S * cg <= (long long)kT * kBlockPieces * V) return kBlock;
    return kTiles;
}

Path bwd_path(int S, int C, int G, bool bf16) {
    const int cg = C / G, W = bf16 ? 8 : 4, V = pieces(C, cg, W) ? W : 1;
    int T, R;
    return S == 1 && rows_shape(cg, V, 4, &T, &R) ? kRows : kTiles;
}

// Whether gn_bwd_sums leaves dw and db in a part per sample and range (8 bytes a channel, against
// 6 or more a channel and row of the range), or gn_bwd_affine reads x and dy again for 1024 parts
// at most. M x S x C bf16, parts against reading again: 4096 x 8 x 64 53 us and 102, 4096 x 8 x 1024
// 91 and 136, 262144 x 8 x 64 3.6 ms and 6.5, 4096 x 512 x 320 1.3 ms and 4.1. The parts grow with
// M all the same; only short ranges of C taken value by value lose (16384 x 8 x 33: 113 and 94).
bool parts_by_range(const Tiles& t) { return t.rows >= 8; }

// Workgroups that sum the parts of dw and db.
int sum_groups(int C) { return (2 * C + 15) / 16; }

int row_parts(long long rows) { return (int)std::min<long long>(kParts, std::max<long long>(1, (rows + 7) / 8)); }

template <bool BF16, int V>
hipError_t rows_fwd(const GroupNormArgs& a, hipStream_t st) {
    const int cg = a.C / a.G;
    const long long groups = (long long)a.M * a.G;
    int T, R;
    rows_shape(cg, V, 8, &T, &R);
    const dim3 grid = fold((groups + kT / T - 1) / (kT / T));
#define SSM_GN_ROWS(t, r) \
    if (T == t && R == r) launch((gn_rows_fwd<BF16, V, t, r>), grid, dim3(kT), 0, st, a, groups, cg);
    SSM_GN_ROWS(1, 1) SSM_GN_ROWS(2, 1) SSM_GN_ROWS(4, 1) SSM_GN_ROWS(8, 1) SSM_GN_ROWS(16, 1) SSM_GN_ROWS(32, 1)
    SSM_GN_ROWS(64, 1) SSM_GN_ROWS(64, 2) SSM_GN_ROWS(64, 4) SSM_GN_ROWS(64, 8)
#undef SSM_GN_ROWS
    return hipGetLastError();
}

template <bool BF16, int V, bool GATE>
hipError_t rows_bwd(const GroupNormBwdArgs& a, float* part, int parts, hipStream_t st) {
    const int cg = a.C / a.G;
    int T, R;
    rows_shape(cg, V, 4, &T, &R);
    const dim3 grid((unsigned)((a.G + kT / T - 1) / (kT / T)), (unsigned)parts);
#define SSM_GN_ROWS(t, r) \
    if (T == t && R == r) launch((gn_rows_bwd<BF16, V, t, r, GATE>), grid, dim3(kT), 0, st, a, cg, part);
    SSM_GN_ROWS(1, 1) SSM_GN_ROWS(2, 1) SSM_GN_ROWS(4, 1) SSM_GN_ROWS(8, 1) SSM_GN_ROWS(16, 1) SSM_GN_ROWS(32, 1)
    SSM_GN_ROWS(64, 1) SSM_GN_ROWS(64, 2) SSM_GN_ROWS(64, 4)
#undef SSM_GN_ROWS
    return hipGetLastError();
}

template <bool BF16>
hipError_t block_fwd(const GroupNormArgs& a, hipStream_t st) {
    constexpr int V = BF16 ? 8 : 4;
    const int cg = a.C / a.G;
    const long long n = ((long long)a.S * (cg / V) + kT - 1) / kT;
    const dim3 grid = fold((long long)a.M * a.G);
    if (n <= 1) launch((gn_block_fwd<BF16, V, 1>), grid, dim3(kT), 0, st, a, cg);
    else if (n <= 4) launch((gn_block_fwd<BF16, V, 4>), grid, dim3(kT), 0, st, a, cg);
    else launch((gn_block_fwd<BF16, V, kBlockPieces>), grid, dim3(kT), 0, st, a, cg);
    return hipGetLastError();
}

template <bool BF16, int V>
hipError_t tiles_fwd(const GroupNormArgs& a, const Tiles& t, hipStream_t st) {
    const dim3 grid = fold((long long)t.tiles * a.M, t.splits);
    float2* stat = static_cast<float2*>(a.ws);
    launch((gn_stats<BF16, V>), grid, dim3(kT), 0, st, a, t, stat);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    launch((gn_apply<BF16, V>), grid, dim3(kT), (uint32_t)(t.gt * sizeof(float2)), st, a, t, stat);
    return hipGetLastError();
}

template <bool BF16, int V, bool GATE>
hipError_t tiles_bwd(const GroupNormBwdArgs& a, const Tiles& t, float* part, hipStream_t st) {
    const dim3 grid = fold((long long)t.tiles * a.M, t.splits);
    float2* stat = static_cast<float2*>(a.ws);
    launch((gn_bwd_sums<BF16, V, GATE>), grid, dim3(kT), 0, st, a, t, stat, parts_by_range(t) ? part : nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const bool sums = part && parts_by_range(t);
    const dim3 more = fold((long long)t.tiles * a.M + (sums ? (sum_groups(a.C) + t.splits - 1) / t.splits : 0), t.splits);
    launch((gn_bwd_apply<BF16, V, GATE>), more, dim3(kT), (uint32_t)(t.gt * sizeof(float2)), st, a, t, stat, part,
           sums ? a.M * t.splits : 0);
    if ((e = hipGetLastError()) != hipSuccess || !part || sums) return e;
    const long long rows = (long long)a.M * a.S;
    const dim3 ga((unsigned)((a.C / V + kT - 1) / kT), (unsigned)row_parts(rows));
    launch((gn_bwd_affine<BF16, V, GATE>), ga, dim3(kT), 0, st, a, rows, a.C / a.G, part);
    return hipGetLastError();
}

}  // namespace

size_t group_norm_workspace_bytes(int M, int S, int C, int G, bool bf16) {
    if (M == 0 || fwd_path(S, C, G, bf16) != kTiles) return 0;
    int V;
    return stat_bytes(M, G, tiles_of(M, S, C, G, bf16, &V));
}

size_t group_norm_bwd_workspace_bytes(int M, int S, int C, int G, bool bf16) {
    if (M == 0) return 0;
    if (bwd_path(S, C, G, bf16) == kRows) return (size_t)row_parts(M) * 2 * C * 4;
    int V;
    const Tiles t = tiles_of(M, S, C, G, bf16, &V);
    const size_t parts = parts_by_range(t) ? (size_t)M * t.splits : (size_t)row_parts((long long)M * S);
    return stat_bytes(M, G, t) + parts * 2 * C * 4;
}

hipError_t launch_group_norm_fwd(const GroupNormArgs& a, hipStream_t st) {
    if (a.M == 0) return hipSuccess;
    const Path path = fwd_path(a.S, a.C, a.G, a.bf16);
    if (path == kRows) {
        if (a.bf16) return pieces(a.C, a.C / a.G, 8) ? rows_fwd<true, 8>(a, st) : rows_fwd<true, 1>(a, st);
        return pieces(a.C, a.C / a.G, 4) ? rows_fwd<false, 4>(a, st) : rows_fwd<false, 1>(a, st);
    }
    if (path == kBlock) return a.bf16 ? block_fwd<true>(a, st) : block_fwd<false>(a, st);
    int V;
    const Tiles t = tiles_of(a.M, a.S, a.C, a.G, a.bf16, &V);
    if (a.bf16) return V == 8 ? tiles_fwd<true, 8>(a, t, st) : tiles_fwd<true, 1>(a, t, st);
    return V == 4 ? tiles_fwd<false, 4>(a, t, st) : tiles_fwd<false, 1>(a, t, st);
}

hipError_t launch_group_norm_bwd(const GroupNormBwdArgs& a, hipStream_t st) {
    const bool affine = a.dweight || a.dbias, gate = a.z != nullptr;
    float* part = nullptr;
    int n = 0;
    bool summed = false;
    hipError_t e = hipSuccess;
    if (a.M > 0 && bwd_path(a.S, a.C, a.G, a.bf16) == kRows) {
        n = row_parts(a.M);
        part = affine ? static_cast<float*>(a.ws) : nullptr;
        const bool p = pieces(a.C, a.C / a.G, a.bf16 ? 8 : 4);
        if (a.bf16 && p) e = gate ? rows_bwd<true, 8, true>(a, part, n, st) : rows_bwd<true, 8, false>(a, part, n, st);
        else if (a.bf16) e = gate ? rows_bwd<true, 1, true>(a, part, n, st) : rows_bwd<true, 1, false>(a, part, n, st);
        else if (p) e = gate ? rows_bwd<false, 4, true>(a, part, n, st) : rows_bwd<false, 4, false>(a, part, n, st);
        else e = gate ? rows_bwd<false, 1, true>(a, part, n, st) : rows_bwd<false, 1, false>(a, part, n, st);
    } else if (a.M > 0) {
        int V;
        const Tiles t = tiles_of(a.M, a.S, a.C, a.G, a.bf16, &V);
        if (affine) {
            part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + stat_bytes(a.M, a.G, t));
            n = row_parts((long long)a.M * a.S);
            summed = parts_by_range(t);
        }
        if (a.bf16 && V == 8) e = gate ? tiles_bwd<true, 8, true>(a, t, part, st) : tiles_bwd<true, 8, false>(a, t, part, st);
        else if (a.bf16) e = gate ? tiles_bwd<true, 1, true>(a, t, part, st) : tiles_bwd<true, 1, false>(a, t, part, st);
        else if (V == 4) e = gate ? tiles_bwd<false, 4, true>(a, t, part, st) : tiles_bwd<false, 4, false>(a, t, part, st);
        else e = gate ? tiles_bwd<false, 1, true>(a, t, part, st) : tiles_bwd<false, 1, false>(a, t, part, st);
    }
    if (e != hipSuccess || !affine || summed) return e;
    launch(gn_sum_parts, dim3((unsigned)sum_groups(a.C)), dim3(kT), 0, st, part, n, a.C, a.dweight, a.dbias);
    return hipGetLastError();
}

}  // namespace ssm
