// Residual add with dropout and layer norm or RMS norm on gfx950, its gradient, and dropout alone:
//   s = residual + dropout(x),  y = (s - mean) rstd w + b   (rms: s rstd w + b)
//   ds = rstd (dn - mean(dn) - xhat mean(dn xhat)) + dsum,  dn = dy w   (rms: no mean(dn))
//   dresidual = ds,  dx = dropout(ds),  dw = sum dy xhat,  db = sum dy
//
// Bandwidth-bound: every row is read and written once, in registers in between (but for the
// gradient beyond 8192 channels, below). A lane has eight
// neighbouring channels (an octet: the generator's block, and one or two 16-byte accesses); a row
// takes 16 lanes (C <= 128), a wave (C <= 512) or a workgroup of as many waves as its octets
// fill, one octet a lane, two beyond 8192 channels. Workgroups walk rows, so that a lane reads
// its weights once and, in the gradient, sums dw and db of its channels in registers, and the
// next row's loads are under way while the present one is reduced and written. Sums of a row that
// spans waves go through LDS, two sets of slots in turn, one barrier a sum. Octets that start off
// a 16-byte border (odd widths) are loaded as they lie; the last one of a row is taken value by
// value where it is not whole.
// Statistics and sums are fp32, the variance from squared distances to the mean.
// Measured: 32768 x 1536 bf16 on an fp32 stream with dropout 115 us (604 MB, 5.3 TB/s, a copy's
// rate), its gradient 153 us (805 MB, 5.3 TB/s), gradient of 4099 x 1001 fp32 23 us (82 MB, partly
// in the memory-side cache; a second launch that sums the parts takes 4), 64 x 2048 3.2 us (the
// call's host side 10), dropout alone of 32768 x 1536 bf16 33 us (201 MB; 6.2 TB/s, partly in the
// cache). 12 waves a CU walk the rows: 18 or 24 of the forward's were slower at 32768 x 1536 (122,
// 124 us), in the gradient 6 (186) and 15 (161); workgroups that do not all fit at once cost a
// quarter (201). Other widths, bf16 on fp32 without dropout: 65536 x 256, 520 and 768 and 8192 x
// 4096 to 5120 take 42, 94, 121 and 83 to 97 us (4.4 to 5.2 TB/s), their gradients 56, 115, 151 and
// 119 to 138; rows that leave lanes idle run at that share of it (65536 x 32 10 and 18 us, 65536 x
// 136 33 and 49: 1.9 to 3.3 TB/s).
// In the gradient with two octets a lane registers do not hold a row: 22 (fp32) or 19 (bf16 on
// fp32) of them go to scratch beyond 8192 channels, 43 to 106 beyond 12288, and counters show that
// traffic in memory: 4096 x 10000 fp32 252 us (3.2 TB/s of what has to move; 1.3 times that moved),
// 2048 x 16384 318 us (2.1 TB/s; 2.3 times).
#include "add_norm.h"
#include "common.h"
#include "launch.h"

#include <algorithm>

namespace ssm {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// 16 bytes at any element's address
typedef unsigned int u32x4 __attribute__((ext_vector_type(4), aligned(2)));

constexpr int kBwdLanes = 768;  // of a workgroup in the gradient, but where one row takes more

// An octet as it is stored: values beyond the row's end read as 0.
template <bool BF16>
struct Octet {
    static constexpr int N = BF16 ? 4 : 8;
    uint32_t w[N];
    // n: channels of the row from here on
    __device__ __forceinline__ void load(const void* p, size_t i, int n) {
        if (n >= 8) {
            const char* at = static_cast<const char*>(p) + i * (BF16 ? 2 : 4);
#pragma unroll
            for (int k = 0; k < N / 4; ++k) {
                const u32x4 q = *reinterpret_cast<const u32x4*>(at + 16 * k);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * k + j] = q[j];
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = 0;
#pragma unroll
        for (int j = 0; j < 7; ++j) {
            if (j >= n) continue;
            if constexpr (BF16) w[j / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[i + j] << (16 * (j & 1));
            else w[j] = static_cast<const uint32_t*>(p)[i + j];
        }
    }
    __device__ __forceinline__ float operator[](int j) const {
        if constexpr (BF16) return j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
        else return __uint_as_float(w[j]);
    }
};

template <bool BF16>
__device__ __forceinline__ void store(void* p, size_t i, int n, const float (&v)[8]) {
    if (n >= 8) {
        char* at = static_cast<char*>(p) + i * (BF16 ? 2 : 4);
        if constexpr (BF16) {
            u32x4 q;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                q[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * k], v[2 * k + 1]}, bf16x2));
            *reinterpret_cast<u32x4*>(at) = q;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 q;
#pragma unroll
                for (int k = 0; k < 4; ++k) q[k] = __float_as_uint(v[4 * h + k]);
                *reinterpret_cast<u32x4*>(at + 16 * h) = q;
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        if (j >= n) continue;
        if constexpr (BF16) static_cast<uint16_t*>(p)[i + j] = f32_to_bf16(v[j]);
        else static_cast<float*>(p)[i + j] = v[j];
    }
}

// Eight of a vector's values (missing: the vector is NULL; 0 behind its end).
__device__ __forceinline__ void params(const float* p, int c, int n, float missing, float (&v)[8]) {
    Octet<false> q;
    if (p) q.load(p, c, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p ? q[j] : j < n ? missing : 0.0f;
}

// v where the octet's block keeps it, scaled; else 0.
__device__ __forceinline__ void drop(float (&v)[8], const Dropout& d, unsigned long long seed, unsigned long long block) {
    const Philox p(seed, block);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p.bits(j) >= d.least ? v[j] * d.scale : 0.0f;
}

// The lanes of a row: L of a wave, or (L = 0) `waves` whole waves of the workgroup, of which it
// has one or several rows.
template <int L>
struct Row {
    int waves;
    __device__ __forceinline__ int lanes() const { return L == 0 ? waves * 64 : L; }
    __device__ __forceinline__ int rows() const { return blockDim.x / lanes(); }
    // the same in every lane of a wave but with rows of 16 lanes
    __device__ __forceinline__ int row() const {
        if constexpr (L == 16) return threadIdx.x / 16;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        return L == 0 ? wave / waves : wave;
    }
    __device__ __forceinline__ int lane() const { return threadIdx.x - row() * lanes(); }

    template <int CTRL>
    __device__ __forceinline__ static void exchange(float& v) {
        v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, false));
    }

    // Sums over the row's lanes, in every lane and in a fixed order. slots: 16 a value, another set
    // than the last call's, whose values waves that are behind may still read; that they have read
    // those of the call before it, they say at the last call's barrier. Every wave of the workgroup
    // takes part.
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N], float (*slots)[16]) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            exchange<0xb1>(v[k]);   // lanes 1, 0, 3, 2
            exchange<0x4e>(v[k]);   // lanes 2, 3, 0, 1
            exchange<0x141>(v[k]);  // 8 lanes mirrored
            exchange<0x140>(v[k]);  // 16 lanes mirrored
            if constexpr (L != 16) {
                v[k] += __shfl_xor(v[k], 16);
                v[k] += __shfl_xor(v[k], 32);
            }
        }
        if constexpr (L == 0) {
            const int wave = threadIdx.x >> 6, first = row() * waves;
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int k = 0; k < N; ++k) slots[k][wave] = v[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < N; ++k) {
                v[k] = slots[k][first];
                for (int w = 1; w < waves; ++w) v[k] += slots[k][first + w];
            }
        }
    }
};

// ------------------------------------------------------------------ forward
template <bool BF16, bool RES16, int L, int R>
__global__ void __launch_bounds__(L == 0 ? 1024 : 256) add_norm_fwd(AddNormArgs a) {
    __shared__ float slots[2][1][16];
    const Row<L> me{(int)blockDim.x >> 6};  // with whole waves, one row a workgroup
    const int l = me.lane(), lanes = me.lanes(), octets = (a.C + 7) / 8;
    const long long step = (long long)gridDim.x * me.rows();
    float w[R][8], b[R][8];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (l + k * lanes) * 8;
        params(a.weight, c, a.C - c, 1.0f, w[k]);
        params(a.bias, c, a.C - c, 0.0f, b[k]);
    }
    const bool dropping = a.drop.least != 0;
    const unsigned long long seed = dropping ? a.drop.rng[0] : 0, offset = dropping ? a.drop.rng[1] : 0;
    const float inv = 1.0f / (float)a.C;
    Octet<BF16> x[R];
    Octet<RES16> res[R];
    auto fetch = [&](long long m) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (l + k * lanes) * 8;
            x[k].load(a.x, m * a.C + c, a.C - c);
            if (a.residual) res[k].load(a.residual, m * a.C + c, a.C - c);
        }
    };
    // one row a workgroup: m is the same in every lane, no wave leaves the barriers early
    long long m = (long long)blockIdx.x * me.rows() + me.row();
    int turn = 0;
    if (m < a.M) fetch(m);
    for (; m < a.M; m += step) {
        float s[R][8], t[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < R; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) s[k][j] = x[k][j];
            if (dropping) drop(s[k], a.drop, seed, offset + (unsigned long long)m * octets + l + k * lanes);
            if (a.residual)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[k][j] += res[k][j];
        }
        if (m + step < a.M) fetch(m + step);
        float mean = 0.0f;
        if (!a.rms) {
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) t[0] += s[k][j];
            me.sum(t, slots[turn]);
            turn ^= 1;
            mean = t[0] * inv;
            t[0] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int n = a.C - (l + k * lanes) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = j < n ? s[k][j] - mean : 0.0f;
                t[0] = __builtin_fmaf(d, d, t[0]);
            }
        }
        me.sum(t, slots[turn]);
        turn ^= 1;
        const float rstd = 1.0f / sqrtf(t[0] * inv + a.eps);
        if (l == 0) {
            if (a.mean) a.mean[m] = mean;
            if (a.rstd) a.rstd[m] = rstd;
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (l + k * lanes) * 8;
            if (c >= a.C) continue;
            if (a.sum) store<RES16>(a.sum, m * a.C + c, a.C - c, s[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[k][j] = __builtin_fmaf((s[k][j] - mean) * rstd, w[k][j], b[k][j]);
            store<BF16>(a.y, m * a.C + c, a.C - c, s[k]);
        }
    }
}

// ------------------------------------------------------------------ gradient
// Workgroup g leaves its sums of dw and db, those of its rows added in order, in part[g][2][C]
// (NULL: not wanted). joined: 16 values a lane, where a workgroup has several rows.
template <bool BF16, bool RES16, int L, int R, int MOST>
__global__ void __launch_bounds__(MOST) add_norm_bwd(AddNormBwdArgs a, int waves, float* part) {
    __shared__ float slots[2][2][16];
    extern __shared__ float joined[];
    const Row<L> me{waves};
    const int l = me.lane(), lanes = me.lanes(), rows = me.rows(), octets = (a.C + 7) / 8;
    const long long step = (long long)gridDim.x * rows;
    float w[R][8], dw[R][8], db[R][8];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (l + k * lanes) * 8;
        params(a.weight, c, a.C - c, 1.0f, w[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = db[k][j] = 0.0f;
    }
    const bool dropping = a.drop.least != 0;
    const unsigned long long seed = dropping ? a.drop.rng[0] : 0, offset = dropping ? a.drop.rng[1] : 0;
    const float inv = 1.0f / (float)a.C;
    Octet<RES16> sum[R], add[R];
    Octet<BF16> dy[R];
    float mean = 0.0f, rstd = 0.0f;
    // a row behind the last reads as zeros
    auto fetch = [&](long long m) {
        const bool in = m < a.M;
        if (in && !a.rms) mean = a.mean[m];
        rstd = in ? a.rstd[m] : 0.0f;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (l + k * lanes) * 8, n = in ? a.C - c : 0;
            sum[k].load(a.sum, m * a.C + c, n);
            dy[k].load(a.dy, m * a.C + c, n);
            if (a.dsum) add[k].load(a.dsum, m * a.C + c, n);
        }
    };
    // base: the workgroup's first row, the same in every lane: no wave leaves the barriers early
    long long base = (long long)blockIdx.x * rows;
    int turn = 0;
    if (base < a.M) fetch(base + me.row());
    for (; base < a.M; base += step) {
        const long long m = base + me.row();
        float xhat[R][8], d[R][8], t[2] = {0.0f, 0.0f};
        const float r = rstd;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int n = m < a.M ? a.C - (l + k * lanes) * 8 : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xhat[k][j] = j < n ? (sum[k][j] - mean) * r : 0.0f;
                const float g = dy[k][j];
                db[k][j] += g;
                dw[k][j] = __builtin_fmaf(g, xhat[k][j], dw[k][j]);
                d[k][j] = g * w[k][j];
                t[0] += d[k][j];
                t[1] = __builtin_fmaf(d[k][j], xhat[k][j], t[1]);
            }
        }
        Octet<RES16> more[R];
#pragma unroll
        for (int k = 0; k < R; ++k) more[k] = add[k];
        if (base + step < a.M) fetch(m + step);
        me.sum(t, slots[turn]);
        turn ^= 1;
        if (m >= a.M) continue;
        const float s0 = a.rms ? 0.0f : t[0] * inv, s1 = t[1] * inv;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (l + k * lanes) * 8;
            if (c >= a.C) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[k][j] = r * (d[k][j] - s0 - xhat[k][j] * s1);
                if (a.dsum) d[k][j] += more[k][j];
            }
            if (a.dresidual) store<RES16>(a.dresidual, m * a.C + c, a.C - c, d[k]);
            if (!a.dx) continue;
            if (dropping) drop(d[k], a.drop, seed, offset + (unsigned long long)m * octets + l + k * lanes);
            store<BF16>(a.dx, m * a.C + c, a.C - c, d[k]);
        }
    }
    if (!part) return;
    float* p = part + (size_t)blockIdx.x * 2 * a.C;
    if (rows > 1) {  // R = 1 there
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            joined[(me.row() * 16 + j) * lanes + l] = dw[0][j];
            joined[(me.row() * 16 + 8 + j) * lanes + l] = db[0][j];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * lanes; i += blockDim.x) {
            float v = 0.0f;
            for (int q = 0; q < rows; ++q) v += joined[q * 16 * lanes + i];
            const int j = i / lanes, c = (i - j * lanes) * 8 + j % 8;
            if (c < a.C) p[(j < 8 ? 0 : a.C) + c] = v;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (l + k * lanes) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < a.C) {
                p[c + j] = dw[k][j];
                p[a.C + c + j] = db[k][j];
            }
    }
}

// dw and db from n parts: 16 columns a workgroup, 16 lanes on each, in a fixed order.
__global__ void __launch_bounds__(256) add_norm_sum(const float* __restrict__ part, int n, int C, float* dweight,
                                                    float* dbias) {
    __shared__ float sums[16][17];
    const int cl = threadIdx.x & 15, q = threadIdx.x >> 4, c = blockIdx.x * 16 + cl;
    float s = 0.0f;
    if (c < 2 * C)
#pragma unroll 8
        for (int k = q; k < n; k += 16) s += part[(size_t)k * 2 * C + c];
    sums[q][cl] = s;
    __syncthreads();
    if (q != 0 || c >= 2 * C) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += sums[k][cl];
    if (c < C && dweight) dweight[c] = s;
    if (c >= C && dbias) dbias[c - C] = s;
}

// ------------------------------------------------------------------ dropout alone
// An octet a lane at a time; the octets of all rows one after the other.
template <bool BF16>
__global__ void __launch_bounds__(256) dropout_octets(DropoutArgs a, long long total, unsigned octets) {
    const bool dropping = a.drop.least != 0;
    const unsigned long long seed = dropping ? a.drop.rng[0] : 0, offset = dropping ? a.drop.rng[1] : 0;
    for (long long q = (long long)blockIdx.x * 256 + threadIdx.x; q < total; q += (long long)gridDim.x * 256) {
        const long long m = q / octets;
        const int c = (int)(q - m * octets) * 8, n = a.C - c;
        Octet<BF16> x;
        x.load(a.x, m * a.C + c, n);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x[j];
        if (dropping) drop(v, a.drop, seed, offset + (unsigned long long)q);
        store<BF16>(a.y, m * a.C + c, n, v);
    }
}

// ------------------------------------------------------------------ choices
constexpr int kCus = 256;
constexpr int kFwdWaves = 12;                  // of a CU
constexpr int kBwdWaves = 12, kBwdRounds = 2;  // of a CU; rows a lane at least
// Lanes of a row: 16, or whole waves, up to 16 of them; two octets each beyond 1024 octets.
int row_lanes(int C) {
    const int octets = (C + 7) / 8, each = octets > 1024 ? 2 : 1;
    return octets <= 16 ? 16 : ((octets + each - 1) / each + 63) / 64 * 64;
}

// Workgroups of `rows` rows at once for M rows: at least `least` rounds each, and a whole number a
// CU (all of them resident together: one that has to wait for another's end walks its rows alone).
int groups(int M, int rows, int least, int a_cu) {
    const long long most = std::max<long long>(1, ((long long)M + (long long)least * rows - 1) / ((long long)least * rows));
    return (int)std::min<long long>(most, (long long)kCus * std::max(1, a_cu));
}

// Forward: one row of whole waves a workgroup, else 256 lanes.
int fwd_lanes(int C) { return row_lanes(C) < 128 ? 256 : row_lanes(C); }
int fwd_groups(int M, int C) {
    const int lanes = fwd_lanes(C);
    return groups(M, lanes / row_lanes(C), 1, (kFwdWaves * 64 + lanes / 2) / lanes);
}

// Gradient: as many rows a workgroup as kBwdLanes hold; a part of dw and db each.
int bwd_rows(int C) { return std::max(1, kBwdLanes / row_lanes(C)); }
int parts(int M, int C) {
    const int rows = bwd_rows(C);
    const int lanes = rows * row_lanes(C);
    return groups(M, rows, kBwdRounds, (kBwdWaves * 64 + lanes / 2) / lanes);
}

template <bool BF16, bool RES16>
hipError_t fwd(const AddNormArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)fwd_groups(a.M, a.C)), block((unsigned)fwd_lanes(a.C));
    const int lanes = row_lanes(a.C);
    if (lanes == 16) launch((add_norm_fwd<BF16, RES16, 16, 1>), grid, block, 0, s, a);
    else if (lanes == 64) launch((add_norm_fwd<BF16, RES16, 64, 1>), grid, block, 0, s, a);
    else if (a.C <= 8192) launch((add_norm_fwd<BF16, RES16, 0, 1>), grid, block, 0, s, a);
    else launch((add_norm_fwd<BF16, RES16, 0, 2>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <bool BF16, bool RES16>
hipError_t bwd(const AddNormBwdArgs& a, float* part, int n, hipStream_t s) {
    const int lanes = row_lanes(a.C), rows = bwd_rows(a.C), waves = lanes / 64;
    const dim3 grid((unsigned)n), block((unsigned)(lanes * rows));
    const uint32_t lds = rows > 1 ? 16 * lanes * rows * 4 : 0;
    const bool two = a.C > 8192, large = lanes > kBwdLanes;
    if (lanes == 16) launch((add_norm_bwd<BF16, RES16, 16, 1, kBwdLanes>), grid, block, lds, s, a, waves, part);
    else if (lanes == 64) launch((add_norm_bwd<BF16, RES16, 64, 1, kBwdLanes>), grid, block, lds, s, a, waves, part);
    else if (!two && !large) launch((add_norm_bwd<BF16, RES16, 0, 1, kBwdLanes>), grid, block, lds, s, a, waves, part);
    else if (!two) launch((add_norm_bwd<BF16, RES16, 0, 1, 1024>), grid, block, lds, s, a, waves, part);
    else if (!large) launch((add_norm_bwd<BF16, RES16, 0, 2, kBwdLanes>), grid, block, lds, s, a, waves, part);
    else launch((add_norm_bwd<BF16, RES16, 0, 2, 1024>), grid, block, lds, s, a, waves, part);
    return hipGetLastError();
}

}  // namespace

size_t add_norm_bwd_workspace_bytes(int M, int C, bool, bool) { return M == 0 ? 0 : (size_t)parts(M, C) * 2 * C * 4; }

hipError_t launch_add_norm_fwd(const AddNormArgs& a, hipStream_t s) {
    if (a.M == 0) return hipSuccess;
    if (!a.bf16) return fwd<false, false>(a, s);
    return a.res_bf16 ? fwd<true, true>(a, s) : fwd<true, false>(a, s);
}

hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t s) {
    const bool affine = a.dweight || a.dbias;
    float* part = affine ? static_cast<float*>(a.ws) : nullptr;
    const int n = a.M == 0 ? 0 : parts(a.M, a.C);
    hipError_t e = hipSuccess;
    if (a.M > 0) {
        if (!a.bf16) e = bwd<false, false>(a, part, n, s);
        else e = a.res_bf16 ? bwd<true, true>(a, part, n, s) : bwd<true, false>(a, part, n, s);
    }
    if (e != hipSuccess || !affine) return e;
    launch(add_norm_sum, dim3((unsigned)((2 * a.C + 15) / 16)), dim3(256), 0, s, part, n, a.C, a.dweight, a.dbias);
    return hipGetLastError();
}

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s) {
    const unsigned octets = ((unsigned)a.C + 7) / 8;
    const long long total = (long long)a.M * octets;
    if (total == 0) return hipSuccess;
    const dim3 grid((unsigned)std::min<long long>((total + 255) / 256, kCus * 32));
    if (a.bf16) launch((dropout_octets<true>), grid, dim3(256), 0, s, a, total, octets);
    else launch((dropout_octets<false>), grid, dim3(256), 0, s, a, total, octets);
    return hipGetLastError();
}

}  // namespace ssm
