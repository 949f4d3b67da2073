// Gated linear recurrence over whole sequences on gfx950, and its gradient:
//   h_t = a_t h_{t-1} + u_t,   y = h [silu(z)],   g_t = dy_t [silu(z_t)] + a_{t+1} g_{t+1}
//
// Every element is read and written once; its gates cost 45 (forward) to 120 (gradient with
// gate) vector instruction slots, about what the memory takes for its bytes, so neither can be
// done twice. A workgroup has a tile of 64 channels (a lane each) by 128 steps (16 a wave); a
// and u stay in registers from the load to the end. A piece of the sequence maps the state
// entering it to h -> P h + H, and the maps of consecutive pieces compose: of a wave's steps in
// registers, of the waves through LDS, of the tiles of a sequence through memory, from workgroup
// to workgroup of the same launch. A tile leaves its map, then needs the maps of the tiles before
// it: those of its group of 32 tiles, fetched by the eight waves in parallel, and the state at the
// group's start, which the group before leaves. The order of all operations is fixed by the
// shape, so results repeat bit for bit.
//
// Waiting on other workgroups: a workgroup takes the next tile of its sequence from a counter, so
// that the tiles it waits for belong to workgroups that run already, and the first unfinished
// tile of a sequence waits for nothing: every wait ends, whatever else the GPU runs. A map or state
// is one 8- or 4-byte word stored and loaded whole (relaxed atomics at device scope), and says by
// itself that it is there: the words are filled with 1s by a launch of their own before, a NaN that
// no result is written as. No other data passes between workgroups, so no fence is needed. A wait
// gives up after some seconds all the same, and what depends on it becomes NaN.
#include "glr.h"
#include "launch.h"

#include <algorithm>

namespace ssm {
namespace {

constexpr int kWaves = 8, kSteps = 16, kTile = kWaves * kSteps;
constexpr int kPer = 4, kGroup = kWaves * kPer;  // maps a wave fetches; tiles of a group
constexpr int kThreads = kWaves * 64;
static_assert(kTile == kGlrStateSteps, "a tile starts where a state is kept");

constexpr uint32_t kAbsent = 0xffffffffu;
constexpr int kPolls = 1 << 22;

typedef unsigned long long u64;

// How the work is cut, and the workspace. chain = (batch, strip of 64 channels).
struct Cut {
    int tiles, strips, groups;
    unsigned chains;  // times tiles: at most 2^30
    uint32_t* taken;  // [chains], 128 bytes apart: tiles handed out (counts from kAbsent)
    u64* maps;        // [B][tiles][D]: H | P << 32 of a tile
    uint32_t* ends;   // [B][groups][D]: the state behind a group
    float* part;      // [B][tiles][D]: dA's parts (gradient)
};

template <bool BF16>
__device__ __forceinline__ float ld(const void* p, size_t i) {
    if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void st(void* p, size_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
    else static_cast<float*>(p)[i] = v;
}

// a value's bits, never kAbsent
__device__ __forceinline__ uint32_t present(float v) {
    const uint32_t b = __float_as_uint(v);
    return b == kAbsent ? 0x7fc00000u : b;
}

__device__ __forceinline__ u64 peek(const u64* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ float await_state(const uint32_t* p) {
    uint32_t v = kAbsent;
    for (int n = 0; n < kPolls; ++n) {
        v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (v != kAbsent) break;
        __builtin_amdgcn_s_sleep(1);
    }
    return __uint_as_float(v);
}

// The composition of maps[0], maps[stride], ... (n of them, at most kPer), in order.
__device__ __forceinline__ float2 await_maps(const u64* maps, size_t stride, int n) {
    u64 v[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) v[q] = q < n ? peek(maps + q * stride) : (u64)0x3f800000u << 32;
    float2 m = make_float2(1.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        for (int k = 0; k < kPolls && (uint32_t)(v[q] >> 32) == kAbsent; ++k) {
            __builtin_amdgcn_s_sleep(1);
            v[q] = peek(maps + q * stride);
        }
        const float P = __uint_as_float((uint32_t)(v[q] >> 32)), H = __uint_as_float((uint32_t)v[q]);
        m = make_float2(m.x * P, __builtin_fmaf(P, m.y, H));
    }
    return m;
}

__device__ __forceinline__ void leave(u64* p, float P, float H) {
    __hip_atomic_store(p, (u64)present(P) << 32 | __float_as_uint(H), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Workgroups beyond kFold of grid.x go on in grid.z: a grid's dimension holds 2^32 lanes.
constexpr long long kFold = 1 << 22;
__device__ __forceinline__ unsigned folded() { return blockIdx.z * gridDim.x + blockIdx.x; }
dim3 fold(long long n) {
    return dim3((unsigned)std::min(n, kFold), 1, (unsigned)((n + kFold - 1) / kFold));
}

// The tile (in the order they are taken) and chain of this workgroup; false if there is none.
__device__ __forceinline__ bool take(const Cut& c, int* shared, unsigned* chain, int* k) {
    const unsigned id = folded();
    if (id >= c.chains * c.tiles) return false;
    *chain = id % c.chains;
    *k = 0;
    if (c.tiles > 1) {
        if (threadIdx.x == 0) *shared = (int)(atomicAdd(c.taken + (size_t)*chain * 32, 1u) + 1u);
        __syncthreads();
        *k = __builtin_amdgcn_readfirstlane(*shared);
    }
    return true;
}

// The rows of a wave's steps: where they start, how many are in the sequence and in the tensor.
struct Rows {
    size_t first;
    int live, stored;
    __device__ __forceinline__ Rows(const GlrIn& in, int b, int t0) {
        first = (size_t)b * in.L + t0;
        live = min(max(glr_length(in.seqlens, b, in.L) - t0, 0), kSteps);
        stored = min(max(in.L - t0, 0), kSteps);
    }
};

template <bool BF16>
__device__ __forceinline__ void load_rows(const void* p, int stride, const Rows& rows, int d, float (&v)[kSteps]) {
#pragma unroll
    for (int t = 0; t < kSteps; ++t) v[t] = ld<BF16>(p, (rows.first + min(t, rows.live - 1)) * stride + d);
}

// ------------------------------------------------------------------ forward
template <bool BF16, int FORM, bool GATE>
__global__ void __launch_bounds__(kThreads) glr_fwd_tiles(GlrArgs a, Cut c) {
    __shared__ float2 own[kWaves][64], before[kWaves][64];
    __shared__ float start[64];
    __shared__ int shared;
    const GlrIn& in = a.in;
    unsigned chain;
    int tile;
    if (!take(c, &shared, &chain, &tile)) return;
    const int b = (int)(chain / c.strips), lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int d = (int)(chain % c.strips) * 64 + lane, dc = min(d, in.D - 1);
    const bool mine = d < in.D;
    const Rows rows(in, b, tile * kTile + w * kSteps);
    float ca[kSteps], cu[kSteps], z[kSteps];
    float P = 1.0f, H = 0.0f;
    if (rows.live > 0) {
        float r[kSteps], i[kSteps];
        load_rows<BF16>(in.x, in.ldx, rows, dc, cu);
        load_rows<BF16>(in.r, in.ldr, rows, dc, r);
        if constexpr (FORM == 0) load_rows<BF16>(in.i, in.ldi, rows, dc, i);
        if constexpr (GATE) load_rows<BF16>(in.z, in.ldz, rows, dc, z);
        const float A = FORM == 0 ? in.A[dc] : 0.0f, A2 = A * kLog2e, At = 2.0f * A;
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            glr_coefficients<FORM>(cu[t], r[t], FORM == 0 ? i[t] : 0.0f, A2, At, &ca[t], &cu[t]);
            if (t >= rows.live) {
                ca[t] = 1.0f;
                cu[t] = 0.0f;
            }
            P *= ca[t];
            H = __builtin_fmaf(ca[t], H, cu[t]);
        }
    } else {
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            ca[t] = 1.0f;
            cu[t] = z[t] = 0.0f;
        }
    }
    own[w][lane] = make_float2(P, H);
    __syncthreads();

    const int group = tile / kGroup, first = group * kGroup;
    if (c.tiles > 1) {
        const size_t slot = (size_t)b * c.tiles * in.D + dc;
        if (w == kWaves - 1 && tile + 1 < c.tiles && mine) {
            float p = 1.0f, h = 0.0f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) {
                const float2 m = own[q][lane];
                p *= m.x;
                h = __builtin_fmaf(m.x, h, m.y);
            }
            leave(c.maps + slot + (size_t)tile * in.D, p, h);
        }
        const int from = first + w * kPer;
        if (from < tile) before[w][lane] = await_maps(c.maps + slot + (size_t)from * in.D, in.D, min(tile - from, kPer));
    }
    if (w == kWaves - 2)
        start[lane] = group == 0 ? (a.h0 ? a.h0[(size_t)b * in.D + dc] : 0.0f)
                                 : await_state(c.ends + ((size_t)b * c.groups + group - 1) * in.D + dc);
    __syncthreads();

    float h = start[lane];
    for (int q = 0; q * kPer < tile - first; ++q) h = __builtin_fmaf(before[q][lane].x, h, before[q][lane].y);
    if (w == 0 && a.states && mine && rows.stored > 0)
        a.states[((size_t)b * c.tiles + tile) * in.D + d] = h;
    for (int q = 0; q < w; ++q) h = __builtin_fmaf(own[q][lane].x, h, own[q][lane].y);
    if (w == kWaves - 1 && tile + 1 < c.tiles && tile + 1 == first + kGroup && mine)
        __hip_atomic_store(c.ends + ((size_t)b * c.groups + group) * in.D + d, present(__builtin_fmaf(P, h, H)),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
        h = __builtin_fmaf(ca[t], h, cu[t]);
        if (t < rows.stored && mine)
            st<BF16>(a.y, (rows.first + t) * in.D + d, t >= rows.live ? 0.0f : GATE ? h * silu(z[t]) : h);
    }
    if (a.h_final && tile + 1 == c.tiles && w == kWaves - 1 && mine) a.h_final[(size_t)b * in.D + d] = h;
}

// ------------------------------------------------------------------ gradient
// Tiles are taken from the last to the first. own: P, H (forward) and C (what the wave's own dy
// leaves for the step before it).
template <bool BF16, int FORM, bool GATE>
__global__ void __launch_bounds__(kThreads) glr_bwd_tiles(GlrBwdArgs a, Cut c) {
    __shared__ float ownP[kWaves][64], ownH[kWaves][64], ownC[kWaves][64];
    __shared__ float2 after[kWaves][64];
    __shared__ float start[64];
    __shared__ int shared;
    const GlrIn& in = a.in;
    unsigned chain;
    int k;
    if (!take(c, &shared, &chain, &k)) return;
    const int tile = c.tiles - 1 - k;
    const int b = (int)(chain / c.strips), lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int d = (int)(chain % c.strips) * 64 + lane, dc = min(d, in.D - 1);
    const bool mine = d < in.D;
    const Rows rows(in, b, tile * kTile + w * kSteps);
    float x[kSteps], r[kSteps], i[kSteps], z[kSteps], e[kSteps], ca[kSteps], cu[kSteps];
    const float A = FORM == 0 ? in.A[dc] : 0.0f, A2 = A * kLog2e, At = 2.0f * A;
    float P = 1.0f, H = 0.0f, C = 0.0f;
    if (rows.live > 0) {
        load_rows<BF16>(in.x, in.ldx, rows, dc, x);
        load_rows<BF16>(in.r, in.ldr, rows, dc, r);
        if constexpr (FORM == 0) load_rows<BF16>(in.i, in.ldi, rows, dc, i);
        load_rows<BF16>(a.dy, in.D, rows, dc, e);
        if constexpr (GATE) load_rows<BF16>(in.z, in.ldz, rows, dc, z);
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            glr_coefficients<FORM>(x[t], r[t], FORM == 0 ? i[t] : 0.0f, A2, At, &ca[t], &cu[t]);
            if (t >= rows.live) {
                ca[t] = 1.0f;
                cu[t] = e[t] = 0.0f;
                if constexpr (GATE) z[t] = 0.0f;
            }
            P *= ca[t];
            H = __builtin_fmaf(ca[t], H, cu[t]);
        }
#pragma unroll
        for (int t = kSteps - 1; t >= 0; --t) C = ca[t] * (C + (GATE ? e[t] * silu(z[t]) : e[t]));
    }
    ownP[w][lane] = P;
    ownH[w][lane] = H;
    ownC[w][lane] = C;
    __syncthreads();

    const int group = k / kGroup, first = group * kGroup;
    if (c.tiles > 1) {
        const size_t slot = (size_t)b * c.tiles * in.D + dc;
        if (w == 0 && k + 1 < c.tiles && mine) {
            float p = 1.0f, h = 0.0f;
#pragma unroll
            for (int q = kWaves - 1; q >= 0; --q) {
                p *= ownP[q][lane];
                h = __builtin_fmaf(ownP[q][lane], h, ownC[q][lane]);
            }
            leave(c.maps + slot + (size_t)k * in.D, p, h);
        }
        const int from = first + w * kPer;
        if (from < k) after[w][lane] = await_maps(c.maps + slot + (size_t)from * in.D, in.D, min(k - from, kPer));
    }
    if (w == kWaves - 2)
        start[lane] = group == 0 ? (a.dh_final ? a.dh_final[(size_t)b * in.D + dc] : 0.0f)
                                 : await_state(c.ends + ((size_t)b * c.groups + group - 1) * in.D + dc);
    float h = rows.live > 0 ? a.states[((size_t)b * c.tiles + tile) * in.D + dc] : 0.0f;
    for (int q = 0; q < w; ++q) h = __builtin_fmaf(ownP[q][lane], h, ownH[q][lane]);
    __syncthreads();

    float g = start[lane];
    for (int q = 0; q * kPer < k - first; ++q) g = __builtin_fmaf(after[q][lane].x, g, after[q][lane].y);
    for (int q = kWaves - 1; q > w; --q) g = __builtin_fmaf(ownP[q][lane], g, ownC[q][lane]);
    if (w == 0 && k + 1 < c.tiles && k + 1 == first + kGroup && mine)
        __hip_atomic_store(c.ends + ((size_t)b * c.groups + group) * in.D + d, present(__builtin_fmaf(P, g, C)),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    float dA = 0.0f;
    if (rows.live > 0) {
        // cu becomes the state before each step
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            const float n = __builtin_fmaf(ca[t], h, cu[t]);
            cu[t] = h;
            h = n;
        }
#pragma unroll
        for (int t = kSteps - 1; t >= 0; --t) {
            float dx, dr, di, dl, dz = 0.0f;
            float dy = e[t];
            if constexpr (GATE) {
                const Sigmoid s(z[t]);
                dz = dy * h * s.s * __builtin_fmaf(z[t], s.om, 1.0f);  // h: after the step
                dy *= z[t] * s.s;
            }
            g += dy;
            h = cu[t];
            glr_gradient<FORM>(g, h, x[t], r[t], FORM == 0 ? i[t] : 0.0f, A, A2, At, &dx, &dr, &di, &dl);
            g *= ca[t];
            if (t >= rows.live) dx = dr = di = dl = dz = 0.0f;
            dA += dl;
            if (t < rows.stored && mine) {
                const size_t o = (rows.first + t) * in.D + d;
                st<BF16>(a.dx, o, dx);
                st<BF16>(a.dr, o, dr);
                if constexpr (FORM == 0) st<BF16>(a.di, o, di);
                if constexpr (GATE) st<BF16>(a.dz, o, dz);
            }
        }
    } else {
        for (int t = 0; t < rows.stored; ++t) {
            if (!mine) continue;
            const size_t o = (rows.first + t) * in.D + d;
            st<BF16>(a.dx, o, 0.0f);
            st<BF16>(a.dr, o, 0.0f);
            if constexpr (FORM == 0) st<BF16>(a.di, o, 0.0f);
            if constexpr (GATE) st<BF16>(a.dz, o, 0.0f);
        }
    }
    if (a.dh0 && tile == 0 && w == 0 && mine) a.dh0[(size_t)b * in.D + d] = g;
    if constexpr (FORM == 0) {  // ownH was last read before the last barrier
        ownH[w][lane] = dA;
        __syncthreads();
        if (w == 0 && mine) {
            dA = 0.0f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) dA += ownH[q][lane];
            c.part[((size_t)b * c.tiles + tile) * in.D + d] = dA;
        }
    }
}

// dA from its n parts: 16 channels a workgroup, 16 lanes on each, in a fixed order.
__global__ void __launch_bounds__(256) glr_sum_parts(const float* __restrict__ part, long long n, int D, float* dA) {
    __shared__ float sums[16][17];
    const int cl = threadIdx.x & 15, q = threadIdx.x >> 4, d = blockIdx.x * 16 + cl;
    float s = 0.0f;
    if (d < D)
#pragma unroll 4
        for (long long k = q; k < n; k += 16) s += part[(size_t)k * D + d];
    sums[q][cl] = s;
    __syncthreads();
    if (q == 0 && d < D) {
#pragma unroll
        for (int k = 1; k < 16; ++k) s += sums[k][cl];
        dA[d] = s;
    }
}

__global__ void __launch_bounds__(256) glr_fill(uint4* p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
        p[i] = make_uint4(kAbsent, kAbsent, kAbsent, kAbsent);
}

// The cut of a shape; *fill: bytes of the words that have to be absent at the start.
Cut cut_of(int B, int L, int D, char* ws, size_t* fill) {
    Cut c{};
    c.tiles = std::max(1, (L + kTile - 1) / kTile);
    c.strips = (D + 63) / 64;
    c.groups = (c.tiles + kGroup - 1) / kGroup;
    c.chains = (unsigned)B * c.strips;
    size_t at = 0;
    if (c.tiles > 1) {
        c.maps = reinterpret_cast<u64*>(ws);
        at = (size_t)B * c.tiles * D * 8;
        at = (at + 127) / 128 * 128;
        c.taken = reinterpret_cast<uint32_t*>(ws + at);
        at += (size_t)c.chains * 128;
        c.ends = reinterpret_cast<uint32_t*>(ws + at);
        at += ((size_t)B * c.groups * D * 4 + 15) / 16 * 16;
    }
    c.part = reinterpret_cast<float*>(ws + at);
    *fill = at;
    return c;
}

hipError_t fill_words(void* ws, size_t bytes, hipStream_t s) {
    if (bytes == 0) return hipSuccess;
    const size_t n = bytes / 16;
    launch(glr_fill, dim3((unsigned)std::min<size_t>((n + 255) / 256, 2048)), dim3(256), 0, s,
           static_cast<uint4*>(ws), n);
    return hipGetLastError();
}

template <bool BF16, int FORM>
void fwd(const GlrArgs& a, const Cut& c, hipStream_t s) {
    const dim3 grid = fold((long long)c.chains * c.tiles);
    if (a.in.z) launch((glr_fwd_tiles<BF16, FORM, true>), grid, dim3(kThreads), 0, s, a, c);
    else launch((glr_fwd_tiles<BF16, FORM, false>), grid, dim3(kThreads), 0, s, a, c);
}

template <bool BF16, int FORM>
void bwd(const GlrBwdArgs& a, const Cut& c, hipStream_t s) {
    const dim3 grid = fold((long long)c.chains * c.tiles);
    if (a.in.z) launch((glr_bwd_tiles<BF16, FORM, true>), grid, dim3(kThreads), 0, s, a, c);
    else launch((glr_bwd_tiles<BF16, FORM, false>), grid, dim3(kThreads), 0, s, a, c);
}

}  // namespace

size_t glr_workspace_bytes(int B, int L, int D) {
    size_t fill;
    cut_of(B, L, D, nullptr, &fill);
    return fill;
}

size_t glr_bwd_workspace_bytes(int B, int L, int D) {
    size_t fill;
    const Cut c = cut_of(B, L, D, nullptr, &fill);
    return fill + (size_t)B * c.tiles * D * 4;
}

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s) {
    size_t fill;
    const Cut c = cut_of(a.in.B, a.in.L, a.in.D, static_cast<char*>(a.ws), &fill);
    const hipError_t e = fill_words(a.ws, fill, s);
    if (e != hipSuccess) return e;
    if (a.in.bf16) a.in.form == 0 ? fwd<true, 0>(a, c, s) : fwd<true, 1>(a, c, s);
    else a.in.form == 0 ? fwd<false, 0>(a, c, s) : fwd<false, 1>(a, c, s);
    return hipGetLastError();
}

hipError_t launch_glr_bwd(const GlrBwdArgs& a, hipStream_t s) {
    size_t fill;
    const Cut c = cut_of(a.in.B, a.in.L, a.in.D, static_cast<char*>(a.ws), &fill);
    hipError_t e = fill_words(a.ws, fill, s);
    if (e != hipSuccess) return e;
    if (a.in.bf16) a.in.form == 0 ? bwd<true, 0>(a, c, s) : bwd<true, 1>(a, c, s);
    else a.in.form == 0 ? bwd<false, 0>(a, c, s) : bwd<false, 1>(a, c, s);
    if ((e = hipGetLastError()) != hipSuccess || a.in.form != 0) return e;
    launch(glr_sum_parts, dim3((unsigned)((a.in.D + 15) / 16)), dim3(256), 0, s, c.part, (long long)a.in.B * c.tiles,
           a.in.D, a.dA);
    return hipGetLastError();
}

}  // namespace ssm
