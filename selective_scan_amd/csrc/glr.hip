// Gated linear recurrence over whole sequences on gfx950, and its gradient:
//   h_t = a_t h_{t-1} + u_t,   y = h [silu(z)],   g_t = dy_t [silu(z_t)] + a_{t+1} g_{t+1}
//
// Bandwidth-bound: every element is read and written once, 8 bytes of bf16 forward (10 with the
// gate), 14 (18) in the gradient, beside some 50 (65) and 125 (160) vector instruction slots, a
// third to two thirds of the memory's time: a second pass over the data, or over its arithmetic,
// would show. A workgroup has a tile of 64 channels by 128 steps, 16 a wave; a and u stay in
// registers from the load to the end. A piece of the sequence maps the state entering it to
// h -> P h + H, and the maps of consecutive pieces compose: of a lane's steps in registers, of the
// waves through LDS, of the tiles of a sequence through memory, from workgroup to workgroup of
// the same launch. A tile leaves its map, then needs the maps of the tiles before it: those of its
// group of 32 tiles, fetched by the eight waves in parallel, and the state at the group's start,
// which the group before leaves (a chained scan with look-back). The order of all operations is
// fixed by the shape, the type and whether x, r, i and z hold whole pairs of bf16 (two channels a
// lane, or one), so the same call gives the same bits.
// Measured (with the launch that fills the words, and for the gradient the one that sums dA):
// B8 L32768 D512 bf16 233 us (1.07 GB that have to move, 4.6 TB/s; a copy of that size reaches 4.9
// to 5.1), B1 L4096 D1536 with gate 17.4 us (3 of them the fill), gradient of B4 L4096 D1536 with
// gate 119 us (453 MB, 3.8 TB/s: two workgroups a CU, whose loads, waits and stores take turns;
// counters show no byte moved twice), of B3 L<=2047 D1001 fp32 convex, padded, 31 to 36 us by the
// lengths. Waiting costs nothing that shows (a copy that does not wait takes as long); with one XCD
// of eight slower by 12 % the others end that much earlier. Half as many or twice as many steps,
// wider strips, workgroups that take tile after tile and maps looked at ahead of time were all
// slower, for the registers they take or the lanes that wait.
// Where strips share lines, neighbours run on different XCDs and each fetches the line: B4 L4096
// D1502 bf16 reads 2.0 times its bytes (gradient 169 us, whole lines at D1536 127), D1001 fp32 1.5
// (gradient 1.6). The gradient of the decay form with gate takes 114 registers with pairs; with
// single channels 128 and 6 of them in scratch (B4 L2048 D2048 fp32 144 us, 4.2 TB/s). A sequence
// shorter than a tile leaves waves without steps: B256 D1536 bf16 with gate takes 67 us at L = 1 and
// at L = 16 alike (its gradient 159), B64 L64 D2560 33 (81).
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
#include <initializer_list>

namespace ssm {
namespace {

constexpr int kWaves = 8, kSteps = 16, kTile = kWaves * kSteps;
constexpr int kPer = 4, kGroup = kWaves * kPer;  // maps a wave fetches; tiles of a group
constexpr int kThreads = kWaves * 64;
static_assert(kTile == kGlrStateSteps, "a tile starts where a state is kept");

// Accesses that leave no lines behind in the L2 (PAST 1: stores of pairs, 2: their loads as well).
// Stores gain where every 64 bytes of a row belong to one strip: gradients of B4 L4096 D1536 130 ->
// 127 us, B8 L16384 D96 91 -> 81..89, B8 L8192 D160 71 -> 63 (B4 L4096 D1504 133..138 either way); where
// strips share them, a piece at a time goes to memory: B4 L4096 D1000 110 -> 160, D1502 162 -> 256.
// Loads gain where the call's tensors outgrow the memory-side cache of 256 MiB and strips share no
// line of 128 bytes: B8 L32768 D512 309 -> 300, its gradient 617 -> 595. Within the cache they cost
// (B4 L4096 D1502 78 -> 101), and so do shared lines, fetched twice (B4 L16384 D480 88 -> 98, D1002
// 202 -> 263, its gradient 563 -> 675). (All bf16 decay with gate.) Single channels use neither:
// stores of fp32 gain 0 to 17 % on whole lines (B4 L16384 D1024 282 -> 267) and cost 16 % on shared
// ones (gradient of D1001 728 -> 842).
constexpr int kNonTemporal = 2;
constexpr int kPiece = 64, kLine = 128;  // bytes
constexpr long long kCached = 256LL << 20;

constexpr uint32_t kAbsent = 0xffffffffu;
constexpr int kPolls = 1 << 22;  // some seconds; a wait of this kernel's ends after microseconds

typedef unsigned long long u64;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// How the work is cut, and the workspace. chain = (batch, strip of 64 channels).
struct Cut {
    int tiles, strips, groups;
    unsigned chains;  // times tiles: at most 2^30
    uint32_t* taken;  // [chains], 128 bytes apart: tiles handed out (counts from kAbsent)
    u64* maps;        // [B][tiles][D]: H | P << 32 of a tile
    uint32_t* ends;   // [B][groups][D]: the state behind a group
    float* part;      // [B][tiles][D]: dA's parts (gradient)
};

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

// How the lanes of a wave share its 16 steps of 64 channels: a lane has V neighbouring channels
// (2 where rows hold whole pairs of bf16: one 32-bit access for both) and 16 / V steps, the lanes
// of the wave's first half the earlier ones.
template <int V>
struct Share {
    static constexpr int T = kSteps / V;
    int late, d;  // whether the lane has the later steps; its first channel
    __device__ __forceinline__ Share(int strip) {
        const int lane = threadIdx.x & 63;
        late = V == 1 ? 0 : lane >> 5;
        d = strip * 64 + (V == 1 ? lane : 2 * (lane & 31));
    }
    // whether the lane has the first, or the last, of the wave's steps of its channels
    __device__ __forceinline__ bool first() const { return V == 1 || !late; }
    __device__ __forceinline__ bool last() const { return V == 1 || late; }
    // The value of the lane with the other steps of the same channels.
    __device__ __forceinline__ static float other(float v) { return __shfl_xor(v, 32); }
};

// A lane's elements of an io tensor's row as they are stored.
template <bool BF16, int V>
struct Raw {
    uint32_t w;
    __device__ __forceinline__ float operator[](int v) const {
        if constexpr (!BF16) return __uint_as_float(w);
        else return V == 2 && v == 1 ? bf16_hi(w) : bf16_lo(w);
    }
    // Forgets what was computed from the value: the compiler computes it again.
    __device__ __forceinline__ void anew() { asm volatile("" : "+v"(w)); }
};

// A wave's rows of an io tensor through a buffer that ends behind the last of n rows: rows
// further on read as 0 and are not written, and so does a lane whose channels do not exist (its
// offset lies behind every buffer). One scalar addition a row.
template <bool BF16, int V, int PAST>
struct Rows {
    static constexpr int T = Share<V>::T;
    __amdgpu_buffer_rsrc_t buf;
    uint32_t off, pitch;
    __device__ __forceinline__ Rows(const void* p, int stride, int D, size_t first, int n, const Share<V>& me) {
        constexpr uint32_t es = BF16 ? 2 : 4;
        pitch = (uint32_t)stride * es;
        // the same in every lane, said so that the buffer stays in scalar registers
        const u64 at = (u64)p + (u64)first * pitch;
        const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at), hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
        const uint32_t bytes = __builtin_amdgcn_readfirstlane(n > 0 ? (n - 1) * pitch + D * es : 0);
        buf = make_rsrc(reinterpret_cast<const void*>((u64)hi << 32 | lo), bytes);
        off = me.d < D ? (uint32_t)me.d * es + (me.late ? T * pitch : 0) : 0x80000000u;
    }
    __device__ __forceinline__ void load(Raw<BF16, V> (&v)[T]) const {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            if constexpr (BF16 && V == 1) v[t].w = __builtin_amdgcn_raw_buffer_load_b16(buf, (int)off, (int)(t * pitch), 0);
            else v[t].w = __builtin_amdgcn_raw_buffer_load_b32(buf, (int)off, (int)(t * pitch), PAST > 1 ? kNonTemporal : 0);
        }
    }
    __device__ __forceinline__ void store(int t, const float (&v)[V]) const {
        if constexpr (V == 2) {
            const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2));
            __builtin_amdgcn_raw_buffer_store_b32(w, buf, (int)off, (int)(t * pitch), PAST > 0 ? kNonTemporal : 0);
        } else {
            store_io<BF16>(buf, off, t * pitch, v[0]);
        }
    }
};

// Where a wave's steps are: the first one's row, and how many steps of the lane are in the
// sequence (live) and how many rows of the wave in the sequence and in the tensor.
template <int V>
struct Steps {
    size_t first;
    int wave_live, wave_stored, live;
    __device__ __forceinline__ Steps(const GlrIn& in, int b, int t0, const Share<V>& me) {
        const int n = __builtin_amdgcn_readfirstlane(glr_length(in.seqlens, b, in.L));
        first = (size_t)b * in.L + t0;
        wave_live = min(max(n - t0, 0), kSteps);
        wave_stored = min(max(in.L - t0, 0), kSteps);
        live = wave_live - me.late * Share<V>::T;
    }
};

// Values that exist from here on: left alone, the compiler puts off the gates' arithmetic to where
// its results are needed and spills what it is made of.
template <int V>
__device__ __forceinline__ void computed(float (&v)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) asm volatile("" : "+v"(v[k]));
}

// The state (or gradient) entering a tile: what enters its group, through the maps of the
// tiles between, n of them.
__device__ __forceinline__ float entering(const float (&start)[64], const float2 (&before)[kWaves][64], int n, int ch) {
    float h = start[ch];
    for (int q = 0; q * kPer < n; ++q) h = __builtin_fmaf(before[q][ch].x, h, before[q][ch].y);
    return h;
}

// ------------------------------------------------------------------ forward
template <bool BF16, int V, int PAST, int FORM, bool GATE>
__global__ void __launch_bounds__(kThreads, 4) glr_fwd_tiles(GlrArgs a, Cut c) {
    constexpr int T = Share<V>::T;
    __shared__ float2 own[kWaves][64], before[kWaves][64];
    __shared__ float start[64];
    __shared__ int shared;
    const GlrIn& in = a.in;
    unsigned chain;
    int tile;
    if (!take(c, &shared, &chain, &tile)) return;
    const int b = chain / c.strips, strip = chain % c.strips, lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Share<V> me(strip);
    const Steps<V> at(in, b, tile * kTile + w * kSteps, me);
    const int ch = me.d - strip * 64;
    const bool mine = me.d < in.D;
    float ca[T][V], cu[T][V], P[V], H[V];
    Raw<BF16, V> z[T];
    {
        Raw<BF16, V> x[T], r[T], i[T];
        Rows<BF16, V, PAST>(in.x, in.ldx, in.D, at.first, at.wave_live, me).load(x);
        Rows<BF16, V, PAST>(in.r, in.ldr, in.D, at.first, at.wave_live, me).load(r);
        if constexpr (FORM == 0) Rows<BF16, V, PAST>(in.i, in.ldi, in.D, at.first, at.wave_live, me).load(i);
        float A[V];
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = FORM == 0 ? in.A[min(me.d + v, in.D - 1)] : 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                glr_coefficients<FORM>(x[t][v], r[t][v], FORM == 0 ? i[t][v] : 0.0f, A[v] * kLog2e, A[v], &ca[t][v],
                                       &cu[t][v]);
            computed(ca[t]);
            computed(cu[t]);
        }
    }
    if (at.wave_live < kSteps)  // padding has u = 0 (x = 0); its state stays
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) ca[t][v] = t >= at.live ? 1.0f : ca[t][v];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        P[v] = ca[0][v];
        H[v] = cu[0][v];
#pragma unroll
        for (int t = 1; t < T; ++t) {
            P[v] *= ca[t][v];
            H[v] = __builtin_fmaf(ca[t][v], H[v], cu[t][v]);
        }
    }
    float Po[V], Ho[V];  // of the lane with the other steps
    if constexpr (V == 1) {
        own[w][lane] = make_float2(P[0], H[0]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Po[v] = me.other(P[v]);
            Ho[v] = me.other(H[v]);
            if (me.first()) own[w][ch + v] = make_float2(P[v] * Po[v], __builtin_fmaf(Po[v], H[v], Ho[v]));
        }
    }
    if constexpr (GATE) Rows<BF16, V, PAST>(in.z, in.ldz, in.D, at.first, at.wave_live, me).load(z);
    __syncthreads();

    const int group = tile / kGroup, first = group * kGroup;
    const int dl = strip * 64 + lane, dc = min(dl, in.D - 1);  // a lane a channel
    if (c.tiles > 1) {
        const size_t slot = (size_t)b * c.tiles * in.D + dc;
        if (w == kWaves - 1 && tile + 1 < c.tiles && dl < in.D) {
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

    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = entering(start, before, tile - first, ch + v);
        if (w == 0 && a.states && mine && me.first() && at.wave_stored > 0)
            a.states[((size_t)b * c.tiles + tile) * in.D + me.d + v] = h[v];
        for (int q = 0; q < w; ++q) h[v] = __builtin_fmaf(own[q][ch + v].x, h[v], own[q][ch + v].y);
        if constexpr (V == 2) h[v] = me.late ? __builtin_fmaf(Po[v], h[v], Ho[v]) : h[v];
        if (w == kWaves - 1 && tile + 1 < c.tiles && tile + 1 == first + kGroup && mine && me.last())
            __hip_atomic_store(c.ends + ((size_t)b * c.groups + group) * in.D + me.d + v,
                               present(__builtin_fmaf(P[v], h[v], H[v])), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    const Rows<BF16, V, PAST> out(a.y, in.D, in.D, at.first, at.wave_stored, me);
    auto sweep = [&](auto whole) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = __builtin_fmaf(ca[t][v], h[v], cu[t][v]);
                y[v] = GATE ? h[v] * silu(z[t][v]) : h[v];
                if (!decltype(whole)::value) y[v] = t < at.live ? y[v] : 0.0f;
            }
            out.store(t, y);
        }
    };
    if (at.wave_live == kSteps) sweep(std::true_type{});
    else sweep(std::false_type{});
    if (a.h_final && tile + 1 == c.tiles && w == kWaves - 1 && mine && me.last())
#pragma unroll
        for (int v = 0; v < V; ++v) a.h_final[(size_t)b * in.D + me.d + v] = h[v];
}

// ------------------------------------------------------------------ gradient
// Tiles are taken from the last to the first. The map of a piece on the gradient leaving it at
// its end to that at its start is g -> P g + C. The gates are computed twice: what a step needs
// of them across the wait, held in registers, would cost the second workgroup of a CU.
template <bool BF16, int V, int PAST, int FORM, bool GATE>
__global__ void __launch_bounds__(kThreads, 4) glr_bwd_tiles(GlrBwdArgs a, Cut c) {
    constexpr int T = Share<V>::T;
    __shared__ float ownP[kWaves][64], ownH[kWaves][64], ownC[kWaves][64];
    __shared__ float2 after[kWaves][64];
    __shared__ float start[64];
    __shared__ int shared;
    const GlrIn& in = a.in;
    unsigned chain;
    int k;
    if (!take(c, &shared, &chain, &k)) return;
    const int tile = c.tiles - 1 - k;
    const int b = chain / c.strips, strip = chain % c.strips, lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Share<V> me(strip);
    const Steps<V> at(in, b, tile * kTile + w * kSteps, me);
    const int ch = me.d - strip * 64;
    const bool mine = me.d < in.D;
    Raw<BF16, V> x[T], r[T], i[T], dy[T], z[T];
    float ca[T][V], cu[T][V], A[V], P[V], H[V], C[V];
    Rows<BF16, V, PAST>(in.x, in.ldx, in.D, at.first, at.wave_live, me).load(x);
    Rows<BF16, V, PAST>(in.r, in.ldr, in.D, at.first, at.wave_live, me).load(r);
    if constexpr (FORM == 0) Rows<BF16, V, PAST>(in.i, in.ldi, in.D, at.first, at.wave_live, me).load(i);
    Rows<BF16, V, PAST>(a.dy, in.D, in.D, at.first, at.wave_live, me).load(dy);
    if constexpr (GATE) Rows<BF16, V, PAST>(in.z, in.ldz, in.D, at.first, at.wave_live, me).load(z);
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = FORM == 0 ? in.A[min(me.d + v, in.D - 1)] : 0.0f;
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            glr_coefficients<FORM>(x[t][v], r[t][v], FORM == 0 ? i[t][v] : 0.0f, A[v] * kLog2e, A[v], &ca[t][v],
                                   &cu[t][v]);
        computed(ca[t]);
        computed(cu[t]);
    }
    if (at.wave_live < kSteps)  // padding has u = 0 and dy = 0; state and gradient stay
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) ca[t][v] = t >= at.live ? 1.0f : ca[t][v];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        P[v] = ca[0][v];
        H[v] = cu[0][v];
#pragma unroll
        for (int t = 1; t < T; ++t) {
            P[v] *= ca[t][v];
            H[v] = __builtin_fmaf(ca[t][v], H[v], cu[t][v]);
        }
        C[v] = 0.0f;
#pragma unroll
        for (int t = T - 1; t >= 0; --t) C[v] = ca[t][v] * (C[v] + (GATE ? dy[t][v] * silu(z[t][v]) : dy[t][v]));
    }
    computed(C);
    float Po[V], Ho[V], Co[V];  // of the lane with the other steps
    if constexpr (V == 1) {
        ownP[w][lane] = P[0];
        ownH[w][lane] = H[0];
        ownC[w][lane] = C[0];
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Po[v] = me.other(P[v]);
            Ho[v] = me.other(H[v]);
            Co[v] = me.other(C[v]);
            if (me.first()) {
                ownP[w][ch + v] = P[v] * Po[v];
                ownH[w][ch + v] = __builtin_fmaf(Po[v], H[v], Ho[v]);
                ownC[w][ch + v] = __builtin_fmaf(P[v], Co[v], C[v]);
            }
        }
    }
    __syncthreads();

    const int group = k / kGroup, first = group * kGroup;
    const int dl = strip * 64 + lane, dc = min(dl, in.D - 1);  // a lane a channel
    if (c.tiles > 1) {
        const size_t slot = (size_t)b * c.tiles * in.D + dc;
        if (w == 0 && k + 1 < c.tiles && dl < in.D) {
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
    // cu becomes the state before each step; dz needs the state alone
    float h[V], e[T][V];  // e: dy [silu(z)]
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = at.wave_live > 0 ? a.states[((size_t)b * c.tiles + tile) * in.D + min(me.d + v, in.D - 1)] : 0.0f;
        for (int q = 0; q < w; ++q) h[v] = __builtin_fmaf(ownP[q][ch + v], h[v], ownH[q][ch + v]);
        if constexpr (V == 2) h[v] = me.late ? __builtin_fmaf(Po[v], h[v], Ho[v]) : h[v];
    }
    const Rows<BF16, V, PAST> oz(GATE ? a.dz : a.dx, in.D, in.D, at.first, at.wave_stored, me);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        float dz[V];
        dy[t].anew();
        if constexpr (GATE) z[t].anew();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float n = __builtin_fmaf(ca[t][v], h[v], cu[t][v]);
            cu[t][v] = h[v];
            h[v] = n;
            if constexpr (GATE) {
                const Sigmoid s(z[t][v]);
                const float es = dy[t][v] * s.s;
                e[t][v] = z[t][v] * es;
                dz[v] = at.wave_live == kSteps || t < at.live ? __builtin_fmaf(e[t][v], s.om, es) * h[v] : 0.0f;
            }
        }
        if constexpr (GATE) {
            computed(e[t]);
            oz.store(t, dz);
        }
    }
    __syncthreads();

    float g[V], dA[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        dA[v] = 0.0f;
        g[v] = entering(start, after, k - first, ch + v);
        for (int q = kWaves - 1; q > w; --q) g[v] = __builtin_fmaf(ownP[q][ch + v], g[v], ownC[q][ch + v]);
        if constexpr (V == 2) g[v] = me.late ? g[v] : __builtin_fmaf(Po[v], g[v], Co[v]);
        if (w == 0 && k + 1 < c.tiles && k + 1 == first + kGroup && mine && me.first())
            __hip_atomic_store(c.ends + ((size_t)b * c.groups + group) * in.D + me.d + v,
                               present(__builtin_fmaf(P[v], g[v], C[v])), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    const Rows<BF16, V, PAST> ox(a.dx, in.D, in.D, at.first, at.wave_stored, me), orr(a.dr, in.D, in.D, at.first, at.wave_stored, me);
    const Rows<BF16, V, PAST> oi(FORM == 0 ? a.di : a.dx, in.D, in.D, at.first, at.wave_stored, me);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        x[t].anew();
        r[t].anew();
        if constexpr (FORM == 0) i[t].anew();
    }
    auto sweep = [&](auto whole) {
#pragma unroll
        for (int t = T - 1; t >= 0; --t) {
            float dx[V], dr[V], di[V], dl;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Sigmoid sr(r[t][v]);
                g[v] += GATE ? e[t][v] : dy[t][v];
                glr_gradient<FORM>(g[v], cu[t][v], ca[t][v], x[t][v], sr, FORM == 0 ? Sigmoid(i[t][v]) : sr, A[v],
                                   &dx[v], &dr[v], &di[v], &dl);
                g[v] *= ca[t][v];
                if (!decltype(whole)::value && t >= at.live) dx[v] = dr[v] = di[v] = dl = 0.0f;
                dA[v] += dl;
            }
            ox.store(t, dx);
            orr.store(t, dr);
            if constexpr (FORM == 0) oi.store(t, di);
        }
    };
    if (at.wave_live == kSteps) sweep(std::true_type{});
    else sweep(std::false_type{});
    if (a.dh0 && tile == 0 && w == 0 && mine && me.first())
#pragma unroll
        for (int v = 0; v < V; ++v) a.dh0[(size_t)b * in.D + me.d + v] = g[v];
    if constexpr (FORM == 0) {  // ownH was last read before the last barrier
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (V == 2) dA[v] += me.other(dA[v]);
            if (me.first()) ownH[w][ch + v] = dA[v];
        }
        __syncthreads();
        if (w == 0 && dl < in.D) {
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) sum += ownH[q][lane];
            c.part[((size_t)b * c.tiles + tile) * in.D + dl] = sum;
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

// Bytes of n tensors' elements.
long long bytes(const GlrIn& in, int n) { return (long long)in.B * in.L * in.D * (in.bf16 ? 2 : 4) * n; }

// Whether every row of the tensor starts on a pair of bf16 and holds whole pairs.
bool pairs(const GlrIn& in) {
    const void* p[] = {in.x, in.r, in.i, in.z};
    const int stride[] = {in.ldx, in.ldr, in.ldi, in.ldz};
    if (!in.bf16 || in.D % 2 != 0) return false;
    for (int k = 0; k < 4; ++k)
        if (p[k] && (reinterpret_cast<uintptr_t>(p[k]) % 4 != 0 || stride[k] % 2 != 0)) return false;
    return true;
}

// PAST of a call with pairs: tensors, as many as bytes() is to count, and where its outputs start.
int past(const GlrIn& in, int tensors, std::initializer_list<const void*> outputs) {
    const auto starts = [](const void* p, int at) { return reinterpret_cast<uintptr_t>(p) % at == 0; };
    if (in.D * 2 % kPiece != 0) return 0;
    for (const void* p : outputs)
        if (!starts(p, kPiece)) return 0;
    if (bytes(in, tensors) <= kCached || in.D * 2 % kLine != 0) return 1;
    const void* p[] = {in.x, in.r, in.i, in.z};
    const int stride[] = {in.ldx, in.ldr, in.ldi, in.ldz};
    for (int k = 0; k < 4; ++k)
        if (p[k] && (!starts(p[k], kLine) || stride[k] % (kLine / 2) != 0)) return 1;
    return 2;
}

template <bool BF16, int V, int PAST>
void fwd(const GlrArgs& a, const Cut& c, hipStream_t s) {
    const dim3 grid = fold((long long)c.chains * c.tiles), block(kThreads);
    if (a.in.form == 0) {
        if (a.in.z) launch((glr_fwd_tiles<BF16, V, PAST, 0, true>), grid, block, 0, s, a, c);
        else launch((glr_fwd_tiles<BF16, V, PAST, 0, false>), grid, block, 0, s, a, c);
    } else {
        if (a.in.z) launch((glr_fwd_tiles<BF16, V, PAST, 1, true>), grid, block, 0, s, a, c);
        else launch((glr_fwd_tiles<BF16, V, PAST, 1, false>), grid, block, 0, s, a, c);
    }
}

template <bool BF16, int V, int PAST>
void bwd(const GlrBwdArgs& a, const Cut& c, hipStream_t s) {
    const dim3 grid = fold((long long)c.chains * c.tiles), block(kThreads);
    if (a.in.form == 0) {
        if (a.in.z) launch((glr_bwd_tiles<BF16, V, PAST, 0, true>), grid, block, 0, s, a, c);
        else launch((glr_bwd_tiles<BF16, V, PAST, 0, false>), grid, block, 0, s, a, c);
    } else {
        if (a.in.z) launch((glr_bwd_tiles<BF16, V, PAST, 1, true>), grid, block, 0, s, a, c);
        else launch((glr_bwd_tiles<BF16, V, PAST, 1, false>), grid, block, 0, s, a, c);
    }
}

}  // namespace

size_t glr_workspace_bytes(int B, int L, int D) {
    size_t fill;
    cut_of(B, L, D, nullptr, &fill);
    return fill;
}

size_t glr_bwd_workspace_bytes(int B, int L, int D) {
    size_t fill;
    const size_t parts = (size_t)B * cut_of(B, L, D, nullptr, &fill).tiles;
    return parts == 1 ? 0 : fill + parts * D * 4;
}

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s) {
    size_t fill;
    const Cut c = cut_of(a.in.B, a.in.L, a.in.D, static_cast<char*>(a.ws), &fill);
    const hipError_t e = fill_words(a.ws, fill, s);
    if (e != hipSuccess) return e;
    const int far = past(a.in, 3 + (a.in.i != nullptr) + (a.in.z != nullptr), {a.y});
    if (!a.in.bf16) fwd<false, 1, 0>(a, c, s);
    else if (!pairs(a.in)) fwd<true, 1, 0>(a, c, s);
    else if (far == 0) fwd<true, 2, 0>(a, c, s);
    else if (far == 1) fwd<true, 2, 1>(a, c, s);
    else fwd<true, 2, 2>(a, c, s);
    return hipGetLastError();
}

hipError_t launch_glr_bwd(const GlrBwdArgs& a, hipStream_t s) {
    size_t fill;
    Cut c = cut_of(a.in.B, a.in.L, a.in.D, static_cast<char*>(a.ws), &fill);
    const long long parts = (long long)a.in.B * c.tiles;
    if (parts == 1) c.part = a.dA;  // the whole sum
    hipError_t e = fill_words(a.ws, fill, s);
    if (e != hipSuccess) return e;
    const int far = past(a.in, 5 + 2 * (a.in.i != nullptr) + 2 * (a.in.z != nullptr), {a.dx, a.dr, a.di, a.dz});
    if (!a.in.bf16) bwd<false, 1, 0>(a, c, s);
    else if (!pairs(a.in)) bwd<true, 1, 0>(a, c, s);
    else if (far == 0) bwd<true, 2, 0>(a, c, s);
    else if (far == 1) bwd<true, 2, 1>(a, c, s);
    else bwd<true, 2, 2>(a, c, s);
    if ((e = hipGetLastError()) != hipSuccess || a.in.form != 0 || parts == 1) return e;
    launch(glr_sum_parts, dim3((unsigned)((a.in.D + 15) / 16)), dim3(256), 0, s, c.part, parts, a.in.D, a.dA);
    return hipGetLastError();
}

}  // namespace ssm
