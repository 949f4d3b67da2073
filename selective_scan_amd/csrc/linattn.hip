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
//
// By chunks of 64 steps (rows i, j of a chunk of n <= 64 steps; S the state entering it):
//   forwards   out_i = lam^(i+1) x1_i S + sum_{j <= i} lam^(i-j) (x1_i . x2_j) x3_j
//              S    <- lam^n S + sum_j lam^(n-1-j) x2_j (x) x3_j
//   backwards  out_i = lam^(n-1-i) x1_i S + sum_{j >= i} lam^(j-i) (x1_i . x2_j) x3_j
//              S    <- lam^n S + sum_j lam^(j+1) x2_j (x) x3_j
// Every power has an exponent >= 0, so none can overflow.
//
// Launches. A sequence is cut into super-chunks (runs of chunks), one workgroup per
// (batch, head, super-chunk); runs that need no other's result share a launch:
//   mix_chunks<AGG>   every super-chunk but the last in the run's direction: what it adds to
//                     the state, from a zero start (in pieces where that pays)
//   mix_carry         per state element, over the super-chunks: the state entering each
//   mix_chunks        the outputs, from that state (mix_chunks_shared: dq and dk of two or
//                     three heads that share a group, their sum in registers)
//   sum_heads         dq and dk of other shared groups, from fp32 planes per head
// With one super-chunk only the third runs. All are deterministic.
//
// One wave owns 32 columns of the state (all KD rows, fp32, in its accumulators) and
// the same columns of the output. The state never leaves the registers: an
// accumulator tile of v_mfma_f32_32x32x16_bf16 holds column c = lane % 32 and, per half
// wave hf, rows 8 (r / 4) + 4 hf + r % 4, while an operand wants eight consecutive
// contraction indices per lane. Feeding the operand that makes the tile's rows in the
// order pi(m) = m with bits 2 and 3 exchanged turns registers 0-7 and 8-15 into rows
// 8 hf .. 8 hf + 7 and 16 + 8 hf .. 16 + 8 hf + 7, exactly two operands. The same holds
// for the scores x2_j . x1_i (rows j) that multiply x3, and, with the columns of the
// state in the order pi, for the output tile, whose lanes then hold eight consecutive
// columns of one row: 16-byte stores.
// Operands stored in bf16 enter exactly; those formed in fp32 (state, decayed scores,
// weighted x3) enter as hi = bf16(x) and lo = bf16(x - hi), two products, about 17
// significant bits: one bf16 rounding would cost 1e-3 of the result, two are far below
// the rounding of a bf16 output. Where the state itself is an output (fp32), weighted x3
// enters it with a third part, 24 bits: the final state is then 3e-7 off and not 2e-6,
// for 2% of the time (8% at V = 64). With fp32 storage every product is
// v_mfma_f32_32x32x2_f32.
// The scores are computed once per workgroup (a 32 x 32 tile a wave) and passed on through
// LDS as finished operands; each wave computing all of them was 16 of 100 products and 130
// vector instructions a chunk more. Rows go straight into LDS (no registers between: these
// cost 50 to 80, spills at V = 64, 235 -> 173 us at B4 L8000 H24 K128 V64).
//
// What bounds it (bf16, K = V = 128). A chunk's 84 products of 32 cycles are 1.1 us at
// 2.4 GHz; with the splits, decays and waits a workgroup alone on its CU takes 3.3 us a
// chunk (6900 cycles: 1700 scores and x1 S, 400 passing, 900 barrier and loads' issue, 740
// scores times x3, 650 stores, 2000 state, 430 waiting for rows), one of two on a CU 5.2 us.
// B4 L4096 H16 (one super-chunk, dq, dk and dv side by side): 231 us, 470 MB that have to
// move (92 us at a copy's rate), 800 MB moved. Tried and not kept: both buffers for x1 and
// x3 as well at K = V = 128 (one workgroup a CU; 246 us either way), the state's first
// operands before the read-out (spills), more than 256 registers (AGPR copies: 275 us).
#include "common.h"
#include "launch.h"
#include "linattn.h"

#include <algorithm>

namespace ssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
// LDS-typed pointers keep the address arithmetic in 32 bits
typedef __attribute__((address_space(3))) char lds_t;
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr int kC = 64;  // steps per chunk
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
    const float* init;    // [B, H, KD, VD], transposed ([B, H, VD, KD]) if trans; or NULL
    float* slots;         // [B, H, NS - 1, P, KD, VD] (or transposed): aggregates, then, in each
                          // first piece, entering states
    int trans;
    void* out;            // io dtype, or fp32 if out_f32
    int out_f32;
    float* final_state;   // [B, H, KD, VD] or NULL
    int exact;            // the state to fp32's last bits: x3 weighted enters it in three parts
};

// Up to three runs that one launch does side by side.
struct Jobs {
    Mix m[3];
    int rev[3];  // backwards in time
    int n;
};

struct Geom {
    int NC;   // chunks per sequence
    int cps;  // chunks per super-chunk
    int NS;   // super-chunks per sequence
    int P;    // pieces that a super-chunk's aggregate is computed in
    int cpp;  // chunks per piece
};

// Whether the heads of a group share a workgroup in dq and dk, whose sum over the heads then
// never leaves the registers (they hold the states of three heads of V = 64): B4 L2047 H24 of 8
// K128 V64 takes 200 us with fp32 planes per head and their sum, 159 so.
bool shared_heads(int r, int V, bool bf16) { return bf16 && V == 64 && (r == 2 || r == 3); }

// How many workgroups of mix_chunks fit a CU, by their LDS and registers.
int per_cu(int KD, int VD, bool bf16) {
    const int es = bf16 ? 2 : 4, lds = kC * (3 * KD + VD) * es + 128 * 4 + 3 * 2 * 2048;
    return std::min(163840 / lds, VD == 128 ? 2 : 3);
}

// The number of super-chunks with the least estimated time. The unit is one chunk of a
// bf16 workgroup that has its CU to itself (3.3 us at K = V = 128). Workgroups that share a
// CU slow each other down: by 1.25 while every wave still has a SIMD of its own, by 1.6
// beyond that (measured at B4 L4096 H16 K = V = 128: 3.3 us a chunk alone, 5.2 as one of two;
// B4 L8000 H24 K128 V64: 3.7 and 4.7); fp32 takes three times as long. A workgroup begins and
// ends with its state (2 units). No launch is faster than its rows at 4 TB/s (13 MB a unit;
// rows shared by heads are read once). More than one super-chunk adds the aggregates (half
// a unit a chunk) and the carry; where these have few workgroups of many chunks, each
// aggregate is computed in pieces that the carry joins (B4 L8000 H24 K128 V64: 70 us whole,
// 49 in two). Measured optima are within 4% of what this picks: B1 L4096
// H16 K = V = 128 takes 197 us with one, 55 with 8, 50 with 16, 55 with 32.
Geom geom(int B, int L, int H, int G, int K, int V, bool bf16, bool bwd) {
    const long bh = (long)B * H;
    const int NC = std::max(1, (L + kC - 1) / kC), r = H / G;
    const double rows = (double)B * G * L * (bf16 ? 2 : 4) / 13e6;  // units per value of a group's row
    auto scan = [&](int jobs, int KD, int VD, double values, int NS, int cps) {
        const long wg = jobs * bh * NS, slots = 256L * per_cu(KD, VD, bf16);
        const double share = wg <= 256 ? 1.0 : VD == 64 || slots == 256 ? 1.25 : 1.6;
        const double t = (double)((wg + slots - 1) / slots) * share * (cps * (bf16 ? 1.0 : 3.0) + 2.0);
        return std::max(t, rows * values);
    };
    const int dqk = 2 * (2 * r * V + K + r * K), dv = 2 * K + 2 * r * V;
    Geom best{NC, NC, 1, 1, NC};
    double least = 0.0;
    for (int want = 1; want <= NC && (want == 1 || bh * want <= 1536); ++want) {
        const int cps = (NC + want - 1) / want, NS = (NC + cps - 1) / cps;
        if (NS != want) continue;
        double t;
        int P = 1;
        if (!bwd) t = scan(1, K, V, 2 * K + 2 * r * V, NS, cps);
        else if (shared_heads(r, V, bf16))  // one a CU, 0.8 units a head and chunk
            t = (double)((2 * bh / r * NS + 255) / 256) * (0.8 * r * cps + 2.0) + scan(1, K, V, dv, NS, cps);
        else if (K == V) t = scan(3, K, V, dqk + dv, NS, cps);
        else t = scan(2, V, K, dqk, NS, cps) + scan(1, K, V, dv, NS, cps);
        if (NS > 1) {
            const int dirs = bwd ? 2 : 1;
            const long wg = dirs * bh * (NS - 1);
            P = (int)std::max<long>(1, std::min<long>({768 / wg, cps / 8, 4}));
            t += std::max((double)((wg * P + 511) / 512) * (0.5 * cps / P * (bf16 ? 1.0 : 2.0) + 1.0),
                          dirs * rows * (K + r * V) * (NS - 1) / NS);
            t += 2.4 + 0.14e-6 * dirs * bh * NS * K * V * (1 + P);
        }
        if (want == 1 || t < least) {
            least = t;
            best = Geom{NC, cps, NS, P, (cps + P - 1) / P};
        }
    }
    return best;
}

__device__ __forceinline__ int seq_len(const int* seqlens, int b, int L) {
    return seqlens ? max(0, min(seqlens[b], L)) : L;
}

// log_decay, kept finite so that 0 steps of it are 0 (exp(-1e4) is 0 as well)
__device__ __forceinline__ float log_decay_of(const float* p, int h) {
    const float a = p[h];
    return a < -1e4f ? -1e4f : a;
}

__device__ __forceinline__ int pi(int m) { return (m & 0x13) | ((m & 4) << 1) | ((m & 8) >> 1); }

// A chunk's rows of D values in LDS: kC rows of D es bytes without padding, the 16-byte
// piece p of row r at position p ^ swz(r). Sixteen rows' pieces p, read together as operand
// rows, then cover all 64 banks, and so do the two adjacent pieces of four rows that each
// half wave's transpose read takes. (Loads straight into LDS put a wave's 1 KB down in lane
// order, so the order within a row is chosen by what each lane loads, and rows cannot be
// padded.)
template <int D, bool BF16>
struct Tile {
    static constexpr int RB = D * (BF16 ? 2 : 4);  // bytes per row: 128, 256 or 512
    static constexpr int P = RB / 16;              // pieces per row
    static constexpr int BYTES = kC * RB;
    static __device__ __forceinline__ int swz(int r) {
        if constexpr (P == 8) return ((r << 1) & 4) | ((r >> 2) & 3);  // two rows span the banks
        else return ((r & 3) << 2) | ((r >> 2) & 3);
    }
    static __device__ __forceinline__ int at(int r, int p) { return r * RB + ((p ^ swz(r)) << 4); }
};

// Operands of a 32 x 32 x 16 product: lane l holds row (or column) l % 32 and the eight
// contraction indices 8 (l / 32) + e.
template <bool BF16> struct Types;
template <> struct Types<true> {
    typedef bf16x8 Op;
    struct Formed { bf16x8 hi, lo; };
    static __device__ __forceinline__ f32x16 mma(Op a, Op b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // the two products of a formed operand, apart, so that products into other accumulators
    // can stand between them
    template <int PART> static __device__ __forceinline__ f32x16 part(const Formed& a, Op b, f32x16 c) {
        return mma(PART ? a.lo : a.hi, b, c);
    }
    template <int PART> static __device__ __forceinline__ f32x16 part(Op a, const Formed& b, f32x16 c) {
        return mma(a, PART ? b.lo : b.hi, c);
    }
    static constexpr int PARTS = 2;
    static __device__ __forceinline__ Formed form(f32x8 v) {
        u32x4 hi, lo;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const f32x2 x = {v[2 * p], v[2 * p + 1]};
            const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
            const f32x2 d = {x[0] - bf16_lo(h), x[1] - bf16_hi(h)};
            hi[p] = h;
            lo[p] = __builtin_bit_cast(uint32_t, __builtin_convertvector(d, bf16x2));
        }
        return Formed{__builtin_bit_cast(bf16x8, hi), __builtin_bit_cast(bf16x8, lo)};
    }
    // what hi + lo leave of v, to the last bit of fp32
    static __device__ __forceinline__ Op rest(f32x8 v, const Formed& f) {
        Op r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = (__bf16)((v[e] - (float)f.hi[e]) - (float)f.lo[e]);
        return r;
    }
    static __device__ __forceinline__ f32x8 widen(Op a) {
        f32x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)a[e];
        return v;
    }
    // elements 16 ks + 8 (l / 32) + e of row `row` (tiles: see Tile)
    template <int D> static __device__ __forceinline__ Op row8(const lds_t* t, int row, int ks) {
        return *reinterpret_cast<const lds_bf16x8*>(t + Tile<D, true>::at(row, 2 * ks + ((threadIdx.x >> 5) & 1)));
    }
    // rows r0 + 8 (l / 32) + e of column c0 + pi(l % 32): the LDS transpose read hands lane
    // i of a 16-lane group column i of the group's 16, made of the four 4-column pieces
    // its lanes point at; pointing at the pieces in the order 0, 2, 1, 3 gives pi
    template <int D> static __device__ __forceinline__ Op col8(const lds_t* t, int r0, int c0) {
        const int l = threadIdx.x & 63, i = l & 15, q = i & 3;
        const int row = r0 + 8 * (l >> 5) + (i >> 2), piece = (c0 >> 3) + ((l >> 3) & 2) + (q & 1);
        const lds_t* p = t + 4 * (q & 2);
        const bf16x4 a = __builtin_bit_cast(
            bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + Tile<D, true>::at(row, piece))));
        const bf16x4 b = __builtin_bit_cast(
            bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + Tile<D, true>::at(row + 4, piece))));
        return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
};
template <> struct Types<false> {
    typedef f32x8 Op;
    typedef f32x8 Formed;
    static __device__ __forceinline__ f32x16 mma(const f32x8& a, const f32x8& b, f32x16 c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    template <int PART> static __device__ __forceinline__ f32x16 part(const f32x8& a, const f32x8& b, f32x16 c) {
        return mma(a, b, c);
    }
    static constexpr int PARTS = 1;
    static __device__ __forceinline__ Formed form(f32x8 v) { return v; }
    static __device__ __forceinline__ f32x8 widen(const Op& a) { return a; }
    template <int D> static __device__ __forceinline__ Op row8(const lds_t* t, int row, int ks) {
        const int piece = 4 * ks + 2 * ((threadIdx.x >> 5) & 1);
        const f32x4 a = *reinterpret_cast<const lds_f32x4*>(t + Tile<D, false>::at(row, piece));
        const f32x4 b = *reinterpret_cast<const lds_f32x4*>(t + Tile<D, false>::at(row, piece + 1));
        return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
    template <int D> static __device__ __forceinline__ Op col8(const lds_t* t, int r0, int c0) {
        const int l = threadIdx.x & 63, col = c0 + pi(l & 31);
        f32x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = *reinterpret_cast<const lds_f32*>(t + Tile<D, false>::at(r0 + 8 * (l >> 5) + e, col >> 2) + 4 * (col & 3));
        return v;
    }
};

__device__ __forceinline__ f32x8 half_of(const f32x16& a, int s) {
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = a[8 * s + e];
    return v;
}

// Rows t0 .. t0 + kC - 1 of one head of x1, x2 or x3 into a Tile, straight into LDS, 1 KB per
// wave and instruction. The compiler does not know of these loads: landed() and a barrier
// stand before the tile is read. Rows at or past n are out of the buffer's range (row i
// starts at i row bytes, the range ends inside row n - 1) and are cleared where there are any.
template <int D, int NT, bool BF16>
struct Rows {
    typedef Tile<D, BF16> Ti;
    static constexpr int P = Ti::P, N = kC * P / NT;  // pieces per row, per thread
    static __device__ __forceinline__ void load(const void* x, size_t b, int L, int nh, int h, int t0, int n, lds_t* t) {
        const uint32_t row = (uint32_t)nh * Ti::RB;
        const char* base = static_cast<const char*>(x) + ((b * L + t0) * nh + h) * (size_t)Ti::RB;
        const auto r = make_rsrc(base, (uint32_t)(n - 1) * row + Ti::RB);
        const int tid = threadIdx.x;
        const uint32_t to = (uint32_t)(uintptr_t)t + (uint32_t)__builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int rr = tid / P + k * (NT / P);
            const uint32_t off = (uint32_t)rr * row + (((tid % P) ^ Ti::swz(rr)) << 4);
            // The LDS address goes through m0, which is left as it was. A load into LDS may come no
            // sooner than one wait state after a scalar write of m0, which the compiler sees to
            // only outside asm: hence the s_nop.
            uint32_t m0;
            asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                         "buffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
                         : "=&s"(m0)
                         : "s"(to + k * NT * 16), "v"(off), "s"(r)
                         : "memory");
        }
    }
    // zeros in the rows at or past n
    static __device__ __forceinline__ void clear(lds_t* t, int n) {
        for (int q = n * P + threadIdx.x; q < kC * P; q += NT)
            *reinterpret_cast<lds_u32x4*>(t + q * 16) = u32x4{0u, 0u, 0u, 0u};
    }
};

// all but the last N of this wave's loads and stores are done
template <int N>
__device__ __forceinline__ void landed() {
    static_assert(N == 0 || N == 4 || N == 8, "");
    if constexpr (N == 0) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    else if constexpr (N == 4) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
}

// Workgroup -> (head, super-chunk, batch). Workgroups go round-robin to the 8 XCDs
// (each with its own L2); consecutive coordinates, heads fastest, go to one XCD where
// the count allows, so that heads sharing queries and keys share its L2.
__device__ __forceinline__ void block_coords(int H, int Kp, int& h, int& k, int& b) {
    const int total = (int)gridDim.x, id = (int)blockIdx.x;
    const int idp = (total % 8 == 0) ? (id % 8) * (total / 8) + id / 8 : id;
    h = idp % H;
    const int r = idp / H;
    k = r % Kp;
    b = r / Kp;
}

// The state tiles of one wave: rows k = 32 T + 16 (r / 8) + 8 hf + r % 8, column
// 32 wave + pi(lane % 32). f(T, r, k, column).
template <int KD, typename F>
__device__ __forceinline__ void each_state_element(F&& f) {
    const int lane = threadIdx.x & 63, hf = lane >> 5;
    const int col = 32 * (threadIdx.x >> 6) + pi(lane & 31);
#pragma unroll
    for (int T = 0; T < KD / 32; ++T)
#pragma unroll
        for (int r = 0; r < 16; ++r) f(T, r, 32 * T + 16 * (r >> 3) + 8 * hf + (r & 7), col);
}

// Where a slot holds element (i, j) of a state of I x J: eight i next to each other for
// one j, j next, so that a wave's tile is read and written in whole lines. A run on the
// transposed state (dk on dv's) finds its elements eight lanes to a line.
__device__ __forceinline__ int slot_at(int i, int j, int J) { return ((i >> 3) * J + j) * 8 + (i & 7); }

// lam^64 as the factor of one chunk after another. Rounded once, it would err in the same
// direction on every chunk of a slowly decaying state; so each chunk takes the float that
// brings the product so far nearest to the exact one.
struct ChunkDecay {
    double lam, inv, err;
    __device__ __forceinline__ void set(float a) {
        lam = exp((double)a);
        inv = lam > 0.5 ? 1.0 / lam : 0.0;
        err = 0.0;
    }
    __device__ __forceinline__ float next() {
        const float m = (float)(lam - lam * err);
        err = inv != 0.0 ? (1.0 + err) * ((double)m * inv) - 1.0 : 0.0;
        return m;
    }
};

// The tiles of a workgroup in LDS. Two buffers where they are filled while the other is
// read: of x2, and, if full, of x1 and x3 as well, where that leaves as many workgroups on a
// CU (two, of KD = 64 and VD = 128). Elsewhere it would be one of two, or, at 64 x 64, two of
// three: x1 and x3 have one buffer, filled once the chunk's scores and x1 S are done.
template <int KD, int VD, bool BF16, bool AGG, int R>
struct Lds {
    static constexpr int BK = Tile<KD, BF16>::BYTES, BV = Tile<VD, BF16>::BYTES;
    static constexpr bool FULL = AGG || (BF16 && KD == 64 && VD == 128 && R == 1);
    static constexpr int N2 = 2, N13 = FULL ? 2 : 1;
    static constexpr int X2 = 0, X3 = X2 + N2 * BK, X1 = X3 + N13 * BV, W = X1 + (AGG ? 0 : N13 * BK),
                         M = W + R * 128 * 4, D = M + (AGG ? 0 : 3 * 2 * 2048),
                         TOTAL = D + (R > 1 ? R * 2 * 4096 : 0);
};

// R > 1: the R heads of a group whose x3 they share, one after the other on every chunk, each
// with a state of its own; the output is their sum.
template <int KD, int VD, bool BF16, bool REV, bool AGG, bool EXACT, int R>
__device__ __forceinline__ void run_chunks(const Mix& a, const Geom& geo, lds_t* lds) {
    typedef Types<BF16> Ty;
    typedef typename Ty::Op Op;
    typedef typename Ty::Formed Formed;
    typedef Lds<KD, VD, BF16, AGG, R> Ld;
    constexpr int NT = 2 * VD, KS = KD / 16, KT = KD / 32;
    typedef Rows<KD, NT, BF16> RowsK;
    typedef Rows<VD, NT, BF16> RowsV;
    int h, sc, b;
    block_coords(a.H / R, AGG ? (geo.NS - 1) * geo.P : geo.NS, h, sc, b);
    h *= R;
    const int piece = AGG ? sc % geo.P : 0;
    if (AGG) sc = sc / geo.P + (REV ? 1 : 0);
    const int tid = threadIdx.x, lane = tid & 63, hf = lane >> 5, c = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const size_t bh = (size_t)b * a.H + h;
    const int G = a.H / a.r, hg = h / a.r;
    const int h1 = a.g1 ? hg : h, n1 = a.g1 ? G : a.H;
    const int h2 = a.g2 ? hg : h, n2 = a.g2 ? G : a.H;
    const int h3 = a.g3 ? hg : h, n3 = a.g3 ? G : a.H;
    const int len = seq_len(a.seqlens, b, a.L);

    // chunks [c0, c1) of this super-chunk, of which [c0, ca) hold steps of the sequence
    const int c0 = sc * geo.cps + piece * geo.cpp;
    const int c1 = max(c0, min(min(geo.NC, (sc + 1) * geo.cps), AGG ? c0 + geo.cpp : geo.NC));
    const int ca = max(c0, min(c1, (len + kC - 1) / kC)), nch = ca - c0;
    auto chunk_at = [&](int u) { return REV ? ca - 1 - u : c0 + u; };

    // step u: head u % R of the run's chunk u / R. Its rows into its buffers (x3's with the
    // first head).
    auto load = [&](int u) {
        const int t0 = chunk_at(u / R) * kC, n = min(kC, len - t0), b2 = u % Ld::N2, b13 = u % Ld::N13, hh = u % R;
        RowsK::load(a.x2, b, a.L, n2, h2 + hh, t0, n, lds + Ld::X2 + b2 * Ld::BK);
        if constexpr (!AGG) RowsK::load(a.x1, b, a.L, n1, h1 + hh, t0, n, lds + Ld::X1 + b13 * Ld::BK);
        if (hh == 0) RowsV::load(a.x3, b, a.L, n3, h3, t0, n, lds + Ld::X3 + b13 * Ld::BV);
    };
    if (nch > 0) load(0);

    float la[R];
#pragma unroll
    for (int hh = 0; hh < R; ++hh) la[hh] = log_decay_of(a.log_decay, h + hh);
    auto power = [&](int hh, int n) { return exp2_fast((float)n * (la[hh] * kLog2e)); };

    // the states entering the super-chunk
    f32x16 S[R][KT];
#pragma unroll
    for (int hh = 0; hh < R; ++hh) {
#pragma unroll
        for (int T = 0; T < KT; ++T)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[hh][T][r] = 0.0f;
        if constexpr (!AGG) {
            const bool first = REV ? sc == geo.NS - 1 : sc == 0;
            if (first) {
                const float* src = a.init + (bh + hh) * KD * VD;
                if (a.init)
                    each_state_element<KD>(
                        [&](int T, int r, int k, int j) { S[hh][T][r] = src[a.trans ? j * KD + k : k * VD + j]; });
            } else {
                const float* src = a.slots + ((bh + hh) * (geo.NS - 1) + (REV ? sc : sc - 1)) * geo.P * KD * VD;
                if (a.trans)
                    each_state_element<KD>([&](int T, int r, int k, int j) { S[hh][T][r] = src[slot_at(j, k, KD)]; });
                else each_state_element<KD>([&](int T, int r, int k, int j) { S[hh][T][r] = src[slot_at(k, j, VD)]; });
            }
        }
    }

    // W[x]: weight of row j of x3 in the state's update; forwards lam^(n-1-j) = W[j + 64 - n],
    // backwards lam^(j+1) = W[j]; times kv_scale
    lds_f32* wt = reinterpret_cast<lds_f32*>(lds + Ld::W);
#pragma unroll
    for (int hh = 0; hh < R; ++hh)
        for (int x = tid; x < 128; x += NT)
            wt[hh * 128 + x] = x < kC ? power(hh, REV ? x + 1 : kC - 1 - x) * a.kv_scale : 0.0f;
    // The scores' tiles that count are (J, I) = (0, 0) and (1, 1) on the diagonal and one off
    // it, (0, 1) forwards, (1, 0) backwards. Each is computed by one wave, decayed (this
    // lane's 16 factors: row i = 32 I + c, column j = 32 J + 16 (r / 8) + 8 hf + r % 8),
    // formed and passed to the others through LDS as operands. Of four waves the last
    // repeats tile (0, 0) for nothing; of two, each has a diagonal tile and both the other,
    // which the first passes on.
    const bool off_diag = NT == 256 && wave == 2;
    const int Ja = off_diag ? (REV ? 1 : 0) : wave & 1 & (wave >> 1 ^ 1), Ia = off_diag ? (REV ? 0 : 1) : Ja;
    auto factor = [&](int hh, bool off, int r) {
        const int j = 16 * (r >> 3) + 8 * hf + (r & 7), lag = REV ? j - c : c - j;
        return (off ? power(hh, 32 + lag) : lag >= 0 ? power(hh, lag) : 0.0f) * (a.kv_scale * a.out_scale);
    };
    f32x16 d_a, d_b;  // in registers for one head, in LDS for more ([head][on, off][4][lane])
    lds_f32x4* tab = reinterpret_cast<lds_f32x4*>(lds + Ld::D);
    if constexpr (!AGG && R == 1) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            d_a[r] = factor(0, off_diag, r);
            d_b[r] = factor(0, true, r);
        }
    } else if constexpr (!AGG) {
        if (wave < 2)
#pragma unroll
            for (int hh = 0; hh < R; ++hh)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f32x4 x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = factor(hh, wave, 4 * q + e);
                    tab[((hh * 2 + wave) * 4 + q) * 64 + lane] = x;
                }
    }

    // outputs of this wave's 32 columns of row block I (rows t0 + 32 I + c); rows past the
    // sequence's end are out of range, so the number of stores is always the same
    // A lane holds 32 (or, fp32, 64) bytes of one row in pieces of 16; pieces are exchanged
    // between lanes 16 apart so that a store covers 64 consecutive bytes of 16 rows and not
    // 32 of 32.
    const int ho = h / R, no = a.H / R;  // the output's head of so many
    const uint32_t orow = (uint32_t)no * VD * (BF16 && !a.out_f32 ? 2 : 4);
    auto put = [&](int t0, int I, const f32x16& acc) {
        const int es = BF16 && !a.out_f32 ? 2 : 4;
        const int nr = min(kC, a.L - t0);
        const auto out = make_rsrc(static_cast<char*>(a.out) + (((size_t)b * a.L + t0) * no + ho) * (size_t)(VD * es),
                                   (uint32_t)(nr - 1) * orow + VD * es);
        // pieces x and y of this lane's row; col: where the piece this lane then has begins
        auto pair = [&](u32x4 x, u32x4 y, uint32_t col) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const auto z = __builtin_amdgcn_permlane16_swap(x[e], y[e], false, false);
                x[e] = z[0];
                y[e] = z[1];
            }
            const uint32_t off = (uint32_t)(32 * I + (c & 15)) * orow + (uint32_t)(32 * wave * es) + col;
            __builtin_amdgcn_raw_buffer_store_b128(x, out, (int)off, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b128(y, out, (int)(off + 16 * orow), 0, 0);
        };
        if (BF16 && !a.out_f32) {
            bf16x8 y[2];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e >> 3][e & 7] = (__bf16)acc[e];
            pair(__builtin_bit_cast(u32x4, y[0]), __builtin_bit_cast(u32x4, y[1]), (c >> 4) * 32 + hf * 16);
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                u32x4 y[2];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e >> 2][e & 3] = __float_as_uint(acc[8 * s + e]);
                pair(y[0], y[1], 64 * s + hf * 32 + (c >> 4) * 16);
            }
        }
    };
    if constexpr (!AGG) {  // chunks of padding alone
        f32x16 zero;
#pragma unroll
        for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
        for (int ch = ca; ch < c1; ++ch)
            for (int I = 0; I < 2; ++I)
                if (ch * kC < a.L) put(ch * kC, I, zero);
    }

    // step u's tiles complete and visible to every wave. A chunk's stores of outputs are
    // issued after the loads of the next one's rows and need not be waited for (vmcnt
    // counts both in the order of issue; every wave issues 4 of bf16, 8 of fp32).
    auto stage = [&](int u, bool stores) {
        const int n = min(kC, len - chunk_at(u / R) * kC);
        lds_t* x1 = lds + Ld::X1 + u % Ld::N13 * Ld::BK;
        lds_t* x2 = lds + Ld::X2 + u % Ld::N2 * Ld::BK;
        lds_t* x3 = lds + Ld::X3 + u % Ld::N13 * Ld::BV;
        if (!stores) landed<0>();
        else if (!BF16 || a.out_f32) landed<8>();
        else landed<4>();
        if (n < kC) {
            __syncthreads();
            if constexpr (!AGG) RowsK::clear(x1, n);
            RowsK::clear(x2, n);
            if (u % R == 0) RowsV::clear(x3, n);
        }
        __syncthreads();
    };

    ChunkDecay full[R];
#pragma unroll
    for (int hh = 0; hh < R; ++hh) full[hh].set(la[hh] * (float)kC);
    if (nch > 0) stage(0, false);
    for (int cu = 0; cu < nch; ++cu) {
        const int t0 = chunk_at(cu) * kC, n = min(kC, len - t0);
        Op v[4];
        f32x16 out[2];
#pragma unroll
        for (int hh = 0; hh < R; ++hh) {
            const int u = cu * R + hh;
            const bool more = u + 1 < nch * R;
            const lds_t* x1 = lds + Ld::X1 + u % Ld::N13 * Ld::BK;
            const lds_t* x2 = lds + Ld::X2 + u % Ld::N2 * Ld::BK;
            const lds_t* x3 = lds + Ld::X3 + u % Ld::N13 * Ld::BV;
            if (Ld::FULL && more) load(u + 1);
            auto read_v = [&]() {
#pragma unroll
                for (int s = 0; s < 4; ++s) v[s] = Ty::template col8<VD>(x3, 16 * s, 32 * wave);
            };
            if constexpr (AGG) {
                read_v();
            } else {
                // scores (rows j in the order pi, columns i) and x1 S (rows: columns of S); the
                // operands of step ks + 1 are read while those of ks multiply
                f32x16 acc[2], ma, mb;
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[0][r] = acc[1][r] = ma[r] = mb[r] = 0.0f;
                const lds_t* xj = x2 + Ja * (Ld::BK / 2);
                const lds_t* xi = x1 + Ia * (Ld::BK / 2);
                Op q0, q1, qa{}, ka, kb{};
                auto fetch = [&](int ks) {
                    q0 = Ty::template row8<KD>(x1, c, ks);
                    q1 = Ty::template row8<KD>(x1, 32 + c, ks);
                    ka = Ty::template row8<KD>(xj, pi(c), ks);
                    if constexpr (NT == 256) qa = Ty::template row8<KD>(xi, c, ks);
                    else kb = Ty::template row8<KD>(x2, (REV ? 32 : 0) + pi(c), ks);
                };
                fetch(0);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const Op p0 = q0, p1 = q1, pa = NT == 256 ? qa : (wave ? q1 : q0), la_ = ka, lb = kb;
                    if (ks + 1 < KS) fetch(ks + 1);
                    const Formed sf = Ty::form(half_of(S[hh][ks >> 1], ks & 1));
                    ma = Ty::mma(la_, pa, ma);
                    acc[0] = Ty::template part<0>(sf, p0, acc[0]);
                    acc[1] = Ty::template part<0>(sf, p1, acc[1]);
                    if constexpr (NT != 256) mb = Ty::mma(lb, REV ? p0 : p1, mb);
                    if constexpr (Ty::PARTS == 2) {
                        acc[0] = Ty::template part<1>(sf, p0, acc[0]);
                        acc[1] = Ty::template part<1>(sf, p1, acc[1]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                auto pass = [&](const f32x16& m, const f32x16& d, int slot) {
                    f32x16 x;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = m[r] * d[r];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const Formed f = Ty::form(half_of(x, s));
                        u32x4 q[2];
                        __builtin_memcpy(q, &f, 32);
                        lds_u32x4* to = reinterpret_cast<lds_u32x4*>(lds + Ld::M + (2 * slot + s) * 2048) + lane;
                        to[0] = q[0];
                        to[64] = q[1];
                    }
                };
                auto factors = [&](bool off) {
                    f32x16 d;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 x = tab[((hh * 2 + off) * 4 + q) * 64 + lane];
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[4 * q + e] = x[e];
                    }
                    return d;
                };
                if (wave < 3) pass(ma, R == 1 ? d_a : factors(off_diag), wave);
                if (NT != 256 && wave == 0) pass(mb, R == 1 ? d_b : factors(true), 2);
                if (hh == 0) read_v();
                __syncthreads();  // the scores visible; x1 and x3 read
                if (!Ld::FULL && more) load(u + 1);
                const float w0 = power(hh, REV ? max(n - 1 - c, 0) : c + 1) * a.out_scale;
                const float w1 = power(hh, REV ? max(n - 33 - c, 0) : c + 33) * a.out_scale;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    out[0][r] = hh == 0 ? acc[0][r] * w0 : __builtin_fmaf(acc[0][r], w0, out[0][r]);
                    out[1][r] = hh == 0 ? acc[1][r] * w1 : __builtin_fmaf(acc[1][r], w1, out[1][r]);
                }
                auto formed = [&](int slot, int s) {
                    const lds_u32x4* m = reinterpret_cast<const lds_u32x4*>(lds + Ld::M + (2 * slot + s) * 2048) + lane;
                    const u32x4 q[2] = {m[0], m[64]};
                    Formed f;
                    __builtin_memcpy(&f, q, 32);
                    return f;
                };
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Formed f0 = formed(0, s), f1 = formed(1, s), fx = formed(2, s);
                    f32x16 &ax = out[REV ? 0 : 1], &ay = out[REV ? 1 : 0];
                    const Formed &gx = REV ? f0 : f1, &gy = REV ? f1 : f0;
                    const Op vx = v[REV ? s : 2 + s], vy = v[REV ? 2 + s : s];
                    ax = Ty::template part<0>(vx, gx, ax);
                    ay = Ty::template part<0>(vy, gy, ay);
                    ax = Ty::template part<0>(vy, fx, ax);
                    if constexpr (Ty::PARTS == 2) {
                        ay = Ty::template part<1>(vy, gy, ay);
                        ax = Ty::template part<1>(vx, gx, ax);
                        ax = Ty::template part<1>(vy, fx, ax);
                    }
                }
                if (hh == R - 1) {
                    if (n < kC) {  // rows of padding are 0 whatever the state holds
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            if (c >= n) out[0][r] = 0.0f;
                            if (32 + c >= n) out[1][r] = 0.0f;
                        }
                    }
                    put(t0, 0, out[0]);
                    put(t0, 1, out[1]);
                }
            }
            if (AGG || cu + 1 < nch || (R == 1 && a.final_state)) {
                // the operands of step s + 1 are read and formed while those of step s multiply
                const lds_f32* w0 = wt + hh * 128 + 8 * hf + (REV ? 0 : kC - n);
                Op k[KT];
                f32x8 w;
                auto fetch = [&](int s) {
#pragma unroll
                    for (int T = 0; T < KT; ++T) k[T] = Ty::template col8<KD>(x2, 16 * s, 32 * T);
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = w0[16 * s + e];
                };
                Op rest{};
                auto weighted = [&](int s) {
                    f32x8 x = Ty::widen(v[s]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= w[e];
                    const Formed f = Ty::form(x);
                    if constexpr (BF16 && EXACT) rest = Ty::rest(x, f);
                    return f;
                };
                fetch(0);
                const float m = n == kC ? full[hh].next() : expf(la[hh] * (float)n);  // at most one chunk is shorter
#pragma unroll
                for (int T = 0; T < KT; ++T)
#pragma unroll
                    for (int r = 0; r < 16; ++r) S[hh][T][r] *= m;
                Formed wv = weighted(0);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    Op kn[KT];
#pragma unroll
                    for (int T = 0; T < KT; ++T) kn[T] = k[T];
                    if (s < 3) fetch(s + 1);
#pragma unroll
                    for (int T = 0; T < KT; ++T) S[hh][T] = Ty::template part<0>(kn[T], wv, S[hh][T]);
                    const Op third = rest;
                    const Formed next = s < 3 ? weighted(s + 1) : wv;
                    if constexpr (Ty::PARTS == 2)
#pragma unroll
                        for (int T = 0; T < KT; ++T) S[hh][T] = Ty::template part<1>(kn[T], wv, S[hh][T]);
                    if constexpr (BF16 && EXACT)
#pragma unroll
                        for (int T = 0; T < KT; ++T) S[hh][T] = Ty::mma(kn[T], third, S[hh][T]);
                    wv = next;
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (more) stage(u + 1, !AGG && hh == R - 1);
        }
    }

    if constexpr (AGG) {
        float* dst = a.slots + ((bh * (geo.NS - 1) + (REV ? sc - 1 : sc)) * geo.P + piece) * KD * VD;
        if (a.trans) each_state_element<KD>([&](int T, int r, int k, int j) { dst[slot_at(j, k, KD)] = S[0][T][r]; });
        else each_state_element<KD>([&](int T, int r, int k, int j) { dst[slot_at(k, j, VD)] = S[0][T][r]; });
    } else if (a.final_state && (REV ? sc == 0 : sc == geo.NS - 1)) {
        float* dst = a.final_state + bh * KD * VD;
        each_state_element<KD>([&](int T, int r, int k, int j) { dst[k * VD + j] = S[0][T][r]; });
    }
}

template <int KD, int VD, bool BF16, bool AGG>
__global__ void __launch_bounds__(2 * VD) __attribute__((amdgpu_waves_per_eu(BF16 ? 2 : 1, BF16 ? 2 : 1)))
mix_chunks(Jobs jobs, Geom geo) {
    __shared__ __attribute__((aligned(16))) char lds[Lds<KD, VD, BF16, AGG, 1>::TOTAL];
    const int j = blockIdx.y;
    const Mix& m = jobs.m[j];
    if (BF16 && m.exact) {
        if (jobs.rev[j]) run_chunks<KD, VD, BF16, true, AGG, true, 1>(m, geo, (lds_t*)lds);
        else run_chunks<KD, VD, BF16, false, AGG, true, 1>(m, geo, (lds_t*)lds);
    } else {
        if (jobs.rev[j]) run_chunks<KD, VD, BF16, true, AGG, false, 1>(m, geo, (lds_t*)lds);
        else run_chunks<KD, VD, BF16, false, AGG, false, 1>(m, geo, (lds_t*)lds);
    }
}

// dq and dk of R heads that share a group
template <int VD, int R>
__global__ void __launch_bounds__(2 * VD) __attribute__((amdgpu_waves_per_eu(1, 1)))
mix_chunks_shared(Jobs jobs, Geom geo) {
    __shared__ __attribute__((aligned(16))) char lds[Lds<64, VD, true, false, R>::TOTAL];
    const int j = blockIdx.y;
    if (jobs.rev[j]) run_chunks<64, VD, true, true, false, false, R>(jobs.m[j], geo, (lds_t*)lds);
    else run_chunks<64, VD, true, false, false, false, R>(jobs.m[j], geo, (lds_t*)lds);
}

// Aggregates -> entering states, in the run's direction: what super-chunk s adds, plus
// lam^(its steps) times the state entering it, enters the next. One lane per four
// state elements; eight slots are loaded before any is written.
__global__ void __launch_bounds__(256) mix_carry(Jobs jobs, Geom geo, int n4, int J) {
    const Mix& a = jobs.m[blockIdx.z];
    const int rev = jobs.rev[blockIdx.z];
    const int e = blockIdx.x * 256 + threadIdx.x;
    const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    if (e >= n4) return;
    // piece i in the run's direction: of slot i / P, the same place from the end if backwards
    const int len = seq_len(a.seqlens, b, a.L), n = (geo.NS - 1) * geo.P;
    const float la = log_decay_of(a.log_decay, h);
    float4* slot = reinterpret_cast<float4*>(a.slots) + (size_t)bh * n * n4 + e;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.init) {  // elements 4 e .. 4 e + 3 of a slot: rows i .. i + 3 of column j of [I, J]
        const int j = (e >> 1) % J, i = ((e >> 1) / J) * 8 + 4 * (e & 1);
        const float* p = a.init + ((size_t)bh * (n4 / J * 4) + i) * J + j;
        v = make_float4(p[0], p[J], p[2 * J], p[3 * J]);
    }
    for (int i0 = 0; i0 < n; i0 += 8) {
        float4 sl[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = min(i0 + j, n - 1);
            sl[j] = slot[(size_t)(rev ? n - 1 - i : i) * n4];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j;
            if (i >= n) break;
            const int at = rev ? n - 1 - i : i, sc = at / geo.P + (rev ? 1 : 0), piece = at % geo.P;
            const int c0 = sc * geo.cps + piece * geo.cpp, c1 = min(min(geo.NC, (sc + 1) * geo.cps), c0 + geo.cpp);
            const Decay decay(la * (float)max(0, min(len - c0 * kC, (c1 - c0) * kC)));
            v.x = decay(v.x) + sl[j].x;
            v.y = decay(v.y) + sl[j].y;
            v.z = decay(v.z) + sl[j].z;
            v.w = decay(v.w) + sl[j].w;
            if (piece == (rev ? 0 : geo.P - 1)) slot[(size_t)(at - piece) * n4] = v;
        }
    }
}

// Sum over the r heads of each group of an fp32 [rows, G, r, D] tensor, in head order,
// rounded once to [rows, G, D]; two tensors, one after the other. Four values a lane.
template <bool BF16>
__global__ void __launch_bounds__(256)
sum_heads(const float* __restrict__ p, void* out0, void* out1, size_t n4, int r, int D4) {
    const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= n4) return;
    const f32x4* q = reinterpret_cast<const f32x4*>(p) + blockIdx.y * n4 * r + (e / D4) * r * D4 + e % D4;
    f32x4 s = q[0];
    for (int k = 1; k < r; ++k) s += q[(size_t)k * D4];
    void* out = blockIdx.y ? out1 : out0;
    if constexpr (BF16) {
        const bf16x4 y = {(__bf16)s[0], (__bf16)s[1], (__bf16)s[2], (__bf16)s[3]};
        reinterpret_cast<bf16x4*>(out)[e] = y;
    } else {
        reinterpret_cast<f32x4*>(out)[e] = s;
    }
}

template <int KD, int VD>
hipError_t run_t(const Jobs& jobs, const Geom& g, bool bf16, bool agg, hipStream_t st) {
    const Mix& m = jobs.m[0];
    const dim3 grid((unsigned)m.B * m.H * (agg ? (g.NS - 1) * g.P : g.NS), (unsigned)jobs.n);
    if (bf16 && agg) launch((mix_chunks<KD, VD, true, true>), grid, dim3(2 * VD), 0, st, jobs, g);
    else if (bf16) launch((mix_chunks<KD, VD, true, false>), grid, dim3(2 * VD), 0, st, jobs, g);
    else if (agg) launch((mix_chunks<KD, VD, false, true>), grid, dim3(2 * VD), 0, st, jobs, g);
    else launch((mix_chunks<KD, VD, false, false>), grid, dim3(2 * VD), 0, st, jobs, g);
    return hipGetLastError();
}

hipError_t run(const Jobs& jobs, const Geom& g, int KD, int VD, bool bf16, bool agg, hipStream_t st) {
    if (KD == 64) return VD == 64 ? run_t<64, 64>(jobs, g, bf16, agg, st) : run_t<64, 128>(jobs, g, bf16, agg, st);
    return VD == 64 ? run_t<128, 64>(jobs, g, bf16, agg, st) : run_t<128, 128>(jobs, g, bf16, agg, st);
}

// Aggregates and carry of runs whose states are K x V, or held as such (trans). More than
// one super-chunk means fewer than 4096 (batch, head)s, which the carry's grid.y holds.
hipError_t run_carry(const Jobs& jobs, const Geom& g, int KD, int VD, bool bf16, hipStream_t st) {
    if (g.NS == 1) return hipSuccess;
    const hipError_t e = run(jobs, g, KD, VD, bf16, true, st);
    if (e != hipSuccess) return e;
    const Mix& m = jobs.m[0];
    const int n4 = KD * VD / 4;
    launch(mix_carry, dim3((n4 + 255) / 256, (unsigned)m.B * m.H, (unsigned)jobs.n), dim3(256), 0, st, jobs, g, n4,
           m.trans ? KD : VD);
    return hipGetLastError();
}

hipError_t run_shared(const Jobs& jobs, const Geom& g, int r, int K, hipStream_t st) {
    const Mix& m = jobs.m[0];
    const dim3 grid((unsigned)m.B * (m.H / r) * g.NS, (unsigned)jobs.n), block(2 * K);
    if (K == 64 && r == 2) launch((mix_chunks_shared<64, 2>), grid, block, 0, st, jobs, g);
    else if (K == 64) launch((mix_chunks_shared<64, 3>), grid, block, 0, st, jobs, g);
    else if (r == 2) launch((mix_chunks_shared<128, 2>), grid, block, 0, st, jobs, g);
    else launch((mix_chunks_shared<128, 3>), grid, block, 0, st, jobs, g);
    return hipGetLastError();
}

size_t slot_bytes(int B, int H, int K, int V, const Geom& g) { return (size_t)B * H * (g.NS - 1) * g.P * K * V * 4; }

}  // namespace

bool linattn_supported_dim(int d) { return d == 64 || d == 128; }

void linattn_plan(int B, int L, int H, int G, int K, int V, bool bf16, bool bwd, int plan[6]) {
    const Geom g = geom(B, L, H, G, K, V, bf16, bwd);
    const int p[6] = {g.NC, g.NS, g.cps, g.P, g.cpp, bwd && shared_heads(H / G, V, bf16) ? H / G : 1};
    std::copy(p, p + 6, plan);
}

// entering states of the super-chunks
size_t linattn_workspace_bytes(int B, int L, int H, int G, int K, int V, bool bf16) {
    return slot_bytes(B, H, K, V, geom(B, L, H, G, K, V, bf16, false));
}

// those of both directions, and fp32 dq and dk per head where heads share a group
size_t linattn_bwd_workspace_bytes(int B, int L, int H, int G, int K, int V, bool bf16) {
    return 2 * slot_bytes(B, H, K, V, geom(B, L, H, G, K, V, bf16, true)) +
           (H == G || shared_heads(H / G, V, bf16) ? 0 : 2 * (size_t)B * L * H * K * 4);
}

hipError_t launch_linattn_fwd(const LinattnArgs& a, hipStream_t st) {
    const Geom g = geom(a.B, a.L, a.H, a.G, a.K, a.V, a.bf16, false);
    const Mix m{a.B, a.L, a.H, a.H / a.G, a.q, a.k, a.v, 1, 1, 0, a.log_decay, a.seqlens,
                a.scale, 1.0f, a.h0, static_cast<float*>(a.ws), 0, a.o, 0, a.h_final, a.h_final != nullptr};
    const Jobs jobs{{m}, {0}, 1};
    const hipError_t e = run_carry(jobs, g, a.K, a.V, a.bf16, st);
    return e != hipSuccess ? e : run(jobs, g, a.K, a.V, a.bf16, false, st);
}

hipError_t launch_linattn_bwd(const LinattnBwdArgs& a, hipStream_t st) {
    const Geom g = geom(a.B, a.L, a.H, a.G, a.K, a.V, a.bf16, true);
    const int r = a.H / a.G;
    const bool together = shared_heads(r, a.V, a.bf16), shared = r > 1 && !together;
    const size_t ng = (size_t)a.B * a.L * a.G * a.K, ns = slot_bytes(a.B, a.H, a.K, a.V, g) / 4;
    float* slots = static_cast<float*>(a.ws);
    float* heads = slots + 2 * ns;
    // dq: the state v (x) k of the forward run, held transposed (as [K, V], like h0)
    const Mix mq{a.B, a.L, a.H, r, a.dout, a.v, a.k, 0, 0, 1, a.log_decay, a.seqlens,
                 a.scale, 1.0f, a.h0, slots, 1, shared ? heads : a.dq, shared, nullptr, 0};
    // dv, and dk from the same entering states, read transposed
    const Mix mv{a.B, a.L, a.H, r, a.k, a.q, a.dout, 1, 1, 0, a.log_decay, a.seqlens,
                 1.0f, a.scale, a.dh_final, slots + ns, 0, a.dv, 0, a.dh0, a.dh0 != nullptr};
    Mix mk{a.B, a.L, a.H, r, a.v, a.dout, a.q, 0, 0, 1, a.log_decay, a.seqlens,
           1.0f, a.scale, a.dh_final, slots + ns, 1, shared ? heads + ng * r : a.dk, shared, nullptr, a.dh0 != nullptr};
    hipError_t e;
    // the backwards state's aggregates as those of dk's run: the same orientation as dq's, so
    // that one launch does both
    if ((e = run_carry(Jobs{{mq, mk}, {0, 1}, 2}, g, a.V, a.K, a.bf16, st)) != hipSuccess) return e;
    mk.exact = 0;  // its own state is no output
    if (together) {
        if ((e = run_shared(Jobs{{mq, mk}, {0, 1}, 2}, g, r, a.K, st)) != hipSuccess) return e;
        return run(Jobs{{mv}, {1}, 1}, g, a.K, a.V, a.bf16, false, st);
    }
    if (a.K == a.V) {
        if ((e = run(Jobs{{mq, mk, mv}, {0, 1, 1}, 3}, g, a.V, a.K, a.bf16, false, st)) != hipSuccess) return e;
    } else {  // other workgroup sizes
        if ((e = run(Jobs{{mq, mk}, {0, 1}, 2}, g, a.V, a.K, a.bf16, false, st)) != hipSuccess) return e;
        if ((e = run(Jobs{{mv}, {1}, 1}, g, a.K, a.V, a.bf16, false, st)) != hipSuccess) return e;
    }
    if (!shared || ng == 0) return hipSuccess;
    const dim3 grid((unsigned)((ng / 4 + 255) / 256), 2);
    if (a.bf16) launch(sum_heads<true>, grid, dim3(256), 0, st, heads, a.dq, a.dk, ng / 4, r, a.K / 4);
    else launch(sum_heads<false>, grid, dim3(256), 0, st, heads, a.dq, a.dk, ng / 4, r, a.K / 4);
    return hipGetLastError();
}

}  // namespace ssm
