// Per-head norm and rotation of Q and K rows, and their gradients (formulas in include/vt_attn.h).
//
// Bound by HBM: a row is read once and written once (the backward reads it and its gradient), a handful of
// operations per element.  What the layout is for:
//   - A row is spread over `tpr` threads; each holds VEC elements of the row's rotated part and the VEC
//     elements they pair with, so a rotation needs no other thread and the norm's mean is a shuffle over tpr
//     lanes.  A thread keeps its token and its columns for every head it works on, so the cosines and sines
//     of its pairs live in registers.
//   - A block walks over groups of `tok` consecutive tokens (about one angle per thread) and their heads, Q's and then
//     K's.  The rows come through a ring in shared memory that every thread fills and reads for itself (cp.async, no
//     barrier), several rows ahead and across groups: bytes in flight are what this kernel lives on, and registers
//     hold too few of them.
//   - Angles are formed once per token and pair as 64-bit fixed-point fractions of a turn: the position times the
//     frequency in turns, whose overflow is the reduction by whole turns.  fp32 products lose the phase of
//     positions beyond a few thousand, and fp64 ones keep the (slow) fp64 pipe busy for longer than the loads take
//     when few heads share a token.
//   - VEC is 16 bytes when R and D allow it, else 8 bytes or single elements.
// Measured (8192 tokens of 32 + 8 heads, D = 128, bf16, inputs colder than L2): forward 32 us, 5.3 TB/s of rows read and
// written, schedulers issuing in 73 % of their cycles; backward with both weights' gradients 50 us, 5.0 TB/s, 63 %.  So the
// instructions per row bound both, a little before HBM does.  16 sequences of one token take 5 us, a launch's latency.
#pragma once

#include <cstdint>

#include "vt_attn_common.cuh"

namespace vt {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;
constexpr int kMaxD = 256;
constexpr int kAhead = 4, kAheadBwd = 3;  // rows a thread has under way (32 bytes each, the backward's 64); more gain nothing
constexpr int kBwdMaxBlocks = 608;  // blocks of a backward launch, each leaves one partial weight gradient

struct Params {
    int B, H, H_kv, S, D, half;  // half = R / 2
    int tpr, tok, heads;         // threads per row, tokens per block, heads a block works on at once
    int chunks;                  // chunks of 2 VEC elements in a row
    unsigned tokens;             // B * S
    float eps;
    const void *x[2];            // q, k
    long long x_st[2][3];
    const void *w[2];
    void *y[2];
    long long y_st[2][3];
    const void *g[2];            // backward: gradients of the outputs
    long long g_st[2][3];
    float *part[2];              // backward: partial weight gradients [blocks of the tensor][D], or null
    int blocks_q;                // backward: the first blocks work on Q, the others on K
    const float *freqs;
    const int *pos;
    long long pos_st[3];
    const int *kv_len;           // append, or null
    long long cap;
    int D_v;
    const void *v;
    void *v_out;
    long long v_st[3], vo_st[3];
    unsigned *status;
    uint8_t axis[kMaxPairs];
};

struct bf16 {
    uint16_t u;
};

// A run of VEC elements as 32-bit words (single bf16 elements in the low half of one).
template <typename T, int VEC>
struct Run {
    static constexpr int kBytes = VEC * sizeof(T), kWords = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kBytes == 16) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(p);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (kBytes == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kBytes == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t *>(p) = w[0];
        else *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w[0]);
    }
    // a copy of the run on its way to shared memory, and from there
    __device__ static __forceinline__ void fetch(uint32_t dst, const T *p) {
        if constexpr (kBytes == 16)
            cp_async16(dst, p, 16);
        else if constexpr (kBytes >= 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(p), "n"(kBytes) : "memory");
        else
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst), "h"(*reinterpret_cast<const uint16_t *>(p)) : "memory");
    }
    __device__ __forceinline__ void take(const uint8_t *staged) { load(reinterpret_cast<const T *>(staged)); }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    }
    // elements i and i + 1 (i even; with VEC = 1 the first alone)
    __device__ __forceinline__ void set2(int i, float a, float b) {
        if constexpr (sizeof(T) == 4) {
            w[i] = __float_as_uint(a);
            if constexpr (VEC > 1) w[i + 1] = __float_as_uint(b);
        } else {
            w[i >> 1] = pack_bf16x2(a, b);
        }
    }
};

// The 2 VEC elements of chunk c: the two runs of VEC elements they occupy start at first() and second(), and
// are rotated when c < rotated().  Rotated chunks of the halves form are (i.., i + half..); every other chunk is
// 2 VEC consecutive elements (with pairs (2i, 2i + 1) when rotated).
template <int VEC, bool INTER>
struct Chunk {
    int a, b;
    bool turn;
    __device__ Chunk(const Params &p, int c) {
        if (INTER) {
            a = c * 2 * VEC;
            b = a + VEC;
            turn = a < 2 * p.half;
        } else {
            turn = c * VEC < p.half;
            a = turn ? c * VEC : 2 * p.half + (c - p.half / VEC) * 2 * VEC;
            b = turn ? a + p.half : a + VEC;
        }
    }
};

// A chunk as it lies in memory.
template <typename T, int VEC>
struct Raw {
    Run<T, VEC> lo, hi;

    __device__ __forceinline__ void zero() {
        lo.zero();
        hi.zero();
    }
};
template <typename T, int VEC>
__device__ __forceinline__ void load_raw(Raw<T, VEC> &r, const T *row, int a, int b, int D) {
    r.lo.load(row + a);
    if (VEC > 1 || b < D) r.hi.load(row + b);  // (in single elements an odd D ends inside a chunk)
}

// The ring: `kRuns` runs of a row per thread and stage, each thread's side by side with its neighbours'.
template <typename T, int VEC, int kRuns, int kStages>
struct Ring {
    static constexpr int kBytes = Run<T, VEC>::kBytes;
    static constexpr int kStage = kRuns * kThreads * kBytes;
    uint8_t *mine;
    uint32_t mine_s;
    int put = 0, got = 0;  // byte offsets of the stages to fill and to read next

    __device__ Ring(uint8_t *smem) : mine(smem + threadIdx.x * kBytes), mine_s(smem_u32(smem) + threadIdx.x * kBytes) {}
    __device__ __forceinline__ void fetch(int run, const T *p) {
        Run<T, VEC>::fetch(mine_s + put + run * kThreads * kBytes, p);
    }
    __device__ __forceinline__ void pushed() {
        cp_async_commit();
        put = put == (kStages - 1) * kStage ? 0 : put + kStage;
    }
    __device__ __forceinline__ void take(int run, Run<T, VEC> &r) const {
        r.take(mine + got + run * kThreads * kBytes);
    }
    __device__ __forceinline__ void popped() { got = got == (kStages - 1) * kStage ? 0 : got + kStage; }
};

// The chunk's pairs two by two, for arithmetic on both at once: a[j], b[j] hold the first and the second members of
// pairs 2 j and 2 j + 1 (VEC = 1: of its one pair, and 0).
template <int VEC>
struct Pairs {
    static constexpr int kN = VEC > 1 ? VEC / 2 : 1;
    float2 a[kN], b[kN];
};
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void unpack(const Raw<T, VEC> &r, Pairs<VEC> &x) {
    if constexpr (VEC == 1) {
        x.a[0] = make_float2(r.lo.get(0), 0.0f);
        x.b[0] = make_float2(r.hi.get(0), 0.0f);
    } else {
        auto at = [&](int i) { return i < VEC ? r.lo.get(i) : r.hi.get(i - VEC); };  // the chunk's elements in order
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            x.a[j] = INTER ? make_float2(at(4 * j), at(4 * j + 2)) : make_float2(at(2 * j), at(2 * j + 1));
            x.b[j] = INTER ? make_float2(at(4 * j + 1), at(4 * j + 3)) : make_float2(at(VEC + 2 * j), at(VEC + 2 * j + 1));
        }
    }
}
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void store_raw(T *row, int a, int b, int D, const Pairs<VEC> &x) {
    Run<T, VEC> lo, hi;
    if constexpr (VEC == 1) {
        lo.set2(0, x.a[0].x, 0.0f);
        hi.set2(0, x.b[0].x, 0.0f);
        lo.store(row + a);
        if (b < D) hi.store(row + b);
    } else {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            if (INTER) {
                Run<T, VEC> &run = 4 * j < VEC ? lo : hi;
                run.set2(4 * j % VEC, x.a[j].x, x.b[j].x);
                run.set2(4 * j % VEC + 2, x.a[j].y, x.b[j].y);
            } else {
                lo.set2(2 * j, x.a[j].x, x.a[j].y);
                hi.set2(2 * j, x.b[j].x, x.b[j].y);
            }
        }
        lo.store(row + a);
        hi.store(row + b);
    }
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// The frequency of pair j as a fraction of a turn per position, in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turns_of(const Params &p, int j) {
    const double t = static_cast<double>(p.freqs[j]) * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// The tokens t0 .. t0 + tok - 1 of a block, t0 moving on by `step` tokens at a time without a division.
struct Walk {
    unsigned t0, b0, s0, step, step_b, step_s;

    __device__ Walk(const Params &p, unsigned first, unsigned step_) : t0(first), step(step_) {
        b0 = t0 / p.S;
        s0 = t0 - b0 * p.S;
        step_b = step / p.S;
        step_s = step - step_b * p.S;
    }
    __device__ __forceinline__ void next(const Params &p) {
        t0 += step;
        b0 += step_b;
        s0 += step_s;
        if (s0 >= static_cast<unsigned>(p.S)) {
            s0 -= p.S;
            ++b0;
        }
    }
    // sequence and position in it of token t0 + i
    __device__ __forceinline__ void at(const Params &p, int i, unsigned &b, unsigned &s) const {
        b = b0;
        s = s0 + i;
        while (s >= static_cast<unsigned>(p.S)) {
            s -= p.S;
            ++b;
        }
    }
};

// One angle per thread (tok * half <= kThreads): thread i forms that of token i / half and pair i % half.
struct Angle {
    static constexpr int kLost = 1 << 16;
    int tl, j, slot;  // slot: plus kLost when the frequency is infinite or NaN, which fixed point cannot hold
    bool on;
    long long pos_off;
    unsigned long long turn;

    // A chunk's `vec` angles lie `half / vec` apart, so that neighbouring threads read neighbouring ones.
    __device__ Angle(const Params &p, int vec) {
        tl = threadIdx.x / p.half;
        j = threadIdx.x - tl * p.half;
        slot = tl * p.half + j % vec * (p.half / vec) + j / vec;
        on = tl < p.tok;
        pos_off = on ? p.axis[j] * p.pos_st[0] : 0;
        turn = on ? turns_of(p, j) : 0;
        if (on && !isfinite(p.freqs[j])) slot += kLost;
    }
    __device__ __forceinline__ int position(const Params &p, const Walk &w) const {
        if (!on || w.t0 + tl >= p.tokens) return 0;
        unsigned b, s;
        w.at(p, tl, b, s);
        return p.pos[pos_off + b * p.pos_st[1] + s * p.pos_st[2]];
    }
    // cos and sin into cs[token][pair]
    __device__ __forceinline__ void form(int pos, float2 *cs) const {
        // the product modulo 2^64 is the angle modulo a turn; its high word, read as signed, is in half turns
        const unsigned long long phase = turn * static_cast<unsigned long long>(static_cast<long long>(pos));
        // (the high 32 bits, rounded to 24: an angle is off by at most pi 2^-25, about a cosine's own rounding)
        const float half_turns = static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
        float sn, cn;
        sincospif(half_turns, &sn, &cn);
        if (slot >= kLost) cn = sn = NAN;
        if (on) cs[slot & (kLost - 1)] = make_float2(cn, sn);
    }
};

// cos and sin of the pairs of a chunk (1 and 0 where nothing is rotated), `step` = half / VEC.
template <int VEC>
__device__ __forceinline__ void chunk_angles(int chunk, bool in, const float2 *cs, int step, Pairs<VEC> &ang) {
#pragma unroll
    for (int j = 0; j < Pairs<VEC>::kN; ++j) {
        ang.a[j] = both(1.0f);
        ang.b[j] = both(0.0f);
        if (in) {
            const float2 p0 = cs[chunk + 2 * j * step], p1 = VEC > 1 ? cs[chunk + (2 * j + 1) * step] : p0;
            ang.a[j] = make_float2(p0.x, p1.x);
            ang.b[j] = make_float2(p0.y, p1.y);
        }
    }
}

// Sums of N values over the tpr lanes of a row (a power of two, aligned in the warp); the two usual widths unrolled.
template <int N, int LANES>
__device__ __forceinline__ void row_sums_of(float (&v)[N]) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int tpr) {
    if (tpr == 8) {
        row_sums_of<N, 8>(v);
    } else if (tpr == 16) {
        row_sums_of<N, 16>(v);
    } else {
        for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
}

// NC: chunks per thread (4 covers D = 256 in single elements).
template <typename T, int VEC, int NC, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, NC > 1 ? 1 : 3) fwd_kernel(const __grid_constant__ Params p) {
    using P = Pairs<VEC>;
    __shared__ float2 cs[2][kThreads];  // [tok][half] of this group of tokens and of the next
    extern __shared__ __align__(16) uint8_t ring_mem[];
    Ring<T, VEC, 2 * NC, kAhead> ring(ring_mem);
    const int per_head = p.tpr * p.tok;
    const int hs = threadIdx.x / per_head;
    const int r = threadIdx.x - hs * per_head;
    const int tl = r / p.tpr, lane_c = r - tl * p.tpr;
    const Angle angle(p, VEC);
    int at_a[NC], at_b[NC];  // where this thread's runs start in a row
    bool has[NC], turn[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
        has[c] = lane_c + c * p.tpr < p.chunks;
        turn[c] = has[c] && ch.turn;
        at_a[c] = ch.a;
        at_b[c] = ch.b;
    }
    const float inv_d = 1.0f / static_cast<float>(p.D), eps = p.eps;
    // (copies: the loop's asm statements would have every use of p read again)
    const int tpr = p.tpr, D = p.D, tokens = static_cast<int>(p.tokens), step_cs = p.half / VEC;
    // A token's rows in rounds: round i takes heads hs + i * p.heads of Q, then the K rounds those of K; the rounds
    // are the same for every thread of the block (the norm shuffles), some threads have no row in the last ones.
    const int rounds_q = (p.H + p.heads - 1) / p.heads, rounds = rounds_q + (p.H_kv + p.heads - 1) / p.heads;
    const int rows_q = hs < p.H ? (p.H - hs + p.heads - 1) / p.heads : 0;
    const int rows_k = hs < p.H_kv ? (p.H_kv - hs + p.heads - 1) / p.heads : 0;

    const bool row_thread = hs < p.heads && has[0];

    // ---- the loads' own walk over groups, tensors and rounds, kAhead rows in front
    Walk ahead(p, blockIdx.x * p.tok, gridDim.x * p.tok);
    int ahead_which = 1, ahead_rounds = 0, ahead_rows = 0;  // tensor, its rounds left, this thread's rows left
    long long ahead_step = 0;
    const T *ahead_at = nullptr;
    auto ahead_next = [&](bool move) {  // on to the next tensor with rounds: K after Q, the next group's Q after K
        do {
            ahead_which ^= 1;
            if (ahead_which == 0 && move) ahead.next(p);
            move = true;
            ahead_rounds = ahead_which ? rounds - rounds_q : rounds_q;
        } while (ahead_rounds == 0);
        const int w = ahead_which;
        unsigned b = 0, s = 0;
        const bool in = row_thread && static_cast<int>(ahead.t0 + tl) < tokens;
        if (in) ahead.at(p, tl, b, s);
        ahead_rows = in ? (w ? rows_k : rows_q) : 0;
        ahead_step = p.heads * p.x_st[w][1];
        ahead_at = static_cast<const T *>(p.x[w]) + b * p.x_st[w][0] + s * p.x_st[w][2] + hs * p.x_st[w][1];
    };
    auto fetch = [&]() {
        if (ahead_rows > 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (NC == 1 || has[c]) {
                    ring.fetch(2 * c, ahead_at + at_a[c]);
                    if (VEC > 1 || at_b[c] < D) ring.fetch(2 * c + 1, ahead_at + at_b[c]);
                }
        }
        ring.pushed();
        --ahead_rows;
        ahead_at += ahead_step;
        if (--ahead_rounds == 0) ahead_next(true);
    };
    Walk walk = ahead;
    ahead_next(false);
    int pos_next = angle.position(p, walk);
#pragma unroll 1
    for (int i = 0; i < kAhead - 1; ++i) fetch();
    angle.form(pos_next, cs[0]);
    Walk after = walk;
    after.next(p);
    pos_next = after.t0 < p.tokens ? angle.position(p, after) : 0;

    for (int group = 0; walk.t0 < p.tokens; walk.next(p), ++group) {
        __syncthreads();  // this group's angles are there, and the previous group's have been read
        if (after.t0 < p.tokens) {
            angle.form(pos_next, cs[(group + 1) & 1]);
            after.next(p);
            if (after.t0 < p.tokens) pos_next = angle.position(p, after);
        }
        // (threads without a row take part in the shuffles of the norm)
        const bool live = hs < p.heads && static_cast<int>(walk.t0 + tl) < tokens;
        unsigned b = 0, s = 0;
        if (live) walk.at(p, tl, b, s);
        // the cache row of this token's K and V: written when 0 <= row < cap
        long long row_kv = s;
        bool write_kv = live;
        if (p.kv_len) {
            row_kv = live ? static_cast<long long>(p.kv_len[b]) - p.S + s : -1;
            write_kv = row_kv >= 0 && row_kv < p.cap;
            if (row_kv >= p.cap && lane_c == 0 && hs == 0) atomicOr(p.status, kStatusBounds);
        }

#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const int n = which ? rounds - rounds_q : rounds_q;
            const int mine = has[0] ? (which ? (write_kv ? rows_k : 0) : (live ? rows_q : 0)) : 0;  // rows to write
            T *dst = static_cast<T *>(p.y[which]) + b * p.y_st[which][0] + (which ? row_kv : s) * p.y_st[which][2] +
                     hs * p.y_st[which][1];
            const long long y_step = p.heads * p.y_st[which][1];
            // y_a = a (w_a cos) - b (w_b sin), y_b = a (w_a sin) + b (w_b cos): the weights go into the coefficients
            P ac_bs[NC], as_bc[NC];
            const T *wp = static_cast<const T *>(p.w[which]);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                P ang, w;
                chunk_angles<VEC>(lane_c + c * tpr, live && turn[c], cs[group & 1] + tl * p.half, step_cs, ang);
#pragma unroll
                for (int j = 0; j < P::kN; ++j) w.a[j] = w.b[j] = both(1.0f);
                if (NORM && wp && has[c]) {
                    Raw<T, VEC> raw;
                    raw.zero();
                    load_raw<T, VEC>(raw, wp, at_a[c], at_b[c], p.D);
                    unpack<T, VEC, INTER>(raw, w);
                }
#pragma unroll
                for (int j = 0; j < P::kN; ++j) {
                    ac_bs[c].a[j] = NORM ? mul2(w.a[j], ang.a[j]) : ang.a[j];
                    ac_bs[c].b[j] = NORM ? mul2(w.b[j], neg2(ang.b[j])) : neg2(ang.b[j]);
                    as_bc[c].a[j] = NORM ? mul2(w.a[j], ang.b[j]) : ang.b[j];
                    as_bc[c].b[j] = NORM ? mul2(w.b[j], ang.a[j]) : ang.a[j];
                }
            }
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                fetch();
                cp_async_wait<kAhead - 1>();
                P x[NC];
                float2 ss = both(0.0f);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    Raw<T, VEC> raw;
                    ring.take(2 * c, raw.lo);
                    ring.take(2 * c + 1, raw.hi);
                    if (VEC == 1 && at_b[c] >= D) raw.hi.zero();
                    unpack<T, VEC, INTER>(raw, x[c]);
                    if (NORM && has[c]) {
#pragma unroll
                        for (int j = 0; j < P::kN; ++j) ss = fma2(x[c].a[j], x[c].a[j], fma2(x[c].b[j], x[c].b[j], ss));
                    }
                }
                ring.popped();
                if (NORM) {
                    float sum[1] = {ss.x + ss.y};
                    row_sums(sum, tpr);
                    const float2 rs = both(rsqrtf(sum[0] * inv_d + eps));
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int j = 0; j < P::kN; ++j) {
                            x[c].a[j] = mul2(x[c].a[j], rs);
                            x[c].b[j] = mul2(x[c].b[j], rs);
                        }
                }
                if (i < mine) {
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        P y;
                        if (turn[c]) {
#pragma unroll
                            for (int j = 0; j < P::kN; ++j) {
                                y.a[j] = fma2(x[c].a[j], ac_bs[c].a[j], mul2(x[c].b[j], ac_bs[c].b[j]));
                                y.b[j] = fma2(x[c].a[j], as_bc[c].a[j], mul2(x[c].b[j], as_bc[c].b[j]));
                            }
                        } else {  // columns of their own: 0 times another's infinity would be NaN
#pragma unroll
                            for (int j = 0; j < P::kN; ++j) {
                                y.a[j] = mul2(x[c].a[j], ac_bs[c].a[j]);
                                y.b[j] = mul2(x[c].b[j], as_bc[c].b[j]);
                            }
                        }
                        if (NC == 1 || has[c]) store_raw<T, VEC, INTER>(dst, at_a[c], at_b[c], D, y);
                    }
                }
                dst += y_step;
            }
        }

        if (p.kv_len && p.v && write_kv) {  // V rows are copied, 16 bytes at a time (rows start on 16 bytes)
            constexpr int N = 16 / sizeof(T);
            const T *v0 = static_cast<const T *>(p.v) + b * p.v_st[0] + s * p.v_st[2];
            T *o0 = static_cast<T *>(p.v_out) + b * p.vo_st[0] + row_kv * p.vo_st[2];
            for (int h = hs; h < p.H_kv; h += p.heads)
                for (int e = lane_c * N; e < p.D_v; e += p.tpr * N) {
                    const T *from = v0 + h * p.v_st[1] + e;
                    T *to = o0 + h * p.vo_st[1] + e;
                    if (e + N <= p.D_v) {
                        *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
                    } else {
                        for (int i = 0; i < p.D_v - e; ++i) to[i] = from[i];
                    }
                }
        }
    }
    cp_async_wait<0>();
}

// Backward: dx from the gradient's inverse rotation; a block works on Q or on K, so that one set of weight-gradient
// sums lives in its registers, and leaves its sum of u z per column (see include/vt_attn.h) in its part[], summed in
// a fixed order.  Both means of a row, of x^2 and of w u x, are taken in one pass of shuffles.
template <typename T, int VEC, int NC, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, NC == 1 ? 2 : 1) bwd_kernel(const __grid_constant__ Params p) {
    using P = Pairs<VEC>;
    constexpr int kRuns = (NORM ? 4 : 2) * NC;
    __shared__ float2 cs[2][kThreads];  // [tok][half] of this group of tokens and of the next
    // the ring, and after the loop the weight gradients: float [kThreads / tpr][D]
    extern __shared__ __align__(16) uint8_t ring_mem[];
    Ring<T, VEC, kRuns, kAheadBwd> ring(ring_mem);
    if (NORM) launch_dependents();  // the launch that adds the blocks' sums waits for them
    const int which = blockIdx.x >= static_cast<unsigned>(p.blocks_q);
    const unsigned block = blockIdx.x - (which ? p.blocks_q : 0);
    const unsigned n_blocks = which ? gridDim.x - p.blocks_q : p.blocks_q;
    const int heads = which ? p.H_kv : p.H;
    const int per_head = p.tpr * p.tok;
    const int hs = threadIdx.x / per_head;
    const int r = threadIdx.x - hs * per_head;
    const int tl = r / p.tpr, lane_c = r - tl * p.tpr;
    const Angle angle(p, VEC);
    int at_a[NC], at_b[NC];
    bool has[NC], turn[NC];
    P w[NC], dw[NC];
    const T *wp = static_cast<const T *>(p.w[which]);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
        has[c] = lane_c + c * p.tpr < p.chunks;
        turn[c] = has[c] && ch.turn;
        at_a[c] = ch.a;
        at_b[c] = ch.b;
        if (NORM) {
#pragma unroll
            for (int j = 0; j < P::kN; ++j) {
                w[c].a[j] = w[c].b[j] = both(1.0f);
                dw[c].a[j] = dw[c].b[j] = both(0.0f);
            }
            if (wp && has[c]) {
                Raw<T, VEC> raw;
                raw.zero();
                load_raw<T, VEC>(raw, wp, at_a[c], at_b[c], p.D);
                unpack<T, VEC, INTER>(raw, w[c]);
            }
        }
    }
    const int rounds = (heads + p.heads - 1) / p.heads;  // the same for the whole block: the norm shuffles
    const int rows_of = hs < heads ? (heads - hs + p.heads - 1) / p.heads : 0;
    const float inv_d = 1.0f / static_cast<float>(p.D), eps = p.eps;
    // (copies: the loop's asm statements would have every use of p read again)
    const int tpr = p.tpr, D = p.D, tokens = static_cast<int>(p.tokens), step_cs = p.half / VEC;
    const long long g_step = p.heads * p.g_st[which][1], x_step = p.heads * p.x_st[which][1];
    const long long y_step = p.heads * p.y_st[which][1];
    const bool row_thread = hs < p.heads && has[0];

    // ---- the loads' own walk, kAheadBwd rows in front
    Walk ahead(p, block * p.tok, n_blocks * p.tok);
    int ahead_rounds = 0, ahead_rows = 0;  // rounds left in the group, this thread's rows left
    const T *ahead_g = nullptr, *ahead_x = nullptr;
    auto ahead_group = [&]() {
        unsigned b = 0, s = 0;
        const bool in = row_thread && static_cast<int>(ahead.t0 + tl) < tokens;
        if (in) ahead.at(p, tl, b, s);
        ahead_rounds = rounds;
        ahead_rows = in ? rows_of : 0;
        ahead_g = static_cast<const T *>(p.g[which]) + b * p.g_st[which][0] + s * p.g_st[which][2] + hs * p.g_st[which][1];
        ahead_x = static_cast<const T *>(p.x[which]) + b * p.x_st[which][0] + s * p.x_st[which][2] + hs * p.x_st[which][1];
    };
    auto fetch = [&]() {
        if (ahead_rows > 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (NC == 1 || has[c]) {
                    const bool two = VEC > 1 || at_b[c] < D;
                    ring.fetch(2 * c, ahead_g + at_a[c]);
                    if (two) ring.fetch(2 * c + 1, ahead_g + at_b[c]);
                    if (NORM) {
                        ring.fetch(2 * (NC + c), ahead_x + at_a[c]);
                        if (two) ring.fetch(2 * (NC + c) + 1, ahead_x + at_b[c]);
                    }
                }
        }
        ring.pushed();
        --ahead_rows;
        ahead_g += g_step;
        if (NORM) ahead_x += x_step;
        if (--ahead_rounds == 0) {
            ahead.next(p);
            ahead_group();
        }
    };
    Walk walk = ahead;
    ahead_group();
    int pos_next = angle.position(p, walk);
#pragma unroll 1
    for (int i = 0; i < kAheadBwd - 1; ++i) fetch();
    angle.form(pos_next, cs[0]);
    Walk after = walk;
    after.next(p);
    pos_next = after.t0 < p.tokens ? angle.position(p, after) : 0;

    for (int group = 0; walk.t0 < p.tokens; walk.next(p), ++group) {
        __syncthreads();  // this group's angles are there, and the previous group's have been read
        if (after.t0 < p.tokens) {
            angle.form(pos_next, cs[(group + 1) & 1]);
            after.next(p);
            if (after.t0 < p.tokens) pos_next = angle.position(p, after);
        }
        const bool live = row_thread && static_cast<int>(walk.t0 + tl) < tokens;
        unsigned b = 0, s = 0;
        if (live) walk.at(p, tl, b, s);
        T *y = static_cast<T *>(p.y[which]) + b * p.y_st[which][0] + s * p.y_st[which][2] + hs * p.y_st[which][1];
        const int mine = live ? rows_of : 0;  // rows to write
        P ang[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            chunk_angles<VEC>(lane_c + c * tpr, live && turn[c], cs[group & 1] + tl * p.half, step_cs, ang[c]);
#pragma unroll 1
        for (int i = 0; i < rounds; ++i) {
            fetch();
            cp_async_wait<kAheadBwd - 1>();
            P u[NC], z[NC];
            float2 ss = both(0.0f), dot = both(0.0f);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                Raw<T, VEC> raw;
                P gv;
                ring.take(2 * c, raw.lo);
                ring.take(2 * c + 1, raw.hi);
                if (i >= mine || (NC > 1 && !has[c])) raw.zero();  // no row: nothing may come of what the ring holds
                if (VEC == 1 && at_b[c] >= D) raw.hi.zero();
                unpack<T, VEC, INTER>(raw, gv);
                if (NORM) {
                    ring.take(2 * (NC + c), raw.lo);
                    ring.take(2 * (NC + c) + 1, raw.hi);
                    if (i >= mine || (NC > 1 && !has[c])) raw.zero();
                    if (VEC == 1 && at_b[c] >= D) raw.hi.zero();
                    unpack<T, VEC, INTER>(raw, z[c]);
                }
                if (turn[c]) {
#pragma unroll
                    for (int j = 0; j < P::kN; ++j) {
                        u[c].a[j] = fma2(gv.a[j], ang[c].a[j], mul2(gv.b[j], ang[c].b[j]));
                        u[c].b[j] = fma2(gv.b[j], ang[c].a[j], mul2(gv.a[j], neg2(ang[c].b[j])));
                    }
                } else {
                    u[c] = gv;
                }
            }
            ring.popped();
            if (NORM) {
                // z = rs x:  dx = rs (w u - z mean(w u z)),  dw += u z.  (rs^3 would leave fp32's range long before a row's
                // sum of squares does.)
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int j = 0; j < P::kN; ++j) {
                        ss = fma2(z[c].a[j], z[c].a[j], fma2(z[c].b[j], z[c].b[j], ss));
                        dot = fma2(mul2(w[c].a[j], u[c].a[j]), z[c].a[j],
                                   fma2(mul2(w[c].b[j], u[c].b[j]), z[c].b[j], dot));
                    }
                float sums[2] = {ss.x + ss.y, dot.x + dot.y};
                row_sums(sums, tpr);
                const float rs = rsqrtf(sums[0] * inv_d + eps);
                const float2 rs2 = both(rs), m2 = both(-(rs * sums[1]) * inv_d);
                if (i < mine) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int j = 0; j < P::kN; ++j) {
                            const float2 za = mul2(z[c].a[j], rs2), zb = mul2(z[c].b[j], rs2);
                            dw[c].a[j] = fma2(u[c].a[j], za, dw[c].a[j]);
                            dw[c].b[j] = fma2(u[c].b[j], zb, dw[c].b[j]);
                            u[c].a[j] = mul2(rs2, fma2(w[c].a[j], u[c].a[j], mul2(m2, za)));
                            u[c].b[j] = mul2(rs2, fma2(w[c].b[j], u[c].b[j], mul2(m2, zb)));
                        }
                }
            }
            if (i < mine) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (NC == 1 || has[c]) store_raw<T, VEC, INTER>(y, at_a[c], at_b[c], D, u[c]);
            }
            y += y_step;
        }
    }
    cp_async_wait<0>();

    if (!NORM || !p.part[which]) return;
    // the block's sums: rows of the block (same columns, other tokens and heads) are added in order
    float *sm = reinterpret_cast<float *>(ring_mem);
    const int rows = kThreads / p.tpr;
    const int row = threadIdx.x / p.tpr;
    __syncthreads();  // every thread is done with the ring
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (!has[c]) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int lo = INTER ? at_a[c] + 2 * i : at_a[c] + i, hi = INTER ? lo + 1 : at_b[c] + i;
            sm[row * p.D + lo] = i & 1 ? dw[c].a[i / 2].y : dw[c].a[i / 2].x;
            if (hi < p.D) sm[row * p.D + hi] = i & 1 ? dw[c].b[i / 2].y : dw[c].b[i / 2].x;
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
        float acc = 0.0f;
        for (int k = 0; k < rows; ++k) acc += sm[k * p.D + d];
        p.part[which][static_cast<long long>(block) * p.D + d] = acc;
    }
}

// Sum of the blocks' partial weight gradients, 8 columns of one tensor per block: 64 rows of 8 threads take every
// 64th partial with all their loads in flight, then the rows are added in order.
constexpr int kSumRows = 64;
__global__ void __launch_bounds__(8 * kSumRows) bwd_weights_kernel(const float *part_q, const float *part_k, float *dwq,
                                                                   float *dwk, int n_q, int n_k, int D) {
    __shared__ float sm[kSumRows][9];
    const float *part = blockIdx.y ? part_k : part_q;
    float *dw = blockIdx.y ? dwk : dwq;
    const int n = blockIdx.y ? n_k : n_q;
    const int lane = threadIdx.x & 7, row = threadIdx.x >> 3;
    const int d = blockIdx.x * 8 + lane;
    wait_prerequisites();
    if (!dw) return;
    float v[(kBwdMaxBlocks + kSumRows - 1) / kSumRows];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof v / sizeof v[0]); ++i) {
        const int k = row + i * kSumRows;
        v[i] = d < D && k < n ? part[static_cast<long long>(k) * D + d] : 0.0f;
    }
    float acc = 0.0f;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof v / sizeof v[0]); ++i) acc += v[i];
    sm[row][lane] = acc;
    __syncthreads();
    if (row == 0 && d < D) {
        float sum = 0.0f;
#pragma unroll 16
        for (int k = 0; k < kSumRows; ++k) sum += sm[k][lane];
        dw[d] = sum;
    }
}

}  // namespace rope
}  // namespace vt
