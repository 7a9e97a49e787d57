// Per-head norm and rotation of Q and K rows, and their gradients (formulas in include/vt_attn.h).
//
// Bound by HBM: a row is read once and written once (the backward reads it and its gradient), a handful of
// operations per element.  What the layout is for:
//   - A row is spread over `tpr` threads; each holds VEC elements of the row's rotated part and the VEC
//     elements they pair with, so a rotation needs no other thread and the norm's mean is a shuffle over tpr
//     lanes.  A thread keeps its token and its columns for every head it works on, so the cosines and sines
//     of its pairs live in registers.
//   - A block owns `tok` consecutive tokens (about one angle per thread) and walks over their heads, Q's and then
//     K's, with the next rows' loads in flight while it works on the current ones (kAhead rows a thread): one row per
//     thread keeps too few bytes in flight to cover the memory's latency.
//   - Angles are formed once per token and pair as 64-bit fixed-point fractions of a turn: the position times the
//     frequency in turns, whose overflow is the reduction by whole turns.  fp32 products lose the phase of
//     positions beyond a few thousand, and fp64 ones keep the (slow) fp64 pipe busy for longer than the loads take
//     when few heads share a token.
//   - VEC is 16 bytes when R and D allow it, else 8 bytes or single elements.
#pragma once

#include <cstdint>

#include "vt_attn_common.cuh"

namespace vt {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;
constexpr int kMaxD = 256;
constexpr int kBwdMaxBlocks = 608;  // blocks of a backward launch, each leaves one partial weight gradient
constexpr int kAhead = 2;           // rows a thread has in flight besides the current one

struct Params {
    int B, H, H_kv, S, D, half;  // half = R / 2
    int tpr, tok, heads;         // threads per row, tokens per block, heads a block works on at once
    int chunks;                  // chunks of 2 VEC elements in a row
    long long tokens;            // B * S
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
    // pair index of the chunk's first pair
    __device__ int pair() const { return INTER ? a / 2 : a; }
};

// A chunk as it lies in memory.
template <typename T, int VEC>
struct Raw {
    Run<T, VEC> lo, hi;
};
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void load_raw(Raw<T, VEC> &r, const T *row, const Chunk<VEC, INTER> &ch, int D) {
    r.lo.load(row + ch.a);
    if (VEC > 1 || ch.b < D) r.hi.load(row + ch.b);  // (in single elements an odd D ends inside a chunk)
    else r.hi.zero();
}
// x[i] and x[VEC + i] are the members of pair i for i < VEC.
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void unpack(const Raw<T, VEC> &r, float (&x)[2 * VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (INTER) {
            x[i] = 2 * i < VEC ? r.lo.get(2 * i) : r.hi.get(2 * i - VEC);
            x[VEC + i] = 2 * i + 1 < VEC ? r.lo.get(2 * i + 1) : r.hi.get(2 * i + 1 - VEC);
        } else {
            x[i] = r.lo.get(i);
            x[VEC + i] = r.hi.get(i);
        }
    }
}
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void store_chunk(T *row, const Chunk<VEC, INTER> &ch, int D, const float (&x)[2 * VEC]) {
    Run<T, VEC> lo, hi;
    if constexpr (VEC == 1) {
        lo.set2(0, x[0], 0.0f);
        hi.set2(0, x[1], 0.0f);
        lo.store(row + ch.a);
        if (ch.b < D) hi.store(row + ch.b);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            if (INTER) {
                lo.set2(i, x[i / 2], x[VEC + i / 2]);
                hi.set2(i, x[VEC / 2 + i / 2], x[VEC + VEC / 2 + i / 2]);
            } else {
                lo.set2(i, x[i], x[i + 1]);
                hi.set2(i, x[VEC + i], x[VEC + i + 1]);
            }
        }
        lo.store(row + ch.a);
        hi.store(row + ch.b);
    }
}

// The frequency of pair j as a fraction of a turn per position, in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turns_of(const Params &p, int j) {
    const double t = static_cast<double>(p.freqs[j]) * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// cos and sin of every (token, pair) of the block's tokens, [tok][half]; `turns` holds turns_of every pair.
__device__ __forceinline__ void block_angles(const Params &p, long long t0, const unsigned long long *turns, float2 *cs) {
    const int n = p.tok * p.half;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int tl = i / p.half, j = i - tl * p.half;
        const long long t = t0 + tl;
        if (t >= p.tokens) continue;
        const int b = static_cast<int>(t / p.S), s = static_cast<int>(t - static_cast<long long>(b) * p.S);
        const int pos = p.pos[p.axis[j] * p.pos_st[0] + b * p.pos_st[1] + s * p.pos_st[2]];
        // the product modulo 2^64 is the angle modulo a turn; its high word, read as signed, is in half turns
        const unsigned long long phase = turns[j] * static_cast<unsigned long long>(static_cast<long long>(pos));
        const float half_turns = static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
        float sn, cn;
        sincospif(half_turns, &sn, &cn);
        cs[i] = make_float2(cn, sn);
    }
}

// Sum over the tpr lanes of a row (a power of two, aligned in the warp).
__device__ __forceinline__ float row_sum(float v, int tpr) {
    for (int o = tpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// NC: chunks per thread (4 covers D = 256 in single elements).
template <typename T, int VEC, int NC, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, NC == 1 ? 3 : 1) fwd_kernel(const __grid_constant__ Params p) {
    extern __shared__ float2 cs[];  // [tok][half], then turns_of every pair
    unsigned long long *turns = reinterpret_cast<unsigned long long *>(cs + p.tok * p.half);
    const long long t0 = static_cast<long long>(blockIdx.x) * p.tok;
    const int per_head = p.tpr * p.tok;
    const int hs = threadIdx.x / per_head;
    const int r = threadIdx.x - hs * per_head;
    const int tl = r / p.tpr, lane_c = r - tl * p.tpr;
    const long long t = t0 + tl;
    // (threads without a row take part in the shuffles of the norm)
    const bool live = hs < p.heads && t < p.tokens;
    const int b = live ? static_cast<int>(t / p.S) : 0;
    const int s = live ? static_cast<int>(t - static_cast<long long>(b) * p.S) : 0;
    const int all_heads = p.H + p.H_kv;

    const T *q0 = static_cast<const T *>(p.x[0]) + b * p.x_st[0][0] + s * p.x_st[0][2];
    const T *k0 = static_cast<const T *>(p.x[1]) + b * p.x_st[1][0] + s * p.x_st[1][2];
    // row h of this token: Q's heads, then K's
    auto load_row = [&](int h, Raw<T, VEC> (&raw)[NC]) {
        const bool on = live && h < all_heads;
        const T *row = h < p.H ? q0 + h * p.x_st[0][1] : k0 + (h - p.H) * p.x_st[1][1];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (on && lane_c + c * p.tpr < p.chunks) {
                load_raw<T, VEC, INTER>(raw[c], row, Chunk<VEC, INTER>(p, lane_c + c * p.tpr), p.D);
            } else {
                raw[c].lo.zero();
                raw[c].hi.zero();
            }
        }
    };
    constexpr int kDepth = NC == 1 ? kAhead : 1;
    Raw<T, VEC> ahead[kDepth][NC];
#pragma unroll
    for (int i = 0; i < kDepth; ++i) load_row(hs + i * p.heads, ahead[i]);

    for (int j = threadIdx.x; j < p.half; j += kThreads) turns[j] = turns_of(p, j);
    __syncthreads();
    block_angles(p, t0, turns, cs);
    __syncthreads();
    float2 ang[NC][VEC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
        const bool in = live && lane_c + c * p.tpr < p.chunks && ch.turn;
#pragma unroll
        for (int i = 0; i < VEC; ++i) ang[c][i] = in ? cs[tl * p.half + ch.pair() + i] : make_float2(1.0f, 0.0f);
    }

    // the cache row of this token's K and V: written when 0 <= row < cap
    long long row_kv = s;
    bool write_kv = live;
    if (p.kv_len) {
        row_kv = live ? static_cast<long long>(p.kv_len[b]) - p.S + s : -1;
        write_kv = row_kv >= 0 && row_kv < p.cap;
        if (row_kv >= p.cap && lane_c == 0 && hs == 0) atomicOr(p.status, kStatusBounds);
    }
    T *qo = static_cast<T *>(p.y[0]) + b * p.y_st[0][0] + s * p.y_st[0][2];
    T *ko = static_cast<T *>(p.y[1]) + b * p.y_st[1][0] + row_kv * p.y_st[1][2];

    for (int h0 = 0; h0 < all_heads; h0 += p.heads) {
        const int h = h0 + hs;
        const bool is_q = h < p.H;
        float x[NC][2 * VEC];
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            unpack<T, VEC, INTER>(ahead[0][c], x[c]);
#pragma unroll
            for (int i = 0; i < 2 * VEC; ++i) ss = fmaf(x[c][i], x[c][i], ss);
        }
#pragma unroll
        for (int i = 0; i + 1 < kDepth; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) ahead[i][c] = ahead[i + 1][c];
        load_row(h + kDepth * p.heads, ahead[kDepth - 1]);
        float rs = 1.0f;
        if (NORM) rs = rsqrtf(row_sum(ss, p.tpr) / static_cast<float>(p.D) + p.eps);
        if (!(live && h < all_heads && (is_q || write_kv))) continue;
        T *row = is_q ? qo + h * p.y_st[0][1] : ko + (h - p.H) * p.y_st[1][1];
        const T *wp = static_cast<const T *>(is_q ? p.w[0] : p.w[1]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (lane_c + c * p.tpr >= p.chunks) continue;
            const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
            if (NORM) {
                if (wp) {
                    Raw<T, VEC> raw;
                    float w[2 * VEC];
                    load_raw<T, VEC, INTER>(raw, wp, ch, p.D);
                    unpack<T, VEC, INTER>(raw, w);
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) x[c][i] *= w[i];
                }
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) x[c][i] *= rs;
            }
            float y[2 * VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                y[i] = x[c][i] * ang[c][i].x - x[c][VEC + i] * ang[c][i].y;
                y[VEC + i] = x[c][i] * ang[c][i].y + x[c][VEC + i] * ang[c][i].x;
            }
            store_chunk<T, VEC, INTER>(row, ch, p.D, y);
        }
    }

    if (p.kv_len && p.v && write_kv) {  // V rows are copied, 16 bytes at a time (rows start on 16 bytes)
        constexpr int N = 16 / sizeof(T);
        const T *v0 = static_cast<const T *>(p.v) + b * p.v_st[0] + s * p.v_st[2];
        T *o0 = static_cast<T *>(p.v_out) + b * p.vo_st[0] + row_kv * p.vo_st[2];
        for (int h = hs; h < p.H_kv; h += p.heads)
            for (int e = lane_c * N; e < p.D_v; e += p.tpr * N) {
                const T *src = v0 + h * p.v_st[1] + e;
                T *dst = o0 + h * p.vo_st[1] + e;
                if (e + N <= p.D_v) {
                    *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(src);
                } else {
                    for (int i = 0; i < p.D_v - e; ++i) dst[i] = src[i];
                }
            }
    }
}

// Backward: dx from the gradient's inverse rotation; a block works on Q or on K, so that one set of weight-gradient
// sums lives in its registers, and leaves its sum of u z per column (see include/vt_attn.h) in its part[], summed in
// a fixed order.  Both means of a row, of x^2 and of w u x, are taken in one pass of shuffles.
template <typename T, int VEC, int NC, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, NC == 1 ? 2 : 1) bwd_kernel(const __grid_constant__ Params p) {
    extern __shared__ float2 cs[];  // [tok][half], turns_of every pair; then (weight gradients) float [kThreads / tpr][D]
    unsigned long long *turns = reinterpret_cast<unsigned long long *>(cs + p.tok * p.half);
    if (NORM) launch_dependents();  // the launch that adds the blocks' sums waits for them
    const int which = blockIdx.x >= static_cast<unsigned>(p.blocks_q);
    const int block = static_cast<int>(blockIdx.x) - (which ? p.blocks_q : 0);
    const int n_blocks = which ? static_cast<int>(gridDim.x) - p.blocks_q : p.blocks_q;
    const int heads = which ? p.H_kv : p.H;
    const int per_head = p.tpr * p.tok;
    const int hs = threadIdx.x / per_head;
    const int r = threadIdx.x - hs * per_head;
    const int tl = r / p.tpr, lane_c = r - tl * p.tpr;
    const T *x_base = static_cast<const T *>(p.x[which]), *g_base = static_cast<const T *>(p.g[which]);
    T *y_base = static_cast<T *>(p.y[which]);
    const T *wp = static_cast<const T *>(p.w[which]);

    for (int j = threadIdx.x; j < p.half; j += kThreads) turns[j] = turns_of(p, j);
    float dw[NC][2 * VEC];
    if (NORM) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 2 * VEC; ++i) dw[c][i] = 0.0f;
    }

    const long long groups = (p.tokens + p.tok - 1) / p.tok;
    for (long long tb = block; tb < groups; tb += n_blocks) {
        const long long t = tb * p.tok + tl;
        const bool live = hs < p.heads && t < p.tokens;
        const int b = live ? static_cast<int>(t / p.S) : 0;
        const int s = live ? static_cast<int>(t - static_cast<long long>(b) * p.S) : 0;
        const T *x0 = x_base + b * p.x_st[which][0] + s * p.x_st[which][2];
        const T *g0 = g_base + b * p.g_st[which][0] + s * p.g_st[which][2];
        T *y0 = y_base + b * p.y_st[which][0] + s * p.y_st[which][2];
        Raw<T, VEC> g_next[NC], x_next[NC];
        auto load_row = [&](int h) {
            const bool on = live && h < heads;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (on && lane_c + c * p.tpr < p.chunks) {
                    const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
                    load_raw<T, VEC, INTER>(g_next[c], g0 + h * p.g_st[which][1], ch, p.D);
                    if (NORM) load_raw<T, VEC, INTER>(x_next[c], x0 + h * p.x_st[which][1], ch, p.D);
                } else {
                    g_next[c].lo.zero();
                    g_next[c].hi.zero();
                    x_next[c].lo.zero();
                    x_next[c].hi.zero();
                }
            }
        };
        load_row(hs);
        __syncthreads();  // the frequencies are there, and the previous tokens' angles have been read
        block_angles(p, tb * p.tok, turns, cs);
        __syncthreads();
        float2 ang[NC][VEC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
            const bool in = live && lane_c + c * p.tpr < p.chunks && ch.turn;
#pragma unroll
            for (int i = 0; i < VEC; ++i) ang[c][i] = in ? cs[tl * p.half + ch.pair() + i] : make_float2(1.0f, 0.0f);
        }
        for (int h0 = 0; h0 < heads; h0 += p.heads) {
            const int h = h0 + hs;
            float u[NC][2 * VEC], x[NC][2 * VEC], w[NC][2 * VEC];
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float g[2 * VEC];
                unpack<T, VEC, INTER>(g_next[c], g);
                if (NORM) unpack<T, VEC, INTER>(x_next[c], x[c]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    u[c][i] = g[i] * ang[c][i].x + g[VEC + i] * ang[c][i].y;
                    u[c][VEC + i] = g[VEC + i] * ang[c][i].x - g[i] * ang[c][i].y;
                }
            }
            load_row(h + p.heads);
            if (NORM) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) w[c][i] = 1.0f;
                    if (wp && lane_c + c * p.tpr < p.chunks) {
                        Raw<T, VEC> raw;
                        load_raw<T, VEC, INTER>(raw, wp, Chunk<VEC, INTER>(p, lane_c + c * p.tpr), p.D);
                        unpack<T, VEC, INTER>(raw, w[c]);
                    }
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) {
                        ss = fmaf(x[c][i], x[c][i], ss);
                        dot = fmaf(w[c][i] * u[c][i], x[c][i], dot);
                    }
                }
                for (int o = p.tpr >> 1; o > 0; o >>= 1) {
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    dot += __shfl_xor_sync(0xffffffffu, dot, o);
                }
                const float rs = rsqrtf(ss / static_cast<float>(p.D) + p.eps);
                const float mean = dot * rs / static_cast<float>(p.D);  // of w u z
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) {
                        const float z = x[c][i] * rs;
                        dw[c][i] = fmaf(u[c][i], z, dw[c][i]);
                        u[c][i] = rs * (w[c][i] * u[c][i] - z * mean);
                    }
            }
            if (!(live && h < heads)) continue;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (lane_c + c * p.tpr >= p.chunks) continue;
                store_chunk<T, VEC, INTER>(y0 + h * p.y_st[which][1], Chunk<VEC, INTER>(p, lane_c + c * p.tpr), p.D, u[c]);
            }
        }
    }

    if (!NORM || !p.part[which]) return;
    // the block's sums: rows of the block (same columns, other tokens and heads) are added in order
    float *sm = reinterpret_cast<float *>(cs);
    const int rows = kThreads / p.tpr;
    const int row = threadIdx.x / p.tpr;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (lane_c + c * p.tpr >= p.chunks) continue;
        const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int lo = INTER ? ch.a + 2 * i : ch.a + i, hi = INTER ? lo + 1 : ch.b + i;
            sm[row * p.D + lo] = dw[c][i];
            if (hi < p.D) sm[row * p.D + hi] = dw[c][VEC + i];
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
