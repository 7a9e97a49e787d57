// Per-head norm and rotation of Q and K rows, and their gradients (formulas in include/vt_attn.h).
//
// Bound by HBM: a row is read once and written once (the backward reads it and its gradient), a handful of
// operations per element.  What the layout is for:
//   - A row is spread over `tpr` threads; each holds VEC elements of the row's rotated part and the VEC
//     elements they pair with, so a rotation needs no other thread and the norm's mean is a shuffle over tpr
//     lanes.  A thread keeps its token and its columns for every head it works on, so the cosines and sines
//     of its pairs live in registers.
//   - A block owns `tok` consecutive tokens (about one angle per thread) and walks over their heads.  The
//     angles are formed once per token and pair, in fp64 and reduced to (-1, 1] half turns before they are
//     rounded to fp32: fp32 products lose the phase of positions beyond a few thousand.
//   - VEC is 16 bytes when R and D allow it, else 8 bytes or single elements.
#pragma once

#include <cstdint>

#include "vt_attn_common.cuh"

namespace vt {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;
constexpr int kMaxD = 256;
constexpr int kBwdMaxBlocks = 608;  // blocks of a backward launch: 4 per SM, each leaves one partial weight gradient

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
    float *part[2];              // backward: partial weight gradients [blocks][D], or null
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

template <typename T>
struct Cvt;
template <>
struct Cvt<float> {
    __device__ static float in(float x) { return x; }
    __device__ static float out(float x) { return x; }
};
struct bf16 {
    uint16_t u;
};
template <>
struct Cvt<bf16> {
    __device__ static float in(bf16 x) { return __uint_as_float(static_cast<uint32_t>(x.u) << 16); }
    __device__ static bf16 out(float x) { return {static_cast<uint16_t>(pack_bf16x2(x, 0.0f) & 0xFFFFu)}; }
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T e[N];
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

// x[i] and x[VEC + i] are the members of pair i for i < VEC.
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void load_chunk(const T *row, const Chunk<VEC, INTER> &ch, int D, float (&x)[2 * VEC]) {
    Vec<T, VEC> lo, hi;
    if (VEC == 1) {  // single elements: an odd D ends inside a chunk
        lo.e[0] = row[ch.a];
        hi.e[0] = ch.b < D ? row[ch.b] : T{};
    } else {
        lo = *reinterpret_cast<const Vec<T, VEC> *>(row + ch.a);
        hi = *reinterpret_cast<const Vec<T, VEC> *>(row + ch.b);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (INTER) {
            x[i] = Cvt<T>::in(2 * i < VEC ? lo.e[2 * i] : hi.e[2 * i - VEC]);
            x[VEC + i] = Cvt<T>::in(2 * i + 1 < VEC ? lo.e[2 * i + 1] : hi.e[2 * i + 1 - VEC]);
        } else {
            x[i] = Cvt<T>::in(lo.e[i]);
            x[VEC + i] = Cvt<T>::in(hi.e[i]);
        }
    }
}

template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void store_chunk(T *row, const Chunk<VEC, INTER> &ch, int D, const float (&x)[2 * VEC]) {
    Vec<T, VEC> lo, hi;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (INTER) {
            (2 * i < VEC ? lo.e[2 * i] : hi.e[2 * i - VEC]) = Cvt<T>::out(x[i]);
            (2 * i + 1 < VEC ? lo.e[2 * i + 1] : hi.e[2 * i + 1 - VEC]) = Cvt<T>::out(x[VEC + i]);
        } else {
            lo.e[i] = Cvt<T>::out(x[i]);
            hi.e[i] = Cvt<T>::out(x[VEC + i]);
        }
    }
    if (VEC == 1) {
        row[ch.a] = lo.e[0];
        if (ch.b < D) row[ch.b] = hi.e[0];
    } else {
        *reinterpret_cast<Vec<T, VEC> *>(row + ch.a) = lo;
        *reinterpret_cast<Vec<T, VEC> *>(row + ch.b) = hi;
    }
}

// cos and sin of every (token, pair) of the block's tokens, [tok][half].
__device__ __forceinline__ void block_angles(const Params &p, long long t0, float2 *cs) {
    const int n = p.tok * p.half;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int tl = i / p.half, j = i - tl * p.half;
        const long long t = t0 + tl;
        if (t >= p.tokens) continue;
        const long long b = t / p.S, s = t - b * p.S;
        const int pos = p.pos[p.axis[j] * p.pos_st[0] + b * p.pos_st[1] + s * p.pos_st[2]];
        double turn = static_cast<double>(pos) * static_cast<double>(p.freqs[j]) * 0.31830988618379067154;
        turn -= 2.0 * rint(0.5 * turn);
        float sn, cn;
        sincospif(static_cast<float>(turn), &sn, &cn);
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
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Params p) {
    extern __shared__ float2 cs[];
    const long long t0 = static_cast<long long>(blockIdx.x) * p.tok;
    block_angles(p, t0, cs);
    __syncthreads();

    const int per_head = p.tpr * p.tok;
    const int hs = threadIdx.x / per_head;
    const int r = threadIdx.x - hs * per_head;
    const int tl = r / p.tpr, lane_c = r - tl * p.tpr;
    const long long t = t0 + tl;
    // (threads without a row take part in the shuffles of the norm)
    const bool live = hs < p.heads && t < p.tokens;
    const long long b = live ? t / p.S : 0, s = live ? t - b * p.S : 0;

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

#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const int heads = which ? p.H_kv : p.H;
        const T *x0 = static_cast<const T *>(p.x[which]) + b * p.x_st[which][0] + s * p.x_st[which][2];
        T *y0 = static_cast<T *>(p.y[which]) + b * p.y_st[which][0] + (which ? row_kv : s) * p.y_st[which][2];
        float w[NC][2 * VEC];
        if (NORM) {
            const T *wp = static_cast<const T *>(p.w[which]);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const bool in = lane_c + c * p.tpr < p.chunks;
                const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
                if (wp && in) {
                    load_chunk<T, VEC, INTER>(wp, ch, p.D, w[c]);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) w[c][i] = 1.0f;
                }
            }
        }
        for (int h0 = 0; h0 < heads; h0 += p.heads) {
            const int h = h0 + hs;
            const bool on = live && h < heads;
            float x[NC][2 * VEC];
            float ss = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
                if (on && lane_c + c * p.tpr < p.chunks) {
                    load_chunk<T, VEC, INTER>(x0 + h * p.x_st[which][1], ch, p.D, x[c]);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) x[c][i] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) ss = fmaf(x[c][i], x[c][i], ss);
            }
            float rs = 1.0f;
            if (NORM) rs = rsqrtf(row_sum(ss, p.tpr) / static_cast<float>(p.D) + p.eps);
            if (!(which ? on && write_kv : on)) continue;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (lane_c + c * p.tpr >= p.chunks) continue;
                const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
                float y[2 * VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float u = NORM ? x[c][i] * rs * w[c][i] : x[c][i];
                    const float v = NORM ? x[c][VEC + i] * rs * w[c][VEC + i] : x[c][VEC + i];
                    y[i] = u * ang[c][i].x - v * ang[c][i].y;
                    y[VEC + i] = u * ang[c][i].y + v * ang[c][i].x;
                }
                store_chunk<T, VEC, INTER>(y0 + h * p.y_st[which][1], ch, p.D, y);
            }
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
                    *reinterpret_cast<Vec<T, N> *>(dst) = *reinterpret_cast<const Vec<T, N> *>(src);
                } else {
                    for (int i = 0; i < p.D_v - e; ++i) dst[i] = src[i];
                }
            }
    }
}

// Backward: dx from the gradient's inverse rotation; each block leaves its sum of u z per column (see
// include/vt_attn.h) in part[which][block], summed in a fixed order.
template <typename T, int VEC, int NC, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const Params p) {
    extern __shared__ float2 cs[];  // [tok][half], then (weight gradients) float [kThreads / tpr][D] over it
    const int per_head = p.tpr * p.tok;
    const int hs = threadIdx.x / per_head;
    const int r = threadIdx.x - hs * per_head;
    const int tl = r / p.tpr, lane_c = r - tl * p.tpr;

    float dw[2][NC][2 * VEC];
    if (NORM) {
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) dw[which][c][i] = 0.0f;
    }

    const long long blocks = (p.tokens + p.tok - 1) / p.tok;
    for (long long tb = blockIdx.x; tb < blocks; tb += gridDim.x) {
        const long long t0 = tb * p.tok;
        __syncthreads();  // the previous tokens' angles have been read
        block_angles(p, t0, cs);
        __syncthreads();
        const long long t = t0 + tl;
        const bool live = hs < p.heads && t < p.tokens;
        const long long b = live ? t / p.S : 0, s = live ? t - b * p.S : 0;
        float2 ang[NC][VEC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
            const bool in = live && lane_c + c * p.tpr < p.chunks && ch.turn;
#pragma unroll
            for (int i = 0; i < VEC; ++i) ang[c][i] = in ? cs[tl * p.half + ch.pair() + i] : make_float2(1.0f, 0.0f);
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int heads = which ? p.H_kv : p.H;
            const T *x0 = static_cast<const T *>(p.x[which]) + b * p.x_st[which][0] + s * p.x_st[which][2];
            const T *g0 = static_cast<const T *>(p.g[which]) + b * p.g_st[which][0] + s * p.g_st[which][2];
            T *y0 = static_cast<T *>(p.y[which]) + b * p.y_st[which][0] + s * p.y_st[which][2];
            const T *wp = static_cast<const T *>(p.w[which]);
            for (int h0 = 0; h0 < heads; h0 += p.heads) {
                const int h = h0 + hs;
                const bool on = live && h < heads;
                float u[NC][2 * VEC], x[NC][2 * VEC];
                float ss = 0.0f;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
                    float g[2 * VEC];
                    const bool in = on && lane_c + c * p.tpr < p.chunks;
                    if (in) {
                        load_chunk<T, VEC, INTER>(g0 + h * p.g_st[which][1], ch, p.D, g);
                        if (NORM) load_chunk<T, VEC, INTER>(x0 + h * p.x_st[which][1], ch, p.D, x[c]);
                    }
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        u[c][i] = in ? g[i] * ang[c][i].x + g[VEC + i] * ang[c][i].y : 0.0f;
                        u[c][VEC + i] = in ? g[VEC + i] * ang[c][i].x - g[i] * ang[c][i].y : 0.0f;
                    }
                    if (NORM) {
#pragma unroll
                        for (int i = 0; i < 2 * VEC; ++i) {
                            x[c][i] = in ? x[c][i] : 0.0f;
                            ss = fmaf(x[c][i], x[c][i], ss);
                        }
                    }
                }
                if (NORM) {
                    const float rs = rsqrtf(row_sum(ss, p.tpr) / static_cast<float>(p.D) + p.eps);
                    float dot = 0.0f;
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
                        const bool in = lane_c + c * p.tpr < p.chunks;
                        float w[2 * VEC];
                        if (wp && in) {
                            load_chunk<T, VEC, INTER>(wp, ch, p.D, w);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2 * VEC; ++i) w[i] = 1.0f;
                        }
#pragma unroll
                        for (int i = 0; i < 2 * VEC; ++i) {
                            x[c][i] *= rs;  // z
                            dw[which][c][i] = fmaf(u[c][i], x[c][i], dw[which][c][i]);
                            u[c][i] *= w[i];
                            dot = fmaf(u[c][i], x[c][i], dot);
                        }
                    }
                    const float mean = row_sum(dot, p.tpr) / static_cast<float>(p.D);
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int i = 0; i < 2 * VEC; ++i) u[c][i] = rs * (u[c][i] - x[c][i] * mean);
                }
                if (!on) continue;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if (lane_c + c * p.tpr >= p.chunks) continue;
                    const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
                    store_chunk<T, VEC, INTER>(y0 + h * p.y_st[which][1], ch, p.D, u[c]);
                }
            }
        }
    }

    if (!NORM) return;
    // the block's sums: rows of the block (same columns, other tokens and heads) are added in order
    float *sm = reinterpret_cast<float *>(cs);
    const int rows = kThreads / p.tpr;
    const int row = threadIdx.x / p.tpr;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!p.part[which]) continue;
        __syncthreads();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (lane_c + c * p.tpr >= p.chunks) continue;
            const Chunk<VEC, INTER> ch(p, lane_c + c * p.tpr);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int lo = INTER ? ch.a + 2 * i : ch.a + i, hi = INTER ? lo + 1 : ch.b + i;
                sm[row * p.D + lo] = dw[which][c][i];
                if (hi < p.D) sm[row * p.D + hi] = dw[which][c][VEC + i];
            }
        }
        __syncthreads();
        for (int d = threadIdx.x; d < p.D; d += kThreads) {
            float acc = 0.0f;
            for (int k = 0; k < rows; ++k) acc += sm[k * p.D + d];
            p.part[which][static_cast<long long>(blockIdx.x) * p.D + d] = acc;
        }
    }
}

// Sum of the blocks' partial weight gradients, 32 columns of one tensor per block: 32 rows of threads take
// every 32nd partial, then the rows are added in order.
__global__ void __launch_bounds__(1024) bwd_weights_kernel(const float *part_q, const float *part_k, float *dwq,
                                                           float *dwk, int n, int D) {
    __shared__ float sm[32][33];
    const float *part = blockIdx.y ? part_k : part_q;
    float *dw = blockIdx.y ? dwk : dwq;
    if (!dw) return;
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane;
    float acc = 0.0f;
    if (d < D)
        for (int k = row; k < n; k += 32) acc += part[static_cast<long long>(k) * D + d];
    sm[row][lane] = acc;
    __syncthreads();
    if (row == 0 && d < D) {
        float sum = 0.0f;
        for (int k = 0; k < 32; ++k) sum += sm[k][lane];
        dw[d] = sum;
    }
}

}  // namespace rope
}  // namespace vt
