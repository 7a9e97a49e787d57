// Attention over packed sequences and its gradients, fp32 (contracts in include/vt_attn.h, vt_attn_fwd_packed and
// vt_attn_bwd_packed).  The form for checks and small models: products of two TF32 parts per operand (three MMAs, 21 bits
// of every factor), on mma.sync, whose accumulators' layout lets the scores be the next product's A operand as they lie.
//
// A CTA takes 64 rows of one head (queries, or keys for dK and dV), 16 per warp, and walks the other side in tiles, which
// all warps copy to shared memory one tile ahead.  Rows behind a sequence's end and columns behind D are zeros there.
//
// Shared memory rows are DP floats in 16-byte units, unit u of row r at u ^ swizzle(r).  An MMA's k index may run over the
// columns, and its n index over the rows, in any order that both operands share, so every fragment is a 16-byte load:
//   A B^T (dot): k = t, t + 4 of two steps are columns 4 t, + 1 and 4 t + 2, + 3 of 16; row g of an 8-row tile is row
//   order(g) = g / 2 + 4 (g & 1), so that a thread's accumulators 2 t, 2 t + 1 belong to rows t and t + 4;
//   P B (acc): these rows are k = t, t + 4; n = g of four column tiles is column 4 g + m of 32, so a thread's results are
//   8 consecutive columns 8 t .. 8 t + 7.
// Both loads fall into different banks (swizzle gives 8 lanes' units different low bits).
// Measured (widths 72 on rows of 96): five sequences of 100 to 1000 tokens, 8 heads, 127 to 134 us (26 TFLOP/s; the SMs that
// hold two CTAs of the longest one end last); gradients of three of 77 to 500, window 128: 78 us, 56 of them the keys' walk.
// With 32 rows a CTA and 16-row tiles the forward took 195 us where this took 152 (fewer independent products per warp).
// Errors (norms, random inputs): O 4e-7, dQ and dK 4.6e-7.
#pragma once

#include "vt_attn_bwd_bf16.cuh"
#include "vt_attn_stream.cuh"

namespace vt {

struct PackedF32Params : BwdParams {
    const void *K;
    long long k_sh, k_ss;
};

namespace pf {

constexpr int kThreads = 128;
constexpr int kRows = 64;                         // rows of a CTA
constexpr int kFwdTile = 32, kBwdTile = 16;       // rows of the other side at a time: two CTAs on an SM with each

__device__ __forceinline__ int order(int g) { return (g >> 1) + ((g & 1) << 2); }
__device__ __forceinline__ int swizzle(int r) { return ((r & 3) << 1) ^ (r & 4); }

template <int DP>
__device__ __forceinline__ uint32_t unit_at(int r, int u) {
    return static_cast<uint32_t>(r) * (DP * 4) + ((u ^ swizzle(r)) << 4);
}
__device__ __forceinline__ float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// Rows row0 .. row0 + n - 1 (those below `end`) of D columns into shared memory, by all threads.
template <int DP>
__device__ __forceinline__ void copy_rows(uint32_t dst, const float *src, long long ss, int row0, int n, int end, int D) {
    for (int i = threadIdx.x; i < n * (DP / 4); i += kThreads) {
        const int r = i / (DP / 4), u = i - r * (DP / 4);
        const int bytes = row0 + r < end ? min(16, max(0, (D - 4 * u) * 4)) : 0;
        cp_async16(dst + unit_at<DP>(r, u), bytes > 0 ? src + (row0 + r) * ss + 4 * u : src, bytes);
    }
}

// x as hi + lo: hi rounded to TF32 (10 explicit mantissa bits) in integers, lo the rest, of which the tensor core takes the
// upper bits: what is left out is below 2^-21 of x.  (The conversion instruction runs at an eighth of this rate, and the
// splits, about as many as MMAs, bounded the kernels by it: 146 us for five sequences of up to 1000 tokens, 8 heads of 72.)
// kInf: for a value that may be infinite beside a weight p >= 0: hi is then the largest number and lo the infinity, so that
// p lo is that infinity and no product is NaN.
struct Split {
    uint32_t hi, lo;
};
template <bool kInf = false>
__device__ __forceinline__ Split split(float x) {
    Split s;
    s.hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    if (kInf && fabsf(__uint_as_float(s.hi)) == INFINITY) s.hi -= 0x2000u;
    s.lo = __float_as_uint(x - __uint_as_float(s.hi));
    return s;
}
// d[i] += a b[i] for N accumulators, the small products to low[i] (which may be d[i] itself).  One product of every
// accumulator after the other: an MMA waits for the last one on its accumulator, and for no other.
template <int N>
__device__ __forceinline__ void mma3(float (*d)[4], float (*low)[4], const Split (&a)[4], const Split (&b)[N][2]) {
    const uint32_t ah[4] = {a[0].hi, a[1].hi, a[2].hi, a[3].hi}, al[4] = {a[0].lo, a[1].lo, a[2].lo, a[3].lo};
#pragma unroll
    for (int i = 0; i < N; ++i) st::mma_tf32(low[i], al, b[i][0].hi, b[i][1].hi);
#pragma unroll
    for (int i = 0; i < N; ++i) st::mma_tf32(low[i], ah, b[i][0].lo, b[i][1].lo);
#pragma unroll
    for (int i = 0; i < N; ++i) st::mma_tf32(d[i], ah, b[i][0].hi, b[i][1].hi);
}

// s[n] = A B^T over D columns: 16 rows of this warp at `a`, 8 NT rows at `b`.  Accumulators 0, 1 of tile n are rows 8 n + t and
// 8 n + t + 4 of B for row order(g) of A, 2 and 3 those for row order(g) + 8.
template <int DP, int NT>
__device__ __forceinline__ void dot(float (&s)[NT][4], uint32_t a, uint32_t b, int D, int lane) {
    const int r = order(lane >> 2), t = lane & 3;
    float low[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = low[n][i] = 0.0f;
#pragma unroll 2
    for (int c = 0; c < (D + 15) / 16; ++c) {
        const float4 x = lds4(a + unit_at<DP>(r, 4 * c + t)), y = lds4(a + unit_at<DP>(r + 8, 4 * c + t));
        const Split a0[4] = {split(x.x), split(y.x), split(x.y), split(y.y)};
        const Split a1[4] = {split(x.z), split(y.z), split(x.w), split(y.w)};
        Split b0[NT][2], b1[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float4 z = lds4(b + unit_at<DP>(8 * n + r, 4 * c + t));
            b0[n][0] = split(z.x), b0[n][1] = split(z.y);
            b1[n][0] = split(z.z), b1[n][1] = split(z.w);
        }
        // (16 columns are summed apart, as in acc: gradients 4.6e-7 off where one accumulator for all 72 left 8.5e-7, in the
        // same time; rounding the splits' lo as well changes neither, and takes 5 % more)
        float sum[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[n][i] = 0.0f;
        mma3<NT>(sum, low, a0, b0);
        mma3<NT>(sum, low, a1, b1);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] += sum[n][i];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (beside an infinity the small products may be NaN)
            if (fabsf(s[n][i]) != INFINITY) s[n][i] += low[n][i];
}

// o += P B: the 8 NT rows of B at `b` weighed by accumulators of dot.  o[4 q + m]: columns 32 q + 8 t + m (0), + 4 (1) of
// row order(g), 2 and 3 of row order(g) + 8.  A tile's products are summed apart: the tensor core cuts what it adds to an
// accumulator (1000 keys one after the other: 4e-6 of O, and 5e-7 this way).
template <int DP, int NT, bool kInf>
__device__ __forceinline__ void acc(float (&o)[DP / 8][4], const float (&w)[NT][4], uint32_t b, int lane) {
    const int g = lane >> 2, t = lane & 3;
    Split a[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        a[n][0] = split(w[n][0]);
        a[n][1] = split(w[n][2]);
        a[n][2] = split(w[n][1]);
        a[n][3] = split(w[n][3]);
    }
#pragma unroll
    for (int q = 0; q < DP / 32; ++q) {
        float sum[4][4];
#pragma unroll
        for (int m = 0; m < 4; ++m) sum[m][0] = sum[m][1] = sum[m][2] = sum[m][3] = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float4 x = lds4(b + unit_at<DP>(8 * n + t, 8 * q + g)), y = lds4(b + unit_at<DP>(8 * n + t + 4, 8 * q + g));
            const Split z[4][2] = {{split<kInf>(x.x), split<kInf>(y.x)}, {split<kInf>(x.y), split<kInf>(y.y)},
                                   {split<kInf>(x.z), split<kInf>(y.z)}, {split<kInf>(x.w), split<kInf>(y.w)}};
            mma3<4>(sum, sum, a[n], z);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[4 * q + m][i] += sum[m][i];
    }
}

template <int DP>
__device__ __forceinline__ void zero(float (&o)[DP / 8][4]) {
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
}

// This thread's columns of row order(g) (x = 0) or order(g) + 8 (x = 1), times f.  Rows start on 16 bytes.
template <int DP>
__device__ __forceinline__ void store(float *row, const float (&o)[DP / 8][4], int x, float f, int D, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int q = 0; q < DP / 32; ++q)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int col = 32 * q + 8 * t + 4 * half, e = 2 * x + half;
            const float v[4] = {o[4 * q][e] * f, o[4 * q + 1][e] * f, o[4 * q + 2][e] * f, o[4 * q + 3][e] * f};
            if (col + 4 <= D) {
                *reinterpret_cast<float4 *>(row + col) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (col + m < D) row[col + m] = v[m];
            }
        }
}

// The block of rows that a CTA takes, as bw::decode.
struct Block {
    int slot, h, r0, q0, len_q, k0, len_k, qslot;
    int lo, hi;  // partners [lo, hi), lo on a tile's start
};
template <bool kKeys>
__device__ __forceinline__ Block block_of(const BwdParams &p, int tile) {
    Block B;
    const int heads = kKeys ? p.H / p.groups : p.H;
    const int slot = blockIdx.x / heads, slots = gridDim.x / heads;
    B.h = blockIdx.x - slot * heads;
    B.slot = slot;
    const PackedSeq own = packed_find_warp(kKeys ? p.cu_k : p.cu_q, p.n_seq, kKeys ? p.S_k : p.S_q, kRows,
                                           kKeys ? slot : slots - 1 - slot, threadIdx.x & 31);
    const PackedSeq other = kKeys ? packed_seq(p.cu_q, own.n, p.S_q) : packed_seq(p.cu_k, own.n, p.S_k);
    B.r0 = own.block * kRows;
    B.q0 = kKeys ? other.start : own.start;
    B.len_q = kKeys ? other.len : own.len;
    B.k0 = kKeys ? own.start : other.start;
    B.len_k = kKeys ? own.len : other.len;
    B.qslot = B.q0 / bw::kTile + own.n;
    B.lo = B.hi = 0;
    if (B.r0 < own.len) {
        const long long off = static_cast<long long>(B.len_k) - B.len_q;
        const int last = min(B.r0 + kRows, own.len) - 1;
        const int a = bw::clamp_to(kKeys ? B.r0 - off - p.band_hi : B.r0 + off + p.band_lo, other.len);
        const int e = bw::clamp_to(kKeys ? last - off - p.band_lo + 1 : last + off + p.band_hi + 1, other.len);
        if (a < e) {
            B.lo = a / tile * tile;
            B.hi = e;
        }
    }
    return B;
}

template <int DP>
constexpr int fwd_smem() { return (kRows + 4 * kFwdTile) * DP * 4; }
template <int DP>
constexpr int bwd_smem() { return (2 * kRows + 4 * kBwdTile) * DP * 4 + 2 * 2 * kBwdTile * 4; }

}  // namespace pf

template <int DP>
__global__ void __launch_bounds__(pf::kThreads, 2) attn_packed_f32_kernel(const __grid_constant__ PackedF32Params p) {
    using namespace pf;
    constexpr int kTile = kFwdTile, NT = kTile / 8;
    constexpr uint32_t kTileBytes = kTile * DP * 4;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sQ = smem_u32(smem_raw), sKV = sQ + kRows * DP * 4;  // stages of K, V
    const Block B = block_of<false>(p, kTile);
    const bool check = B.h == 0 && threadIdx.x == 0;  // (behind the block's results, which do not wait for it)
    if (B.r0 >= B.len_q) {
        if (check) packed_check(p, B.slot);
        return;
    }
    const int hk = B.h / p.kv_group;
    const float *Q = static_cast<const float *>(p.Q) + B.h * p.q_sh + B.q0 * p.q_ss;
    const float *K = static_cast<const float *>(p.K) + hk * p.k_sh + B.k0 * p.k_ss;
    const float *V = static_cast<const float *>(p.V) + hk * p.v_sh + B.k0 * p.v_ss;

    auto load = [&](int k, int stage) {
        copy_rows<DP>(sKV + 2 * stage * kTileBytes, K, p.k_ss, k, kTile, B.len_k, p.D_qk);
        copy_rows<DP>(sKV + (2 * stage + 1) * kTileBytes, V, p.v_ss, k, kTile, B.len_k, p.D_v);
    };
    copy_rows<DP>(sQ, Q, p.q_ss, B.r0, kRows, B.len_q, p.D_qk);
    if (B.lo < B.hi) load(B.lo, 0);
    cp_async_commit();

    const int t = lane & 3;
    const int row[2] = {B.r0 + 16 * warp + order(lane >> 2), B.r0 + 16 * warp + order(lane >> 2) + 8};
    const int off = B.len_k - B.len_q;
    int key_lo[2], key_hi[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        key_lo[x] = packed_key_lo(p, off, B.len_k, row[x]);
        key_hi[x] = packed_key_hi(p, off, B.len_k, row[x]);
    }
    float o[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    zero<DP>(o);
    int stage = 0;
    for (int k0 = B.lo; k0 < B.hi; k0 += kTile, stage ^= 1) {
        if (k0 + kTile < B.hi) load(k0 + kTile, stage ^ 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        float s[NT][4];
        dot<DP, NT>(s, sQ + 16 * warp * DP * 4, sKV + 2 * stage * kTileBytes, p.D_qk, lane);
        float alpha[2];
        bool moved = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float mx = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = k0 + 8 * n + t + 4 * e;
                    float &v = s[n][2 * x + e];
                    v = key >= key_lo[x] && key < key_hi[x] ? v * p.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, v);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            alpha[x] = 1.0f;
            if (mx > m[x]) {
                alpha[x] = ex2(m[x] - mx);  // 0 for the first keys
                m[x] = mx;
                moved = true;
            }
            const float ref = m[x] == -INFINITY ? 0.0f : m[x];
            float sum = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &v = s[n][2 * x + e];
                    v = ex2(v - ref);
                    sum += v;
                }
            l[x] = l[x] * alpha[x] + sum;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= alpha[e >> 1];
        }
        acc<DP, NT, true>(o, s, sKV + (2 * stage + 1) * kTileBytes, lane);
        __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        if (row[x] >= B.len_q) continue;
        const long long at = static_cast<long long>(B.q0) + row[x];
        store<DP>(static_cast<float *>(p.O) + B.h * p.o_sh + at * p.o_ss, o, x, l[x] == 0.0f ? 0.0f : 1.0f / l[x], p.D_v, lane);
        if (p.lse && t == 0)
            p.lse[static_cast<long long>(B.h) * p.S_q + at] =
                l[x] == 0.0f ? -INFINITY : (m[x] + log2f(l[x])) * 0.69314718055994531f;
    }
    if (check) packed_check(p, B.slot);
}

template <int DP>
__global__ void __launch_bounds__(pf::kThreads, 2) attn_bwd_q_f32_kernel(const __grid_constant__ PackedF32Params p) {
    using namespace pf;
    constexpr int kTile = kBwdTile, NT = kTile / 8;
    constexpr uint32_t kTileBytes = kTile * DP * 4;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sQ = smem_u32(smem_raw), sG = sQ + kRows * DP * 4, sKV = sG + kRows * DP * 4;
    const Block B = block_of<false>(p, kTile);
    if (B.r0 >= B.len_q) return;
    const int hk = B.h / p.kv_group;
    const float *K = static_cast<const float *>(p.K) + hk * p.k_sh + B.k0 * p.k_ss;
    const float *V = static_cast<const float *>(p.V) + hk * p.v_sh + B.k0 * p.v_ss;
    auto load = [&](int k, int stage) {
        copy_rows<DP>(sKV + 2 * stage * kTileBytes, K, p.k_ss, k, kTile, B.len_k, p.D_qk);
        copy_rows<DP>(sKV + (2 * stage + 1) * kTileBytes, V, p.v_ss, k, kTile, B.len_k, p.D_v);
    };
    copy_rows<DP>(sQ, static_cast<const float *>(p.Q) + B.h * p.q_sh + B.q0 * p.q_ss, p.q_ss, B.r0, kRows, B.len_q, p.D_qk);
    copy_rows<DP>(sG, static_cast<const float *>(p.dO) + B.h * p.do_sh + B.q0 * p.do_ss, p.do_ss, B.r0, kRows, B.len_q, p.D_v);
    if (B.lo < B.hi) load(B.lo, 0);
    cp_async_commit();

    const int t = lane & 3;
    const int row[2] = {B.r0 + 16 * warp + order(lane >> 2), B.r0 + 16 * warp + order(lane >> 2) + 8};
    const int off = B.len_k - B.len_q;
    int key_lo[2], key_hi[2];
    float nl[2], nd[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        key_lo[x] = packed_key_lo(p, off, B.len_k, row[x]);
        key_hi[x] = packed_key_hi(p, off, B.len_k, row[x]);
        nl[x] = -INFINITY;
        nd[x] = 0.0f;
        // (a query that sees one key: dS is 0, or dLSE, and not the rounding of dP - delta)
        if (row[x] < B.len_q && (key_hi[x] - key_lo[x] > 1 || p.dlse)) {
            const float *st = p.stat + (static_cast<long long>(B.h) * p.slots_q + B.qslot + row[x] / bw::kTile) * (2 * bw::kTile) +
                              row[x] % bw::kTile;
            nl[x] = st[0];
            nd[x] = st[bw::kTile];
        }
    }
    float o[DP / 8][4];
    zero<DP>(o);
    int stage = 0;
    for (int k0 = B.lo; k0 < B.hi; k0 += kTile, stage ^= 1) {
        if (k0 + kTile < B.hi) load(k0 + kTile, stage ^ 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        float s[NT][4], d[NT][4];
        dot<DP, NT>(s, sQ + 16 * warp * DP * 4, sKV + 2 * stage * kTileBytes, p.D_qk, lane);
        dot<DP, NT>(d, sG + 16 * warp * DP * 4, sKV + (2 * stage + 1) * kTileBytes, p.D_v, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = i >> 1, key = k0 + 8 * n + t + 4 * (i & 1);
                const float w = key >= key_lo[x] && key < key_hi[x] ? ex2(fmaf(s[n][i], p.scale_log2, nl[x])) : 0.0f;
                s[n][i] = w * (d[n][i] + nd[x]);
            }
        acc<DP, NT, false>(o, s, sKV + 2 * stage * kTileBytes, lane);
        __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
        if (row[x] < B.len_q)
            store<DP>(static_cast<float *>(p.dQ) + B.h * p.dq_sh + (static_cast<long long>(B.q0) + row[x]) * p.dq_ss, o, x,
                      p.scale, p.D_qk, lane);
}

template <int DP>
__global__ void __launch_bounds__(pf::kThreads, 2) attn_bwd_kv_f32_kernel(const __grid_constant__ PackedF32Params p) {
    using namespace pf;
    constexpr int kTile = kBwdTile, NT = kTile / 8;
    constexpr uint32_t kTileBytes = kTile * DP * 4;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sK = smem_u32(smem_raw), sV = sK + kRows * DP * 4, sQG = sV + kRows * DP * 4;
    float *const stat = reinterpret_cast<float *>(smem_raw + (2 * kRows + 4 * kTile) * DP * 4);  // [stage][2][kTile]
    const Block B = block_of<true>(p, kTile);
    if (p.S_q == 0 && B.h == 0 && threadIdx.x == 0) packed_check(p, B.slot);  // (else the statistics' launch does)
    if (B.r0 >= B.len_k) return;
    const int hk = B.h / p.head_units;
    copy_rows<DP>(sK, static_cast<const float *>(p.K) + hk * p.k_sh + B.k0 * p.k_ss, p.k_ss, B.r0, kRows, B.len_k, p.D_qk);
    copy_rows<DP>(sV, static_cast<const float *>(p.V) + hk * p.v_sh + B.k0 * p.v_ss, p.v_ss, B.r0, kRows, B.len_k, p.D_v);
    const int tiles = (B.hi - B.lo + kTile - 1) / kTile, total = tiles * p.groups;
    int g = 0, q_next = B.lo;  // of the next tile to load
    auto load = [&](int stage) {
        const int h = B.h * p.groups + g;
        copy_rows<DP>(sQG + 2 * stage * kTileBytes, static_cast<const float *>(p.Q) + h * p.q_sh + B.q0 * p.q_ss, p.q_ss, q_next,
                      kTile, B.len_q, p.D_qk);
        copy_rows<DP>(sQG + (2 * stage + 1) * kTileBytes, static_cast<const float *>(p.dO) + h * p.do_sh + B.q0 * p.do_ss,
                      p.do_ss, q_next, kTile, B.len_q, p.D_v);
        if (threadIdx.x < 2 * kTile) {  // a tile lies in one slot
            const int what = threadIdx.x / kTile, i = threadIdx.x % kTile;
            stat[2 * kTile * stage + threadIdx.x] =
                p.stat[(static_cast<long long>(h) * p.slots_q + B.qslot + q_next / bw::kTile) * (2 * bw::kTile) +
                       what * bw::kTile + q_next % bw::kTile + i];
        }
        q_next += kTile;
        if (q_next >= B.hi) {
            q_next = B.lo;
            ++g;
        }
    };
    if (total > 0) load(0);
    cp_async_commit();

    const int t = lane & 3;
    const int row[2] = {B.r0 + 16 * warp + order(lane >> 2), B.r0 + 16 * warp + order(lane >> 2) + 8};
    const long long off = static_cast<long long>(B.len_k) - B.len_q;
    int q_lo[2], q_hi[2], q_lone[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {  // queries [q_lo, q_hi) see the key; q_lone sees no other
        q_lo[x] = bw::clamp_to(row[x] - off - p.band_hi, B.len_q);
        q_hi[x] = bw::clamp_to(row[x] - off - p.band_lo + 1, B.len_q);
        q_lone[x] = row[x] == 0 && q_lo[x] + off + p.band_hi == 0 ? q_lo[x] : -1;
    }
    const bool lone = B.len_k == 1 || p.band_lo == p.band_hi;
    float dk[DP / 8][4], dv[DP / 8][4];
    zero<DP>(dk);
    zero<DP>(dv);
    int stage = 0, q0 = B.lo;
    for (int i = 0; i < total; ++i, stage ^= 1) {
        if (i + 1 < total) load(stage ^ 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const uint32_t tq = sQG + 2 * stage * kTileBytes, tg = tq + kTileBytes;
        const float *st = stat + 2 * kTile * stage;
        float s[NT][4], d[NT][4];
        dot<DP, NT>(s, sK + 16 * warp * DP * 4, tq, p.D_qk, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int x = e >> 1, at = 8 * n + t + 4 * (e & 1), q = q0 + at;
                s[n][e] = q >= q_lo[x] && q < q_hi[x] ? ex2(fmaf(s[n][e], p.scale_log2, st[at])) : 0.0f;
            }
        acc<DP, NT, false>(dv, s, tg, lane);
        dot<DP, NT>(d, sV + 16 * warp * DP * 4, tg, p.D_v, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = 8 * n + t + 4 * (e & 1);
                s[n][e] *= d[n][e] + st[kTile + at];
                if (!p.dlse && (lone || q0 + at == q_lone[e >> 1])) s[n][e] = 0.0f;
            }
        acc<DP, NT, false>(dk, s, tq, lane);
        __syncthreads();
        q0 += kTile;
        if (q0 >= B.hi) q0 = B.lo;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if (row[x] >= B.len_k) continue;
        const long long at = static_cast<long long>(B.k0) + row[x], part = static_cast<long long>(B.h) * p.S_k + at;
        if (p.part_k) {
            store<DP>(p.part_k + part * p.part_ldk, dk, x, 1.0f, p.part_ldk, lane);
            store<DP>(p.part_v + part * p.part_ldv, dv, x, 1.0f, p.part_ldv, lane);
        } else {
            store<DP>(static_cast<float *>(p.dK) + B.h * p.dk_sh + at * p.dk_ss, dk, x, p.scale, p.D_qk, lane);
            store<DP>(static_cast<float *>(p.dV) + B.h * p.dv_sh + at * p.dv_ss, dv, x, 1.0f, p.D_v, lane);
        }
    }
}

}  // namespace vt
