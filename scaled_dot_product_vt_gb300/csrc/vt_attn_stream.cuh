// Attention of few query rows over many keys: the keys stream past 16 query rows held in registers
// (contract in include/vt_attn.h, vt_attn_fwd_prefix).
//
// A work unit is 16 query rows that read the same keys: rows (s, g) of one sequence and key/value head over the
// prefix and/or that sequence's cache, or rows (b, s, g) of one key/value head over the prefix alone.  With a few
// rows per key the work is bound by the bytes of K and V (4 flops per row and byte against ~280 that the card
// balances at), so everything serves the loads:
//   - The unit's keys are cut over the CTAs of a cluster and over the grid's shares, and a CTA's keys over its
//     four warps in blocks of 16.  Every warp runs its own ring of cp.async stages and its own online softmax, so
//     the loop has no barrier; rows past the end are filled with zeros instead of being read (a cache row that
//     holds NaN never meets a probability of 0).
//   - Products are mma.sync: 16 rows is a quarter of the smallest tcgen05 tile, and the tensor pipe is not what
//     bounds this kernel.  bf16 with fp32 accumulation; fp32 operands as two TF32 parts each, three products
//     (hi hi + hi lo + lo hi), which keeps 21 bits of every factor.
//   - At the end the warps of the cluster leave (max, sum, unnormalised O) in shared memory; each CTA combines its
//     share of the rows over all of them through distributed shared memory, adds partial results of the prefix
//     that an earlier launch left in the workspace, and writes O.  No merge launch and no atomics: the order of
//     every sum is fixed.
#pragma once

#include <type_traits>

#include "vt_attn_common.cuh"

namespace vt {
namespace st {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRowsTile = 16;
constexpr int kKeys = 16;        // keys per block of a warp
constexpr int kMaxClusterCtas = 8;
constexpr float kTau = 8.0f;     // the reference max moves when the running max exceeds it by 2^8 (see kTau of vt_attn_bf16_2q.cuh)

struct Params {
    int B, H, H_kv, G, S_q, S_p, S_c, D_qk, D_v;
    int all_rows;     // 1: a unit's rows are (b, s, g) and its keys the prefix; 0: rows (s, g) of one sequence
    int with_prefix;  // (all_rows = 0) the unit's keys start with the prefix
    int row_tiles, shares, cluster;
    float scale_log2;
    const void *Q, *Kp, *Vp, *Kc, *Vc;
    long long q_sb, q_sh, q_ss, kp_sh, kp_ss, vp_sh, vp_ss, kc_sb, kc_sh, kc_ss, vc_sb, vc_sh, vc_ss;
    const int *kv_len;  // [B], or null: S_c
    // partial results: [share][rows], rows = H_kv * B * S_q * G indexed ((hk * B + b) * S_q + s) * G + g
    float *part_o, *part_m, *part_l, *part_c;
    long long rows;
    int prior;  // shares in the workspace to add (all_rows = 0)
    void *O;
    long long o_sb, o_sh, o_ss;
    float *lse;
    unsigned *status;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x as hi + lo, both rounded to TF32 (10 explicit mantissa bits): what hi + lo leaves out is below 2^-23 of x.
__device__ __forceinline__ uint32_t tf32_of(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t &hi, uint32_t &lo) {
    hi = tf32_of(__uint_as_float(x));
    lo = tf32_of(__uint_as_float(x) - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_3xtf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_tf32(a[i], ah[i], al[i]);
    split_tf32(b0, bh[0], bl[0]);
    split_tf32(b1, bh[1], bl[1]);
    mma_tf32(d, al, bh[0], bh[1]);
    mma_tf32(d, ah, bl[0], bl[1]);
    mma_tf32(d, ah, bh[0], bh[1]);
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Shared memory of one warp: `stages` blocks of K [16][DQ] then V [16][DV], and after the loop over it the warp's
// result: O [16][DV] fp32, then m, l, c [16].
template <typename T, int DQ, int DV>
struct Tile {
    static constexpr int kElt = sizeof(T);
    static constexpr uint32_t kRowK = DQ * kElt, kRowV = DV * kElt;
    static constexpr uint32_t kBytesK = kKeys * kRowK;
    static constexpr uint32_t kStage = kBytesK + kKeys * kRowV;
    // three blocks in flight per warp at 8 KB a block and more, six below
    static constexpr int kStages = kStage <= 4096 ? 6 : (kStage <= 8192 ? 3 : 3);
    static constexpr uint32_t kWarpBytes = kStages * kStage;
    static constexpr uint32_t kSmem = kWarps * kWarpBytes;
    static_assert(kRowsTile * DV * 4 + 3 * kRowsTile * 4 <= kWarpBytes, "a warp's result takes the place of its stages");
};

template <typename T, int DQ, int DV>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) attn_stream_kernel(const Params p) {
    using L = Tile<T, DQ, DV>;
    constexpr bool kBf = sizeof(T) == 2;
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    const uint32_t wbase = base + warp * L::kWarpBytes;

    // the launch that adds this one's partial results may start; it waits for them where it needs them
    if (p.all_rows) launch_dependents();

    // ---- the unit: 16 rows, and the keys of this CTA's share of them
    const int rank = static_cast<int>(blockIdx.x) % p.cluster;
    long long u = blockIdx.x / p.cluster;
    int share = 0;
    if (p.all_rows) {
        share = static_cast<int>(u % p.shares);
        u /= p.shares;
    }
    const int rt = static_cast<int>(u % p.row_tiles);
    u /= p.row_tiles;
    const int hk = static_cast<int>(u % p.H_kv);
    const int b = static_cast<int>(u / p.H_kv);  // 0 with all_rows
    const int per_b = p.S_q * p.G;
    const int group_rows = p.all_rows ? p.B * per_b : per_b;
    const int f0 = rt * kRowsTile;
    const int n_rows = min(kRowsTile, group_rows - f0);

    const int nP = (p.all_rows || p.with_prefix) ? p.S_p : 0;
    int len = 0;
    if (!p.all_rows) {
        len = p.kv_len ? p.kv_len[b] : p.S_c;
        if (len < 0 || len > p.S_c) {  // a length outside the cache: as many keys as it has
            if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
            len = len < 0 ? 0 : p.S_c;
        }
    }
    // keys seen by row f (concatenated prefix and cache): those below limit(f)
    auto limit = [&](int f) {
        if (p.all_rows) return nP;
        const int c = len - p.S_q + f / p.G + 1;
        return nP + max(0, c);
    };
    const int total = limit(f0 + n_rows - 1), all_see = limit(f0);
    const int blocks = (total + kKeys - 1) / kKeys;
    const int cuts = p.cluster * p.shares;
    const int per = (blocks + cuts - 1) / cuts;
    const int first = min(blocks, (share * p.cluster + rank) * per), last = min(blocks, first + per);

    const T *kp = static_cast<const T *>(p.Kp) + hk * p.kp_sh, *vp = static_cast<const T *>(p.Vp) + hk * p.vp_sh;
    const T *kc = static_cast<const T *>(p.Kc) + b * p.kc_sb + hk * p.kc_sh;
    const T *vc = static_cast<const T *>(p.Vc) + b * p.vc_sb + hk * p.vc_sh;

    // ---- loads: block i of the share into stage s, 16 bytes per lane and row; chunks of a row are permuted by
    // the row's low bits, so that the reads below touch every bank once
    auto load = [&](int blk, int s) {
        const int k0 = blk * kKeys;
        const uint32_t dk = wbase + s * L::kStage, dv = dk + L::kBytesK;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int D = half ? DV : DQ;
            const int cpr = D * L::kElt / 16;  // chunks per row
            const int used = (half ? p.D_v : p.D_qk) * L::kElt;
            const T *pre = half ? vp : kp, *own = half ? vc : kc;
            const long long pre_s = half ? p.vp_ss : p.kp_ss, own_s = half ? p.vc_ss : p.kc_ss;
            const uint32_t d0 = half ? dv : dk;
#pragma unroll
            for (int i = 0; i < kKeys * cpr / 32; ++i) {
                const int idx = i * 32 + lane;
                const int row = idx / cpr, c = idx % cpr;
                const int key = k0 + row;
                int bytes = min(16, used - c * 16);
                if (key >= total || bytes < 0) bytes = 0;
                const T *src = key < nP ? pre + key * pre_s : own + (key - nP) * own_s;
                const int sw = kBf || !half ? (row & 7) : (row & 6);
                const void *from = bytes > 0 ? reinterpret_cast<const uint8_t *>(src) + c * 16 : p.Q;
                cp_async16(d0 + row * (D * L::kElt) + ((c ^ sw) << 4), from, bytes);
            }
        }
    };

    const int n_mine = last > first + warp ? (last - first - warp + kWarps - 1) / kWarps : 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < n_mine) load(first + warp + i * kWarps, i);
        cp_async_commit();
    }

    // ---- the rows' queries, in the layout of an MMA's A operand: rows lane / 4 and lane / 4 + 8
    const int g8 = lane >> 2, t4 = lane & 3;
    constexpr int kSteps = kBf ? DQ / 16 : DQ / 8;
    uint32_t q[kSteps][4];
    const T *qrow[2];
    int lim[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int i = g8 + 8 * r;
        const int f = f0 + (i < n_rows ? i : 0);
        const int bb = p.all_rows ? f / per_b : b;
        const int fs = p.all_rows ? f - bb * per_b : f;
        const int s = fs / p.G, g = fs - s * p.G;
        qrow[r] = i < n_rows ? static_cast<const T *>(p.Q) + bb * p.q_sb + static_cast<long long>(hk * p.G + g) * p.q_sh +
                                   s * p.q_ss
                             : nullptr;
        lim[r] = i < n_rows ? limit(f) : 0;
    }
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const T *row = qrow[j & 1];
            if (kBf) {
                const int d = ks * 16 + (j >> 1) * 8 + t4 * 2;
                uint32_t v = 0;
                if (row && d + 1 < p.D_qk) v = *reinterpret_cast<const uint32_t *>(row + d);
                else if (row && d < p.D_qk) v = *reinterpret_cast<const uint16_t *>(row + d);
                q[ks][j] = v;
            } else {
                const int d = ks * 8 + (j >> 1) * 4 + t4;
                q[ks][j] = row && d < p.D_qk ? *reinterpret_cast<const uint32_t *>(row + d) : 0u;
            }
        }

    float o[DV / 8][4];
#pragma unroll
    for (int n = 0; n < DV / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, c[2] = {0.f, 0.f};

    for (int it = 0; it < n_mine; ++it) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        if (it + kStages - 1 < n_mine) load(first + warp + (it + kStages - 1) * kWarps, (it + kStages - 1) % kStages);
        cp_async_commit();
        const int k0 = (first + warp + it * kWarps) * kKeys;
        const uint32_t sk = wbase + (it % kStages) * L::kStage, sv = sk + L::kBytesK;

        // ---- scores of 16 rows x 16 keys: s[n] holds keys 8 n + 2 t4, + 1 of rows g8 (0, 1) and g8 + 8 (2, 3)
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        {
            // lane 8 j + i addresses row i of matrix j: keys 0-7 and 8-15, chunks 2 ks and 2 ks + 1
            const int key = (lane & 7) + ((lane >> 4) << 3);
            const uint32_t row = sk + key * L::kRowK;
            const int odd = (lane >> 3) & 1;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                uint32_t kb[4];
                ldsm4(kb, row + (((2 * ks + odd) ^ (key & 7)) << 4));
                if (kBf) {
                    mma_bf16(s[0], q[ks], kb[0], kb[1]);
                    mma_bf16(s[1], q[ks], kb[2], kb[3]);
                } else {
                    mma_3xtf32(s[0], q[ks], kb[0], kb[1]);
                    mma_3xtf32(s[1], q[ks], kb[2], kb[3]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] *= p.scale_log2;
        if (k0 + kKeys > all_see) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (k0 + 8 * n + 2 * t4 + (i & 1) >= lim[i >> 1]) s[n][i] = -INFINITY;
        }

        // ---- online softmax of the two rows
        float alpha[2];
        bool moved = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float mx = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            alpha[r] = 1.0f;
            if (mx > m[r] + kTau || (m[r] == -INFINITY && mx > -INFINITY)) {
                alpha[r] = ex2(m[r] - mx);  // 0 for the first keys
                m[r] = mx;
                moved = true;
            }
            const float ref = m[r] == -INFINITY ? 0.0f : m[r];
            float sum = 0.0f, fix = 0.0f;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 2 * r; i < 2 * r + 2; ++i) {
                    s[n][i] = ex2(s[n][i] - ref);
                    sum += s[n][i];
                    // bf16: P V weighs P as rounded to bf16; c makes l + c the sum of those weights
                    if (kBf) fix += __uint_as_float(pack_bf16x2(0.0f, s[n][i]) & 0xFFFF0000u) - s[n][i];
                }
            l[r] = l[r] * alpha[r] + sum;
            c[r] = c[r] * alpha[r] + fix;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int n = 0; n < DV / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] *= alpha[i >> 1];
        }

        // ---- O += P V
        if (kBf) {
            const uint32_t a[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                                   pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
            // matrices: keys 0-7 and 8-15 of column chunk n, then of chunk n + 1
            const int key = lane & 15;
            const uint32_t row = sv + key * L::kRowV;
            const int odd = lane >> 4;
#pragma unroll
            for (int n = 0; n < DV / 8; n += 2) {
                uint32_t vb[4];
                ldsm4_t(vb, row + (((n + odd) ^ (key & 7)) << 4));
                mma_bf16(o[n], a, vb[0], vb[1]);
                mma_bf16(o[n + 1], a, vb[2], vb[3]);
            }
        } else {
            // the k index of the product runs over keys in the order 0, 2, 4, 6, 1, 3, 5, 7, so the scores are
            // the A operand as they lie
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t a[4] = {__float_as_uint(s[j][0]), __float_as_uint(s[j][2]), __float_as_uint(s[j][1]),
                                       __float_as_uint(s[j][3])};
                const int key = 8 * j + 2 * t4;
                const uint8_t *r0 = smem + (sv - base) + key * L::kRowV, *r1 = r0 + L::kRowV;
#pragma unroll
                for (int n = 0; n < DV / 8; ++n) {
                    const int col = n * 8 + g8;
                    const uint32_t at = (((col >> 2) ^ (key & 6)) << 4) + (col & 3) * 4;
                    mma_3xtf32(o[n], a, *reinterpret_cast<const uint32_t *>(r0 + at),
                               *reinterpret_cast<const uint32_t *>(r1 + at));
                }
            }
        }
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- the warp's result
    float *wo = reinterpret_cast<float *>(smem + warp * L::kWarpBytes);
    float *wm = wo + kRowsTile * DV;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
            c[r] += __shfl_xor_sync(0xffffffffu, c[r], x);
        }
        if (t4 == 0) {
            wm[g8 + 8 * r] = m[r];
            wm[kRowsTile + g8 + 8 * r] = l[r];
            wm[2 * kRowsTile + g8 + 8 * r] = c[r];
        }
#pragma unroll
        for (int n = 0; n < DV / 8; ++n)
            *reinterpret_cast<float2 *>(wo + (g8 + 8 * r) * DV + n * 8 + 2 * t4) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    if (!p.all_rows) wait_prerequisites();  // (the whole grid waits, so that it ends after the prefix's launch)

    // ---- combine: this CTA takes rows rank, rank + cluster, ... of the unit, one warp per row
    constexpr int kCols = DV / 32;
    const uint32_t o_off = base, m_off = base + kRowsTile * DV * 4;
    for (int i = rank + p.cluster * warp; i < n_rows; i += p.cluster * kWarps) {
        const int f = f0 + i;
        const long long flat = static_cast<long long>(hk) * p.B * per_b + static_cast<long long>(b) * per_b + f;
        float M = -INFINITY, Ls = 0.0f, Lo = 0.0f, acc[kCols];
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] = 0.0f;
        auto add = [&](float ms, float ls, float cs, const float (&v)[kCols]) {
            if (ms == -INFINITY) return;  // no key there
            const float Mn = fmaxf(M, ms);
            const float a = M == -INFINITY ? 0.0f : ex2(M - Mn), w = ex2(ms - Mn);
            Ls = Ls * a + w * ls;
            Lo = Lo * a + w * (ls + cs);
#pragma unroll
            for (int k = 0; k < kCols; ++k) acc[k] = acc[k] * a + w * v[k];
            M = Mn;
        };
        for (int r = 0; r < p.cluster; ++r)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const uint32_t at = w * L::kWarpBytes;
                const uint32_t mo = p.cluster > 1 ? cluster_map(m_off + at, r) : m_off + at;
                const uint32_t oo = p.cluster > 1 ? cluster_map(o_off + at, r) : o_off + at;
                float v[kCols];
#pragma unroll
                for (int k = 0; k < kCols; ++k) v[k] = ld_cluster(oo + (i * DV + lane + 32 * k) * 4);
                add(ld_cluster(mo + i * 4), ld_cluster(mo + (kRowsTile + i) * 4), ld_cluster(mo + (2 * kRowsTile + i) * 4), v);
            }
        for (int r = 0; r < p.prior; ++r) {
            const long long at = r * p.rows + flat;
            float v[kCols];
#pragma unroll
            for (int k = 0; k < kCols; ++k) {
                const int col = lane + 32 * k;
                v[k] = col < p.D_v ? p.part_o[at * p.D_v + col] : 0.0f;
            }
            add(p.part_m[at], p.part_l[at], p.part_c[at], v);
        }
        if (p.all_rows) {
            const long long at = share * p.rows + flat;
#pragma unroll
            for (int k = 0; k < kCols; ++k)
                if (lane + 32 * k < p.D_v) p.part_o[at * p.D_v + lane + 32 * k] = acc[k];
            if (lane == 0) {
                p.part_m[at] = M;
                p.part_l[at] = Ls;
                p.part_c[at] = Lo - Ls;
            }
        } else {
            const int s = f / p.G, g = f - s * p.G;
            const int h = hk * p.G + g;
            const float inv = Ls > 0.0f ? 1.0f / Lo : 0.0f;  // a row without keys is 0
            T *orow = static_cast<T *>(p.O) + b * p.o_sb + h * p.o_sh + s * p.o_ss;
#pragma unroll
            for (int k = 0; k < kCols; ++k) {
                const int col = lane + 32 * k;
                if (col >= p.D_v) continue;
                const float v = acc[k] * inv;
                if constexpr (kBf) {
                    reinterpret_cast<uint16_t *>(orow)[col] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
                } else {
                    reinterpret_cast<float *>(orow)[col] = v;
                }
            }
            if (p.lse && lane == 0)
                p.lse[(static_cast<long long>(b) * p.H + h) * p.S_q + s] = lse_from(M, Ls);
        }
    }
    if (p.cluster > 1) cluster_sync();  // the other CTAs have read this one's results
}

}  // namespace st
}  // namespace vt
