// Attention of few query rows over many keys: the keys stream past 16 query rows held in registers
// (contract in include/vt_attn.h, vt_attn_fwd_prefix).
//
// A work unit is 16 query rows that read the same keys: rows (s, g) of one sequence and key/value head over the
// prefix and/or that sequence's cache, or rows (b, s, g) of one key/value head over the prefix alone.  With a few
// rows per key the work is bound by the bytes of K and V (4 flops per row and byte against ~280 that the card
// balances at), so everything serves the loads:
//   - The unit's keys are cut over the CTAs of a cluster and over the grid's shares, and a CTA's keys over its
//     four warps in blocks of 16.  Every warp runs its own ring of TMA loads (one lane issues them; loads by all lanes
//     spent more instructions on addresses than the products take) and its own online softmax, so the loop has no
//     barrier between warps.  V rows past the end of a sequence are set to zero in shared memory: they may hold
//     NaN, which a probability of 0 does not hide.
//   - Products are mma.sync: 16 rows is a quarter of the smallest tcgen05 tile, and the tensor pipe is not what
//     bounds this kernel.  bf16 with fp32 accumulation; fp32 operands as two TF32 parts each, three products
//     (hi hi + hi lo + lo hi), which keeps 21 bits of every factor.
//   - At the end the warps of the cluster leave (max, sum, unnormalised O) in shared memory; each CTA combines its
//     share of the rows over all of them through distributed shared memory.  Then either it adds the partial results of
//     the prefix that an earlier launch leaves in the workspace and writes O, or (more CTAs than fit at once: those that
//     wait for the earlier launch would keep the others out) it leaves one there itself and attn_shares_kernel adds
//     them all.  No atomics: the order of every sum is fixed.
// Measured (bf16, 64 sequences, 8 key/value heads, D = 128, GPU time per call): 53 us with caches of 1024 tokens each
// (268 MB, 5.1 TB/s), 30 us with 512 (4.4 TB/s), 9.2 us with one token each (in L2).  A CTA takes 4.8 us besides its keys (setup,
// first loads, combine), which is what short caches pay; long ones are bound by HBM.
#pragma once

#include <climits>
#include <type_traits>

#include "vt_attn_common.cuh"
#include "vt_attn_tree.cuh"

namespace vt {
namespace st {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRowsTile = 16;
constexpr int kKeys = 16;        // keys per block of a warp
constexpr int kMaxClusterCtas = 8;
constexpr int kMaxShares = 32;       // partial results of the prefix, at most
constexpr int kMaxCacheShares = 32;  // and of the caches
constexpr int kMaxSources = kWarps * kMaxClusterCtas + kMaxShares;
static_assert(kMaxSources >= kMaxShares + kMaxCacheShares, "attn_shares_kernel reads both");
static_assert(kMaxSources == 64, "a lane holds the weights of two sources");
constexpr int kMaxSorted = 32;   // sequences that every warp ranks by their lengths
constexpr float kTau = 8.0f;     // the reference max moves when the running max exceeds it by 2^8 (see kTau of vt_attn_bf16_2q.cuh)

struct Params {
    int B, H, H_kv, G, S_q, S_p, S_c, D_qk, D_v;
    int all_rows;     // 1: a unit's rows are (b, s, g) and its keys the prefix; 0: rows (s, g) of one sequence
    int with_prefix;  // (all_rows = 0) the unit's keys start with the prefix
    int row_tiles, shares, cluster;
    float scale_log2;
    const void *Q;
    long long q_sb, q_sh, q_ss;
    const int *kv_len;  // [B], or null: S_c
    const int *parents;  // kTree: [B][S_q]
    // partial results: [share][rows], rows = H_kv * B * S_q * G indexed ((hk * B + b) * S_q + s) * G + g
    float *part_o, *part_m, *part_l, *part_c;
    long long rows;
    int part_ld;  // floats between partial O rows
    int partial, share0;  // 1: write a partial result, to share0 and on; 0: write O
    int prior;            // shares in the workspace to add (partial = 0)
    int follows;          // started ahead of the prefix's launch's end
    int longest_first;    // units in the order of their sequences' lengths (B <= kMaxSorted)
    void *O;
    long long o_sb, o_sh, o_ss;
    float *lse;
    unsigned long long timeout_ns;
    unsigned *status;
};

// Tensor maps of the prefix and of the caches, boxes of 16 rows x 128 bytes with the 128-byte swizzle.
struct Maps {
    CUtensorMap kp, vp, kc, vc;
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
// (hi in integers, which is the conversion's value at eight times its rate; of a NaN lo alone is left.)
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t &hi, uint32_t &lo) {
    hi = (x + 0x1000u) & 0xFFFFE000u;
    lo = tf32_of(__uint_as_float(x) - __uint_as_float(hi));
}
// The same for a value that may be infinite beside a factor p >= 0: hi is then the largest number and lo the infinity, so
// that p lo is that infinity and no product is NaN (as hi it would meet p's lo, which may be 0 or of either sign).  Rounding
// in integers is the conversion's, without its slow unit (all NaN bits overflow to 0; lo is NaN then).
__device__ __forceinline__ void split_tf32_inf(uint32_t x, uint32_t &hi, uint32_t &lo) {
    hi = (x + 0x1000u) & 0xFFFFE000u;
    if (fabsf(__uint_as_float(hi)) == INFINITY) hi -= 0x2000u;
    lo = tf32_of(__uint_as_float(x) - __uint_as_float(hi));
}
// d += a b by three products; the two small ones go to `low`, which may be d itself.
template <bool kInfB>
__device__ __forceinline__ void mma_3xtf32(float (&d)[4], float (&low)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_tf32(a[i], ah[i], al[i]);
    if constexpr (kInfB) {
        split_tf32_inf(b0, bh[0], bl[0]);
        split_tf32_inf(b1, bh[1], bl[1]);
    } else {
        split_tf32(b0, bh[0], bl[0]);
        split_tf32(b1, bh[1], bl[1]);
    }
    mma_tf32(low, al, bh[0], bh[1]);
    mma_tf32(low, ah, bl[0], bl[1]);
    mma_tf32(d, ah, bh[0], bh[1]);
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
template <typename V>
__device__ __forceinline__ V ld_cluster_vec(uint32_t addr) {
    V v;
    if constexpr (sizeof(V) == 16)
        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// Wait for the phase of `bar` with `parity`, giving up after the time limit (which the status word then records).
__device__ __forceinline__ bool wait_limited(uint32_t bar, uint32_t parity, const Params &p) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 63u) == 0 && globaltimer_ns() - t0 > p.timeout_ns) {
            atomicOr(p.status, kStatusTimeout);
            return false;
        }
    }
}

// Shared memory: each warp's `stages` blocks of K [pieces of 128 bytes][16 keys] then V, which its result takes the
// place of after the loop (O [16][DV + 8] fp32, then m, l, c [16]); then the queries, as pieces of 16 rows.
template <typename T, int DQ, int DV>
struct Tile {
    static constexpr int kElt = sizeof(T);
    static constexpr int kCols = 128 / kElt;  // columns of a 128-byte piece
    static constexpr uint32_t kPiece = kKeys * 128;
    static constexpr uint32_t kBytesK = DQ / kCols * kPiece, kBytesV = DV / kCols * kPiece, kBytesQ = kBytesK;
    static constexpr uint32_t kStage = kBytesK + kBytesV;
    // Two or three blocks a warp (16 KB at full width), so that three CTAs share an SM, four with narrow values, and
    // one's start and end hide behind the others' loads: 37 sequences of 32 heads over up to 333 keys, D 96 and 64,
    // take 22 us with four and 28 us with three.  (fp32 at full width: 32 KB, one CTA.)
    static constexpr int kStages = kStage <= 4096 ? 3 : 2;
    static constexpr int kPerSm = kElt == 2 ? (DV == 64 ? 4 : 3) : 1;
    static constexpr uint32_t kWarpBytes = kStages * kStage;
    static constexpr uint32_t kQ = kWarps * kWarpBytes;
    static constexpr uint32_t kSmem = 1024 + kQ + kBytesQ;  // pieces start on 1024 bytes
    static constexpr int kLdO = DV + 8;  // floats between result rows: eight rows' stores fall into different banks
    static_assert(kRowsTile * kLdO * 4 + 3 * kRowsTile * 4 <= kWarpBytes, "a warp's result takes the place of its stages");
};

// One row's answer from its sources (partial results), by one warp: every lane holds the weights of sources lane and
// lane + 32 and sums DV / 32 columns over the sources in order, eight loads at a time.
template <typename T, int DV>
struct Combine {
    static constexpr int kCols = DV / 32;
    using Vec = typename std::conditional<kCols == 4, float4, float2>::type;
    float M, Ls, Lo;   // max (log2 units), sum, and the sum as P V weighed it
    float acc[kCols];
    int col;

    __device__ __forceinline__ Vec vec() const {
        if constexpr (kCols == 4) return make_float4(acc[0], acc[1], acc[2], acc[3]);
        else return make_float2(acc[0], acc[1]);
    }

    // row(src, col, v) loads a source's columns, stats(src, m, l, fix) its statistics
    template <typename Row, typename Stats>
    __device__ __forceinline__ void run(int lane, int n_src, Row row, Stats stats) {
        constexpr int kAtOnce = 8, kPer = kMaxSources / 32;
        col = lane * kCols;
        Vec v[kAtOnce];
        auto load_rows = [&](int s0) {
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                v[j] = Vec{};
                if (s0 + j < n_src) row(s0 + j, col, v[j]);
            }
        };
        load_rows(0);  // on their way while the weights are formed
        float ms[kPer], ls[kPer], cs[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            ms[k] = -INFINITY;
            ls[k] = cs[k] = 0.0f;
            if (lane + 32 * k < n_src) stats(lane + 32 * k, ms[k], ls[k], cs[k]);
        }
        M = ms[0];
#pragma unroll
        for (int k = 1; k < kPer; ++k) M = fmaxf(M, ms[k]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        Ls = Lo = 0.0f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            // the source's weight: 0 without keys (a sum that is NaN without a maximum stays NaN)
            ms[k] = ms[k] == -INFINITY && ls[k] == 0.0f ? 0.0f : ex2(ms[k] - M);
            Ls += ms[k] * ls[k];
            Lo += ms[k] * (ls[k] + cs[k]);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) {
            Ls += __shfl_xor_sync(0xffffffffu, Ls, x);
            Lo += __shfl_xor_sync(0xffffffffu, Lo, x);
        }
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] = 0.0f;
#pragma unroll 1
        for (int s0 = 0; s0 < n_src; s0 += kAtOnce) {
            if (s0 > 0) load_rows(s0);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const float w = __shfl_sync(0xffffffffu, s0 < 32 ? ms[0] : ms[1], (s0 + j) & 31);
#pragma unroll
                for (int x = 0; x < kCols; ++x) acc[x] = fmaf(w, reinterpret_cast<const float *>(&v[j])[x], acc[x]);
            }
        }
    }

    // O and LSE of row f of sequence b
    __device__ __forceinline__ void store(const Params &p, int lane, int b, int hk, int f) {
        const int s = f / p.G, h = hk * p.G + f - s * p.G;
        const float inv = Ls == 0.0f ? 0.0f : 1.0f / Lo;  // a row without keys is 0
        T *orow = static_cast<T *>(p.O) + b * p.o_sb + h * p.o_sh + s * p.o_ss + col;
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] *= inv;
        if (col + kCols <= p.D_v) {  // rows start on 16 bytes
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int k = 0; k < kCols; k += 2)
                    *reinterpret_cast<uint32_t *>(orow + k) = pack_bf16x2(acc[k], acc[k + 1]);
            } else {
                *reinterpret_cast<Vec *>(orow) = vec();
            }
        } else {
            for (int k = 0; k < kCols && col + k < p.D_v; ++k) {
                if constexpr (sizeof(T) == 2)
                    reinterpret_cast<uint16_t *>(orow)[k] = static_cast<uint16_t>(pack_bf16x2(acc[k], 0.0f) & 0xFFFFu);
                else
                    reinterpret_cast<float *>(orow)[k] = acc[k];
            }
        }
        if (p.lse && lane == 0)
            p.lse[(static_cast<long long>(b) * p.H + h) * p.S_q + s] =
                Ls == 0.0f ? -INFINITY : (M + log2f(Ls)) * 0.69314718055994531f;
    }
};

// The workspace's shares of every row combined into O: one warp per row.
constexpr int kMergeWarps = 4;
template <typename T, int DV>
__global__ void __launch_bounds__(32 * kMergeWarps) attn_shares_kernel(const __grid_constant__ Params p) {
    using C = Combine<T, DV>;
    wait_prerequisites();
    const int lane = threadIdx.x & 31;
    const long long flat = static_cast<long long>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
    if (flat >= p.rows) return;
    C c;
    c.run(
        lane, p.prior,
        [&](int src, int col, typename C::Vec &v) {
            if (col < p.part_ld)
                v = *reinterpret_cast<const typename C::Vec *>(p.part_o + (src * p.rows + flat) * p.part_ld + col);
        },
        [&](int src, float &m, float &l, float &fix) {
            const long long at = src * p.rows + flat;
            m = p.part_m[at];
            l = p.part_l[at];
            fix = p.part_c[at];
        });
    const int per_b = p.S_q * p.G, seq = static_cast<int>(flat) / per_b, hk = seq / p.B;  // rows stay below 2^30
    c.store(p, lane, seq - hk * p.B, hk, static_cast<int>(flat) - seq * per_b);
}

// kTree: the S_q tokens of a sequence are the nodes of a tree, and its keys its cache (or with the prefix).  Four trees of 8
// behind 333 keys: 8.3 us, as for tokens in a row.
template <typename T, int DQ, int DV, bool kTree = false>
__global__ void __launch_bounds__(kThreads, Tile<T, DQ, DV>::kPerSm)
    attn_stream_kernel(const __grid_constant__ Maps maps, const Params p) {
    using L = Tile<T, DQ, DV>;
    constexpr bool kBf = sizeof(T) == 2;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kWarps][kStages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - raw);
    const uint32_t wbase = base + warp * L::kWarpBytes;

    // the launch that adds this one's partial results may start; it waits for them where it needs them
    if (p.all_rows) launch_dependents();

    // ---- the unit: 16 rows, and the keys of this CTA's share of them
    unsigned u = blockIdx.x / p.cluster;
    const int rank = static_cast<int>(blockIdx.x - u * p.cluster);
    int share = 0;
    if (p.shares > 1) {
        share = static_cast<int>(u % p.shares);
        u /= p.shares;
    }
    const int rt = static_cast<int>(u % p.row_tiles);
    u /= p.row_tiles;
    int b = static_cast<int>(u / p.H_kv);  // 0 with all_rows
    const int hk = static_cast<int>(u) - b * p.H_kv;
    // When the CTAs of a launch do not all fit at once, those of the longest sequences start first and the short ones fill the
    // end (16 sequences of up to 8192 tokens: 51 us against 56 us; ranking more of them costs every CTA more than it gains).
    if (p.longest_first) b = nth_longest(p.kv_len, p.B, b, lane);
    const int per_b = p.S_q * p.G;
    const int group_rows = p.all_rows ? p.B * per_b : per_b;
    const int f0 = rt * kRowsTile;
    const int n_rows = min(kRowsTile, group_rows - f0);

    int len = p.all_rows ? 0 : (p.kv_len ? p.kv_len[b] : p.S_c);  // (asked for first: the keys wait for it)
    TreeNodes tree;
    if constexpr (kTree) tree.load(p.parents + static_cast<long long>(b) * p.S_q, p.S_q, lane);
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(p.all_rows ? &maps.kp : &maps.kc);
        tma_prefetch_desc(p.all_rows ? &maps.vp : &maps.vc);
    }
    // the queries on their way to shared memory: 16 bytes per thread and step, swizzled as the keys are, zeros past
    // the last row and past D_qk
    {
        constexpr int kUnitsRow = DQ * L::kElt / 16;
        for (int i = threadIdx.x; i < kRowsTile * kUnitsRow; i += kThreads) {
            const int r = i / kUnitsRow, c = i % kUnitsRow;
            const int f = f0 + r;
            const int bytes = r < n_rows ? min(16, max(0, p.D_qk * L::kElt - c * 16)) : 0;
            const void *src = p.Q;
            if (bytes > 0) {
                const int bb = p.all_rows ? f / per_b : b;
                const int fs = p.all_rows ? f - bb * per_b : f;
                const int s = fs / p.G, g = fs - s * p.G;
                src = static_cast<const T *>(p.Q) + bb * p.q_sb + static_cast<long long>(hk * p.G + g) * p.q_sh +
                      s * p.q_ss + c * (16 / L::kElt);
            }
            cp_async16(base + L::kQ + (c >> 3) * L::kPiece + r * 128 + (((c & 7) ^ (r & 7)) << 4), src, bytes);
        }
        cp_async_commit();
    }

    if (!p.all_rows) {
        if (len < 0 || len > p.S_c) {  // a length outside the cache counts as the nearest one inside
            if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
            len = len < 0 ? 0 : p.S_c;
        }
    }
    // The key axis: the prefix's blocks, then the cache's.  Row f sees the prefix and the first own(f) cache rows.
    const int nP = (p.all_rows || p.with_prefix) ? p.S_p : 0;
    const int c0 = (nP + kKeys - 1) / kKeys * kKeys;  // where the cache starts on it
    auto own = [&](int f) { return p.all_rows ? 0 : max(0, len - p.S_q + f / p.G + 1); };
    const int context = kTree ? max(0, len - p.S_q) : 0;  // keys before the tree
    const int own_last = own(f0 + n_rows - 1), own_first = kTree ? context : own(f0);
    const int blocks = (c0 + own_last + kKeys - 1) / kKeys;
    const int cuts = p.cluster * p.shares;
    const int per = (blocks + cuts - 1) / cuts;
    const int first = min(blocks, (share * p.cluster + rank) * per), last = min(blocks, first + per);

    // ---- loads: block blk into stage s, issued by one lane
    auto load = [&](int blk, int s) {
        const int k0 = blk * kKeys;
        const uint32_t dk = wbase + s * L::kStage, dv = dk + L::kBytesK, bar = smem_u32(&full[warp][s]);
        const bool pre = k0 < c0;
        const CUtensorMap *mk = pre ? &maps.kp : &maps.kc, *mv = pre ? &maps.vp : &maps.vc;
        const int row = pre ? k0 : k0 - c0, seq = pre ? 0 : b;
        mbar_arrive_expect_tx(bar, L::kStage);
#pragma unroll
        for (int i = 0; i < DQ / L::kCols; ++i) tma_load_4d(dk + i * L::kPiece, mk, bar, i * L::kCols, row, hk, seq);
#pragma unroll
        for (int i = 0; i < DV / L::kCols; ++i) tma_load_4d(dv + i * L::kPiece, mv, bar, i * L::kCols, row, hk, seq);
    };

    const int n_mine = last > first + warp ? (last - first - warp + kWarps - 1) / kWarps : 0;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
        fence_mbar_init();
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            if (i < n_mine) load(first + warp + i * kWarps, i);
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- the queries in the layout of an MMA's A operand: this thread's rows are lane / 4 and lane / 4 + 8
    const int g8 = lane >> 2, t4 = lane & 3;
    constexpr int kSteps = kBf ? DQ / 16 : DQ / 8;
    uint32_t q[kSteps][4];
    {
        // matrices: rows 0-7 and 8-15 of 16-byte column 2 ks, then of column 2 ks + 1
        const int r = lane & 15;
        const uint32_t row = base + L::kQ + r * 128, odd = lane >> 4;
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
            ldsm4(q[ks], row + (ks >> 2) * L::kPiece + (((2 * (ks & 3) + odd) ^ (r & 7)) << 4));
    }
    // The scale is folded into the exponent (one rounding, near 0 for the keys that count), so it has to be positive:
    // its sign goes to the queries, and with a scale of 0 they become 0.
    const float scale = p.scale_log2 == 0.0f ? 1.0f : fabsf(p.scale_log2);
    if (p.scale_log2 <= 0.0f) {
        const uint32_t keep = p.scale_log2 == 0.0f ? 0u : ~0u, sign = keep & (kBf ? 0x80008000u : 0x80000000u);
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
            for (int j = 0; j < 4; ++j) q[ks][j] = (q[ks][j] & keep) ^ sign;
    }
    const int lim[2] = {g8 < n_rows ? own(f0 + g8) : 0, g8 + 8 < n_rows ? own(f0 + g8 + 8) : 0};
    unsigned long long seen[2] = {0, 0};  // kTree: the nodes that the two rows see
    if constexpr (kTree) {
        tree.follow(p.S_q, lane, p.status);
#pragma unroll
        for (int r = 0; r < 2; ++r) seen[r] = tree.of(min(f0 + g8 + 8 * r, per_b - 1) / p.G);
    }

    float o[DV / 8][4];
#pragma unroll
    for (int n = 0; n < DV / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, c[2] = {0.f, 0.f};

    bool ok = true;
    int stage = 0, issued = min(n_mine, kStages - 1);
    uint32_t parity = 0;
    for (int it = 0; it < n_mine; ++it) {
        ok = __all_sync(0xffffffffu, wait_limited(smem_u32(&full[warp][stage]), parity, p)) != 0;
        if (!ok) break;
        if (issued < n_mine) {  // into the stage read last time (every lane has passed it)
            if (lane == 0) load(first + warp + issued * kWarps, stage == 0 ? kStages - 1 : stage - 1);
            ++issued;
        }
        const int k0 = (first + warp + it * kWarps) * kKeys;
        const uint32_t sk = wbase + stage * L::kStage, sv = sk + L::kBytesK;
        // keys of the block that exist
        const int n_keys = k0 < c0 ? nP - k0 : c0 + own_last - k0;
        if (k0 >= c0 && n_keys < kKeys) {  // the cache's last block (the prefix's is filled with zeros by the map)
            constexpr int kUnits = static_cast<int>(L::kBytesV / 16);
            for (int i = lane; i < kUnits; i += 32)
                if (((i >> 3) & (kKeys - 1)) >= n_keys)
                    *reinterpret_cast<uint4 *>(smem + (sv - base) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
        }
        if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
        }

        // ---- scores of 16 rows x 16 keys: s[n] holds keys 8 n + 2 t4, + 1 of rows g8 (0, 1) and g8 + 8 (2, 3)
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        float low[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // fp32: the small products' own sums
        {
            // lane 8 j + i addresses row i of matrix j: keys 0-7 and 8-15, 16-byte columns 2 ks and 2 ks + 1
            const int key = (lane & 7) + ((lane >> 4) << 3);
            const uint32_t row = sk + key * 128;
            const uint32_t odd = (lane >> 3) & 1;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                uint32_t kb[4];
                ldsm4(kb, row + (ks >> 2) * L::kPiece + (((2 * (ks & 3) + odd) ^ (key & 7)) << 4));
                if (kBf) {
                    mma_bf16(s[0], q[ks], kb[0], kb[1]);
                    mma_bf16(s[1], q[ks], kb[2], kb[3]);
                } else {
                    mma_3xtf32<false>(s[0], low[0], q[ks], kb[0], kb[1]);
                    mma_3xtf32<false>(s[1], low[1], q[ks], kb[2], kb[3]);
                }
            }
        }
        if (!kBf) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)  // (beside an infinity the small products may be NaN)
                    if (fabsf(s[n][i]) != INFINITY) s[n][i] += low[n][i];
        }
        if (k0 < c0 ? n_keys < kKeys : k0 + kKeys > c0 + own_first) {  // some row does not see every key
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = k0 + 8 * n + 2 * t4 + (i & 1);
                    if (key >= (k0 < c0 ? nP : c0 + lim[i >> 1])) s[n][i] = -INFINITY;
                    if (kTree && k0 >= c0) {
                        const int node = key - c0 - (len - p.S_q);
                        if (node >= 0 && !((seen[i >> 1] >> (node & 63)) & 1ull)) s[n][i] = -INFINITY;
                    }
                }
        }

        // ---- online softmax of the two rows
        float alpha[2];
        bool moved = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float mx = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx *= scale;
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
                    s[n][i] = ex2(fmaf(s[n][i], scale, -ref));
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
            // P goes in as bf16, as in the library's other bf16 kernels: an error of 1.2e-3 of O beside its own rounding's
            // 1.66e-3 (2.05e-3 in all; norms, random inputs).  The rest of P in a second product would leave the rounding
            // alone, and take 0.5 to 1.5 % more time (ragged caches 40.9 -> 41.5 us).
            const uint32_t a[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                                   pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
            // matrices: keys 0-7 and 8-15 of 16-byte column n, then of column n + 1
            const int key = lane & 15;
            const uint32_t row = sv + key * 128;
            const uint32_t odd = lane >> 4;
#pragma unroll
            for (int n = 0; n < DV / 8; n += 2) {
                uint32_t vb[4];
                ldsm4_t(vb, row + (n >> 3) * L::kPiece + ((((n & 7) + odd) ^ (key & 7)) << 4));
                mma_bf16(o[n], a, vb[0], vb[1]);
                mma_bf16(o[n + 1], a, vb[2], vb[3]);
            }
        } else {
            // the k index of the product runs over keys in the order 0, 2, 4, 6, 1, 3, 5, 7, so the scores are
            // the A operand as they lie
            const uint32_t a[2][4] = {
                {__float_as_uint(s[0][0]), __float_as_uint(s[0][2]), __float_as_uint(s[0][1]), __float_as_uint(s[0][3])},
                {__float_as_uint(s[1][0]), __float_as_uint(s[1][2]), __float_as_uint(s[1][1]), __float_as_uint(s[1][3])}};
            // d += the products of keys 8 j and on with columns 8 n and on
            auto pv = [&](int n, int j, float (&d)[4]) {
                const int col = (n & 3) * 8 + g8, key = 8 * j + 2 * t4;
                const uint32_t in = (n >> 2) * L::kPiece + (col & 3) * 4, unit = col >> 2;
                const uint8_t *r0 = smem + (sv - base) + key * 128, *r1 = r0 + 128;
                mma_3xtf32<true>(d, d, a[j], *reinterpret_cast<const uint32_t *>(r0 + in + ((unit ^ (key & 7)) << 4)),
                                 *reinterpret_cast<const uint32_t *>(r1 + in + ((unit ^ ((key + 1) & 7)) << 4)));
            };
            if constexpr (kTree) {
                // a block's products are summed apart, because the tensor core cuts what it adds to an accumulator
                // (eight trees of 13 behind 1000 keys: 1.1e-6 of O and 39 us on one accumulator, 4.5e-7 and 41 us this way)
#pragma unroll
                for (int n = 0; n < DV / 8; ++n) {
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    pv(n, 0, sum);
                    pv(n, 1, sum);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][i] += sum[i];
                }
            } else {
                // (columns inside: the products after each other belong to different accumulators)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int n = 0; n < DV / 8; ++n) pv(n, j, o[n]);
            }
        }
        __syncwarp();
    }
    if (!ok && lane == 0) {  // gave up: the copies in flight land before their memory is used otherwise
        for (int it = max(0, issued - kStages); it < issued; ++it)
            wait_limited(smem_u32(&full[warp][it % kStages]), (it / kStages) & 1, p);
    }
    __syncwarp();

    // ---- the warp's result
    float *wo = reinterpret_cast<float *>(smem + warp * L::kWarpBytes);
    float *wm = wo + kRowsTile * L::kLdO;
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
            *reinterpret_cast<float2 *>(wo + (g8 + 8 * r) * L::kLdO + n * 8 + 2 * t4) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    if (p.prior) wait_prerequisites();

    // ---- combine: this CTA takes rows rank, rank + cluster, ... of the unit, one warp per row, over the cluster's warps
    // and the workspace's shares
    using C = Combine<T, DV>;
    const uint32_t o_off = base, m_off = base + kRowsTile * L::kLdO * 4;
    const int n_smem = kWarps * p.cluster, n_src = n_smem + p.prior;
#pragma unroll 1
    for (int i = rank + p.cluster * warp; i < n_rows; i += p.cluster * kWarps) {
        const int f = f0 + i;
        const long long flat = static_cast<long long>(hk) * p.B * per_b + static_cast<long long>(b) * per_b + f;
        auto warp_part = [&](uint32_t off, int src) {  // a warp's part of the cluster's shared memory
            const uint32_t at = off + (src % kWarps) * L::kWarpBytes;
            return p.cluster > 1 ? cluster_map(at, src / kWarps) : at;
        };
        C c;
        c.run(
            lane, n_src,
            [&](int src, int col, typename C::Vec &v) {
                if (src < n_smem) v = ld_cluster_vec<typename C::Vec>(warp_part(o_off, src) + (i * L::kLdO + col) * 4);
                else if (col < p.part_ld)
                    v = *reinterpret_cast<const typename C::Vec *>(p.part_o + ((src - n_smem) * p.rows + flat) * p.part_ld + col);
            },
            [&](int src, float &m, float &l, float &fix) {
                if (src < n_smem) {
                    const uint32_t at = warp_part(m_off, src) + i * 4;
                    m = ld_cluster(at);
                    l = ld_cluster(at + kRowsTile * 4);
                    fix = ld_cluster(at + 2 * kRowsTile * 4);
                } else {
                    const long long at = (src - n_smem) * p.rows + flat;
                    m = p.part_m[at];
                    l = p.part_l[at];
                    fix = p.part_c[at];
                }
            });
        if (p.partial) {
            const long long at = (p.share0 + share) * p.rows + flat;
            if (c.col < p.part_ld)
                *reinterpret_cast<typename C::Vec *>(p.part_o + at * p.part_ld + c.col) = c.vec();
            if (lane == 0) {
                p.part_m[at] = c.M;
                p.part_l[at] = c.Ls;
                p.part_c[at] = c.Lo - c.Ls;
            }
        } else {
            c.store(p, lane, b, hk, f);
        }
    }
    if (p.cluster > 1) cluster_sync();  // the other CTAs have read this one's results
    if (!p.all_rows && p.partial) {
        // The launch that adds the shares may start, and waits for this one to end.  That has to be after the prefix's
        // launch ends too, which nothing else sees to: one cluster stays until then.
        launch_dependents();
        if (p.follows && blockIdx.x < static_cast<unsigned>(p.cluster)) wait_prerequisites();
    }
}

}  // namespace st
}  // namespace vt
