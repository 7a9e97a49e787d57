// Gradients of the attention over packed sequences, bf16, for sm_103a (contract in include/vt_attn.h, vt_attn_bwd_packed).
//
// With s = scale q . k, P = exp(s - LSE), g = dO, delta = sum_e g_e O_e - dLSE:
//   dV = P^T g,   dS = P o (g V^T - delta),   dQ = scale dS K,   dK = scale dS^T Q.
// Three launches, or four.  attn_bwd_stats_kernel forms -LSE log2(e) and -delta of every query; attn_bwd_kv_bf16_kernel walks
// the queries of a 128-key block (dK, dV); attn_bwd_q_bf16_kernel walks the keys of a 128-query block (dQ).  The two walks
// form S and dO V^T twice, 7 products of 128 x 128 x D per pair of blocks where one walk would take 5; in return no sum of a
// query head crosses CTAs: no atomics, no fp32 dQ in memory, the same result in every call.  Where blocks of keys are few and
// heads share them, the keys' walk takes one query head per CTA and leaves its dK and dV in the workspace (fp32), and
// attn_bwd_heads_kernel, the fourth launch, adds a group's in the order of its heads: the same result in every call again.
//
// Every tensor core operand lies as TMA left it or as a warpgroup wrote it to TMEM: the keys' walk forms the transposed
// S^T = K Q^T and dP^T = V dO^T, whose rows are keys, so that P^T and dS^T are A operands from TMEM; Q and dO are K-major B
// operands of the first two products and N-major ones of the last two, from one copy in shared memory.
//
// Measured (16 texts of 128 to 4096 tokens, 32 heads on 8, D = 128, causal): statistics 59 us, keys' walk 498 us (1.49
// PFLOP/s of its four products), queries' walk 437 us (1.27 of its three).  Sequences of 4096 keep the tensor pipe 75 and 64 %
// busy (ncu).  A tile's products take the pipe 2048 and 1536 cycles; a tile takes 2830 and 2160 (clock64): the pipe waits
// for the warpgroups' exponentials (about 1000 cycles for 64 columns a thread) in the keys' walk, whose next scores need
// P's place in TMEM, and a unit's end and start cost 4200 cycles beside its 9 tiles in the queries' walk.
// Widths up to 64 halve the products and not the exponentials: 9 images of 256 to 2048 patches, 16 heads, 182 to 190 us in all.
//
// Errors of dQ and dK (norms, random inputs, 40 to 2000 keys): 1.66e-3 is their own rounding to bf16; dS rounded to bf16, as
// the tensor core takes it, makes that 2.3e-3 to 2.4e-3, and delta from an O that was rounded 2.4e-3 to 2.6e-3.  The rest of dS
// in a product of its own would leave out the first, for 9 products where there are 7; delta from P and dP in fp32 the second,
// for a walk more.
//
// Warps (both kernels, 12): 0 loads (TMA, one lane) and draws the units (cluster launch control, as in
// vt_attn_bf16_2q.cuh); 1 allocates TMEM and issues every MMA (one lane); 4-7 and 8-11 compute, columns 0-63 and 64-127
// of a tile, one row per thread.  A warpgroup writes its bf16 P or dS over the first half of the columns it read itself.
#pragma once

#include <cstring>

#include "vt_attn_packed.cuh"

namespace vt {

// What the gradients' kernels take beside the attention's parameters.
struct BwdParams : AttnParams {
    float scale;
    float *stat;      // [H][slots_q][2][128]: -LSE log2(e), then -delta, of the slot's rows (-inf and 0 past the end)
    int slots_q;      // slots of 128 query rows
    int units;        // work units of a launch
    // The keys' walk: query heads of a unit and units of a key/value head.  All heads of the group in one unit, or (few
    // blocks of keys) one head a unit, whose results go to part_k and part_v for attn_bwd_heads_kernel to add.
    int groups, head_units;
    float *part_k, *part_v;  // [H][T_k][part_ldk], [H][T_k][part_ldv]; null with one unit
    int part_ldk, part_ldv;
    int n_qk;         // MMA N of dQ and dK: D_qk rounded up to 16
    int q_slots, v_slots;  // ring slots: of Q and dO (keys' walk), or of K and V (queries' walk)
    const void *dO;
    long long do_sh, do_ss;
    const float *dlse;
    void *dQ, *dK, *dV;
    long long dq_sh, dq_ss, dk_sh, dk_ss, dv_sh, dv_ss;
    int dq_vec32, dk_vec32, dv_vec32;  // rows start on 32 bytes
};

namespace bw {

constexpr int kTile = 128;  // rows of a block, on both sides
constexpr int kThreads = 384;
constexpr int kRegsControl = 72, kRegsCompute = 216;
static_assert(128 * kRegsControl + 256 * kRegsCompute <= kThreads * 168, "register split exceeds the launch");
constexpr int kChunk = 64;                       // bf16 elements of a 128-byte chunk
constexpr uint32_t kChunkBytes = kTile * 128;    // a 128-byte column chunk of a tile
constexpr uint32_t kStatBytes = 2 * kTile * 4;
constexpr int kMaxSlots = 4;  // of one ring
constexpr int kUnitRing = 4, kUnitReaders = 1 + 8;
constexpr uint32_t kTmemCols = 512;

// A block of 128 rows of one head of a sequence, and the tiles of the other side that it walks.
struct Unit {
    int u;               // -1: no more units
    int h;               // query head (dQ) or key/value head (dK, dV)
    int r0;              // the block's first row in its sequence
    int q0, len_q, k0, len_k;
    int qslot;           // the sequence's first slot of 128 queries
    int lo, n;           // first tile, and tiles
};

struct Ctl {
    // the walked side's two rings: [0] Q or K, with the queries' statistics, [1] dO or V
    uint64_t full[2][kMaxSlots], empty[2][kMaxSlots];
    uint64_t own_full, own_empty;   // the unit's own tiles (K and V, or Q and dO)
    uint64_t s_full[2], dp_full, p_full, ds_full, done;
    uint64_t unit_full[kUnitRing], unit_empty[kUnitRing];
    Unit unit[kUnitRing];
    uint4 clc_resp;
    uint64_t clc_full;
    uint64_t drain;
    uint32_t tmem_base;
    volatile uint32_t abort_flag;
};

__device__ __forceinline__ int clamp_to(long long x, int most) {
    return static_cast<int>(x < 0 ? 0 : (x > most ? most : x));
}

// kKeys: a block of keys and the queries that see one of them; otherwise a block of queries and the keys they see.  The heads
// of a block are adjacent, and blocks with more work come first (a causal mask gives early keys and late queries the most
// partners).
template <bool kKeys>
__device__ __forceinline__ int unit_heads(const BwdParams &p) { return kKeys ? p.H / p.groups : p.H; }
// The block of unit u, by one lane or (first units) by a whole warp.
template <bool kKeys, bool kWarp>
__device__ __forceinline__ PackedSeq unit_block(const BwdParams &p, int u) {
    const int slot = u / unit_heads<kKeys>(p);
    const int *cu = kKeys ? p.cu_k : p.cu_q;
    const int T = kKeys ? p.S_k : p.S_q, at = kKeys ? slot : p.slots_q - 1 - slot;
    if constexpr (kWarp) return packed_find_warp(cu, p.n_seq, T, kTile, at, threadIdx.x & 31);
    return packed_find(cu, p.n_seq, T, kTile, at);
}
template <bool kKeys>
__device__ __forceinline__ Unit decode(const BwdParams &p, int u, const PackedSeq &own) {
    Unit U;
    U.u = u;
    U.h = u % unit_heads<kKeys>(p);
    if (kKeys && p.S_q == 0 && U.h == 0) packed_check(p, u / unit_heads<kKeys>(p));  // (else the statistics' launch does)
    const PackedSeq other = kKeys ? packed_seq(p.cu_q, own.n, p.S_q) : packed_seq(p.cu_k, own.n, p.S_k);
    U.r0 = own.block * kTile;
    U.q0 = kKeys ? other.start : own.start;
    U.len_q = kKeys ? other.len : own.len;
    U.k0 = kKeys ? own.start : other.start;
    U.len_k = kKeys ? own.len : other.len;
    U.qslot = U.q0 / kTile + own.n;
    U.lo = U.n = 0;
    if (U.r0 < own.len) {
        const long long off = static_cast<long long>(U.len_k) - U.len_q;
        const int last = min(U.r0 + kTile, own.len) - 1;
        // partners [a, e) of rows r0..last
        const int a = clamp_to(kKeys ? U.r0 - off - p.band_hi : U.r0 + off + p.band_lo, other.len);
        const int e = clamp_to(kKeys ? last - off - p.band_lo + 1 : last + off + p.band_hi + 1, other.len);
        if (a < e) {
            U.lo = a / kTile;
            U.n = (e + kTile - 1) / kTile - U.lo;
        }
    }
    return U;
}

// Invariants of a decoded unit, checked by the debug build.
template <bool kKeys>
__device__ __forceinline__ bool valid(const BwdParams &p, const Unit &U) {
    const int other = kKeys ? U.len_q : U.len_k;
    return U.h >= 0 && U.h < p.H && U.r0 >= 0 && U.q0 >= 0 && U.len_q >= 0 && U.len_q <= p.S_q - U.q0 && U.k0 >= 0 &&
           U.len_k >= 0 && U.len_k <= p.S_k - U.k0 && U.lo >= 0 && U.n >= 0 && U.lo + U.n <= (other + kTile - 1) / kTile &&
           U.qslot + (U.len_q + kTile - 1) / kTile <= p.slots_q;
}

__device__ __forceinline__ bool next_unit(Ctl &ctl, int n, Unit *out, const BwdParams &p, int lane) {
    const int k = n % kUnitRing;
    bool ok = true;
    if (lane == 0) ok = wait_bounded(smem_u32(&ctl.unit_full[k]), (n / kUnitRing) & 1, ctl.abort_flag, p);
    if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
    __syncwarp();
    const volatile Unit *src = &ctl.unit[k];
    out->u = src->u;
    out->h = src->h;
    out->r0 = src->r0;
    out->q0 = src->q0;
    out->len_q = src->len_q;
    out->k0 = src->k0;
    out->len_k = src->len_k;
    out->qslot = src->qslot;
    out->lo = src->lo;
    out->n = src->n;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ctl.unit_empty[k]));
    return true;
}

// A ring of shared-memory slots, as one role follows it: slot s, and for each slot the parity of its next phase.
struct Ring {
    int s = 0, n;
    uint32_t phase = 0;
    __device__ __forceinline__ explicit Ring(int slots) : n(slots) {}
    __device__ __forceinline__ uint32_t parity() const { return (phase >> s) & 1u; }
    __device__ __forceinline__ void next() {
        phase ^= 1u << s;
        if (++s == n) s = 0;
    }
};
// The producer's side: the slot to load next, free once its previous tile has been read.
struct LoadRing : Ring {
    int loads = 0;
    __device__ __forceinline__ explicit LoadRing(int slots) : Ring(slots) {}
    __device__ __forceinline__ bool wait(Ctl &ctl, int which, const BwdParams &p) {
        // (the first round finds every slot free: its phases are not waited for)
        return loads < n || wait_bounded(smem_u32(&ctl.empty[which][s]), parity(), ctl.abort_flag, p);
    }
    __device__ __forceinline__ void loaded() {
        if (loads >= n) phase ^= 1u << s;
        ++loads;
        if (++s == n) s = 0;
    }
    // Every copy lands before the CTA's memory goes away.
    __device__ __forceinline__ void drain(Ctl &ctl, int which, const BwdParams &p) const {
        for (int k = max(0, loads - n); k < loads; ++k) wait_drain(smem_u32(&ctl.full[which][k % n]), (k / n) & 1, p);
    }
};

// The producer lane draws the n-th unit of this CTA and publishes it; false on abort.  `first`: the block of the first.
template <bool kKeys>
__device__ __forceinline__ bool draw_unit(Ctl &ctl, int n, const PackedSeq &first, Unit *out, bool *clc_done, uint32_t *clc_par,
                                          const BwdParams &p) {
    const int k = n % kUnitRing;
    if (n >= kUnitRing && !wait_bounded(smem_u32(&ctl.unit_empty[k]), ((n / kUnitRing) - 1) & 1, ctl.abort_flag, p))
        return false;
    int u = -1;
    if (n == 0) {
        u = static_cast<int>(blockIdx.x);
    } else if (!*clc_done) {
        mbar_arrive_expect_tx(smem_u32(&ctl.clc_full), 16);
        clc_try_cancel(smem_u32(&ctl.clc_resp), smem_u32(&ctl.clc_full));
        if (!wait_bounded(smem_u32(&ctl.clc_full), *clc_par, ctl.abort_flag, p)) return false;
        *clc_par ^= 1u;
        u = clc_cancelled_x(smem_u32(&ctl.clc_resp));
        if (u < 0) *clc_done = true;
    }
    Unit U{};
    U.u = -1;
    if (u >= 0 && u < p.units) {
        U = decode<kKeys>(p, u, n == 0 ? first : unit_block<kKeys, false>(p, u));
        if (!VT_DEV_CHECK(valid<kKeys>(p, U), ctl.abort_flag, p)) return false;
    }
    volatile Unit *dst = &ctl.unit[k];
    dst->u = U.u;
    dst->h = U.h;
    dst->r0 = U.r0;
    dst->q0 = U.q0;
    dst->len_q = U.len_q;
    dst->k0 = U.k0;
    dst->len_k = U.len_k;
    dst->qslot = U.qslot;
    dst->lo = U.lo;
    dst->n = U.n;
    mbar_arrive(smem_u32(&ctl.unit_full[k]));
    *out = U;
    return true;
}

__device__ __forceinline__ void init(Ctl &ctl) {
    for (int r = 0; r < 2; ++r)
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(smem_u32(&ctl.full[r][i]), 1);
            mbar_init(smem_u32(&ctl.empty[r][i]), 1);
        }
    mbar_init(smem_u32(&ctl.own_full), 1);
    mbar_init(smem_u32(&ctl.own_empty), 1);
    mbar_init(smem_u32(&ctl.s_full[0]), 1);
    mbar_init(smem_u32(&ctl.s_full[1]), 1);
    mbar_init(smem_u32(&ctl.dp_full), 1);
    mbar_init(smem_u32(&ctl.p_full), 256);
    mbar_init(smem_u32(&ctl.ds_full), 256);
    mbar_init(smem_u32(&ctl.done), 1);
    for (int k = 0; k < kUnitRing; ++k) {
        mbar_init(smem_u32(&ctl.unit_full[k]), 1);
        mbar_init(smem_u32(&ctl.unit_empty[k]), kUnitReaders);
    }
    mbar_init(smem_u32(&ctl.clc_full), 1);
    mbar_init(smem_u32(&ctl.drain), 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
}

// Zero rows n and on of a tile in shared memory (the whole warp): rows behind a sequence's end may hold NaN, which a
// factor of 0 does not hide.  The tensor core sees the zeros afterwards.
__device__ __forceinline__ void clear_rows(uint32_t tile, int chunks, int n, int lane) {
    for (int c = 0; c < chunks; ++c)
        for (int i = n * 8 + lane; i < kTile * 8; i += 32)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + c * kChunkBytes + i * 16), "r"(0) : "memory");
    fence_async_shared();
    __syncwarp();
}

// A tile of 128 rows: `chunks` boxes from row `row` of head h.
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *m, uint32_t bar, int chunks, int row, int h) {
    for (int c = 0; c < chunks; ++c) tma_load_4d(dst + c * kChunkBytes, m, bar, c * kChunk, row, h, 0);
}

// D columns of this thread's TMEM row, times f, as a bf16 row of global memory.
__device__ __forceinline__ void store_row(uint32_t tmem, bool any, uint16_t *row, bool ok, int D, float f, bool vec32) {
    for (int cc = 0; cc < D; cc += 16) {
        uint32_t o[16];
        __syncwarp();  // (lanes part below)
        if (any) {
            tmem_ld16(tmem + cc, o);
            tmem_wait_ld();
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0u;
        }
        if (!ok) continue;
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * f, __uint_as_float(o[2 * k + 1]) * f);
        if (cc + 16 <= D) {
            if (vec32) {
                st_global_v8(row + cc, w);
            } else {
                uint4 *dst = reinterpret_cast<uint4 *>(row + cc);
                dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (cc + k < D) row[cc + k] = static_cast<uint16_t>((w[k >> 1] >> ((k & 1) * 16)) & 0xFFFFu);
        }
    }
}

// The same row of fp32, `ld` columns (a multiple of 8).
__device__ __forceinline__ void store_part(uint32_t tmem, bool any, float *row, bool ok, int ld) {
    for (int cc = 0; cc < ld; cc += 16) {
        uint32_t o[16];
        __syncwarp();  // (lanes part below)
        if (any) {
            tmem_ld16(tmem + cc, o);
            tmem_wait_ld();
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0u;
        }
        if (!ok) continue;
        const uint32_t a[8] = {o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]};
        const uint32_t b[8] = {o[8], o[9], o[10], o[11], o[12], o[13], o[14], o[15]};
        st_global_v8(row + cc, a);
        if (cc + 16 <= ld) st_global_v8(row + cc + 8, b);
    }
}

// Products D (+)= A B^T of K-steps of 16 columns, A and B K-major tiles in shared memory.
template <int KS>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t lead) {
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        const uint32_t off = (kk >> 2) * (kChunkBytes >> 4) + (kk & 3) * 2;
        mma_ss_lead(d, a_lo + off, hi, b_lo + off, hi, idesc, kk > 0, lead);
    }
}
// D (+)= A B over 128 rows of B (N-major tile): A is the bf16 tile that the warpgroups wrote, 32 columns at `a` and 32 at
// a + 64.
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc0,
                                         uint32_t lead) {
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk)
        mma_ts_lead(d, a + (kk >> 2) * 64 + (kk & 3) * 8, b_lo + kk * 128, hi, idesc, (acc0 | kk) ? 1u : 0u, lead);
}

}  // namespace bw

// -LSE log2(e) and -delta of every query, by slots of 128 rows, so that a tile's lie together on 16 bytes.  Bound by the
// bytes of O and dO; 32 rows a CTA, two or four a thread at once, keep enough of them on their way.
constexpr int kStatThreads = 256;
constexpr int kStatRows = 32;
template <typename T>
__global__ void __launch_bounds__(kStatThreads) attn_bwd_stats_kernel(const __grid_constant__ BwdParams p) {
    constexpr int kVec = 16 / sizeof(T), kLanes = 128 / kVec;  // lanes of a row: 16 (bf16) or 32
    constexpr int kStep = kStatThreads / kLanes, kEach = kStatRows / kStep;  // rows at a time, and of a thread
    constexpr int kParts = bw::kTile / kStatRows;
    const int part = blockIdx.x % kParts, unit = blockIdx.x / kParts, slot = unit / p.H, h = unit - slot * p.H;
    const PackedSeq s = packed_find_warp(p.cu_q, p.n_seq, p.S_q, bw::kTile, slot, threadIdx.x & 31);
    const int lane = threadIdx.x % kLanes, col = lane * kVec;
    float *out = p.stat + (static_cast<long long>(h) * p.slots_q + slot) * (2 * bw::kTile);
    const int n = min(s.len - s.block * bw::kTile, bw::kTile);  // rows of the slot
    const long long first = static_cast<long long>(s.start) + s.block * bw::kTile;
    const T *o = static_cast<const T *>(p.O) + h * p.o_sh, *g = static_cast<const T *>(p.dO) + h * p.do_sh;
    const int r0 = part * kStatRows + threadIdx.x / kLanes;
    uint4 x[kEach], y[kEach];
    float lse[kEach], dl[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int r = r0 + i * kStep;
        const long long at = first + r;
        x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
        lse[i] = -INFINITY;
        dl[i] = 0.0f;
        if (r < n && col < p.D_v) {
            const T *a = o + at * p.o_ss + col, *b = g + at * p.do_ss + col;
            if (col + kVec <= p.D_v) {
                x[i] = __ldg(reinterpret_cast<const uint4 *>(a));
                y[i] = __ldg(reinterpret_cast<const uint4 *>(b));
            } else {  // (columns behind the last one are not read)
                T ta[kVec] = {}, tb[kVec] = {};
#pragma unroll
                for (int k = 0; k < kVec; ++k)
                    if (col + k < p.D_v) ta[k] = a[k], tb[k] = b[k];
                memcpy(&x[i], ta, 16);
                memcpy(&y[i], tb, 16);
            }
        }
        if (r < n && lane == 0) {
            lse[i] = p.lse[static_cast<long long>(h) * p.S_q + at];
            if (p.dlse) dl[i] = p.dlse[static_cast<long long>(h) * p.S_q + at];
        }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 2) {
                sum = fmaf(__uint_as_float(xs[k] << 16), __uint_as_float(ys[k] << 16), sum);
                sum = fmaf(__uint_as_float(xs[k] & 0xFFFF0000u), __uint_as_float(ys[k] & 0xFFFF0000u), sum);
            } else {
                sum = fmaf(__uint_as_float(xs[k]), __uint_as_float(ys[k]), sum);
            }
        }
#pragma unroll
        for (int m = kLanes / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const int r = r0 + i * kStep;
        if (lane == 0) {  // (a row without keys has no weight at all, and 0 times its delta would not hide a NaN)
            out[r] = lse[i] == -INFINITY ? -INFINITY : -lse[i] * 1.4426950408889634f;
            out[bw::kTile + r] = lse[i] == -INFINITY ? 0.0f : dl[i] - sum;
        }
    }
    if (part == 0 && h == 0 && threadIdx.x == 0) packed_check(p, slot);
}

// dK and dV of ROWS keys of one key/value head, from those of its query heads, added in their order.
constexpr int kHeadsThreads = 256, kHeadsRows = 8;  // rows of a CTA: a thread adds four columns of one, for dK and for dV
template <typename T, int ROWS>
__global__ void __launch_bounds__(kHeadsThreads) attn_bwd_heads_kernel(const __grid_constant__ BwdParams p) {
    constexpr int kParts = ROWS / kHeadsRows;
    const int part = blockIdx.x % kParts, unit = blockIdx.x / kParts;
    const int heads = p.H / p.kv_group, slot = unit / heads, hk = unit - slot * heads;
    const PackedSeq s = packed_find_warp(p.cu_k, p.n_seq, p.S_k, ROWS, slot, threadIdx.x & 31);
    const int r = part * kHeadsRows + threadIdx.x / 32, c = threadIdx.x % 32 * 4;
    if (r >= min(s.len - s.block * ROWS, ROWS)) return;
    const long long row = static_cast<long long>(s.start) + s.block * ROWS + r;
    auto add = [&](const float *from, int ld, int D, float f, T *out) {
        if (c >= D) return;
        const float *src = from + (static_cast<long long>(hk) * p.kv_group * p.S_k + row) * ld + c;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int g = 0; g < p.kv_group; ++g) {
            const float4 x = *reinterpret_cast<const float4 *>(src + static_cast<long long>(g) * p.S_k * ld);
            sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
        }
        const float v[4] = {sum.x * f, sum.y * f, sum.z * f, sum.w * f};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c + k < D) {
                if constexpr (sizeof(T) == 2) out[c + k] = static_cast<T>(pack_bf16x2(v[k], 0.0f) & 0xFFFFu);
                else out[c + k] = v[k];
            }
    };
    add(p.part_k, p.part_ldk, p.D_qk, p.scale, static_cast<T *>(p.dK) + hk * p.dk_sh + row * p.dk_ss);
    add(p.part_v, p.part_ldv, p.D_v, 1.0f, static_cast<T *>(p.dV) + hk * p.dv_sh + row * p.dv_ss);
}

// dK and dV of 128 keys of one key/value head.  Shared memory: K, V, then rings of Q (with its
// queries' statistics) and of dO.
// TMEM: S^T (P^T over it), dP^T (dS^T over it), dV, dK.  The tensor pipe's order per tile i is
//   dV += P_i^T dO_i,  S_{i+1} = K Q_{i+1}^T,  dK += dS_i^T Q_i,  dP_{i+1} = V dO_{i+1}^T,
// so that two products run while the warpgroups form dS_i, and two while they form P_{i+1}.
// KQ, KV: K-steps of 16 columns of D_qk and D_v (rounded up; the TMA fills zeros).
template <int KQ, int KV>
__global__ void __launch_bounds__(bw::kThreads, 1)
    attn_bwd_kv_bf16_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                            const __grid_constant__ BwdParams p) {
    using namespace bw;
    __shared__ Ctl ctl;
    extern __shared__ uint8_t smem_raw[];
    launch_dependents();  // the queries' walk takes the SMs that this one no longer fills
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t q_bytes = p.q_chunks * kChunkBytes, v_bytes = p.v_chunks * kChunkBytes;
    const uint32_t sK = base, sV = sK + q_bytes, sQ = sV + v_bytes, sG = sQ + p.q_slots * q_bytes;
    const uint32_t sStat = sG + p.v_slots * v_bytes;
    uint8_t *const smem = smem_raw + (base - raw);

    if (threadIdx.x == 0) init(ctl);
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmG);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctl.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    const uint32_t tS = tmem, tP = tmem + 128, tDV = tmem + 256, tDK = tmem + 384;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
        if (warp == 0) {
            const PackedSeq first = unit_block<true, true>(p, blockIdx.x);
            if (lane == 0) {
                bool ok = true, clc_done = false;
                uint32_t clc_par = 0;
                int owns = 0;
                LoadRing rq(p.q_slots), rg(p.v_slots);
                for (int n = 0; ok; ++n) {
                    Unit U;
                    if (!draw_unit<true>(ctl, n, first, &U, &clc_done, &clc_par, p) || U.u < 0) break;
                    if (U.n == 0) continue;
                    if (owns > 0 && !wait_bounded(smem_u32(&ctl.own_empty), (owns - 1) & 1, ctl.abort_flag, p)) break;
                    mbar_arrive_expect_tx(smem_u32(&ctl.own_full), q_bytes + v_bytes);
                    load_tile(sK, &tmK, smem_u32(&ctl.own_full), p.q_chunks, U.k0 + U.r0, U.h / p.head_units);
                    load_tile(sV, &tmV, smem_u32(&ctl.own_full), p.v_chunks, U.k0 + U.r0, U.h / p.head_units);
                    ++owns;
                    for (int g = 0; ok && g < p.groups; ++g) {
                        const int h = U.h * p.groups + g;
                        for (int t = U.lo; t < U.lo + U.n; ++t) {
                            if (!(ok = rq.wait(ctl, 0, p))) break;
                            uint32_t bar = smem_u32(&ctl.full[0][rq.s]);
                            mbar_arrive_expect_tx(bar, q_bytes + kStatBytes);
                            load_tile(sQ + rq.s * q_bytes, &tmQ, bar, p.q_chunks, U.q0 + t * kTile, h);
                            bulk_load(sStat + rq.s * kStatBytes,
                                      p.stat + (static_cast<long long>(h) * p.slots_q + U.qslot + t) * (2 * kTile), kStatBytes,
                                      bar);
                            rq.loaded();
                            if (!(ok = rg.wait(ctl, 1, p))) break;
                            bar = smem_u32(&ctl.full[1][rg.s]);
                            mbar_arrive_expect_tx(bar, v_bytes);
                            load_tile(sG + rg.s * v_bytes, &tmG, bar, p.v_chunks, U.q0 + t * kTile, h);
                            rg.loaded();
                        }
                    }
                }
                if (ctl.abort_flag) {
                    if (owns > 0) wait_drain(smem_u32(&ctl.own_full), (owns - 1) & 1, p);
                    rq.drain(ctl, 0, p);
                    rg.drain(ctl, 1, p);
                }
            }
        } else if (warp == 1) {
            const uint32_t idesc_s = instr_desc(1, kTile, kTile, 0);
            const uint32_t idesc_v = instr_desc(1, kTile, p.n_pv, 1), idesc_k = instr_desc(1, kTile, p.n_qk, 1);
            const uint64_t rows0 = smem_desc_sw128(sQ, 16, 1024), cols0 = smem_desc_sw128(sQ, kChunkBytes, 1024);
            const uint32_t r_hi = static_cast<uint32_t>(rows0 >> 32), c_hi = static_cast<uint32_t>(cols0 >> 32);
            const uint32_t k_lo = static_cast<uint32_t>(smem_desc_sw128(sK, 16, 1024));
            const uint32_t v_lo = static_cast<uint32_t>(smem_desc_sw128(sV, 16, 1024));
            // low words of slot 0 as rows (K-major) and as columns (N-major): Q, and dO behind it
            const uint32_t r_lo = static_cast<uint32_t>(rows0), c_lo = static_cast<uint32_t>(cols0), g_off = (sG - sQ) >> 4;
            const uint32_t q_step = q_bytes >> 4, g_step = v_bytes >> 4;
            const uint32_t lead = elect_leader();
            bool ok = true, any = false;
            uint32_t own_par = 0, p_par = 0, ds_par = 0;
            // The warp stays together: its lanes part in a wait, in clear_rows and where one of them arrives for all (next_unit),
            // and meet again in the __all_sync of the wait or the __syncwarp of clear_rows that stands between each of these and
            // the next MMA or commit.  All lanes come to these with the same operands, and the elected one issues them.
            auto wait1 = [&](uint32_t bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, wait_bounded(bar, parity, ctl.abort_flag, p)) != 0;
            };
            Ring rq(p.q_slots), rg(p.v_slots);   // the next tile's slots
            for (int n = 0; ok; ++n) {
                Unit U;
                if (!(ok = next_unit(ctl, n, &U, p, lane)) || U.u < 0) break;
                if (U.n == 0) continue;
                if (!(ok = wait1(smem_u32(&ctl.own_full), own_par))) break;
                own_par ^= 1u;
                const int total = U.n * p.groups;
                int tile = 0, rows = 0;  // of the head's tiles, and the rows of the next one that exist
                int q_at = 0, g_at = 0;  // slots of the current tile
                // S^T and dP^T of the next tile, once it has landed; rows behind the sequence's end become zeros
                auto scores = [&]() -> bool {
                    if (!wait1(smem_u32(&ctl.full[0][rq.s]), rq.parity())) return false;
                    rows = U.len_q - (U.lo + tile) * kTile;
                    if (++tile == U.n) tile = 0;
                    q_at = rq.s;
                    rq.next();
                    if (rows < kTile) clear_rows(sQ + q_at * q_bytes, p.q_chunks, rows, lane);
                    mma_rows<KQ>(tS, k_lo, r_lo + q_at * q_step, r_hi, idesc_s, lead);
                    mma_commit_lead(smem_u32(&ctl.s_full[0]), lead);
                    return true;
                };
                auto dscores = [&]() -> bool {
                    if (!wait1(smem_u32(&ctl.full[1][rg.s]), rg.parity())) return false;
                    g_at = rg.s;
                    rg.next();
                    if (rows < kTile) clear_rows(sG + g_at * v_bytes, p.v_chunks, rows, lane);
                    mma_rows<KV>(tP, v_lo, r_lo + g_off + g_at * g_step, r_hi, idesc_s, lead);
                    mma_commit_lead(smem_u32(&ctl.dp_full), lead);
                    return true;
                };
                any = true;
                if (!(ok = scores() && dscores())) break;
                if (total == 1) mma_commit_lead(smem_u32(&ctl.own_empty), lead);
                for (int i = 0; i < total; ++i) {
                    const bool more = i + 1 < total;
                    const int q_now = q_at;
                    if (!(ok = wait1(smem_u32(&ctl.p_full), p_par))) break;
                    p_par ^= 1u;
                    tc_fence_after();
                    mma_cols(tDV, tS, c_lo + g_off + g_at * g_step, c_hi, idesc_v, i > 0, lead);
                    mma_commit_lead(smem_u32(&ctl.empty[1][g_at]), lead);
                    if (more && !(ok = scores())) break;
                    if (!(ok = wait1(smem_u32(&ctl.ds_full), ds_par))) break;
                    ds_par ^= 1u;
                    tc_fence_after();
                    mma_cols(tDK, tP, c_lo + q_now * q_step, c_hi, idesc_k, i > 0, lead);
                    mma_commit_lead(smem_u32(&ctl.empty[0][q_now]), lead);
                    if (more) {
                        if (!(ok = dscores())) break;
                        if (i + 2 == total) mma_commit_lead(smem_u32(&ctl.own_empty), lead);  // K and V are read
                    } else {
                        mma_commit_lead(smem_u32(&ctl.done), lead);
                    }
                }
            }
            if (!ok && any) {
                mma_commit_lead(smem_u32(&ctl.drain), lead);
                if (lane == 0) wait_drain(smem_u32(&ctl.drain), 0, p);
                __syncwarp();
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
        const int wg = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t aS = tS + lanes + wg * 64, aP = tP + lanes + wg * 64;
        const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
        uint32_t s_par = 0, dp_par = 0, done_par = 0;
        Ring rq(p.q_slots);
        bool ok = true;
        auto wait1 = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, wait_bounded(bar, parity, ctl.abort_flag, p)) != 0;
        };
        for (int n = 0; ok; ++n) {
            Unit U;
            if (!(ok = next_unit(ctl, n, &U, p, lane)) || U.u < 0) break;
            const int total = U.n * p.groups;
            // queries [q_lo, q_hi) see this thread's key
            const long long at = static_cast<long long>(U.r0) + row - (static_cast<long long>(U.len_k) - U.len_q);
            const int q_lo = clamp_to(at - p.band_hi, U.len_q), q_hi = clamp_to(at - p.band_lo + 1, U.len_q);
            // tiles that every key of the block sees in whole
            const int all_lo = clamp_to(at - row + kTile - 1 - p.band_hi, U.len_q);
            const int all_hi = clamp_to(at - row - p.band_lo + 1, U.len_q);
            // A query that sees one key has P = 1 whatever its score: dS is 0 (or dLSE), and not the rounding of dP - delta.
            // That is every query (window of 1, one key), or the one whose band ends at key 0.
            const bool lone = !p.dlse && (U.len_k == 1 || p.band_lo == p.band_hi);
            const int q_lone = !p.dlse && U.r0 + row == 0 && q_lo - at + p.band_hi == 0 ? q_lo : -1;
            int tile = U.lo;
            for (int i = 0; i < total; ++i) {
                const int q_first = tile * kTile;
                if (++tile == U.lo + U.n) tile = U.lo;
                const bool cut = q_first < all_lo || min(q_first + kTile, U.len_q) > all_hi;
                const float4 *stat = reinterpret_cast<const float4 *>(smem + (sStat - base) + rq.s * kStatBytes) + wg * 16;
                if (!(ok = wait1(smem_u32(&ctl.full[0][rq.s]), rq.parity()))) break;  // the statistics
                rq.next();
                if (!(ok = wait1(smem_u32(&ctl.s_full[0]), s_par))) break;
                s_par ^= 1u;
                tc_fence_after();
                uint32_t x[64];
                tmem_ld32(aS, x);
                tmem_ld32(aS + 32, x + 32);
                tmem_wait_ld();
                float2 pr[32];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float4 nl = stat[k];
                    const float2 a = __ffma2_rn(make_float2(__uint_as_float(x[4 * k]), __uint_as_float(x[4 * k + 1])), c2,
                                                make_float2(nl.x, nl.y));
                    const float2 b = __ffma2_rn(make_float2(__uint_as_float(x[4 * k + 2]), __uint_as_float(x[4 * k + 3])), c2,
                                                make_float2(nl.z, nl.w));
                    pr[2 * k] = make_float2(ex2(a.x), ex2(a.y));
                    pr[2 * k + 1] = make_float2(ex2(b.x), ex2(b.y));
                }
                if (cut) {
                    const int q = q_first + wg * 64;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (q + 2 * k < q_lo || q + 2 * k >= q_hi) pr[k].x = 0.0f;
                        if (q + 2 * k + 1 < q_lo || q + 2 * k + 1 >= q_hi) pr[k].y = 0.0f;
                    }
                }
                // P goes into dV's product as bf16 (2^-9 of each weight), dS below into dK's the same way
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) w[k] = pack_bf16x2(pr[16 * half + k].x, pr[16 * half + k].y);
                    tmem_st16(aS + 16 * half, w);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&ctl.p_full));
                if (lone || (q_lone >= q_first && q_lone < q_first + kTile)) {
                    const int q = q_first + wg * 64;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (lone || q + 2 * k == q_lone) pr[k].x = 0.0f;
                        if (lone || q + 2 * k + 1 == q_lone) pr[k].y = 0.0f;
                    }
                }

                if (!(ok = wait1(smem_u32(&ctl.dp_full), dp_par))) break;
                dp_par ^= 1u;
                tc_fence_after();
                tmem_ld32(aP, x);
                tmem_ld32(aP + 32, x + 32);
                tmem_wait_ld();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 nd = stat[32 + 8 * half + k];
                        const uint32_t *d = x + 32 * half + 4 * k;
                        const float2 *pp = pr + 16 * half + 2 * k;
                        const float2 a = __fmul2_rn(pp[0], __fadd2_rn(make_float2(__uint_as_float(d[0]), __uint_as_float(d[1])),
                                                                      make_float2(nd.x, nd.y)));
                        const float2 b = __fmul2_rn(pp[1], __fadd2_rn(make_float2(__uint_as_float(d[2]), __uint_as_float(d[3])),
                                                                      make_float2(nd.z, nd.w)));
                        w[2 * k] = pack_bf16x2(a.x, a.y);
                        w[2 * k + 1] = pack_bf16x2(b.x, b.y);
                    }
                    tmem_st16(aP + 16 * half, w);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&ctl.ds_full));
            }
            if (!ok) break;
            if (total > 0) {
                if (!(ok = wait1(smem_u32(&ctl.done), done_par))) break;
                done_par ^= 1u;
                tc_fence_after();
            }
            // warpgroup 0 stores dV, warpgroup 1 dK
            const bool mine = U.r0 + row < U.len_k;
            const long long key = static_cast<long long>(U.k0) + U.r0 + row;
            if (p.part_k) {
                const long long at = static_cast<long long>(U.h) * p.S_k + key;
                if (wg == 0) store_part(tDV + lanes, total > 0, p.part_v + at * p.part_ldv, mine, p.part_ldv);
                else store_part(tDK + lanes, total > 0, p.part_k + at * p.part_ldk, mine, p.part_ldk);
            } else if (wg == 0) {
                store_row(tDV + lanes, total > 0, static_cast<uint16_t *>(p.dV) + U.h * p.dv_sh + key * p.dv_ss, mine, p.D_v,
                          1.0f, p.dv_vec32);
            } else {
                store_row(tDK + lanes, total > 0, static_cast<uint16_t *>(p.dK) + U.h * p.dk_sh + key * p.dk_ss, mine, p.D_qk,
                          p.scale, p.dk_vec32);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// dQ of 128 queries of one head.  Shared memory: Q, dO, then rings of K and of V.
// TMEM: S of even and of odd key tiles (dS over them), dP, dQ.  The tensor pipe's order per tile j is
//   dP_{j+1} = dO V_{j+1}^T,  dQ += dS_j K_j,  S_{j+2} = Q K_{j+2}^T,
// so that the warpgroups, once past dS_j, wait for one product at most.
template <int KQ, int KV>
__global__ void __launch_bounds__(bw::kThreads, 1)
    attn_bwd_q_bf16_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                           const __grid_constant__ BwdParams p) {
    using namespace bw;
    __shared__ Ctl ctl;
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t q_bytes = p.q_chunks * kChunkBytes, v_bytes = p.v_chunks * kChunkBytes;
    const uint32_t sQ = base, sG = sQ + q_bytes, sK = sG + v_bytes, sV = sK + p.q_slots * q_bytes;

    if (threadIdx.x == 0) init(ctl);
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmG);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctl.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    const uint32_t tS = tmem, tP = tmem + 256, tDQ = tmem + 384;  // S of tile j at tS + 128 (j & 1)

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
        if (warp == 0) {
            const PackedSeq first = unit_block<false, true>(p, blockIdx.x);
            if (lane == 0) {
                bool ok = true, clc_done = false;
                uint32_t clc_par = 0;
                int owns = 0;
                LoadRing rk(p.q_slots), rv(p.v_slots);
                for (int n = 0; ok; ++n) {
                    Unit U;
                    if (!draw_unit<false>(ctl, n, first, &U, &clc_done, &clc_par, p) || U.u < 0) break;
                    if (U.n == 0) continue;
                    // the unit's Q and dO replace the previous one's, once those have been read: into L2 until then
                    for (int c = 0; c < p.q_chunks; ++c) tma_prefetch_l2_4d(&tmQ, c * kChunk, U.q0 + U.r0, U.h, 0);
                    for (int c = 0; c < p.v_chunks; ++c) tma_prefetch_l2_4d(&tmG, c * kChunk, U.q0 + U.r0, U.h, 0);
                    if (owns > 0 && !wait_bounded(smem_u32(&ctl.own_empty), (owns - 1) & 1, ctl.abort_flag, p)) break;
                    mbar_arrive_expect_tx(smem_u32(&ctl.own_full), q_bytes + v_bytes);
                    load_tile(sQ, &tmQ, smem_u32(&ctl.own_full), p.q_chunks, U.q0 + U.r0, U.h);
                    load_tile(sG, &tmG, smem_u32(&ctl.own_full), p.v_chunks, U.q0 + U.r0, U.h);
                    ++owns;
                    const int hk = U.h / p.kv_group;
                    for (int j = 0; j < U.n; ++j) {
                        const int key = U.k0 + (U.lo + j) * kTile;
                        if (!(ok = rk.wait(ctl, 0, p))) break;
                        uint32_t bar = smem_u32(&ctl.full[0][rk.s]);
                        mbar_arrive_expect_tx(bar, q_bytes);
                        load_tile(sK + rk.s * q_bytes, &tmK, bar, p.q_chunks, key, hk);
                        rk.loaded();
                        if (!(ok = rv.wait(ctl, 1, p))) break;
                        bar = smem_u32(&ctl.full[1][rv.s]);
                        mbar_arrive_expect_tx(bar, v_bytes);
                        load_tile(sV + rv.s * v_bytes, &tmV, bar, p.v_chunks, key, hk);
                        rv.loaded();
                    }
                }
                if (ctl.abort_flag) {
                    if (owns > 0) wait_drain(smem_u32(&ctl.own_full), (owns - 1) & 1, p);
                    rk.drain(ctl, 0, p);
                    rv.drain(ctl, 1, p);
                }
            }
        } else if (warp == 1) {
            const uint32_t idesc_s = instr_desc(1, kTile, kTile, 0), idesc_q = instr_desc(1, kTile, p.n_qk, 1);
            const uint64_t rows0 = smem_desc_sw128(sK, 16, 1024), cols0 = smem_desc_sw128(sK, kChunkBytes, 1024);
            const uint32_t r_hi = static_cast<uint32_t>(rows0 >> 32), c_hi = static_cast<uint32_t>(cols0 >> 32);
            const uint32_t q_lo = static_cast<uint32_t>(smem_desc_sw128(sQ, 16, 1024));
            const uint32_t g_lo = static_cast<uint32_t>(smem_desc_sw128(sG, 16, 1024));
            const uint32_t r_lo = static_cast<uint32_t>(rows0), c_lo = static_cast<uint32_t>(cols0), v_off = (sV - sK) >> 4;
            const uint32_t k_step = q_bytes >> 4, v_step = v_bytes >> 4;
            const uint32_t lead = elect_leader();
            bool ok = true, any = false;
            uint32_t own_par = 0, ds_par = 0, g = 0;  // g: key tiles of this CTA so far
            // (the warp stays together, as in the keys' walk)
            auto wait1 = [&](uint32_t bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, wait_bounded(bar, parity, ctl.abort_flag, p)) != 0;
            };
            Ring rk(p.q_slots), rv(p.v_slots);  // the next tiles' slots
            int k_at = 0;                       // slot of K_j
            for (int n = 0; ok; ++n) {
                Unit U;
                if (!(ok = next_unit(ctl, n, &U, p, lane)) || U.u < 0) break;
                if (U.n == 0) continue;
                if (!(ok = wait1(smem_u32(&ctl.own_full), own_par))) break;
                own_par ^= 1u;
                // S_j and dP_j, once K_j and V_j have landed; rows behind the sequence's end become zeros (dQ multiplies K by
                // weights of 0)
                auto scores = [&](int j) -> bool {
                    if (!wait1(smem_u32(&ctl.full[0][rk.s]), rk.parity())) return false;
                    const int rows = U.len_k - (U.lo + j) * kTile;
                    if (rows < kTile) clear_rows(sK + rk.s * q_bytes, p.q_chunks, rows, lane);
                    mma_rows<KQ>(tS + ((g + j) & 1u) * 128, q_lo, r_lo + rk.s * k_step, r_hi, idesc_s, lead);
                    mma_commit_lead(smem_u32(&ctl.s_full[(g + j) & 1u]), lead);
                    rk.next();
                    return true;
                };
                auto dscores = [&](int j) -> bool {
                    if (!wait1(smem_u32(&ctl.full[1][rv.s]), rv.parity())) return false;
                    const int rows = U.len_k - (U.lo + j) * kTile;
                    if (rows < kTile) clear_rows(sV + rv.s * v_bytes, p.v_chunks, rows, lane);
                    mma_rows<KV>(tP, g_lo, r_lo + v_off + rv.s * v_step, r_hi, idesc_s, lead);
                    mma_commit_lead(smem_u32(&ctl.dp_full), lead);
                    mma_commit_lead(smem_u32(&ctl.empty[1][rv.s]), lead);
                    rv.next();
                    return true;
                };
                any = true;
                if (!(ok = scores(0) && dscores(0))) break;
                if (U.n == 1) mma_commit_lead(smem_u32(&ctl.own_empty), lead);
                else if (!(ok = scores(1))) break;
                for (int j = 0; j < U.n; ++j) {
                    if (!(ok = wait1(smem_u32(&ctl.ds_full), ds_par))) break;
                    ds_par ^= 1u;
                    tc_fence_after();
                    if (j + 1 < U.n) {
                        if (!(ok = dscores(j + 1))) break;
                        if (j + 2 == U.n) mma_commit_lead(smem_u32(&ctl.own_empty), lead);  // Q and dO are read
                    }
                    mma_cols(tDQ, tS + ((g + j) & 1u) * 128, c_lo + k_at * k_step, c_hi, idesc_q, j > 0, lead);
                    mma_commit_lead(smem_u32(&ctl.empty[0][k_at]), lead);
                    if (++k_at == p.q_slots) k_at = 0;
                    if (j + 1 == U.n) mma_commit_lead(smem_u32(&ctl.done), lead);
                    if (j + 2 < U.n && !(ok = scores(j + 2))) break;
                }
                g += U.n;
            }
            if (!ok && any) {
                mma_commit_lead(smem_u32(&ctl.drain), lead);
                if (lane == 0) wait_drain(smem_u32(&ctl.drain), 0, p);
                __syncwarp();
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
        const int wg = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
        uint32_t dp_par = 0, done_par = 0, g = 0;
        bool ok = true;
        auto wait1 = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, wait_bounded(bar, parity, ctl.abort_flag, p)) != 0;
        };
        for (int n = 0; ok; ++n) {
            Unit U;
            if (!(ok = next_unit(ctl, n, &U, p, lane)) || U.u < 0) break;
            const int off = U.len_k - U.len_q;
            const int last = min(U.r0 + kTile, U.len_q) - 1;
            const int key_lo = packed_key_lo(p, off, U.len_k, U.r0 + row), key_hi = packed_key_hi(p, off, U.len_k, U.r0 + row);
            const int all_lo = packed_key_lo(p, off, U.len_k, last), all_hi = packed_key_hi(p, off, U.len_k, U.r0);
            float2 nl = make_float2(-INFINITY, -INFINITY), nd = make_float2(0.0f, 0.0f);
            if (U.n > 0 && (key_hi - key_lo > 1 || p.dlse)) {  // (a query that sees one key: dS is 0, and not the rounding of dP - delta)
                const float *st = p.stat + (static_cast<long long>(U.h) * p.slots_q + U.qslot + U.r0 / kTile) * (2 * kTile) + row;
                nl.x = nl.y = st[0];
                nd.x = nd.y = st[kTile];
            }
            for (int j = 0; j < U.n; ++j, ++g) {
                const uint32_t aS = tS + lanes + (g & 1u) * 128 + wg * 64, aP = tP + lanes + wg * 64;
                const int k0 = (U.lo + j) * kTile;
                if (!(ok = wait1(smem_u32(&ctl.s_full[g & 1u]), (g >> 1) & 1u))) break;
                tc_fence_after();
                uint32_t x[64];
                tmem_ld32(aS, x);
                tmem_ld32(aS + 32, x + 32);
                tmem_wait_ld();
                float2 pr[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float2 a = __ffma2_rn(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), c2, nl);
                    pr[k] = make_float2(ex2(a.x), ex2(a.y));
                }
                if (k0 < all_lo || k0 + kTile > all_hi) {
                    const int k1 = k0 + wg * 64;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (k1 + 2 * k < key_lo || k1 + 2 * k >= key_hi) pr[k].x = 0.0f;
                        if (k1 + 2 * k + 1 < key_lo || k1 + 2 * k + 1 >= key_hi) pr[k].y = 0.0f;
                    }
                }
                if (!(ok = wait1(smem_u32(&ctl.dp_full), dp_par))) break;
                dp_par ^= 1u;
                tc_fence_after();
                tmem_ld32(aP, x);
                tmem_ld32(aP + 32, x + 32);
                tmem_wait_ld();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint32_t *d = x + 32 * half + 2 * k;
                        const float2 a = __fmul2_rn(pr[16 * half + k], __fadd2_rn(make_float2(__uint_as_float(d[0]),
                                                                                              __uint_as_float(d[1])), nd));
                        w[k] = pack_bf16x2(a.x, a.y);
                    }
                    tmem_st16(aS + 16 * half, w);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&ctl.ds_full));
            }
            if (!ok) break;
            if (U.n > 0) {
                if (!(ok = wait1(smem_u32(&ctl.done), done_par))) break;
                done_par ^= 1u;
                tc_fence_after();
            }
            // each warpgroup stores half of the columns, whole groups of 16
            const bool mine = U.r0 + row < U.len_q;
            const int half = min((p.n_qk / 16 + 1) / 2 * 16, p.D_qk), c0 = wg ? half : 0, cols = wg ? p.D_qk - half : half;
            uint16_t *dst = static_cast<uint16_t *>(p.dQ) + U.h * p.dq_sh +
                            (static_cast<long long>(U.q0) + U.r0 + row) * p.dq_ss + c0;
            store_row(tDQ + lanes + c0, U.n > 0, dst, mine, cols, p.scale, p.dq_vec32);
        }
    }

    // This launch ends after the one it was started ahead of: the next one may read the results of both.  (Every CTA waits:
    // which of them run, and which are drawn by others as units, is the hardware's choice.)
    if (p.follows && threadIdx.x == 0) wait_prerequisites();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace vt
