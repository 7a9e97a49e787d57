// Packed sequences: rows of sequences of different lengths behind each other in one tensor, cu[n] the first row of
// sequence n and cu[N] the end of the last (contracts of vt_attn_fwd_packed and vt_attn_bwd_packed in include/vt_attn.h).
//
// Work is cut into blocks of R rows that start at a sequence's first row.  Lengths are known on the device only, so the
// host launches for every block that could exist: sequence n owns the slots cu[n] / R + n and on, up to
// cu[n + 1] / R + n + 1.  That is enough room for its blocks (it is one more than whole blocks between multiples of R),
// no two sequences meet, and a slot is found by searching cu itself, with nothing to prepare: T / R + N slots in all, at
// most one or two of each sequence empty.
#pragma once

#include <cstdint>

#include "vt_attn_common.cuh"

namespace vt {

struct PackedSeq {
    int n, block;    // sequence, and block of its rows
    int start, len;  // its first row and its rows
};

// Slots for T rows of N sequences.
__host__ __device__ constexpr long long packed_slots(long long T, long long N, int R) { return T / R + N; }

// First row n, brought into [0, T].
__device__ __forceinline__ int packed_cu(const int *cu, int n, int T) { return min(max(__ldg(cu + n), 0), T); }

// Rows of sequence n.  Ends outside [0, T] count as the nearest inside, an end before its start as the start.
__device__ __forceinline__ PackedSeq packed_seq(const int *cu, int n, int T) {
    PackedSeq s;
    s.n = n;
    s.block = 0;
    s.start = packed_cu(cu, n, T);
    s.len = max(packed_cu(cu, n + 1, T) - s.start, 0);
    return s;
}

// What is wrong with sequence n's first rows goes to the status word.  Every sequence is looked at by the unit of the slot of
// its number (there are as many slots as sequences, and more), whether or not an array that decreases leaves it one of its own.
__device__ __forceinline__ void packed_check(const AttnParams &p, int n) {
    if (n >= p.n_seq) return;
    const int a = __ldg(p.cu_q + n), b = __ldg(p.cu_q + n + 1), c = __ldg(p.cu_k + n), d = __ldg(p.cu_k + n + 1);
    if (a < 0 || b > p.S_q || b < a || c < 0 || d > p.S_k || d < c) atomicOr(p.status, kStatusBounds);
}

// The search for a slot takes 32 candidates lo, lo + step, ... at a time and halves them: `before(i)` says whether candidate
// i's sequence starts at the slot or before it.  By a lane alone or (a call's first units) by a whole warp, it looks at the
// same candidates and finds the same sequence, in arrays that decrease too.  A lane reads for two halvings at once.
template <typename Before>
__device__ __forceinline__ int packed_halve(Before before) {
    int i = 0;
#pragma unroll
    for (int b = 8; b > 1; b /= 4) {
        const bool quarter = before(i + b), half = before(i + 2 * b), three = before(i + 3 * b);
        i += half ? (three ? 3 * b : 2 * b) : (quarter ? b : 0);
    }
    return before(i + 1) ? i + 1 : i;
}
template <typename Round>
__device__ __forceinline__ PackedSeq packed_search(const int *cu, int N, int T, int R, int slot, Round round) {
    int lo = 0, hi = N;  // sequence lo starts at the slot or before it, sequence hi behind it
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        lo += step * round([&](int i) {
            const int at = lo + i * step;
            return (at < hi) & (packed_cu(cu, min(at, hi - 1), T) / R + at <= slot);
        });
        hi = min(hi, lo + step);
    }
    PackedSeq s = packed_seq(cu, lo, T);
    s.block = slot - (s.start / R + lo);
    if (s.block < 0) s.block = s.len = 0;  // ahead of the first sequence
    return s;
}

// The sequence and block of a slot (its rows may end before the block), by one lane.
__device__ __forceinline__ PackedSeq packed_find(const int *cu, int N, int T, int R, int slot) {
    return packed_search(cu, N, T, R, slot, [](auto before) { return packed_halve(before); });
}

// The same by a whole warp, which reads 32 candidates at once: one or two reads after each other where a lane alone makes
// log2(N).
__device__ __forceinline__ PackedSeq packed_find_warp(const int *cu, int N, int T, int R, int slot, int lane) {
    return packed_search(cu, N, T, R, slot, [lane](auto before) {
        const unsigned set = __ballot_sync(0xffffffffu, before(lane));
        return packed_halve([set](int i) { return (set >> i & 1u) != 0; });
    });
}

// First key that query i of a packed sequence of `len` keys sees, and one past its last: the band around its own
// position i + off (empty when lo >= hi).
__device__ __forceinline__ int packed_key_lo(const AttnParams &p, int off, int len, int i) {
    const long long x = static_cast<long long>(i) + off + p.band_lo;
    return static_cast<int>(x < 0 ? 0 : (x > len ? len : x));
}
__device__ __forceinline__ int packed_key_hi(const AttnParams &p, int off, int len, int i) {
    const long long x = static_cast<long long>(i) + off + p.band_hi + 1;
    return static_cast<int>(x < 0 ? 0 : (x > len ? len : x));
}

}  // namespace vt
