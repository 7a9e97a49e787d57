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

// Rows of sequence n.  Ends outside [0, T] count as the nearest inside, an end before its start as the start, and the
// status word records both.
__device__ __forceinline__ PackedSeq packed_seq(const int *cu, int n, int T, unsigned *status) {
    const int a = __ldg(cu + n), e = __ldg(cu + n + 1);
    PackedSeq s;
    s.n = n;
    s.block = 0;
    s.start = min(max(a, 0), T);
    s.len = max(min(max(e, 0), T) - s.start, 0);
    if (a < 0 || e > T || e < a) atomicOr(status, kStatusBounds);
    return s;
}

// The sequence and block of a slot (its rows may end before the block).
__device__ __forceinline__ PackedSeq packed_find(const int *cu, int N, int T, int R, int slot, unsigned *status) {
    int lo = 0, hi = N;  // sequence lo starts at the slot or before it, sequence hi behind it
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (packed_cu(cu, mid, T) / R + mid <= slot) lo = mid;
        else hi = mid;
    }
    PackedSeq s = packed_seq(cu, lo, T, status);
    s.block = slot - (s.start / R + lo);
    if (s.block < 0) s.block = s.len = 0;  // ahead of the first sequence
    return s;
}

// The same by a whole warp, 32 candidates at a time: one or two reads after each other where a lane alone makes log2(N).
__device__ __forceinline__ PackedSeq packed_find_warp(const int *cu, int N, int T, int R, int slot, int lane, unsigned *status) {
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool before = lane == 0 || (at < hi && packed_cu(cu, min(at, hi - 1), T) / R + at <= slot);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));
        lo += last * step;
        hi = min(hi, lo + step);
    }
    PackedSeq s = packed_seq(cu, lo, T, status);
    s.block = slot - (s.start / R + lo);
    if (s.block < 0) s.block = s.len = 0;  // ahead of the first sequence
    return s;
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
