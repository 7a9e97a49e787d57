// Trees of drafted tokens: the last n <= 64 cached tokens of a sequence are the nodes of a tree (or of several), and a node
// sees, of these, itself and its ancestors (contract of vt_attn_fwd_tree in include/vt_attn.h).  What a node sees is a
// 64-bit word, formed from the parents by each warp that masks with it.
#pragma once

#include <climits>
#include <cstdint>

#include "vt_attn_common.cuh"

namespace vt {

constexpr int kMaxNodes = 64;

// What this lane's nodes, lane and lane + 32, see (bit j: node j).
struct TreeNodes {
    unsigned long long sees[2];
    int up[2];  // an ancestor whose own ancestors are not in `sees` yet, or -1

    // The nodes' parents, on their way from memory.
    __device__ __forceinline__ void load(const int *parents, int n, int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) up[i] = lane + 32 * i < n ? parents[lane + 32 * i] : -1;
    }
    // The whole warp: in every step a node takes over what its furthest known ancestor sees and jumps to that one's, so a
    // depth of 64 takes 6 steps.  A parent below -1 or not before its child counts as -1, and the status word records it.
    __device__ __forceinline__ void follow(int n, int lane, unsigned *status) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int node = lane + 32 * i;
            sees[i] = node < n ? 1ull << node : 0ull;
            if (up[i] < -1 || up[i] >= node) {
                atomicOr(status, kStatusBounds);
                up[i] = -1;
            }
        }
        for (int step = 1; step < n; step *= 2) {
            unsigned long long add[2];
            int next[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                add[i] = of(up[i]);
                const int from = up[i] & 31;
                const int u0 = __shfl_sync(0xffffffffu, up[0], from), u1 = __shfl_sync(0xffffffffu, up[1], from);
                next[i] = up[i] < 32 ? u0 : u1;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (up[i] < 0) continue;
                sees[i] |= add[i];
                up[i] = next[i];
            }
        }
    }
    // What node s of this lane's choice sees (the whole warp).
    __device__ __forceinline__ unsigned long long of(int s) const {
        const unsigned long long a = __shfl_sync(0xffffffffu, sees[0], s & 31), b = __shfl_sync(0xffffffffu, sees[1], s & 31);
        return s < 32 ? a : b;
    }
};

// The place of this lane's sequence in the order of B <= 32 lengths, longest first (equal ones in order), by a whole warp.
__device__ __forceinline__ int length_rank(const int *kv_len, int B, int lane) {
    const int mine = lane < B ? kv_len[lane] : INT_MIN;
    int rank = 0;
    for (int j = 0; j < B; ++j) {
        const int other = __shfl_sync(0xffffffffu, mine, j);
        rank += other > mine || (other == mine && j < lane);
    }
    return rank;
}
// The sequence with the n-th longest cache.
__device__ __forceinline__ int nth_longest(const int *kv_len, int B, int n, int lane) {
    const int rank = length_rank(kv_len, B, lane);
    return __ffs(__ballot_sync(0xffffffffu, lane < B && rank == n)) - 1;
}

// 32 keys from the `from`-th node on, as bits: the keys before the tree (from < 0) are seen, those behind it are not.
__device__ __forceinline__ uint32_t tree_window(unsigned long long seen, int from) {
    if (from <= -32) return 0xffffffffu;
    if (from >= kMaxNodes) return 0u;
    return static_cast<uint32_t>(from < 0 ? (seen << -from) | ((1ull << -from) - 1ull) : seen >> from);
}

}  // namespace vt
