// Host side of vt_attn_fwd_prefix and vt_attn_fwd_tree: argument checks, the plan of a call, launches (contract in include/vt_attn.h).
#include <cmath>
#include <cstring>

#include "vt_attn_bf16_2q.cuh"
#include "vt_attn_stream.cuh"
#include "vt_host.h"

namespace vt {
namespace prefix {
namespace {

using Args = vt_attn_prefix_args;

// How a call runs.  With prefix_shares > 0 a first launch leaves that many partial results of the prefix in the
// workspace, from the two-tile tcgen05 kernel (`tiles`) or from the key-streaming kernel; the second launch streams
// the caches and adds them.  Otherwise one launch streams the prefix and the cache of every sequence, or
// (`seq_tiles`: many rows per sequence) takes them on the tcgen05 kernel.
// (`merge`: the streaming launch leaves its results in the workspace too, and a last one adds them.)
struct Plan {
    bool tiles, seq_tiles, with_prefix, merge;
    int prefix_shares, prefix_cluster, cluster;
    int shares;  // of the streaming launch's keys, beyond a cluster's CTAs (more than 1: merge)
    int tree_shares;  // (seq_tiles) partial results of each sequence's own launch: its cache where the prefix has shares of
                      // its own, else all its keys; a last launch adds them.  0: one launch writes the answer
    size_t workspace;
};

struct Sizes {
    int64_t G, per_b, rows, tiles_all, tiles_b;
};

vt_status check_shape(const Args &a, bool *empty) {
    *empty = false;
    if (a.struct_bytes != sizeof(Args)) return VT_ERR_INVALID_ARG;
    if (a.dtype != VT_F32 && a.dtype != VT_BF16) return VT_ERR_INVALID_ARG;
    if (a.B < 0 || a.H < 0 || a.S_q < 0 || a.S_p < 0 || a.S_c < 0 || a.D_qk <= 0 || a.D_v <= 0) return VT_ERR_INVALID_ARG;
    if (a.H_kv < 1 || a.H % a.H_kv != 0 || !std::isfinite(a.scale)) return VT_ERR_INVALID_ARG;
    if (a.D_qk > kMaxD || a.D_v > kMaxD || a.B > kMaxExtent || a.H > kMaxExtent || a.S_q > kMaxSeq) return VT_ERR_UNSUPPORTED;
    if (a.S_p > kMaxSeq || a.S_c > kMaxSeq || a.S_p + a.S_c > kMaxSeq) return VT_ERR_UNSUPPORTED;
    *empty = a.B == 0 || a.H == 0 || a.S_q == 0;
    // rows are counted in 32 bits
    int64_t n = 0;
    if (__builtin_mul_overflow(a.B, a.H, &n) || __builtin_mul_overflow(n, a.S_q, &n) || n > kMaxSeq) return VT_ERR_UNSUPPORTED;
    return VT_OK;
}

Sizes sizes_of(const Args &a) {
    Sizes z;
    z.G = a.H / a.H_kv;
    z.per_b = a.S_q * z.G;
    z.rows = a.B * a.H * a.S_q;
    z.tiles_all = (a.B * z.per_b + st::kRowsTile - 1) / st::kRowsTile;
    z.tiles_b = (z.per_b + st::kRowsTile - 1) / st::kRowsTile;
    return z;
}

// More rows that share the prefix's keys than this take the tcgen05 kernel (bf16): 37 rows of 32 heads over 8191 keys,
// 52 us against 74 us streamed; with 64 rows of 8 heads over 2048 keys the two are level (59 us).
constexpr int64_t kTileRows = 32;
// More rows per sequence and key/value head than this take it for all their keys, one CTA for 256 rows.  Measured on both
// sides, 8 key/value heads of D = 128 and caches of up to 512: with many sequences it pays (64 sequences over 2048 shared
// keys: 96 rows 128 us here and 139 us with the prefix in a launch of its own, 256 rows 133 and 349 us; 8 sequences of 256
// rows 36 and 54 us), and with few rows or few sequences it loses, most behind a long prefix (8 sequences of 65 rows 37 and
// 28 us; one sequence of 256 rows over 32768 keys 356 and 44 us), where its CTAs are fewer than SMs and share no keys.
constexpr int64_t kSeqTileRows = 64;
// Bytes of the prefix that the streaming launch may read again, once per sequence and row tile, to spare a launch
// (4 sequences of 16 rows over 333 keys: 6.6 us against 9 us).  fp32 multiplies three times as much, and gains
// from the prefix's own launch earlier (8 sequences over 1000 keys: 12.8 us against 19.7 us).
constexpr int64_t kReadAgainBf16 = int64_t(16) << 20, kReadAgainF32 = int64_t(2) << 20;

size_t partial_bytes(int64_t rows, int64_t D_v, int shares) {
    return ((static_cast<size_t>(rows) * shares * (partial_ld(D_v) + 3) * sizeof(float)) + 255) & ~size_t(255);
}

// CTAs of a cluster that share a unit's keys: two CTAs per SM in all, as long as every CTA keeps `least` keys.  The
// fp32 kernel fills an SM per CTA, and clusters of 8 then wait for room (26 us against 20 us with 4).
// (`one_wave`: no more CTAs than SMs, where the fp32 kernel has several row tiles per sequence and its second wave of CTAs,
// each of a few keys, takes as long as the first: trees, which have no results of earlier plans to keep.  Eight trees of 13
// in 4 heads behind 1000 keys, fp32: 51 us with two waves, 41 us with one.)
int cluster_for(int64_t units, int64_t keys, int64_t least, bool f32, bool one_wave, int sms) {
    int c = 1;
    const int most = f32 ? 4 : st::kMaxClusterCtas;
    while (c < most && (one_wave ? 2 * units * c <= sms : units * c < 2LL * sms) && keys >= 2 * least * c) c *= 2;
    return c;
}

// Shares of the prefix for the tcgen05 kernel.  A unit takes 1.6 us per 128-key tile (1 us when its rows fill one query
// tile only) and 8 us besides; a streaming CTA takes 4.8 us besides its keys' time at 6 bytes per ns for all, three or four on
// an SM.  The two launches run beside each other: the first should be done when both are, without more overhead
// than that needs.
int tile_shares(const Args &a, const Sizes &z, int cluster, int sms) {
    const int64_t tiles = (a.S_p + q2::kBN - 1) / q2::kBN, rows = a.B * z.per_b;
    const int64_t blocks = a.H_kv * ((rows + q2::kRows - 1) / q2::kRows);
    const double tile_us = rows > kBM ? 1.6 : 1.0;
    const double stream_us = static_cast<double>(a.B * a.H_kv) * (a.S_c / 2) * (a.D_qk + a.D_v) * 2.0 / 6e6 +
                             static_cast<double>(a.B * a.H_kv * z.tiles_b * cluster) * 4.8 /
                                 static_cast<double>((a.D_v <= 64 ? 4 : 3) * sms);
    int best = 1;
    double best_us = 0.0;
    for (int n = 1; n <= st::kMaxShares && n <= tiles; ++n) {
        const double unit_us = 8.0 + tile_us * static_cast<double>((tiles + n - 1) / n);
        const double latency = static_cast<double>((blocks * n + sms - 1) / sms) * unit_us;
        const double machine = static_cast<double>(blocks * n) * unit_us / sms + stream_us;
        const double us = (latency > machine ? latency : machine) + 0.1 * n;
        if (n == 1 || us < best_us) {
            best = n;
            best_us = us;
        }
    }
    return best;
}

// Lengths live on the device, so the plan takes every cache as half full.  Where caches are mostly empty it gives the
// prefix too few shares (64 sequences of up to 100 tokens behind 8192 shared keys: 23 us in caches of 128 rows, 35 us in
// 1024, 99 us in 8192 and 32768).

// Streaming CTAs that share an SM (Tile::kPerSm).
int64_t ctas_per_sm(const Args &a) { return a.dtype == VT_F32 ? 1 : (a.D_v <= 64 ? 4 : 3); }

// Trees of many rows (Plan::seq_tiles): whether the prefix is taken once for the rows of all sequences, and into how many
// shares the keys are cut.  A 128-key step of the two-tile kernel takes 1.6 us and a unit 5 us besides, caches count as half
// full, and a partial result is written and read at 5 bytes per ns.  32 trees of 25 nodes in 4 heads, behind 8192 shared keys
// and caches of 1024: 221 us in one launch (256 units of 68 steps on 152 SMs, and 100 rows fill one tile of two), 124 us with
// the prefix in a launch of its own; 16 trees of 64 over up to 8192 keys: 101 us in one launch of 128 units, 94 us in two
// shares, longest first (114 us in the order of the batch).  Without a cache, one sequence of 64 nodes, 32 heads on 8, behind
// 8192 keys: 28 us in shares, 94 us in one launch; behind 1024 keys 23 and 19 us; 16 sequences behind 8192 keys 107 and 97 us.
// (vt_attn_fwd_prefix keeps its plan, and so the rounding of its results.)
void tree_plan(const Args &a, const Sizes &z, int sms, Plan *p) {
    const double step = 1.6, unit = 5.0;
    const int64_t tp = (a.S_p + q2::kBN - 1) / q2::kBN, tc = (a.S_c / 2 + q2::kBN - 1) / q2::kBN;
    const int64_t own = a.B * a.H_kv * ((z.per_b + q2::kRows - 1) / q2::kRows);
    const int64_t all = a.H_kv * ((a.B * z.per_b + q2::kRows - 1) / q2::kRows);
    const double share_us = static_cast<double>(z.rows) * static_cast<double>(partial_ld(a.D_v) + 3) * 8.0 / 5e6;
    // units of `tiles` steps, the longest of `most`
    auto launch_us = [&](int64_t units, int64_t tiles, int64_t most, int n) {
        const double waves = static_cast<double>((units * n + sms - 1) / sms);
        const double longest = unit + step * static_cast<double>((most + n - 1) / n);
        const double all_of_them = waves * (unit + step * static_cast<double>((tiles + n - 1) / n));
        return longest > all_of_them ? longest : all_of_them;
    };
    // the best number of shares of a launch, and its time with theirs
    auto best = [&](int64_t units, int64_t tiles, int64_t most, int *n) {
        double us = 0.0;
        for (int k = 1; k <= st::kMaxShares && (k == 1 || k <= most); ++k) {
            const double t = launch_us(units, tiles, most, k) + share_us * k;
            if (k == 1 || t < us) us = t, *n = k;
        }
        return us;
    };
    const int64_t full = (a.S_c + q2::kBN - 1) / q2::kBN;
    double least = launch_us(own, tp + tc, tp + full, 1);
    int n = 0, n_prefix = 0;
    if (const double us = 4.0 + best(own, tp + tc, tp + full, &n); us < least) least = us, p->tree_shares = n;
    if (tp > 0 && a.S_c > 0) {
        const double us = 8.0 + best(all, tp, tp, &n_prefix) + best(own, tc, full, &n);
        if (us < least) p->tree_shares = n, p->prefix_shares = n_prefix;
    }
    if (p->tree_shares) p->workspace = partial_bytes(z.rows, a.D_v, p->prefix_shares + p->tree_shares);
}

Plan plan_of(const Args &a, bool tree, int sms) {
    const Sizes z = sizes_of(a);
    Plan p{};
    const int64_t kv_units = a.B * a.H_kv * z.tiles_b;
    const int64_t elt = a.dtype == VT_BF16 ? 2 : 4;
    // (a double: up to 2^70)
    const double again = static_cast<double>(kv_units) * static_cast<double>(a.S_p * (a.D_qk + a.D_v) * elt);
    const bool f32 = a.dtype == VT_F32, one_wave = f32 && tree;
    p.shares = 1;
    p.seq_tiles = !f32 && z.per_b > kSeqTileRows;
    if (p.seq_tiles) {
        if (tree) tree_plan(a, z, sms, &p);
        return p;
    }
    p.tiles = !f32 && a.B * z.per_b > kTileRows;
    p.with_prefix = again <= static_cast<double>(f32 ? kReadAgainF32 : kReadAgainBf16) || (!p.tiles && z.tiles_all >= a.B * z.tiles_b);
    // keys a CTA should keep: with one launch latency counts (16 rows over 460 keys: 6.6 us with 4 CTAs, 7.1 us with
    // 2), beside the tcgen05 kernel overhead does (256 keys: 38 us with 1, 43 us with 2); fp32 is bound by its products
    const int64_t least = f32 ? 32 : (p.with_prefix || !p.tiles ? 96 : 192);
    p.cluster = cluster_for(kv_units, (p.with_prefix ? a.S_p : 0) + a.S_c / 2, least, f32, one_wave, sms);
    const int64_t keys = (p.with_prefix ? a.S_p : 0) + a.S_c / 2;
    if (kv_units * p.cluster < sms && keys >= 2 * 256LL * p.cluster) {
        // few units of many keys (one sequence of 65536 tokens: 105 us without): shares of 256 keys a CTA or more
        int64_t n = 2LL * sms / (kv_units * p.cluster);
        if (n > keys / (256LL * p.cluster)) n = keys / (256LL * p.cluster);
        if (n > st::kMaxCacheShares) n = st::kMaxCacheShares;
        p.shares = static_cast<int>(n);
    }
    if (p.with_prefix) {
        p.tiles = false;
        p.merge = p.shares > 1;
        p.workspace = p.merge ? partial_bytes(z.rows, a.D_v, p.shares) : 0;
        return p;
    }
    if (p.tiles) {
        p.prefix_shares = tile_shares(a, z, p.cluster, sms);
    } else {
        const int64_t units = a.H_kv * z.tiles_all;
        p.prefix_cluster = cluster_for(units, a.S_p, f32 ? 32 : 96, f32, one_wave, sms);
        int64_t shares = (one_wave ? sms : 2LL * sms) / (units * p.prefix_cluster);
        const int64_t most = a.S_p / ((f32 ? 64LL : 256LL) * p.prefix_cluster);
        if (shares > most) shares = most;
        if (shares > st::kMaxShares) shares = st::kMaxShares;
        p.prefix_shares = shares < 1 ? 1 : static_cast<int>(shares);
    }
    // Streaming CTAs wait for the prefix's shares only where every CTA of both launches has room at once.
    const int64_t per_sm = ctas_per_sm(a);
    const int64_t first = p.tiles ? per_sm * a.H_kv * ((a.B * z.per_b + q2::kRows - 1) / q2::kRows) * p.prefix_shares
                                  : a.H_kv * z.tiles_all * p.prefix_shares * p.prefix_cluster;
    p.merge = p.shares > 1 || first + kv_units * p.cluster > per_sm * sms;
    p.workspace = partial_bytes(z.rows, a.D_v, p.prefix_shares + (p.merge ? p.shares : 0));
    return p;
}

vt_status check_memory(const Args &a, const int32_t *parents, const Plan &plan) {
    const int elt = a.dtype == VT_BF16 ? 2 : 4;
    Span in[7], out[3];
    int n_in = 0, n_out = 0;
    VT_TRY(tensor(a.q, a.q_stride, a.B, a.H, a.S_q, a.D_qk, elt, false, &in[n_in++]));
    if (a.S_p > 0) {
        const int64_t ks[3] = {1, a.kp_stride[0], a.kp_stride[1]}, vs[3] = {1, a.vp_stride[0], a.vp_stride[1]};
        VT_TRY(tensor(a.k_prefix, ks, 1, a.H_kv, a.S_p, a.D_qk, elt, false, &in[n_in++]));
        VT_TRY(tensor(a.v_prefix, vs, 1, a.H_kv, a.S_p, a.D_v, elt, false, &in[n_in++]));
    }
    if (a.S_c > 0) {
        VT_TRY(tensor(a.k_cache, a.kc_stride, a.B, a.H_kv, a.S_c, a.D_qk, elt, false, &in[n_in++]));
        VT_TRY(tensor(a.v_cache, a.vc_stride, a.B, a.H_kv, a.S_c, a.D_v, elt, false, &in[n_in++]));
    }
    if (a.kv_len) {
        if (reinterpret_cast<uintptr_t>(a.kv_len) % 4) return VT_ERR_MISALIGNED;
        if (!span_bytes(a.kv_len, a.B * 4, &in[n_in++])) return VT_ERR_INVALID_ARG;
    }
    if (parents) {
        if (reinterpret_cast<uintptr_t>(parents) % 4) return VT_ERR_MISALIGNED;
        if (!span_bytes(parents, a.B * a.S_q * 4, &in[n_in++])) return VT_ERR_INVALID_ARG;
    }
    VT_TRY(tensor(a.o, a.o_stride, a.B, a.H, a.S_q, a.D_v, elt, true, &out[n_out++]));
    if (a.lse) {
        if (reinterpret_cast<uintptr_t>(a.lse) % 4) return VT_ERR_INVALID_ARG;
        if (!span_bytes(a.lse, a.B * a.H * a.S_q * 4, &out[n_out++])) return VT_ERR_INVALID_ARG;
    }
    if (plan.workspace) {
        if (!a.workspace || a.workspace_bytes < plan.workspace) return VT_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(a.workspace) % 256) return VT_ERR_MISALIGNED;
        if (!span_bytes(a.workspace, static_cast<int64_t>(plan.workspace), &out[n_out++])) return VT_ERR_INVALID_ARG;
    }
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(out[i], in[j])) return VT_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return VT_ERR_INVALID_ARG;
    }
    return VT_OK;
}

st::Params params_of(const Args &a, const Plan &plan, const Sizes &z, unsigned *status) {
    st::Params p{};
    p.B = static_cast<int>(a.B);
    p.H = static_cast<int>(a.H);
    p.H_kv = static_cast<int>(a.H_kv);
    p.G = static_cast<int>(z.G);
    p.S_q = static_cast<int>(a.S_q);
    p.S_p = static_cast<int>(a.S_p);
    p.S_c = static_cast<int>(a.S_c);
    p.D_qk = static_cast<int>(a.D_qk);
    p.D_v = static_cast<int>(a.D_v);
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.Q = a.q;
    p.q_sb = a.q_stride[0]; p.q_sh = a.q_stride[1]; p.q_ss = a.q_stride[2];
    p.kv_len = a.S_c > 0 ? a.kv_len : nullptr;
    p.rows = z.rows;
    if (plan.workspace) {
        const int64_t n = z.rows * (plan.prefix_shares + (plan.merge ? plan.shares : 0) + plan.tree_shares);
        p.part_o = static_cast<float *>(a.workspace);
        p.part_ld = static_cast<int>(partial_ld(a.D_v));
        p.part_m = p.part_o + n * p.part_ld;
        p.part_l = p.part_m + n;
        p.part_c = p.part_l + n;
    }
    p.O = a.o;
    p.o_sb = a.o_stride[0]; p.o_sh = a.o_stride[1]; p.o_ss = a.o_stride[2];
    p.lse = a.lse;
    p.timeout_ns = kDefaultTimeoutNs;
    p.status = status;
    return p;
}

// A tensor map of a prefix or cache tensor, boxes of `rows` rows; strides of an index with one value are replaced.
bool kv_map(CUtensorMap *map, const void *ptr, const int64_t st[3], int64_t B, int64_t H_kv, int64_t S, int64_t D,
            int elt, int rows) {
    const int64_t row = (D * elt + 15) / 16 * 16 / elt;
    const int64_t strides[3] = {B > 1 ? st[0] : row, H_kv > 1 ? st[1] : row, S > 1 ? st[2] : row};
    return make_map(map, ptr, strides, B, H_kv, S, D, elt, rows);
}

// The four maps with boxes of `rows` keys (an absent prefix or cache gets the other's, and where both are absent the queries'
// stand in: they are not read, but the kernels ask for the descriptors).
bool kv_maps(const Args &a, int rows, st::Maps *m) {
    const int elt = a.dtype == VT_BF16 ? 2 : 4;
    if (a.S_p == 0 && a.S_c == 0) {
        if (!kv_map(&m->kp, a.q, a.q_stride, a.B, a.H, a.S_q, a.D_qk, elt, rows)) return false;
        m->vp = m->kc = m->vc = m->kp;
        return true;
    }
    const int64_t kp[3] = {0, a.kp_stride[0], a.kp_stride[1]}, vp[3] = {0, a.vp_stride[0], a.vp_stride[1]};
    if (a.S_p > 0 && (!kv_map(&m->kp, a.k_prefix, kp, 1, a.H_kv, a.S_p, a.D_qk, elt, rows) ||
                      !kv_map(&m->vp, a.v_prefix, vp, 1, a.H_kv, a.S_p, a.D_v, elt, rows)))
        return false;
    if (a.S_c > 0 && (!kv_map(&m->kc, a.k_cache, a.kc_stride, a.B, a.H_kv, a.S_c, a.D_qk, elt, rows) ||
                      !kv_map(&m->vc, a.v_cache, a.vc_stride, a.B, a.H_kv, a.S_c, a.D_v, elt, rows)))
        return false;
    if (a.S_p == 0) m->kp = m->kc, m->vp = m->vc;
    if (a.S_c == 0) m->kc = m->kp, m->vc = m->vp;
    return true;
}

using Kern = void (*)(const st::Maps, const st::Params);

template <typename T, bool TREE>
Kern pick(const Args &a, int *smem) {
    const bool k64 = a.D_qk <= 64, v64 = a.D_v <= 64;
    if (k64 && v64) { *smem = st::Tile<T, 64, 64>::kSmem; return st::attn_stream_kernel<T, 64, 64, TREE>; }
    if (k64) { *smem = st::Tile<T, 64, 128>::kSmem; return st::attn_stream_kernel<T, 64, 128, TREE>; }
    if (v64) { *smem = st::Tile<T, 128, 64>::kSmem; return st::attn_stream_kernel<T, 128, 64, TREE>; }
    *smem = st::Tile<T, 128, 128>::kSmem;
    return st::attn_stream_kernel<T, 128, 128, TREE>;
}

vt_status launch_stream(const Args &a, const st::Maps &maps, const st::Params &p, int64_t units, int cluster, bool follows, int dev,
                        cudaStream_t stream) {
    int smem = 0;
    // (the prefix's own launch reads no cache; in fp32 it takes the trees' sums)
    const bool tree = p.parents && (a.dtype == VT_F32 || !p.all_rows);
    const Kern kern = a.dtype == VT_BF16 ? (tree ? pick<uint16_t, true>(a, &smem) : pick<uint16_t, false>(a, &smem))
                                         : (tree ? pick<float, true>(a, &smem) : pick<float, false>(a, &smem));
    if (!ensure_smem(reinterpret_cast<const void *>(kern), dev, smem)) return VT_ERR_CUDA;
    const int64_t ctas = units * cluster;
    if (ctas > 0x7FFFFFFFll) return VT_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(st::kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (follows) {  // start as the prefix's CTAs leave room; the kernel waits for them before it adds their results
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, kern, maps, p) != cudaSuccess) return VT_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? VT_OK : VT_ERR_CUDA;
}

using TileKern = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const AttnParams);

template <int EPI, int ROWS>
TileKern pick_tiles(const AttnParams &p) {
    const int ksteps = (p.D_qk + 15) / 16;
    auto pick = [&](auto ring_c) -> TileKern {
        constexpr bool R = decltype(ring_c)::value;
        if (p.scale_log2 > 0.0f)
            return ksteps <= 4   ? attn_fwd_bf16_2q_kernel<4, R, EPI, true, ROWS>
                   : ksteps <= 6 ? attn_fwd_bf16_2q_kernel<6, R, EPI, true, ROWS>
                                 : attn_fwd_bf16_2q_kernel<8, R, EPI, true, ROWS>;
        return ksteps <= 4 ? attn_fwd_bf16_2q_kernel<4, R, EPI, false, ROWS>
                           : attn_fwd_bf16_2q_kernel<8, R, EPI, false, ROWS>;
    };
    return p.n_pv <= 64 ? pick(std::true_type{}) : pick(std::false_type{});
}

// The two-tile tcgen05 kernel on gathered rows: the prefix for the rows of all sequences (partial results), or
// (`seq`) the prefix and the cache for the rows of each sequence (the whole answer).
vt_status launch_tiles(const Args &a, const Plan &plan, const Sizes &z, const st::Params &sp, bool seq,
                       const DeviceInfo &info, int dev, cudaStream_t stream) {
    st::Maps m{};
    if (!kv_maps(a, q2::kBN, &m)) return VT_ERR_CUDA;
    AttnParams p{};
    p.B = seq ? sp.B : 1;
    p.H = sp.H_kv;
    p.S_q = static_cast<int>(seq ? z.per_b : a.B * z.per_b);
    const bool own_only = seq && plan.prefix_shares > 0;  // (the prefix has its own launch)
    p.prefix_tiles = own_only ? 0 : (sp.S_p + q2::kBN - 1) / q2::kBN;
    p.prefix_keys = own_only ? 0 : sp.S_p;
    p.cache_keys = sp.S_c;
    p.kv_len = sp.kv_len;
    p.parents = sp.parents;
    p.S_k = seq ? (p.prefix_tiles + (sp.S_c + q2::kBN - 1) / q2::kBN) * q2::kBN : sp.S_p;
    p.D_qk = sp.D_qk;
    p.D_v = sp.D_v;
    p.n_qblocks = (p.S_q + q2::kRows - 1) / q2::kRows;
    p.q_chunks = (p.D_qk + q2::kChunk - 1) / q2::kChunk;
    p.v_chunks = (p.D_v + q2::kChunk - 1) / q2::kChunk;
    p.n_pv = (p.D_v + 15) / 16 * 16;
    p.band_lo = -kBandInf;
    p.band_hi = kBandInf;
    p.kv_group = 1;
    p.scale_log2 = sp.scale_log2;
    p.Q = sp.Q;
    p.q_sb = sp.q_sb;
    p.q_sh = sp.q_sh;
    p.q_ss = sp.q_ss;
    p.row_heads = sp.G;
    p.row_tokens = sp.S_q;
    p.O = sp.O;
    p.o_sb = sp.o_sb;
    p.o_sh = sp.o_sh;
    p.o_ss = sp.o_ss;
    p.o_vec32 = reinterpret_cast<uintptr_t>(sp.O) % 32 == 0 && (sp.B < 2 || sp.o_sb % 16 == 0) &&
                (sp.H < 2 || sp.o_sh % 16 == 0) && (sp.S_q < 2 || sp.o_ss % 16 == 0);
    p.lse = sp.lse;
    p.tiles_per_unit = 2;
    p.cluster = 1;
    p.n_split = !seq ? plan.prefix_shares : plan.tree_shares ? plan.tree_shares : 1;
    p.part_share0 = plan.prefix_shares;
    p.part_o = sp.part_o;
    p.part_ld = sp.part_ld;
    p.part_m = sp.part_m;
    p.part_l = sp.part_l;
    p.part_c = sp.part_c;
    p.timeout_ns = kDefaultTimeoutNs;
    p.status = sp.status;
    const int q_bytes = 2 * p.q_chunks * static_cast<int>(q2::kChunkBytes);
    const int slot_bytes = (p.q_chunks > p.v_chunks ? p.q_chunks : p.v_chunks) * static_cast<int>(q2::kChunkBytes);
    p.stages = (kSmemLimit - 1024 - static_cast<int>(sizeof(q2::Ctl)) - 256 - q_bytes) / slot_bytes;
    if (p.stages > q2::kMaxSlots) p.stages = q2::kMaxSlots;
    const int smem = 1024 + q_bytes + p.stages * slot_bytes;
    const int64_t heads = static_cast<int64_t>(p.B) * p.H;
    const int64_t per_head = static_cast<int64_t>(p.n_qblocks) * p.n_split;
    p.head_group = 1;
    const int64_t units = per_head * heads;
    if (units > 0x7FFFFFFFll) return VT_ERR_UNSUPPORTED;
    p.n_units = static_cast<int>(units);
    // (kRowsTree reads the parents of every sequence, without a cache too; plan_of cuts a sequence's keys for trees alone)
    const TileKern kern = !seq               ? pick_tiles<q2::kEpiSplit, q2::kRowsAll>(p)
                          : !p.parents       ? pick_tiles<q2::kEpiPlain, q2::kRowsSeq>(p)
                          : plan.tree_shares ? pick_tiles<q2::kEpiSplit, q2::kRowsTree>(p)
                                             : pick_tiles<q2::kEpiPlain, q2::kRowsTree>(p);
    if (!ensure_smem(reinterpret_cast<const void *>(kern), dev, smem)) return VT_ERR_CUDA;
    p.follows = own_only ? 1 : 0;
    p.longest_first = seq && p.parents && p.kv_len && sp.B > 1 && sp.B <= st::kMaxSorted && units > info.sms;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units));
    cfg.blockDim = dim3(q2::kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];  // takes the SMs that the prefix's launch no longer fills
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.follows ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, m.kc, m.kp, m.vp, m.vc, p) != cudaSuccess) return VT_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? VT_OK : VT_ERR_CUDA;
}

// The workspace's `n` shares of every row combined into O (by a kernel that waits for the launch before it itself).
vt_status launch_shares(const Args &a, const Sizes &z, st::Params p, int n, cudaStream_t stream) {
    p.prior = n;
    const unsigned blocks = static_cast<unsigned>((z.rows + st::kMergeWarps - 1) / st::kMergeWarps);
    const bool bf = a.dtype == VT_BF16;
    void (*kern)(const st::Params) = a.D_v <= 64 ? (bf ? st::attn_shares_kernel<uint16_t, 64> : st::attn_shares_kernel<float, 64>)
                                                 : (bf ? st::attn_shares_kernel<uint16_t, 128> : st::attn_shares_kernel<float, 128>);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * st::kMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return VT_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? VT_OK : VT_ERR_CUDA;
}

// (`parents`: the sequences' new tokens are the nodes of trees)
vt_status forward(const Args &a, const int32_t *parents, cudaStream_t stream) {
    bool empty = false;
    VT_TRY(check_shape(a, &empty));
    if (empty) return VT_OK;
    int dev = 0;
    DeviceInfo info;
    const bool have = cudaGetDevice(&dev) == cudaSuccess && device_info(dev, &info);
    const Plan plan = plan_of(a, parents != nullptr, have ? info.sms : 152);
    VT_TRY(check_memory(a, parents, plan));
    if (!have) return VT_ERR_CUDA;
    const Sizes z = sizes_of(a);
    st::Params p = params_of(a, plan, z, info.status + status_slot(stream));
    p.parents = parents;
    if (plan.seq_tiles) {
        if (plan.prefix_shares) VT_TRY(launch_tiles(a, plan, z, p, false, info, dev, stream));
        VT_TRY(launch_tiles(a, plan, z, p, true, info, dev, stream));
        if (plan.tree_shares) VT_TRY(launch_shares(a, z, p, plan.prefix_shares + plan.tree_shares, stream));
        return env_check() ? read_status(stream) : VT_OK;
    }
    st::Maps maps{};
    if (!kv_maps(a, st::kKeys, &maps)) return VT_ERR_CUDA;
    if (plan.tiles) {
        VT_TRY(launch_tiles(a, plan, z, p, false, info, dev, stream));
    } else if (plan.prefix_shares) {
        p.all_rows = 1;
        p.partial = 1;
        p.row_tiles = static_cast<int>(z.tiles_all);
        p.shares = plan.prefix_shares;
        p.cluster = plan.prefix_cluster;
        VT_TRY(launch_stream(a, maps, p, a.H_kv * z.tiles_all * p.shares, p.cluster, false, dev, stream));
    }
    p.all_rows = 0;
    p.with_prefix = plan.with_prefix ? 1 : 0;
    p.row_tiles = static_cast<int>(z.tiles_b);
    p.shares = plan.shares;
    p.cluster = plan.cluster;
    p.partial = plan.merge ? 1 : 0;
    p.share0 = plan.merge ? plan.prefix_shares : 0;
    p.prior = plan.merge ? 0 : plan.prefix_shares;
    p.follows = plan.prefix_shares > 0 ? 1 : 0;
    const int64_t units = a.B * a.H_kv * z.tiles_b * p.shares;
    p.longest_first = p.kv_len && a.B > 1 && a.B <= st::kMaxSorted && (plan.tiles || units * p.cluster > ctas_per_sm(a) * info.sms);
    VT_TRY(launch_stream(a, maps, p, units, p.cluster, p.follows != 0, dev, stream));
    if (plan.merge) VT_TRY(launch_shares(a, z, p, plan.prefix_shares + plan.shares, stream));
    return env_check() ? read_status(stream) : VT_OK;
}

size_t workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t S_q, int64_t S_p, int64_t S_c, int64_t D_qk, int64_t D_v,
                      vt_dtype dtype, bool tree) {
    Args a{};
    a.struct_bytes = sizeof a;
    a.B = B; a.H = H; a.H_kv = H_kv; a.S_q = S_q; a.S_p = S_p; a.S_c = S_c; a.D_qk = D_qk; a.D_v = D_v;
    a.dtype = dtype;
    bool empty = false;
    if (check_shape(a, &empty) != VT_OK || empty) return 0;
    int dev = 0;
    DeviceInfo info;
    const bool have = cudaGetDevice(&dev) == cudaSuccess && device_info(dev, &info);
    return plan_of(a, tree, have ? info.sms : 152).workspace;
}

}  // namespace
}  // namespace prefix
}  // namespace vt

extern "C" {

vt_status vt_attn_fwd_prefix(const vt_attn_prefix_args *args, vt_stream_t stream) {
    const vt::NvtxRange range("vt_attn_fwd_prefix");
    if (!args) return VT_ERR_INVALID_ARG;
    return vt::prefix::forward(*args, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

vt_status vt_attn_fwd_tree(const vt_attn_prefix_args *args, const int32_t *parents, vt_stream_t stream) {
    const vt::NvtxRange range("vt_attn_fwd_tree");
    if (!args) return VT_ERR_INVALID_ARG;
    bool empty = false;
    VT_TRY(vt::prefix::check_shape(*args, &empty));
    if (empty) return VT_OK;
    if (args->S_q > vt::kMaxNodes) return VT_ERR_UNSUPPORTED;
    if (!parents) return VT_ERR_INVALID_ARG;
    return vt::prefix::forward(*args, parents, reinterpret_cast<cudaStream_t>(stream));
}

size_t vt_attn_prefix_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t S_q, int64_t S_p, int64_t S_c,
                                     int64_t D_qk, int64_t D_v, vt_dtype dtype) {
    return vt::prefix::workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, dtype, false);
}

size_t vt_attn_tree_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t S_q, int64_t S_p, int64_t S_c, int64_t D_qk,
                                   int64_t D_v, vt_dtype dtype) {
    return S_q > vt::kMaxNodes ? 0 : vt::prefix::workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, dtype, true);
}

}  // extern "C"
