// Host side of vt_attn_fwd_packed and vt_attn_bwd_packed: argument checks and launches (contract in include/vt_attn.h).
#include <cmath>

#include "vt_attn_bf16_2q.cuh"
#include "vt_attn_bwd_bf16.cuh"
#include "vt_attn_packed.cuh"
#include "vt_attn_packed_f32.cuh"
#include "vt_host.h"
#include "vt_pieces.h"

namespace vt {
namespace packed {
namespace {

using Args = vt_attn_packed_args;
using Grads = vt_attn_packed_grads;

constexpr int kLeastRows = 32;  // rows of the smallest block a launch is cut into

vt_status check_shape(const Args &a) {
    if (a.struct_bytes != sizeof(Args) || a.reserved != 0) return VT_ERR_INVALID_ARG;
    if (a.dtype != VT_F32 && a.dtype != VT_BF16) return VT_ERR_INVALID_ARG;
    if (a.N < 0 || a.H < 0 || a.T_q < 0 || a.T_k < 0 || a.D_qk <= 0 || a.D_v <= 0) return VT_ERR_INVALID_ARG;
    if (a.H_kv < 1 || a.H % a.H_kv != 0 || !std::isfinite(a.scale)) return VT_ERR_INVALID_ARG;
    if (a.mask < VT_MASK_NONE || a.mask > VT_MASK_WINDOW_COMPLEMENT) return VT_ERR_INVALID_ARG;
    const bool window = a.mask == VT_MASK_WINDOW || a.mask == VT_MASK_WINDOW_COMPLEMENT;
    if (window && a.window < 1) return VT_ERR_INVALID_ARG;
    if (window && a.window > (int64_t(1) << 40)) return VT_ERR_UNSUPPORTED;
    if (a.D_qk > kMaxD || a.D_v > kMaxD || a.N > kMaxSeq || a.T_q > kMaxSeq || a.T_k > kMaxSeq || a.H > kMaxExtent)
        return VT_ERR_UNSUPPORTED;
    int64_t units = 0;
    const int64_t T = a.T_q > a.T_k ? a.T_q : a.T_k;
    if (__builtin_mul_overflow(4 * packed_slots(T, a.N, kLeastRows), a.H, &units) || units > kMaxExtent) return VT_ERR_UNSUPPORTED;
    return VT_OK;
}

// The pieces of a call, and their checks.
struct Memory {
    Pieces ps;
    const Args &a;
    const int elt;
    explicit Memory(const Args &args) : a(args), elt(args.dtype == VT_BF16 ? 2 : 4) {}

    vt_status rows(const void *p, const int64_t st[2], int64_t H, int64_t T, int64_t D, bool out) {
        if (H == 0 || T == 0) return VT_OK;  // no element
        Piece x{};
        const int64_t s3[3] = {1, st[0], st[1]};
        VT_TRY(tensor(p, s3, 1, H, T, D, elt, out, &x.span));
        x.p = p;
        x.st = st;
        x.out = out;
        x.n[0] = H;
        x.n[1] = T;
        x.n[2] = 1;  // (its stride is not looked at)
        x.D = D;
        ps.add(x);
        return VT_OK;
    }
    vt_status vector(const void *p, int64_t bytes, int align, bool out) {
        Piece x{};
        if (!p) return VT_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(p) % align) return VT_ERR_MISALIGNED;
        if (!span_bytes(p, bytes, &x.span)) return VT_ERR_INVALID_ARG;
        x.out = out;
        ps.add(x);
        return VT_OK;
    }
    vt_status inputs() {
        VT_TRY(rows(a.q, a.q_stride, a.H, a.T_q, a.D_qk, false));
        VT_TRY(rows(a.k, a.k_stride, a.H_kv, a.T_k, a.D_qk, false));
        VT_TRY(rows(a.v, a.v_stride, a.H_kv, a.T_k, a.D_v, false));
        VT_TRY(vector(a.cu_q, (a.N + 1) * 4, 4, false));
        return vector(a.cu_k, (a.N + 1) * 4, 4, false);
    }
    // No output meets another piece.
    vt_status clear() const {
        for (int i = 0; i < ps.n; ++i)
            for (int j = 0; j < ps.n; ++j) {
                const Piece &x = ps.at[i], &y = ps.at[j];
                if (i != j && x.out && overlap(x.span, y.span) && !beside(x, y, elt)) return VT_ERR_INVALID_ARG;
            }
        return VT_OK;
    }
};

// A tensor map of [H,T,D] rows, boxes of `rows` of them.
bool rows_map(CUtensorMap *map, const void *p, const int64_t st[2], int64_t H, int64_t T, int64_t D, int elt, int rows) {
    const int64_t row = (D * elt + 15) / 16 * 16 / elt;
    const int64_t s3[3] = {row, H > 1 ? st[0] : row, T > 1 ? st[1] : row};
    return make_map(map, p, s3, 1, H, T, D, elt, rows);
}

void band_of(const Args &a, long long *lo, long long *hi) {
    *lo = a.mask == VT_MASK_WINDOW ? 1 - a.window : -kBandInf;
    *hi = a.mask == VT_MASK_NONE ? kBandInf : a.mask == VT_MASK_WINDOW_COMPLEMENT ? -a.window : 0;
}

// What the kernels of both directions share.
AttnParams params_of(const Args &a, unsigned *status) {
    AttnParams p{};
    p.B = 1;
    p.H = static_cast<int>(a.H);
    p.S_q = static_cast<int>(a.T_q);
    p.S_k = static_cast<int>(a.T_k);
    p.D_qk = static_cast<int>(a.D_qk);
    p.D_v = static_cast<int>(a.D_v);
    p.cu_q = a.cu_q;
    p.cu_k = a.cu_k;
    p.n_seq = static_cast<int>(a.N);
    band_of(a, &p.band_lo, &p.band_hi);
    p.kv_group = static_cast<int>(a.H / a.H_kv);
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.lse = a.lse;
    p.O = a.o;
    p.o_sh = a.o_stride[0];
    p.o_ss = a.o_stride[1];
    p.timeout_ns = kDefaultTimeoutNs;
    p.status = status;
    return p;
}

// ---------------------------------------------------------------- forward

using TileKern = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const AttnParams);

TileKern pick_tiles(const AttnParams &p) {
    const int ksteps = (p.D_qk + 15) / 16;
    auto pick = [&](auto ring_c) -> TileKern {
        constexpr bool R = decltype(ring_c)::value;
        constexpr int E = q2::kEpiPlain, P = q2::kRowsPacked;
        if (p.scale_log2 > 0.0f)
            return ksteps <= 4   ? attn_fwd_bf16_2q_kernel<4, R, E, true, P>
                   : ksteps <= 6 ? attn_fwd_bf16_2q_kernel<6, R, E, true, P>
                                 : attn_fwd_bf16_2q_kernel<8, R, E, true, P>;
        return ksteps <= 4 ? attn_fwd_bf16_2q_kernel<4, R, E, false, P> : attn_fwd_bf16_2q_kernel<8, R, E, false, P>;
    };
    return p.n_pv <= 64 ? pick(std::true_type{}) : pick(std::false_type{});
}

vt_status forward_bf16(const Args &a, AttnParams p, int dev, cudaStream_t stream) {
    CUtensorMap tq, tk, tv;
    if (!rows_map(&tq, a.q, a.q_stride, a.H, a.T_q, a.D_qk, 2, kBM)) return VT_ERR_CUDA;
    tk = tv = tq;  // (without keys they are not read)
    if (a.T_k > 0 && (!rows_map(&tk, a.k, a.k_stride, a.H_kv, a.T_k, a.D_qk, 2, q2::kBN) ||
                      !rows_map(&tv, a.v, a.v_stride, a.H_kv, a.T_k, a.D_v, 2, q2::kBN)))
        return VT_ERR_CUDA;
    p.q_chunks = (p.D_qk + q2::kChunk - 1) / q2::kChunk;
    p.v_chunks = (p.D_v + q2::kChunk - 1) / q2::kChunk;
    p.n_pv = (p.D_v + 15) / 16 * 16;
    p.o_vec32 = reinterpret_cast<uintptr_t>(a.o) % 32 == 0 && (a.H < 2 || p.o_sh % 16 == 0) && (a.T_q < 2 || p.o_ss % 16 == 0);
    p.tiles_per_unit = 2;
    p.cluster = 1;
    p.n_split = 1;
    const int q_bytes = 2 * p.q_chunks * static_cast<int>(q2::kChunkBytes);
    const int slot_bytes = (p.q_chunks > p.v_chunks ? p.q_chunks : p.v_chunks) * static_cast<int>(q2::kChunkBytes);
    p.stages = (kSmemLimit - 1024 - static_cast<int>(sizeof(q2::Ctl)) - 256 - q_bytes) / slot_bytes;
    if (p.stages > q2::kMaxSlots) p.stages = q2::kMaxSlots;
    const int smem = 1024 + q_bytes + p.stages * slot_bytes;
    p.n_qblocks = static_cast<int>(packed_slots(a.T_q, a.N, q2::kRows));
    p.n_units = p.n_qblocks * p.H;
    const TileKern kern = pick_tiles(p);
    if (!ensure_smem(reinterpret_cast<const void *>(kern), dev, smem)) return VT_ERR_CUDA;
    kern<<<static_cast<unsigned>(p.n_units), q2::kThreads, smem, stream>>>(tq, tk, tv, tv, p);
    return cudaGetLastError() == cudaSuccess ? VT_OK : VT_ERR_CUDA;
}

// The fp32 kernels' parameters beside those of params_of.
void set_inputs(const Args &a, PackedF32Params *p) {
    p->Q = a.q;
    p->q_sh = a.q_stride[0];
    p->q_ss = a.q_stride[1];
    p->K = a.k;
    p->k_sh = a.k_stride[0];
    p->k_ss = a.k_stride[1];
    p->V = a.v;
    p->v_sh = a.v_stride[0];
    p->v_ss = a.v_stride[1];
}

using F32Kern = void (*)(const PackedF32Params);

vt_status launch_f32(F32Kern kern, int smem, int64_t ctas, const PackedF32Params &p, int dev, cudaStream_t stream) {
    if (!ensure_smem(reinterpret_cast<const void *>(kern), dev, smem)) return VT_ERR_CUDA;
    kern<<<static_cast<unsigned>(ctas), pf::kThreads, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? VT_OK : VT_ERR_CUDA;
}

// Columns of shared memory rows: a multiple of 32 that holds both widths.
int padded(const Args &a) {
    const int64_t D = a.D_qk > a.D_v ? a.D_qk : a.D_v;
    return D <= 64 ? 64 : D <= 96 ? 96 : 128;
}

vt_status forward_f32(const Args &a, const AttnParams &base, int dev, cudaStream_t stream) {
    PackedF32Params p{};
    static_cast<AttnParams &>(p) = base;
    set_inputs(a, &p);
    const int64_t ctas = packed_slots(a.T_q, a.N, pf::kRows) * a.H;
    switch (padded(a)) {
        case 64: return launch_f32(attn_packed_f32_kernel<64>, pf::fwd_smem<64>(), ctas, p, dev, stream);
        case 96: return launch_f32(attn_packed_f32_kernel<96>, pf::fwd_smem<96>(), ctas, p, dev, stream);
        default: return launch_f32(attn_packed_f32_kernel<128>, pf::fwd_smem<128>(), ctas, p, dev, stream);
    }
}

vt_status forward(const Args &a, cudaStream_t stream) {
    VT_TRY(check_shape(a));
    if (a.N == 0 || a.H == 0 || a.T_q == 0) return VT_OK;
    Memory m(a);
    VT_TRY(m.inputs());
    VT_TRY(m.rows(a.o, a.o_stride, a.H, a.T_q, a.D_v, true));
    if (a.lse) VT_TRY(m.vector(a.lse, a.H * a.T_q * 4, 4, true));
    VT_TRY(m.clear());
    int dev = 0;
    DeviceInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || !device_info(dev, &info)) return VT_ERR_CUDA;
    const AttnParams p = params_of(a, info.status + status_slot(stream));
    VT_TRY(a.dtype == VT_BF16 ? forward_bf16(a, p, dev, stream) : forward_f32(a, p, dev, stream));
    return env_check() ? read_status(stream) : VT_OK;
}

// ---------------------------------------------------------------- gradients

// The workspace: the queries' statistics, and (split) dK and dV of every query head.
struct Layout {
    bool split;
    size_t part_k, part_v, bytes;
};

// Few blocks of keys are walked by one CTA per query head, whose results another launch adds, so that more SMs take part:
// where the key/value heads' blocks would not give every SM one (bf16, one CTA on an SM), or two (fp32).  Six texts of up to
// 333 tokens, 16 heads on 4: keys' walk 30 us with 44 units, 17 us and 6 us for the sums with 176; fp32, three of up to 500,
// 8 heads on 2: 198 us with 30 CTAs, 56 and 5 us with 120.  With more blocks the sums' bytes only add.
Layout layout_of(const Args &a, int sms) {
    const bool bf = a.dtype == VT_BF16;
    const int64_t G = a.H / a.H_kv, blocks = packed_slots(a.T_k, a.N, bf ? bw::kTile : pf::kRows) * a.H_kv;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    Layout l{};
    l.split = G > 1 && a.T_k > 0 && blocks < (bf ? 1 : 2) * sms;
    l.bytes = l.part_k = up(static_cast<size_t>(a.H * packed_slots(a.T_q, a.N, bw::kTile)) * bw::kStatBytes);
    if (l.split) {
        const size_t rows = static_cast<size_t>(a.H * a.T_k) * sizeof(float);
        l.part_v = up(l.part_k + rows * partial_ld(a.D_qk));
        l.bytes = up(l.part_v + rows * partial_ld(a.D_v));
    }
    return l;
}

// Rows start on 32 bytes.
bool vec32(const void *p, const int64_t st[2], int64_t H, int64_t T, int elt) {
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 && (H < 2 || st[0] * elt % 32 == 0) && (T < 2 || st[1] * elt % 32 == 0);
}

using GradKern = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const BwdParams);

template <template <int, int> class K>
GradKern pick_grad(const BwdParams &p) {
    const int kq = (p.D_qk + 15) / 16;
    if (p.D_v <= 64) return kq <= 4 ? K<4, 4>::kern() : kq <= 6 ? K<6, 4>::kern() : K<8, 4>::kern();
    return kq <= 4 ? K<4, 8>::kern() : kq <= 6 ? K<6, 8>::kern() : K<8, 8>::kern();
}
template <int KQ, int KV>
struct KeysKern {
    static GradKern kern() { return attn_bwd_kv_bf16_kernel<KQ, KV>; }
};
template <int KQ, int KV>
struct QueriesKern {
    static GradKern kern() { return attn_bwd_q_bf16_kernel<KQ, KV>; }
};

template <typename T, int ROWS>
vt_status launch_heads(const Args &a, const BwdParams &p, cudaStream_t stream) {
    const int64_t blocks = packed_slots(a.T_k, a.N, ROWS) * a.H_kv * (ROWS / kHeadsRows);
    if (blocks > kMaxExtent) return VT_ERR_UNSUPPORTED;
    attn_bwd_heads_kernel<T, ROWS><<<static_cast<unsigned>(blocks), kHeadsThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? VT_OK : VT_ERR_CUDA;
}

vt_status backward_bf16(const Args &a, const Grads &g, BwdParams p, int dev, cudaStream_t stream) {
    CUtensorMap tq, tk, tv, tg;
    const int64_t H_kv = a.H_kv;
    if (a.T_q > 0 && (!rows_map(&tq, a.q, a.q_stride, a.H, a.T_q, a.D_qk, 2, bw::kTile) ||
                      !rows_map(&tg, g.d_o, g.do_stride, a.H, a.T_q, a.D_v, 2, bw::kTile)))
        return VT_ERR_CUDA;
    if (a.T_k > 0 && (!rows_map(&tk, a.k, a.k_stride, H_kv, a.T_k, a.D_qk, 2, bw::kTile) ||
                      !rows_map(&tv, a.v, a.v_stride, H_kv, a.T_k, a.D_v, 2, bw::kTile)))
        return VT_ERR_CUDA;
    if (a.T_q == 0) tq = tk, tg = tv;  // (a side without rows is not read)
    if (a.T_k == 0) tk = tq, tv = tg;
    p.q_chunks = (p.D_qk + bw::kChunk - 1) / bw::kChunk;
    p.v_chunks = (p.D_v + bw::kChunk - 1) / bw::kChunk;
    p.n_pv = (p.D_v + 15) / 16 * 16;
    p.n_qk = (p.D_qk + 15) / 16 * 16;
    const int q_bytes = p.q_chunks * static_cast<int>(bw::kChunkBytes), v_bytes = p.v_chunks * static_cast<int>(bw::kChunkBytes);
    const int room = kSmemLimit - 1024 - static_cast<int>(sizeof(bw::Ctl)) - 256 - q_bytes - v_bytes;
    // slots of the two rings: as many as fit, the second ring's first where both are as long
    auto rings = [&](int first_bytes, int second_bytes, int q_least, int v_least) {
        p.q_slots = q_least;
        p.v_slots = v_least;
        int left = room - q_least * first_bytes - v_least * second_bytes;
        for (;;) {
            const bool second = p.v_slots - v_least < p.q_slots - q_least + 1 && p.v_slots < p.q_slots;
            int &slots = second ? p.v_slots : p.q_slots;
            const int bytes = second ? second_bytes : first_bytes;
            if (slots == bw::kMaxSlots || left < bytes) break;
            ++slots;
            left -= bytes;
        }
        return 1024 + q_bytes + v_bytes + p.q_slots * first_bytes + p.v_slots * second_bytes;
    };
    if (a.T_k > 0) {
        const int smem = rings(q_bytes + static_cast<int>(bw::kStatBytes), v_bytes, 2, 2);
        p.units = static_cast<int>(packed_slots(a.T_k, a.N, bw::kTile) * (a.H / p.groups));
        const GradKern kern = pick_grad<KeysKern>(p);
        if (!ensure_smem(reinterpret_cast<const void *>(kern), dev, smem)) return VT_ERR_CUDA;
        kern<<<static_cast<unsigned>(p.units), bw::kThreads, smem, stream>>>(tq, tk, tv, tg, p);
        if (cudaGetLastError() != cudaSuccess) return VT_ERR_CUDA;
    }
    if (a.T_q > 0) {
        const int smem = rings(q_bytes, v_bytes, 3, 2);
        p.units = static_cast<int>(p.slots_q * a.H);
        const GradKern kern = pick_grad<QueriesKern>(p);
        if (!ensure_smem(reinterpret_cast<const void *>(kern), dev, smem)) return VT_ERR_CUDA;
        p.follows = a.T_k > 0 ? 1 : 0;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(p.units));
        cfg.blockDim = dim3(bw::kThreads);
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = p.follows ? 1 : 0;
        if (cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, tg, p) != cudaSuccess) return VT_ERR_CUDA;
        if (cudaGetLastError() != cudaSuccess) return VT_ERR_CUDA;
    }
    return p.part_k ? launch_heads<uint16_t, bw::kTile>(a, p, stream) : VT_OK;
}

vt_status backward_f32(const Args &a, const BwdParams &base, int dev, cudaStream_t stream) {
    PackedF32Params p{};
    static_cast<BwdParams &>(p) = base;
    set_inputs(a, &p);
    const int D = padded(a);
    const int smem = D == 64 ? pf::bwd_smem<64>() : D == 96 ? pf::bwd_smem<96>() : pf::bwd_smem<128>();
    if (a.T_k > 0) {
        const int64_t slots = packed_slots(a.T_k, a.N, pf::kRows);
        VT_TRY(launch_f32(D == 64   ? attn_bwd_kv_f32_kernel<64>
                          : D == 96 ? attn_bwd_kv_f32_kernel<96>
                                    : attn_bwd_kv_f32_kernel<128>,
                          smem, slots * (a.H / p.groups), p, dev, stream));
        if (p.part_k) VT_TRY((launch_heads<float, pf::kRows>(a, p, stream)));
    }
    if (a.T_q > 0)
        VT_TRY(launch_f32(D == 64   ? attn_bwd_q_f32_kernel<64>
                          : D == 96 ? attn_bwd_q_f32_kernel<96>
                                    : attn_bwd_q_f32_kernel<128>,
                          smem, packed_slots(a.T_q, a.N, pf::kRows) * a.H, p, dev, stream));
    return VT_OK;
}

vt_status backward(const Args &a, const Grads &g, cudaStream_t stream) {
    VT_TRY(check_shape(a));
    if (g.struct_bytes != sizeof(Grads)) return VT_ERR_INVALID_ARG;
    if (a.N == 0 || a.H == 0 || (a.T_q == 0 && a.T_k == 0)) return VT_OK;
    Memory m(a);
    VT_TRY(m.inputs());
    if (a.T_q > 0) {
        VT_TRY(m.rows(a.o, a.o_stride, a.H, a.T_q, a.D_v, false));
        VT_TRY(m.vector(a.lse, a.H * a.T_q * 4, 4, false));
        VT_TRY(m.rows(g.d_o, g.do_stride, a.H, a.T_q, a.D_v, false));
        if (g.d_lse) VT_TRY(m.vector(g.d_lse, a.H * a.T_q * 4, 4, false));
    }
    VT_TRY(m.rows(g.dq, g.dq_stride, a.H, a.T_q, a.D_qk, true));
    VT_TRY(m.rows(g.dk, g.dk_stride, a.H_kv, a.T_k, a.D_qk, true));
    VT_TRY(m.rows(g.dv, g.dv_stride, a.H_kv, a.T_k, a.D_v, true));
    int dev = 0;
    DeviceInfo info;
    const bool have = cudaGetDevice(&dev) == cudaSuccess && device_info(dev, &info);
    const Layout lay = layout_of(a, have ? info.sms : 152);
    if (g.workspace_bytes < lay.bytes) return VT_ERR_INVALID_ARG;
    VT_TRY(m.vector(g.workspace, static_cast<int64_t>(lay.bytes), 256, true));
    VT_TRY(m.clear());
    if (!have) return VT_ERR_CUDA;
    BwdParams p{};
    static_cast<AttnParams &>(p) = params_of(a, info.status + status_slot(stream));
    const int elt = a.dtype == VT_BF16 ? 2 : 4;
    p.scale = a.scale;
    p.stat = static_cast<float *>(g.workspace);
    p.groups = lay.split ? 1 : p.kv_group;
    p.head_units = lay.split ? p.kv_group : 1;
    if (lay.split) {
        p.part_k = reinterpret_cast<float *>(static_cast<uint8_t *>(g.workspace) + lay.part_k);
        p.part_v = reinterpret_cast<float *>(static_cast<uint8_t *>(g.workspace) + lay.part_v);
        p.part_ldk = static_cast<int>(partial_ld(a.D_qk));
        p.part_ldv = static_cast<int>(partial_ld(a.D_v));
    }
    p.slots_q = static_cast<int>(packed_slots(a.T_q, a.N, bw::kTile));
    p.dO = g.d_o;
    p.do_sh = g.do_stride[0];
    p.do_ss = g.do_stride[1];
    p.dlse = g.d_lse;
    p.dQ = g.dq;
    p.dq_sh = g.dq_stride[0];
    p.dq_ss = g.dq_stride[1];
    p.dK = g.dk;
    p.dk_sh = g.dk_stride[0];
    p.dk_ss = g.dk_stride[1];
    p.dV = g.dv;
    p.dv_sh = g.dv_stride[0];
    p.dv_ss = g.dv_stride[1];
    p.dq_vec32 = vec32(g.dq, g.dq_stride, a.H, a.T_q, elt);
    p.dk_vec32 = vec32(g.dk, g.dk_stride, a.H_kv, a.T_k, elt);
    p.dv_vec32 = vec32(g.dv, g.dv_stride, a.H_kv, a.T_k, elt);
    if (a.T_q > 0) {
        const unsigned ctas = static_cast<unsigned>(p.slots_q * a.H * (bw::kTile / kStatRows));
        if (a.dtype == VT_BF16) attn_bwd_stats_kernel<uint16_t><<<ctas, kStatThreads, 0, stream>>>(p);
        else attn_bwd_stats_kernel<float><<<ctas, kStatThreads, 0, stream>>>(p);
        if (cudaGetLastError() != cudaSuccess) return VT_ERR_CUDA;
    }
    VT_TRY(a.dtype == VT_BF16 ? backward_bf16(a, g, p, dev, stream) : backward_f32(a, p, dev, stream));
    return env_check() ? read_status(stream) : VT_OK;
}

}  // namespace
}  // namespace packed
}  // namespace vt

extern "C" {

vt_status vt_attn_fwd_packed(const vt_attn_packed_args *args, vt_stream_t stream) {
    const vt::NvtxRange range("vt_attn_fwd_packed");
    if (!args) return VT_ERR_INVALID_ARG;
    return vt::packed::forward(*args, reinterpret_cast<cudaStream_t>(stream));
}

vt_status vt_attn_bwd_packed(const vt_attn_packed_args *args, const vt_attn_packed_grads *grads, vt_stream_t stream) {
    const vt::NvtxRange range("vt_attn_bwd_packed");
    if (!args || !grads) return VT_ERR_INVALID_ARG;
    return vt::packed::backward(*args, *grads, reinterpret_cast<cudaStream_t>(stream));
}

size_t vt_attn_bwd_packed_workspace_size(int64_t N, int64_t H, int64_t H_kv, int64_t T_q, int64_t T_k, int64_t D_qk,
                                         int64_t D_v, vt_dtype dtype) {
    vt_attn_packed_args a{};
    a.struct_bytes = sizeof a;
    a.N = N; a.H = H; a.H_kv = H_kv; a.T_q = T_q; a.T_k = T_k; a.D_qk = D_qk; a.D_v = D_v;
    a.dtype = dtype;
    if (vt::packed::check_shape(a) != VT_OK || N == 0 || H == 0 || (T_q == 0 && T_k == 0)) return 0;
    int dev = 0;
    vt::DeviceInfo info;
    const bool have = cudaGetDevice(&dev) == cudaSuccess && vt::device_info(dev, &info);
    return vt::packed::layout_of(a, have ? info.sms : 152).bytes;
}

}  // extern "C"
