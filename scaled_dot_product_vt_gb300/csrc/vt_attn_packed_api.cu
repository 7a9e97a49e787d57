// Host side of vt_attn_fwd_packed: argument checks and launches (contract in include/vt_attn.h).
#include <cmath>

#include "vt_attn_bf16_2q.cuh"
#include "vt_attn_packed.cuh"
#include "vt_host.h"
#include "vt_pieces.h"

namespace vt {
namespace packed {
namespace {

using Args = vt_attn_packed_args;

constexpr int kLeastRows = 64;  // rows of the smallest block a launch is cut into

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
    if (__builtin_mul_overflow(packed_slots(T, a.N, kLeastRows), a.H, &units) || units > kMaxExtent) return VT_ERR_UNSUPPORTED;
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
    if (a.dtype != VT_BF16) return VT_ERR_UNSUPPORTED;
    VT_TRY(forward_bf16(a, p, dev, stream));
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

}  // extern "C"
