// Host side of vt_qk_rope_fwd and vt_qk_rope_bwd: argument checks and launches (contract in include/vt_attn.h).
#include <cmath>
#include <cstring>

#include "vt_host.h"
#include "vt_pieces.h"
#include "vt_qk_rope.cuh"

namespace vt {
namespace rope {
namespace {

using Args = vt_qk_rope_args;

// No output overlaps another piece, but for an output that is the same tensor as one of these inputs.
bool outputs_clear(const Pieces &ps, int elt, const void *in0, const void *in1, const void *in2 = nullptr,
                   const void *in3 = nullptr) {
    for (int i = 0; i < ps.n; ++i)
        for (int j = 0; j < ps.n; ++j) {
            const Piece &x = ps.at[i], &y = ps.at[j];
            if (i == j || !x.out || !overlap(x.span, y.span)) continue;
            const bool named = y.p == in0 || y.p == in1 || y.p == in2 || y.p == in3;
            if (named && !y.out && x.side == y.side && same_tensor(x, y)) continue;
            if (beside(x, y, elt)) continue;
            return false;
        }
    return true;
}

vt_status check_shape(const Args &a, bool *empty) {
    *empty = false;
    if (a.struct_bytes != sizeof(Args) || a.reserved != 0) return VT_ERR_INVALID_ARG;
    if (a.dtype != VT_F32 && a.dtype != VT_BF16) return VT_ERR_INVALID_ARG;
    if (a.B < 0 || a.H < 0 || a.H_kv < 0 || a.S < 0 || a.D <= 0) return VT_ERR_INVALID_ARG;
    if (a.R < 2 || a.R % 2 || a.R > a.D || a.axes < 1) return VT_ERR_INVALID_ARG;
    if (a.normalize && !(std::isfinite(a.eps) && a.eps >= 0.0f)) return VT_ERR_INVALID_ARG;
    if (a.kv_len && (a.cap < 0 || (a.v && a.D_v <= 0))) return VT_ERR_INVALID_ARG;
    if (a.D > kMaxD || a.axes > VT_ROPE_MAX_AXES || (a.kv_len && a.v && a.D_v > kMaxD)) return VT_ERR_UNSUPPORTED;
    if (a.B > kMaxExtent || a.H > kMaxExtent || a.H_kv > kMaxExtent || a.S > kMaxSeq || (a.kv_len && a.cap > kMaxSeq))
        return VT_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < a.R / 2; ++i)
        if (a.pair_axis[i] >= a.axes) return VT_ERR_INVALID_ARG;
    // tokens, and the next group's past the last one, are counted in 32 bits (B < 2^31 and S <= 2^30 here)
    if (a.B * a.S > kMaxSeq) return VT_ERR_UNSUPPORTED;
    *empty = a.B == 0 || a.S == 0 || (a.H == 0 && a.H_kv == 0);
    return VT_OK;
}

// A [B,H,S,D] tensor: present, 16-byte rows, strides in range (that of an index with one value is not looked
// at); an output also has rows of its own.
vt_status add_tensor(Pieces *ps, const void *p, const int64_t st[3], int64_t B, int64_t H, int64_t S, int64_t D, int elt,
                     bool out, int side) {
    if (!p || !st) return VT_ERR_INVALID_ARG;
    const int64_t n[3] = {B, H, S};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && st[i] <= 0) return VT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(p) % 16) return VT_ERR_MISALIGNED;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && st[i] >= kMaxStrideBytes / elt) return VT_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (st[i] * elt) % 16) return VT_ERR_MISALIGNED;
    Span s;
    if (!span_of(p, st, B, H, S, D, elt, &s)) return VT_ERR_INVALID_ARG;
    if (out && !rows_disjoint(st, B, H, S, D)) return VT_ERR_INVALID_ARG;
    ps->add({s, p, st, out, side, {B, H, S}, D});
    return VT_OK;
}

vt_status add_vector(Pieces *ps, const void *p, int64_t n, int elt, int align, bool out) {
    if (!p) return VT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(p) % align) return VT_ERR_MISALIGNED;
    Span s;
    if (!span_bytes(p, n * elt, &s)) return VT_ERR_INVALID_ARG;
    ps->add({s, p, nullptr, out, 0, {}, 0});
    return VT_OK;
}

#define VT_TRY(expr)                                \
    do {                                            \
        const vt_status vt_try_ = (expr);           \
        if (vt_try_ != VT_OK) return vt_try_;       \
    } while (0)

// The vectors both directions read: weights, frequencies and positions.
vt_status add_common(const Args &a, int elt, Pieces *ps) {
    if (a.normalize && a.q_weight && a.H > 0) VT_TRY(add_vector(ps, a.q_weight, a.D, elt, 16, false));
    if (a.normalize && a.k_weight && a.H_kv > 0) VT_TRY(add_vector(ps, a.k_weight, a.D, elt, 16, false));
    VT_TRY(add_vector(ps, a.freqs, a.R / 2, 4, 4, false));
    if (!a.positions) return VT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a.positions) % 4) return VT_ERR_MISALIGNED;
    for (int i = 0; i < 3; ++i) {
        if (a.pos_stride[i] < 0) return VT_ERR_INVALID_ARG;
        if (a.pos_stride[i] >= kMaxStrideBytes / 4) return VT_ERR_UNSUPPORTED;
    }
    Span s;
    if (!span_of(a.positions, a.pos_stride, a.axes, a.B, a.S, 1, 4, &s)) return VT_ERR_INVALID_ARG;
    ps->add({s, a.positions, nullptr, false, 0, {}, 0});
    return VT_OK;
}

// How a call's rows are spread over the threads (see vt_qk_rope.cuh), for `vec` elements per run.
struct Shape {
    int vec, nc;
};
Shape shape_of(const Args &a, int elt) {
    // 16-byte runs need the halves of the rotated part, and what follows it, to be whole runs
    for (int vec = 16 / elt; vec >= 4; vec /= 2) {
        const bool fits = a.interleaved ? a.R % (2 * vec) == 0 : (a.R / 2) % vec == 0;
        if (fits && (a.D - a.R) % (2 * vec) == 0) return {vec, 1};
    }
    return {1, (a.D + 1) / 2 <= 32 ? 1 : 4};
}

int pow2_at_least(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// Fill what both directions share; `sms` sets how far tokens are gathered into a block.
Params common_params(const Args &a, const Shape &sh, int sms) {
    Params p{};
    p.B = static_cast<int>(a.B);
    p.H = static_cast<int>(a.H);
    p.H_kv = static_cast<int>(a.H_kv);
    p.S = static_cast<int>(a.S);
    p.D = static_cast<int>(a.D);
    p.half = static_cast<int>(a.R / 2);
    p.chunks = (p.D + 2 * sh.vec - 1) / (2 * sh.vec);
    const int lanes = (p.chunks + sh.nc - 1) / sh.nc;
    // the norm's shuffles want a power of two; without it a row takes exactly the threads it needs
    p.tpr = a.normalize ? pow2_at_least(lanes) : lanes;
    p.tokens = static_cast<unsigned>(a.B * a.S);
    // at most one angle per thread, while every SM still has a few blocks
    int tok = kThreads / p.half;
    if (tok > 8) tok = 8;
    if (tok > kThreads / p.tpr) tok = kThreads / p.tpr;
    while (tok > 1 && a.B * a.S / tok < 4LL * sms) tok /= 2;
    p.tok = tok < 1 ? 1 : tok;
    p.heads = kThreads / (p.tpr * p.tok);
    p.eps = a.eps;
    p.x[0] = a.q;
    p.x[1] = a.k;
    p.y[0] = a.q_out;
    p.y[1] = a.k_out;
    p.w[0] = a.normalize ? a.q_weight : nullptr;
    p.w[1] = a.normalize ? a.k_weight : nullptr;
    for (int i = 0; i < 3; ++i) {
        p.x_st[0][i] = a.q_stride[i];
        p.x_st[1][i] = a.k_stride[i];
        p.y_st[0][i] = a.q_out_stride[i];
        p.y_st[1][i] = a.k_out_stride[i];
        p.pos_st[i] = a.pos_stride[i];
    }
    p.freqs = a.freqs;
    p.pos = a.positions;
    std::memcpy(p.axis, a.pair_axis, sizeof p.axis);
    return p;
}

// A kernel variant and the shared memory of its ring.
struct Variant {
    void (*kern)(const Params);
    int smem;
};

template <typename T, int VEC, int NC, bool BWD>
Variant pick_form(bool inter, bool norm) {
    if constexpr (BWD) {
        const int smem = norm ? kAheadBwd * Ring<T, VEC, 4 * NC, kAheadBwd>::kStage : kAheadBwd * Ring<T, VEC, 2 * NC, kAheadBwd>::kStage;
        return {inter ? (norm ? bwd_kernel<T, VEC, NC, true, true> : bwd_kernel<T, VEC, NC, true, false>)
                      : (norm ? bwd_kernel<T, VEC, NC, false, true> : bwd_kernel<T, VEC, NC, false, false>),
                smem};
    } else {
        return {inter ? (norm ? fwd_kernel<T, VEC, NC, true, true> : fwd_kernel<T, VEC, NC, true, false>)
                      : (norm ? fwd_kernel<T, VEC, NC, false, true> : fwd_kernel<T, VEC, NC, false, false>),
                kAhead * Ring<T, VEC, 2 * NC, kAhead>::kStage};
    }
}

template <bool BWD>
Variant pick(const Args &a, const Shape &sh) {
    const bool in = a.interleaved != 0, no = a.normalize != 0;
    if (a.dtype == VT_BF16) {
        if (sh.vec == 8) return pick_form<bf16, 8, 1, BWD>(in, no);
        if (sh.vec == 4) return pick_form<bf16, 4, 1, BWD>(in, no);
        return sh.nc == 1 ? pick_form<bf16, 1, 1, BWD>(in, no) : pick_form<bf16, 1, 4, BWD>(in, no);
    }
    if (sh.vec == 4) return pick_form<float, 4, 1, BWD>(in, no);
    return sh.nc == 1 ? pick_form<float, 1, 1, BWD>(in, no) : pick_form<float, 1, 4, BWD>(in, no);
}

vt_status launch(const Variant &v, int smem, unsigned blocks, const Params &p, int dev, cudaStream_t stream) {
    if (!ensure_smem(reinterpret_cast<const void *>(v.kern), dev, smem)) return VT_ERR_CUDA;
    v.kern<<<blocks, kThreads, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? VT_OK : VT_ERR_CUDA;
}

vt_status device_of(int *dev, DeviceInfo *info) {
    return cudaGetDevice(dev) == cudaSuccess && device_info(*dev, info) ? VT_OK : VT_ERR_CUDA;
}

vt_status forward(const Args &a, cudaStream_t stream) {
    bool empty = false;
    VT_TRY(check_shape(a, &empty));
    if (empty) return VT_OK;
    const int elt = a.dtype == VT_BF16 ? 2 : 4;
    Pieces ps;
    VT_TRY(add_common(a, elt, &ps));
    if (a.H > 0) {
        VT_TRY(add_tensor(&ps, a.q, a.q_stride, a.B, a.H, a.S, a.D, elt, false, 1));
        VT_TRY(add_tensor(&ps, a.q_out, a.q_out_stride, a.B, a.H, a.S, a.D, elt, true, 1));
    }
    const bool append = a.kv_len != nullptr;
    if (a.H_kv > 0) {
        VT_TRY(add_tensor(&ps, a.k, a.k_stride, a.B, a.H_kv, a.S, a.D, elt, false, 2));
        // (an append writes no row of a cache without rows: its tokens are all past the end)
        const int64_t rows = append ? (a.cap > 0 ? a.cap : 1) : a.S;
        VT_TRY(add_tensor(&ps, a.k_out, a.k_out_stride, a.B, a.H_kv, rows, a.D, elt, true, 2));
        if (append && a.v) {
            VT_TRY(add_tensor(&ps, a.v, a.v_stride, a.B, a.H_kv, a.S, a.D_v, elt, false, 3));
            VT_TRY(add_tensor(&ps, a.v_out, a.v_out_stride, a.B, a.H_kv, rows, a.D_v, elt, true, 3));
        }
    }
    if (append) VT_TRY(add_vector(&ps, a.kv_len, a.B, 4, 4, false));
    // Q and (without an append) K may be rotated in place
    if (!outputs_clear(ps, elt, a.q, append ? nullptr : a.k)) return VT_ERR_INVALID_ARG;

    int dev = 0;
    DeviceInfo info;
    VT_TRY(device_of(&dev, &info));
    const Shape sh = shape_of(a, elt);
    Params p = common_params(a, sh, info.sms);
    p.kv_len = a.kv_len;
    p.cap = append ? a.cap : 0;
    p.v = append && a.H_kv > 0 ? a.v : nullptr;
    p.v_out = a.v_out;
    p.D_v = static_cast<int>(append && a.v ? a.D_v : 0);
    for (int i = 0; i < 3; ++i) {
        p.v_st[i] = a.v_stride[i];
        p.vo_st[i] = a.v_out_stride[i];
    }
    p.status = info.status + status_slot(stream);
    const int64_t groups = (a.B * a.S + p.tok - 1) / p.tok, most = 3LL * info.sms;
    const unsigned blocks = static_cast<unsigned>(groups < most ? groups : most);
    const Variant v = pick<false>(a, sh);
    VT_TRY(launch(v, v.smem, blocks, p, dev, stream));
    return env_check() ? read_status(stream) : VT_OK;
}

size_t bwd_workspace(int64_t D) {
    return D < 1 || D > kMaxD ? 0 : static_cast<size_t>(2 * kBwdMaxBlocks * D) * sizeof(float);
}

vt_status backward(const Args &a, const void *gq, const int64_t gq_st[3], const void *gk, const int64_t gk_st[3],
                   float *dwq, float *dwk, void *ws, size_t ws_bytes, cudaStream_t stream) {
    bool empty = false;
    VT_TRY(check_shape(a, &empty));
    if (a.kv_len) return VT_ERR_INVALID_ARG;
    const int elt = a.dtype == VT_BF16 ? 2 : 4;
    const bool norm = a.normalize != 0;
    if (!norm) dwq = dwk = nullptr;
    Pieces ps;
    if (!empty) {
        VT_TRY(add_common(a, elt, &ps));
        if (a.H > 0) {
            VT_TRY(add_tensor(&ps, gq, gq_st, a.B, a.H, a.S, a.D, elt, false, 1));
            VT_TRY(add_tensor(&ps, a.q_out, a.q_out_stride, a.B, a.H, a.S, a.D, elt, true, 1));
            if (norm) VT_TRY(add_tensor(&ps, a.q, a.q_stride, a.B, a.H, a.S, a.D, elt, false, 1));
        }
        if (a.H_kv > 0) {
            VT_TRY(add_tensor(&ps, gk, gk_st, a.B, a.H_kv, a.S, a.D, elt, false, 2));
            VT_TRY(add_tensor(&ps, a.k_out, a.k_out_stride, a.B, a.H_kv, a.S, a.D, elt, true, 2));
            if (norm) VT_TRY(add_tensor(&ps, a.k, a.k_stride, a.B, a.H_kv, a.S, a.D, elt, false, 2));
        }
    }
    if (dwq) VT_TRY(add_vector(&ps, dwq, a.D, 4, 4, true));
    if (dwk) VT_TRY(add_vector(&ps, dwk, a.D, 4, 4, true));
    const bool weights = !empty && (dwq || dwk);
    if (weights) {
        if (!ws || ws_bytes < bwd_workspace(a.D)) return VT_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(ws) % 256) return VT_ERR_MISALIGNED;
        Span s;
        if (!span_bytes(ws, static_cast<int64_t>(bwd_workspace(a.D)), &s)) return VT_ERR_INVALID_ARG;
        ps.add({s, ws, nullptr, true, 0, {}, 0});
    }
    // dq may take the place of q or of dq_out, dk that of k or of dk_out
    if (!outputs_clear(ps, elt, gq, gk, a.q, a.k)) return VT_ERR_INVALID_ARG;
    if (empty) {  // no token: the weights' gradients are 0
        if (dwq && cudaMemsetAsync(dwq, 0, a.D * sizeof(float), stream) != cudaSuccess) return VT_ERR_CUDA;
        if (dwk && cudaMemsetAsync(dwk, 0, a.D * sizeof(float), stream) != cudaSuccess) return VT_ERR_CUDA;
        return env_check() ? read_status(stream) : VT_OK;
    }

    int dev = 0;
    DeviceInfo info;
    VT_TRY(device_of(&dev, &info));
    const Shape sh = shape_of(a, elt);
    Params p = common_params(a, sh, info.sms);
    p.g[0] = gq;
    p.g[1] = gk;
    for (int i = 0; i < 3; ++i) {
        p.g_st[0][i] = a.H > 0 ? gq_st[i] : 0;
        p.g_st[1][i] = a.H_kv > 0 ? gk_st[i] : 0;
    }
    // Two blocks per SM in all (they fit at once), for Q and for K in proportion to what a group of tokens costs them:
    // its rounds of rows, and about two rounds' time for its angles and addresses.
    const int64_t groups = (a.B * a.S + p.tok - 1) / p.tok;
    const int most = 2 * info.sms < kBwdMaxBlocks ? 2 * info.sms : kBwdMaxBlocks;
    const int cost_q = p.H > 0 ? (p.H + p.heads - 1) / p.heads + 2 : 0;
    const int cost_k = p.H_kv > 0 ? (p.H_kv + p.heads - 1) / p.heads + 2 : 0;
    int n_k = static_cast<int>(static_cast<int64_t>(most) * cost_k / (cost_q + cost_k));
    if (p.H_kv > 0 && n_k < 1) n_k = 1;
    if (p.H > 0 && n_k > most - 1) n_k = most - 1;
    int n_q = most - n_k;
    if (n_q > groups) n_q = static_cast<int>(groups);
    if (n_k > groups) n_k = static_cast<int>(groups);
    p.blocks_q = n_q;
    float *part = static_cast<float *>(ws);
    p.part[0] = dwq ? part : nullptr;
    p.part[1] = dwk ? part + static_cast<long long>(kBwdMaxBlocks) * p.D : nullptr;
    const Variant v = pick<true>(a, sh);
    const int sums = norm ? kThreads / p.tpr * p.D * static_cast<int>(sizeof(float)) : 0;
    VT_TRY(launch(v, v.smem > sums ? v.smem : sums, static_cast<unsigned>(n_q + n_k), p, dev, stream));
    if (!weights) return env_check() ? read_status(stream) : VT_OK;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((p.D + 7) / 8, 2);
    cfg.blockDim = dim3(8 * kSumRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const float *part_q = p.part[0], *part_k = p.part[1];
    const int D = p.D;
    if (cudaLaunchKernelEx(&cfg, bwd_weights_kernel, part_q, part_k, dwq, dwk, n_q, n_k, D) != cudaSuccess)
        return VT_ERR_CUDA;
    if (cudaGetLastError() != cudaSuccess) return VT_ERR_CUDA;
    return env_check() ? read_status(stream) : VT_OK;
}

}  // namespace
}  // namespace rope
}  // namespace vt

extern "C" {

vt_status vt_qk_rope_fwd(const vt_qk_rope_args *args, vt_stream_t stream) {
    const vt::NvtxRange range("vt_qk_rope_fwd");
    if (!args) return VT_ERR_INVALID_ARG;
    return vt::rope::forward(*args, reinterpret_cast<cudaStream_t>(stream));
}

vt_status vt_qk_rope_bwd(const vt_qk_rope_args *args, const void *dq_out, const int64_t dq_out_stride[3],
                         const void *dk_out, const int64_t dk_out_stride[3], float *dq_weight, float *dk_weight,
                         void *workspace, size_t workspace_bytes, vt_stream_t stream) {
    const vt::NvtxRange range("vt_qk_rope_bwd");
    if (!args) return VT_ERR_INVALID_ARG;
    return vt::rope::backward(*args, dq_out, dq_out_stride, dk_out, dk_out_stride, dq_weight, dk_weight, workspace,
                              workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t vt_qk_rope_bwd_workspace_size(int64_t D) { return vt::rope::bwd_workspace(D); }

}  // extern "C"
