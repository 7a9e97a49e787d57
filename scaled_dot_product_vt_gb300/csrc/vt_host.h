// Host-side helpers shared by the library's translation units: argument spans, per-device facts, status
// words, shared-memory grants and tensor maps.  Defined in vt_attn_api.cu unless inline here.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "../../include/vt_attn.h"

#define VT_TRY(expr)                          \
    do {                                      \
        const vt_status vt_try_ = (expr);     \
        if (vt_try_ != VT_OK) return vt_try_; \
    } while (0)

#pragma GCC visibility push(hidden)
namespace vt {

// An NVTX range over one public call (named after the entry point), for profilers that record NVTX;
// without one attached, push and pop return at once.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

constexpr int64_t kMaxD = 128;
constexpr int64_t kMaxExtent = 0x7FFFFFFF;  // B and H (their product is bounded by the work-unit count)
// S_q and S_k: the kernels form row and key indices a few tiles past an extent in 32-bit ints
constexpr int64_t kMaxSeq = int64_t(1) << 30;
constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
constexpr int kSmemLimit = 232448;  // 227 KiB per CTA on sm_100-class parts
constexpr int64_t kMaxStrideBytes = int64_t(1) << 40;  // (b, h, s) strides stay below what a TMA tensor map accepts

struct Span {
    uintptr_t lo, hi;  // [lo, hi) bytes touched by a tensor's logical elements
};

inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// The bytes a tensor's logical elements touch; false when the extent arithmetic overflows (no such
// tensor fits in an address space).  Extents and strides are positive here.
bool span_of(const void *p, const int64_t st[3], int64_t B, int64_t H, int64_t S, int64_t D, int elt, Span *out);

// `bytes` contiguous bytes from p; false on overflow.
inline bool span_bytes(const void *p, int64_t bytes, Span *out) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (bytes < 0 || static_cast<uint64_t>(bytes) > UINTPTR_MAX - lo) return false;
    *out = {lo, lo + static_cast<uintptr_t>(bytes)};
    return true;
}

// True when no two logical elements of a [B, H, S, D] tensor with (b, h, s) strides st and unit stride
// along D share an address: with the extents of size 1 left out and the rest taken in order of
// increasing stride, each stride reaches past everything the smaller ones span.  This accepts every
// nesting of the three indices ([B,H,S,D], [B,S,H,D], ...) without gaps or overlap, and any padding.
bool rows_disjoint(const int64_t st[3], int64_t B, int64_t H, int64_t S, int64_t D);

bool env_check();  // VT_CHECK is set: every call reads its status word

// Per-device facts that do not change while the process runs, looked up once: the SM count, the L2
// size and the device address of the status words.
struct DeviceInfo {
    bool ready = false;
    int sms = 0;
    long long l2_bytes = 0;
    unsigned *status = nullptr;  // g_status on this device
};
constexpr int kMaxDevices = 64;
bool device_info(int dev, DeviceInfo *out);

// The status slot of a stream (see its definition).
int status_slot(cudaStream_t s);

// Grant a kernel `bytes` of dynamic shared memory on a device (once per kernel, device and size).
bool ensure_smem(const void *kern, int dev, int bytes);

// 4-D map over [B][H][S][D] (D innermost), box = 128-byte chunk of D x `rows` rows of S.
bool make_map(CUtensorMap *map, const void *ptr, const int64_t st[3], int64_t B, int64_t H, int64_t S, int64_t D,
              int elt, int rows);

// A tensor's checks (strides of an index with one value are not looked at).
inline vt_status tensor(const void *p, const int64_t st[3], int64_t B, int64_t H, int64_t S, int64_t D, int elt, bool out,
                        Span *span) {
    if (!p) return VT_ERR_INVALID_ARG;
    const int64_t n[3] = {B, H, S};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && st[i] <= 0) return VT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(p) % 16) return VT_ERR_MISALIGNED;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && st[i] >= kMaxStrideBytes / elt) return VT_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (st[i] * elt) % 16) return VT_ERR_MISALIGNED;
    if (!span_of(p, st, B, H, S, D, elt, span)) return VT_ERR_INVALID_ARG;
    if (out && !rows_disjoint(st, B, H, S, D)) return VT_ERR_INVALID_ARG;
    return VT_OK;
}

// Wait for `stream`, then read and clear its status word on the current device.
vt_status read_status(cudaStream_t stream);

}  // namespace vt
#pragma GCC visibility pop
