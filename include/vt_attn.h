/*
 * vt_attn — scaled dot-product attention forward on one GB300 GPU (sm_103a).
 *
 * The operation (VeriTile page "VeriTile.Examples.FlashAttention1.NaiveRefinement":
 * fa1NaiveReference4D and fa1NaiveCausalReference4D, with the sequence-boundary and
 * head-dimension-tail write contract of fa1_boundaryD_refines_naive_reference_views;
 * separate query/key and value widths as in the accy page
 * "tiny.accy.kernel.library.attention", spec fields `qk` and `value`):
 *
 *   for every batch b < B, head h < H, query row i < S_q and value column e < D_v
 *     O[b,h,i,e] = sum_{j in A_i} softmax_j( scale * sum_{d<D_qk} Q[b,h,i,d] K[b,h,j,d] ) V[b,h,j,e]
 *   where A_i = { j < S_k } (causal = 0) or { j < S_k : j <= i } (causal != 0; key j
 *   <= query i counted from index 0 of both sequences).
 *
 * Layouts.  Q is [B,H,S_q,D_qk], K is [B,H,S_k,D_qk], V is [B,H,S_k,D_v] and O is
 * [B,H,S_q,D_v], the last index contiguous (stride 1).  vt_attn_fwd takes the packed
 * row-major layout; vt_attn_fwd_strided takes element strides for the (b, h, s)
 * indices of each tensor.  All four pointers are DEVICE pointers (CUDA global memory
 * of the current device).
 *
 * Element types.  VT_BF16: bf16 in, bf16 out, products accumulated in fp32 on the
 * tensor cores (probabilities are rounded to bf16 before the P*V product; the row sum
 * that normalises O counts each key tile's largest probability at its bf16 value, so a
 * row dominated by one key reproduces that key's value row up to the output rounding.
 * That holds for one dominating key per tile: when two or more keys of a tile carry most
 * of a row's weight, the bf16 rounding of the others' probabilities stays in the result,
 * an error of up to about 2^-9 of |O| on top of the output rounding; for |V| in [4, 8)
 * that is about 0.03).
 * VT_F32: fp32 in, fp32 out, products on the TF32 tensor-core path with fp32
 * accumulation (inputs and probabilities keep the TF32 subset of their bits).
 *
 * Ownership.  The caller owns every buffer.  The library allocates no device memory
 * per call: tensor maps are built on the host and passed by value to the kernel.
 *
 * Writes.  Only O's logical elements (i < S_q, e < D_v of each (b, h)) are written;
 * memory between rows or heads of a strided O is never touched.  O must not overlap
 * Q, K or V, and no two of O's logical elements may share an address (the strides may
 * nest the b, h and s indices in any order, e.g. [B,S,H,D], with any padding).
 *
 * Asynchrony.  Calls enqueue work on `stream` and return without waiting.  A kernel
 * that detects a problem on the device (a pipeline wait that exceeds its time limit)
 * records it in the device status word of the stream it was launched on instead of
 * faulting; vt_last_device_status(stream) synchronises that stream and returns (and
 * clears) that stream's status only.  If the environment variable VT_CHECK is set to a
 * non-zero value, every call does this itself.
 *
 * Argument errors are detected on the host before anything is launched:
 *   VT_ERR_INVALID_ARG   a NULL pointer, a negative extent, S_k, D_qk or D_v equal to 0,
 *                        an unknown dtype, a non-finite scale, O overlapping Q/K/V or
 *                        itself, a non-positive stride, or (vt_attn_fwd) extents whose
 *                        packed element count overflows 64 bits;
 *   VT_ERR_UNSUPPORTED   D_qk or D_v above 128, S_q or S_k above 2^30, B or H above
 *                        2^31 - 1, a (b, h, s) stride of 2^40 bytes or more (beyond a TMA
 *                        tensor map), or more than 2^31 - 1 work units (query blocks x heads x
 *                        batches x split-KV shares);
 *   (also VT_ERR_INVALID_ARG: extents and strides whose byte span overflows 64 bits);
 *   VT_ERR_MISALIGNED    a pointer not 16-byte aligned, or a (b, h, s) stride whose
 *                        byte size is not a multiple of 16 (the TMA engine's rule);
 *   VT_ERR_CUDA          a CUDA runtime or driver call failed (no device, launch error).
 * B, H or S_q equal to 0 is a valid empty problem: VT_OK, nothing launched.
 */
#ifndef VT_ATTN_H
#define VT_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *vt_stream_t;

typedef enum { VT_F32 = 0, VT_BF16 = 1 } vt_dtype;

typedef enum {
    VT_OK = 0,
    VT_ERR_INVALID_ARG = 1,
    VT_ERR_UNSUPPORTED = 2,
    VT_ERR_MISALIGNED = 3,
    VT_ERR_CUDA = 4,
    VT_ERR_DEVICE_TIMEOUT = 5,
    VT_ERR_DEVICE_BOUNDS = 6
} vt_status;

/*
 * Attention forward on packed [B,H,S,D] tensors (the operation above).
 * Q, K, V: device pointers to the inputs (read only).  O: device pointer to the output.
 * scale: the factor applied to every dot product (the VeriTile reference's `scale`
 * parameter; 1/sqrt(D_qk) is the usual choice).  causal: 0 or non-zero.
 */
vt_status vt_attn_fwd(const void *Q, const void *K, const void *V, void *O,
                      int64_t B, int64_t H, int64_t S_q, int64_t S_k,
                      int64_t D_qk, int64_t D_v,
                      float scale, int causal, vt_dtype dtype, vt_stream_t stream);

/*
 * The same operation on strided tensors.  x_stride[0..2] are the element strides of
 * the b, h and s indices of tensor x; its last index has stride 1.  Every stride must
 * be positive and its byte size a multiple of 16.
 */
vt_status vt_attn_fwd_strided(const void *Q, const int64_t q_stride[3],
                              const void *K, const int64_t k_stride[3],
                              const void *V, const int64_t v_stride[3],
                              void *O, const int64_t o_stride[3],
                              int64_t B, int64_t H, int64_t S_q, int64_t S_k,
                              int64_t D_qk, int64_t D_v,
                              float scale, int causal, vt_dtype dtype, vt_stream_t stream);

/*
 * Options for vt_attn_fwd_ex.  A zeroed struct gives the defaults of vt_attn_fwd.
 *   wait_timeout_ns  limit for any single pipeline wait inside the kernel before it
 *                    gives up, records VT_ERR_DEVICE_TIMEOUT and exits cleanly
 *                    (0: 2 seconds).
 *   flags            VT_OPT_TEST_STALL makes the kernel wait on a barrier that is never
 *                    signalled, so that the time-limit path can be tested; it does no
 *                    attention work and leaves O unwritten.
 *                    VT_OPT_TEST_BOUNDS (debug library only, libvt_attn_debug.so, built
 *                    with VT_DEBUG) makes the first device index check of the producer
 *                    report a failure, so that the VT_ERR_DEVICE_BOUNDS path can be tested:
 *                    the kernel stops before any access and leaves O unwritten.  The
 *                    release library ignores it.
 *
 * The debug library exports the same entry points.  Its kernels check their index invariants
 * (decoded work units, key-tile ranges, ring slots, output rows) before each access they guard;
 * a failed check records VT_ERR_DEVICE_BOUNDS for vt_last_device_status, skips the access and
 * stops the kernel through the same clean path as a time-out.
 */
#define VT_OPT_TEST_STALL 1u
#define VT_OPT_TEST_BOUNDS 2u
typedef struct {
    uint64_t wait_timeout_ns;
    uint32_t flags;
    uint32_t reserved;
} vt_attn_opts;

/* vt_attn_fwd_strided with options (opts may be NULL). */
vt_status vt_attn_fwd_ex(const void *Q, const int64_t q_stride[3],
                         const void *K, const int64_t k_stride[3],
                         const void *V, const int64_t v_stride[3],
                         void *O, const int64_t o_stride[3],
                         int64_t B, int64_t H, int64_t S_q, int64_t S_k,
                         int64_t D_qk, int64_t D_v,
                         float scale, int causal, vt_dtype dtype,
                         const vt_attn_opts *opts, vt_stream_t stream);

/*
 * Split-KV forward: the same operation, with the key range of every query block cut into
 * n_split contiguous shares that separate CTAs process at the same time.  Each share writes an
 * unnormalised partial output with its row max, its row sum and that sum's correction for the
 * bf16 rounding of P (bf16 I/O) to `workspace`; a merge kernel then
 * combines the shares of each row into O (the continuation step of the VeriTile coverage table's
 * attention_fwd_triton3 row, case 4, which reads a previous M, L and Out and merges further keys).
 * It pays off when B * H * ceil(S_q / 256) is below the number of SMs (long keys, few queries).
 *
 *   n_split          1 .. 64; 1 is the plain forward (workspace unused, may be NULL).
 *   workspace        DEVICE memory owned by the caller, 256-byte aligned, at least
 *                    vt_attn_splitkv_workspace_size(B, H, S_q, D_v, n_split) bytes, not overlapping
 *                    Q, K, V or O.  Its contents are scratch: overwritten by every call, and two
 *                    calls that share a workspace must not overlap on the GPU.
 * Both element types (the fp32 shares cut 64-key tiles, the bf16 shares 128-key tiles).  Other
 * arguments and errors as for vt_attn_fwd_strided; a too small or NULL workspace is
 * VT_ERR_INVALID_ARG.
 */
vt_status vt_attn_fwd_splitkv(const void *Q, const int64_t q_stride[3],
                              const void *K, const int64_t k_stride[3],
                              const void *V, const int64_t v_stride[3],
                              void *O, const int64_t o_stride[3],
                              int64_t B, int64_t H, int64_t S_q, int64_t S_k,
                              int64_t D_qk, int64_t D_v,
                              float scale, int causal, vt_dtype dtype,
                              int n_split, void *workspace, size_t workspace_bytes,
                              vt_stream_t stream);

/* Bytes of workspace that serve vt_attn_fwd_splitkv (0 when n_split <= 1, an extent is not positive, or the size
 * overflows: no such workspace can exist, and such a call is rejected).  For D_v that is no multiple of 4 it counts
 * partial rows rounded up to 8 floats; a call with D_v below 16 (bf16) or below 4 (fp32) takes packed rows of D_v
 * floats, and with them a smaller workspace.
 * Host-only arithmetic: no GPU call. */
size_t vt_attn_splitkv_workspace_size(int64_t B, int64_t H, int64_t S_q, int64_t D_v, int n_split);

/* The number of shares this library would pick on the current device: the most that still fit
 * one wave of CTAs with at least four key tiles each (128 keys for bf16, 64 for fp32); 1 when
 * splitting does not pay.  Queries the current device's SM count. */
int vt_attn_splitkv_choose(int64_t B, int64_t H, int64_t S_q, int64_t S_k, int causal, vt_dtype dtype);

/*
 * vt_attn_fwd_splitkv without a caller-provided workspace, for callers that cannot allocate
 * device memory: for example a plugin running inside a host framework that owns every byte of
 * device memory and does not let extensions call cudaMalloc, or a latency-critical service that
 * must not allocate after start-up because an allocation can block and synchronise the device.
 * The pages describe no such call; it has no counterpart in them.
 *
 * The shares' partial results live in a fixed 32 MiB array inside this library (a static
 * __device__ array: every GPU that loads the library holds it until the process exits).  The call
 * itself allocates nothing.  Arguments and errors are those of vt_attn_fwd_splitkv without the
 * workspace; in addition, a problem whose partial results need more than 32 MiB (33554432 bytes; see
 * vt_attn_splitkv_workspace_size) is rejected with VT_ERR_UNSUPPORTED before anything runs.  n_split = 1 uses no scratch at all.
 *
 * The first call with n_split > 1 on a device looks up the array's device address
 * (cudaGetSymbolAddress) and remembers it; make that first call before any stream capture.  All
 * calls share the one array, which keeps whatever the last call left there: every call writes all
 * the partial results it reads, so nothing has to start at zero, but calls that overlap on the GPU
 * (concurrent streams, or several host threads) race on the array and must be serialised by the
 * caller.
 */
vt_status vt_attn_fwd_splitkv_noalloc(const void *Q, const int64_t q_stride[3],
                                      const void *K, const int64_t k_stride[3],
                                      const void *V, const int64_t v_stride[3],
                                      void *O, const int64_t o_stride[3],
                                      int64_t B, int64_t H, int64_t S_q, int64_t S_k,
                                      int64_t D_qk, int64_t D_v,
                                      float scale, int causal, vt_dtype dtype,
                                      int n_split, vt_stream_t stream);

/*
 * General form.  Everything above is a special case of vt_attn_fwd_general, which adds:
 *
 * Grouped key/value heads (GQA; H_kv = 1 is multi-query attention).  K is [B,H_kv,S_k,D_qk] and V
 * is [B,H_kv,S_k,D_v]; query head h < H reads key/value head h / (H / H_kv), the num_kv_heads
 * indexing of the VeriTile coverage table's block-sparse attention row.  H must be a multiple of
 * H_kv; k_stride and v_stride are the strides of (b, h_kv, s).
 *
 * A mask choosing the keys A_i of query row i (o = offset >= 0, w = window >= 1):
 *   VT_MASK_NONE               A_i = { j < S_k }
 *   VT_MASK_CAUSAL             A_i = { j < S_k : j <= i + o }; query i sits at key position i + o
 *                              (the start_position of the coverage table's attention_llama causal
 *                              row; o = S_k - S_q aligns the last query with the last key)
 *   VT_MASK_WINDOW             A_i = { j < S_k : i + o - w < j <= i + o }: the w most recent keys
 *                              (the sliding window of the coverage table's attention_fwd_triton3
 *                              row, case 1)
 *   VT_MASK_WINDOW_COMPLEMENT  A_i = { j < S_k : j <= i + o - w }: the causal keys the window leaves
 *                              out (case 2 of the same row)
 * Key tiles outside every row's A_i are skipped, not masked.  A row whose A_i is empty (possible
 * with the window kinds only) is written as 0.
 *
 * An optional log-sum-exp output: lse, if not NULL, is a DEVICE fp32 array [B,H,S_q] (packed,
 * row-major) that receives LSE[b,h,i] = log(sum_{j in A_i} exp(scale * Q_i . K_j)), natural log,
 * -inf for an empty row.  With it, two calls over disjoint key sets (a window and its complement,
 * or two key ranges) combine into the call over their union: O = sum_k e^{LSE_k} O_k / sum_k e^{LSE_k}
 * (the continuation case 4 of the attention_fwd_triton3 row).  Must be 4-byte aligned and must not
 * overlap Q, K, V, O or the workspace.
 *
 * n_split, workspace and workspace_bytes are those of vt_attn_fwd_splitkv;
 * opts those of vt_attn_fwd_ex (may be NULL); mask may be NULL (VT_MASK_NONE).  Errors as for
 * vt_attn_fwd_splitkv, and VT_ERR_INVALID_ARG for H_kv < 1, H not a multiple of H_kv, an unknown mask
 * kind, offset < 0, window < 1 with a window kind, or a misplaced lse; VT_ERR_UNSUPPORTED for
 * offset or window above 2^40.
 */
typedef enum {
    VT_MASK_NONE = 0,
    VT_MASK_CAUSAL = 1,
    VT_MASK_WINDOW = 2,
    VT_MASK_WINDOW_COMPLEMENT = 3
} vt_mask_kind;

typedef struct {
    int32_t kind;     /* vt_mask_kind */
    int32_t reserved; /* 0 */
    int64_t offset;   /* o >= 0 */
    int64_t window;   /* w >= 1 for the window kinds; ignored otherwise */
} vt_attn_mask;

vt_status vt_attn_fwd_general(const void *Q, const int64_t q_stride[3],
                              const void *K, const int64_t k_stride[3],
                              const void *V, const int64_t v_stride[3],
                              void *O, const int64_t o_stride[3], float *lse,
                              int64_t B, int64_t H, int64_t H_kv, int64_t S_q, int64_t S_k,
                              int64_t D_qk, int64_t D_v, float scale, vt_dtype dtype,
                              const vt_attn_mask *mask, int n_split,
                              void *workspace, size_t workspace_bytes,
                              const vt_attn_opts *opts, vt_stream_t stream);

/*
 * Token preparation: the per-head norm of Q and K and their rotation by the token's position, in one
 * pass over the rows, with an optional append of K and V to a cache.  It produces the Q and K that the
 * attention calls of this header read.
 *
 * For every token (b, s) and head h the row x[0..D) of Q or K becomes y[0..D):
 *   n = x                                                        normalize = 0
 *   n_j = w_j x_j / sqrt(mean_j(x_j^2) + eps)                    normalize != 0 (w = 1 when the weight is NULL)
 *   angle_i = positions[pair_axis[i], b, s] * freqs[i],  i < R/2
 *   (y_u, y_v) = (n_u cos(angle_i) - n_v sin(angle_i), n_u sin(angle_i) + n_v cos(angle_i))
 *       with (u, v) = (i, i + R/2)   interleaved = 0
 *            (u, v) = (2i, 2i + 1)   interleaved != 0
 *   y_j = n_j for j >= R.
 * Everything between x and y is fp32 and y is rounded once.  The angle keeps its phase at any position: it is reduced to
 * a fraction of a turn in 64 bits, and that fraction is rounded to 24 (an error of the angle of at most pi 2^-25).  A
 * frequency that is infinite or NaN makes its pairs NaN.  A row of numbers whose squares add up to more than fp32 holds
 * becomes 0; with eps = 0 a row of zeros becomes NaN, and one whose squares are too small for fp32 infinite.  Without the
 * norm, what a column holds reaches its pair alone, and itself alone where it is not rotated.  The weights are not looked
 * at when normalize is 0.  Several position axes (time, height, width of a video patch) need one row of `positions` each;
 * pair_axis names the axis of every frequency pair, in any order.
 *
 * Append (kv_len not NULL): token s of sequence b belongs at cache row kv_len[b] - S + s, kv_len[b] being the
 * sequence's length after these S tokens, so that the same array serves vt_attn_fwd_prefix.  The K row is
 * written there in k_out [B,H_kv,cap,D] and the V row is copied there in v_out [B,H_kv,cap,D_v] (v may be NULL).
 * A token whose row is negative is padding on the left: its K and V are not written (its Q is).  A row at or past
 * `cap` is not written either and records VT_ERR_DEVICE_BOUNDS in the stream's status word.  No other row of the
 * cache is read or written.
 *
 * Arguments, as a struct whose first field is its size.
 *   q, k          [B,H,S,D] and [B,H_kv,S,D]; k may be NULL with H_kv = 0 (one tensor only)
 *   q_out, k_out  as q and k, or (append) k_out the cache.  An output may be the same tensor as its input (same
 *                 pointer and strides); it must not overlap any input or output in another way.  Heads beside each other
 *                 in one tensor (Q, K and V of one projection) do not overlap.
 *   weights       [D] in the tensors' dtype, or NULL
 *   freqs         fp32 [R/2]; R even, 2 <= R <= D
 *   positions     int32, element strides pos_stride over (axis, b, s), 0 allowed (one row for the whole batch)
 * Strides, dtypes, alignment and their errors are those of vt_attn_fwd_strided (16-byte rule; the stride of an
 * index with one value is not looked at, and an append's K and V outputs count `cap` rows); D <= 256 and
 * D_v <= 256, at most 4 axes, B * S at most 2^30.  eps must be finite and not negative.  B or S equal to 0 is a valid empty
 * problem.
 */
#define VT_ROPE_MAX_AXES 4
#define VT_ROPE_MAX_PAIRS 128
typedef struct {
    uint64_t struct_bytes; /* sizeof(vt_qk_rope_args) */
    const void *q, *k;
    const void *q_weight, *k_weight;
    const float *freqs;
    const int32_t *positions;
    void *q_out, *k_out;
    const int32_t *kv_len; /* [B]; NULL: no append, and v, v_out, cap and D_v are ignored */
    const void *v;
    void *v_out;
    int64_t B, H, H_kv, S, D, R;
    int64_t cap, D_v;
    int32_t dtype; /* vt_dtype */
    int32_t interleaved;
    int32_t normalize;
    int32_t axes;
    float eps;
    int32_t reserved; /* 0 */
    int64_t q_stride[3], k_stride[3];
    int64_t q_out_stride[3], k_out_stride[3];
    int64_t v_stride[3], v_out_stride[3];
    int64_t pos_stride[3];
    uint8_t pair_axis[VT_ROPE_MAX_PAIRS]; /* pair_axis[i] < axes for i < R/2 */
} vt_qk_rope_args;

vt_status vt_qk_rope_fwd(const vt_qk_rope_args *args, vt_stream_t stream);

/*
 * Gradients of vt_qk_rope_fwd (without the append).  With g the gradient of an output row, u its rotation by
 * the opposite angles, r = 1 / sqrt(mean(x^2) + eps) and z = r x:
 *   dw_j = sum over tokens and heads of u_j z_j,   dx = r (w u - z mean_j(w_j u_j z_j)),
 * and dx = u when normalize is 0.  The products w u x of a row are summed in fp32, like its squares.  In `args`: q, k
 * are the forward's inputs (not read, and may be NULL, when normalize is 0); q_out, k_out are dq and dk, written;
 * kv_len must be NULL.  dq_out, dk_out are the gradients of the forward's outputs, with their strides; dq may be dq_out,
 * or q (same pointer and strides), and dk the same way.  dq_weight, dk_weight: fp32 [D], written (each may be NULL),
 * summed in fp32, in an order that does not change from call to call.  The workspace (256-byte aligned, at least
 * vt_qk_rope_bwd_workspace_size bytes) holds partial sums of the weight gradients; it is not used, and may be NULL, when
 * normalize is 0 or both are NULL.
 */
vt_status vt_qk_rope_bwd(const vt_qk_rope_args *args, const void *dq_out, const int64_t dq_out_stride[3],
                         const void *dk_out, const int64_t dk_out_stride[3], float *dq_weight, float *dk_weight,
                         void *workspace, size_t workspace_bytes, vt_stream_t stream);

/* Bytes of workspace vt_qk_rope_bwd needs for the weight gradients of rows of D elements (0 when D is outside
 * 1..256).  Host-only arithmetic. */
size_t vt_qk_rope_bwd_workspace_size(int64_t D);

/*
 * Attention of a batch of sequences behind a prefix that all of them share, each with its own cache: decoding
 * (S_q = 1), checking a few drafted tokens, or a chunk of a prompt.  K and V of the prefix are stored and read
 * once for the batch, not once per sequence.
 *
 * Query (b, h, s) attends to every prefix row j < S_p of K_p[h_kv], V_p[h_kv] and to the rows
 *   j <= kv_len[b] - S_q + s,  j >= 0
 * of its own cache K_c[b, h_kv], V_c[b, h_kv], h_kv = h / (H / H_kv): the S_q queries are the last S_q tokens of
 * the sequence's kv_len[b] cached ones (vt_qk_rope_fwd appends them), each seeing the tokens up to itself.
 *   O = softmax(scale q . k) v over the union,  LSE = log(sum exp(scale q . k)) (natural log).
 * A query with kv_len[b] - S_q + s < 0 sees the prefix alone; with no prefix either, O = 0 and LSE = -inf.
 *
 * Arguments, as a struct whose first field is its size.
 *   q, o                 [B,H,S_q,D_qk] and [B,H,S_q,D_v]
 *   k_prefix, v_prefix   [H_kv,S_p,D_qk] and [H_kv,S_p,D_v], strides (h_kv, s); not read when S_p = 0
 *   k_cache, v_cache     [B,H_kv,S_c,D_qk] and [B,H_kv,S_c,D_v]; not read when S_c = 0.  What the rows at
 *                        or past kv_len[b] hold has no influence.
 *   kv_len               int32 [B], 0 <= kv_len[b] <= S_c, read on the device (a captured call replays with new
 *                        lengths); NULL: S_c for every sequence.  A length outside that range counts as the nearest
 *                        one inside and records VT_ERR_DEVICE_BOUNDS in the stream's status word; not read when
 *                        S_c = 0.
 *   lse                  fp32 [B,H,S_q] or NULL
 *   workspace            DEVICE scratch, 256-byte aligned, at least vt_attn_prefix_workspace_size bytes (may be
 *                        NULL when that is 0).  Every call writes what it reads there; two calls that share it must
 *                        not overlap on the GPU, replays of captured ones included.
 * Element types: VT_BF16, with probabilities rounded to bf16 as in the other calls, and VT_F32 with products of two TF32
 * parts per operand (about 2^-21 of every factor is lost, against 2^-11 in the other fp32 calls).  Sums and statistics are
 * fp32.  An infinite value fills its column of O with that infinity for every query that gives it a weight fp32 holds, and
 * a key whose score is -inf has no weight.  A key that a query may not see but that another query of the same sequence does must be finite, as in the other
 * calls.
 * Strides, alignment and errors as for vt_attn_fwd_strided (the stride of an index with one value is not looked at);
 * VT_ERR_INVALID_ARG also for H not a multiple of H_kv or a workspace that is too small, VT_ERR_UNSUPPORTED also for
 * S_p + S_c or B * H * S_q above 2^30.  B, H or S_q equal to 0 is a valid empty problem.
 */
typedef struct {
    uint64_t struct_bytes; /* sizeof(vt_attn_prefix_args) */
    const void *q;
    const void *k_prefix, *v_prefix;
    const void *k_cache, *v_cache;
    const int32_t *kv_len;
    void *o;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
    int64_t B, H, H_kv, S_q, S_p, S_c, D_qk, D_v;
    int32_t dtype; /* vt_dtype */
    float scale;
    int64_t q_stride[3];
    int64_t kp_stride[2], vp_stride[2];
    int64_t kc_stride[3], vc_stride[3];
    int64_t o_stride[3];
} vt_attn_prefix_args;

vt_status vt_attn_fwd_prefix(const vt_attn_prefix_args *args, vt_stream_t stream);

/* Bytes of workspace vt_attn_fwd_prefix needs on the current device (0: none, or the call would be refused). */
size_t vt_attn_prefix_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t S_q, int64_t S_p, int64_t S_c,
                                     int64_t D_qk, int64_t D_v, vt_dtype dtype);

/*
 * vt_attn_fwd_prefix for trees of drafted tokens: the S_q <= 64 new tokens of a sequence are the nodes of a tree, or of
 * several, that are checked in one call.  Node s lies in cache row kv_len[b] - S_q + s, as vt_qk_rope_fwd appends it (its
 * position is the caller's: that of its depth), and parents[b * S_q + s] is the node that it continues, an earlier one, or
 * -1 where it continues the tokens before the tree.  Its queries attend to the prefix, to the cache's rows before the tree
 * (those below kv_len[b] - S_q), to the node's ancestors and to the node itself, and to no other node.  With parents s - 1
 * the call is vt_attn_fwd_prefix.
 * `parents` is int32 [B,S_q], packed, on the device, read there (a captured call replays with new trees).  A parent that is
 * neither -1 nor an earlier node counts as -1 and records VT_ERR_DEVICE_BOUNDS in the stream's status word.  A node whose
 * row is negative (a sequence shorter than the tree) has no key: its queries see the prefix alone.
 * Without a cache (S_c equal to 0) every node's queries see the prefix alone; kv_len is not read, parents are.
 * The workspace has vt_attn_tree_workspace_size bytes; other arguments and errors as for vt_attn_fwd_prefix,
 * VT_ERR_INVALID_ARG also for parents NULL,
 * VT_ERR_UNSUPPORTED also for S_q above 64.
 */
vt_status vt_attn_fwd_tree(const vt_attn_prefix_args *args, const int32_t *parents, vt_stream_t stream);

/* Bytes of workspace vt_attn_fwd_tree needs on the current device (0: none, or the call would be refused). */
size_t vt_attn_tree_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t S_q, int64_t S_p, int64_t S_c,
                                   int64_t D_qk, int64_t D_v, vt_dtype dtype);

/*
 * Attention over packed sequences: N sequences of different lengths whose rows lie behind each other in one tensor, as a
 * batch of prompts or of training texts is laid out without padding.
 *
 * Sequence n has the queries cu_q[n] <= t < cu_q[n + 1] and the keys cu_k[n] <= t < cu_k[n + 1]; queries see keys of their
 * own sequence only.  Its queries are the last of its keys' positions: query i of len_q sits at position
 * i + len_k - len_q, and with o = len_k - len_q the mask kinds keep the keys that vt_attn_fwd_general's keep at offset o
 * (here o may be negative: the first queries then see no key of a causal mask).
 *   O = softmax(scale q . k) v over the keys a query sees,  LSE = log(sum exp(scale q . k)) (natural log);
 * a query that sees no key has O = 0 and LSE = -inf.  Query head h reads key/value head h / (H / H_kv).
 *
 * Arguments, as a struct whose first field is its size.
 *   q, o        [H,T_q,D_qk] and [H,T_q,D_v], strides (h, t); T_q >= cu_q[N].  Rows of O and of LSE that belong to no
 *               sequence are not written.
 *   k, v        [H_kv,T_k,D_qk] and [H_kv,T_k,D_v], strides (h, t); T_k >= cu_k[N].  What rows of other sequences, or of
 *               none, hold has no influence.
 *   cu_q, cu_k  int32 [N + 1], not decreasing, read on the device (a captured call replays with new lengths); they may
 *               be one array.  First rows outside [0, T] count as the nearest ones inside and record VT_ERR_DEVICE_BOUNDS in
 *               the stream's status word.  So does an array that decreases anywhere: every access stays inside the tensors
 *               then and rows of no sequence are left as they were, but the sequences' results are not specified.
 *   lse         fp32 [H,T_q] packed, or NULL
 *   mask        a vt_mask_kind, with its `window`
 * Element types: VT_BF16, with probabilities rounded to bf16 as in the other calls, and VT_F32 with products of two TF32
 * parts per operand (about 2^-21 of every factor is lost).  Sums and statistics are fp32.  A key that a query may not see
 * but that another query of the same sequence does must be finite, as in the other calls.
 * Strides, alignment and errors as for vt_attn_fwd_strided (the stride of an index with one value is not looked at);
 * VT_ERR_INVALID_ARG also for H not a multiple of H_kv, an unknown mask or a window below 1 with a window kind,
 * VT_ERR_UNSUPPORTED also for a window above 2^40, N, T_q or T_k above 2^30, or 4 (T / 32 + N) H above 2^31 - 1.  N, H or T_q
 * equal to 0 is a valid empty problem.
 */
typedef struct {
    uint64_t struct_bytes; /* sizeof(vt_attn_packed_args) */
    const void *q, *k, *v;
    const int32_t *cu_q, *cu_k;
    void *o;
    float *lse;
    int64_t N, H, H_kv, T_q, T_k, D_qk, D_v;
    int64_t window;
    int32_t dtype; /* vt_dtype */
    float scale;
    int32_t mask;     /* vt_mask_kind */
    int32_t reserved; /* 0 */
    int64_t q_stride[2], k_stride[2], v_stride[2], o_stride[2];
} vt_attn_packed_args;

vt_status vt_attn_fwd_packed(const vt_attn_packed_args *args, vt_stream_t stream);

/*
 * Gradients of vt_attn_fwd_packed.  `args` are the forward's, with its results: o and lse are read (both are required).
 * With P = exp(scale q . k - LSE) over the pairs the mask keeps, g = d_o and delta = sum_e g_e o_e - d_lse of every query,
 *   dv = sum P g,   dS = P (g . v - delta),   dq = scale sum dS k,   dk = scale sum dS q;
 * sums for a key run over the queries of all the heads that share it.  A query or key without a partner has a gradient
 * of 0; rows that belong to no sequence are not written.  A query without a key adds nothing to any gradient, whatever its
 * d_lse; d_o is finite in every row of a sequence, as q, k and v are.
 *   d_o          [H,T_q,D_v]: the gradient of O
 *   d_lse        fp32 [H,T_q] packed: the gradient of LSE, or NULL (0)
 *   dq, dk, dv   as q, k and v.  They may lie beside each other in one tensor (the gradient of one projection); they must
 *                not overlap the inputs.
 *   workspace    DEVICE scratch, 256-byte aligned, at least vt_attn_bwd_packed_workspace_size bytes.  Every call writes
 *                what it reads there; two calls that share it must not overlap on the GPU, replays of captured ones
 *                included.
 * Every sum is fp32 in an order that does not change from call to call; VT_BF16 rounds P and dS to bf16 before they are
 * multiplied.  N or H equal to 0, or no row at all, is a valid empty problem; with T_q equal to 0, dk and dv are written
 * as 0.
 */
typedef struct {
    uint64_t struct_bytes; /* sizeof(vt_attn_packed_grads) */
    const void *d_o;
    const float *d_lse;
    void *dq, *dk, *dv;
    void *workspace;
    size_t workspace_bytes;
    int64_t do_stride[2], dq_stride[2], dk_stride[2], dv_stride[2];
} vt_attn_packed_grads;

vt_status vt_attn_bwd_packed(const vt_attn_packed_args *args, const vt_attn_packed_grads *grads, vt_stream_t stream);

/* Bytes of workspace vt_attn_bwd_packed needs on the current device (0: none, or the call would be refused). */
size_t vt_attn_bwd_packed_workspace_size(int64_t N, int64_t H, int64_t H_kv, int64_t T_q, int64_t T_k, int64_t D_qk,
                                         int64_t D_v, vt_dtype dtype);

/* A static, human-readable name for a status code (never NULL). */
const char *vt_status_str(vt_status status);

/*
 * Synchronise `stream`, then return and clear the device status word that the kernels launched on
 * `stream` (on the current device) write: VT_OK, VT_ERR_DEVICE_TIMEOUT or VT_ERR_DEVICE_BOUNDS;
 * VT_ERR_CUDA if the synchronisation itself reports an error.  Other streams' words are neither read
 * nor cleared, and no other stream is waited for.
 *
 * Words are kept per stream handle: the first 255 distinct handles a process passes to this library get
 * a word each, in order of first use, and any later handle shares one common word (a destroyed stream's
 * handle keeps its word, which a new stream that receives the same handle inherits).  The per-thread
 * default stream is one handle for all threads.  A launch captured into a CUDA graph writes the word of
 * the stream it was captured on, whichever stream the graph is later launched into.
 */
vt_status vt_last_device_status(vt_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* VT_ATTN_H */
