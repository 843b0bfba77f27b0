/*
 * ep.h -- MoE expert-parallel token routing on one AMD Instinct MI355X
 * (gfx950): prepare, dispatch, combine and their two backward ops, plus a
 * fused weighted combine and its backward, and the experts' own work between
 * dispatch and combine: products grouped by expert, with their gradients and
 * with 4-bit weights, and the gated activation with its gradient; the same in 8
 * bits with scales, from the norm in front of the layer on; and a whole layer
 * for a few tokens.
 *
 * The five per-step calls follow the per-step part of the common C API in
 * "Expert Parallelism: common C API + NCCL EP backend" (section "Per-step
 * (allocation-free, CUDA-graph capturable)"), at one GPU's share of the work:
 * prepare builds the routing maps of a handle, dispatch moves token rows and
 * their routing weights into an expert-major receive buffer, combine sums the
 * expert outputs of each token back into a token row without weighting them
 * (the caller has already multiplied by the received weights), and
 * dispatch_bwd / combine_bwd are the adjoints of dispatch / combine.
 *
 * Conventions shared by every call
 *  - Routes are numbered s = t*K + k over the [T,K] routing table.
 *  - A route is valid iff 0 <= topk_idx[s] < E. The id -1 marks a masked
 *    route (one whose expert lives elsewhere; see the masking of
 *    "Expert-parallel implementations for ep_dispatch_experts", table
 *    "Implementations"). Any other id is an error: the device raises
 *    EP_STATUS_BAD_EXPERT and the route is then treated as masked.
 *  - Expert e owns the received rows [offsets[e], offsets[e+1]). Its valid
 *    routes fill the first counts[e] rows in ascending s; the segment is then
 *    padded up to a multiple of the alignment A. The pad rows of every
 *    expert-major output are written as zeros, unless the layout sets
 *    EP_LAYOUT_NO_PAD_FILL: then they are not written at all. An expert with
 *    no route has an empty segment. total = offsets[E].
 *  - Payload rows hold the layout's payload type: bf16 (the default, and the
 *    only type of the PyTorch wrapper in "[PyTorch] Expert Parallelism:
 *    PyTorch wrapper + autograd ops with symm-mem zero-copy", section
 *    "Public Python API"), fp16 or fp32 (the types the C++ tests of "Expert
 *    Parallelism: common C API + NCCL EP backend" cover, per its section
 *    "Important Files Changed"). They are passed as raw bit patterns through
 *    void pointers. Routing ids are int64, routing weights fp32. Rows are
 *    contiguous, H elements each, row-major.
 *  - Sums are taken in fp32 and rounded once to the payload type: round to
 *    nearest, ties to even, subnormals kept, overflow to infinity, and any
 *    NaN becomes the canonical quiet NaN (bf16 0x7FC0, fp16 0x7E00, fp32
 *    0x7FC00000). For fp32 payloads the only change is that NaN rule.
 *  - All pointers are device pointers unless stated otherwise. Payload
 *    pointers must be 16-byte aligned and H must be a multiple of 8. A
 *    pointer to a buffer with no element (T == 0 for [T,...] buffers,
 *    recv_capacity == 0 for [recv_capacity,...] buffers) may be NULL; every
 *    other required pointer must not be, whatever the other sizes are.
 *  - Work is enqueued on `stream` and nothing waits for it: no call below
 *    synchronises, allocates, frees or keeps a pointer after it returns,
 *    except ep_read_status, which waits for the stream. The caller owns
 *    every buffer. Outputs must not overlap inputs or each other, but where
 *    a call says that they may.
 *  - Host-detectable errors return an ep_status_t before any HIP call is
 *    made; nothing is enqueued then. Data-dependent errors raise sticky bits
 *    in the handle's status word (see ep_read_status).
 *  - Calls on one handle must be ordered on the GPU (same stream, or events)
 *    with prepare first. Several handles may be in flight at once.
 */
#ifndef EP_MI355X_EP_H
#define EP_MI355X_EP_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ep_status {
  EP_OK = 0,
  EP_ERR_NULL = 1,        /* a required pointer is NULL */
  EP_ERR_SHAPE = 2,       /* a size is out of range (see ep_layout_t) */
  EP_ERR_ALIGN = 3,       /* a payload pointer is not 16-byte aligned */
  EP_ERR_HANDLE_SIZE = 4, /* handle_bytes < ep_handle_mem_size(layout) */
  EP_ERR_CAPACITY = 5,    /* recv_capacity < 0 or >= 2^31 */
  EP_ERR_DEVICE = 6,      /* the current device is not gfx950 */
  EP_ERR_HIP = 7,         /* a HIP runtime call or kernel launch failed */
  EP_ERR_SCRATCH = 8,     /* ep_prepare_static: the layout's prepare scratch
                             exceeds EP_PREPARE_STATIC_SCRATCH_BYTES */
  EP_ERR_WORKSPACE = 9    /* workspace_bytes is below what the call's query
                             (ep_rms_norm_bwd_workspace,
                             ep_expert_layer_workspace) returns */
} ep_status_t;

/* Sticky device-side bits of a handle's status word. */
enum {
  EP_STATUS_BAD_EXPERT = 1u, /* prepare saw an id outside [0,E) other than -1 */
  EP_STATUS_OVERFLOW = 2u,   /* prepare: total > recv_capacity; routes whose row
                                would lie at or past the capacity were dropped */
  EP_STATUS_LAYOUT = 4u      /* a payload op was given a layout other than the
                                one the handle was prepared with, or a handle
                                that was never prepared; the op wrote nothing */
};

/* Payload element types (ep_layout_t.dtype). */
enum {
  EP_DTYPE_BF16 = 0,
  EP_DTYPE_FP16 = 1,
  EP_DTYPE_FP32 = 2
};

/* Layout flags (ep_layout_t.flags). EP_LAYOUT_NO_PAD_FILL: the payload ops
 * leave pad rows unwritten instead of zeroing them (dispatch's rows and
 * weights, combine_bwd's rows, the weighted backward's rows and weight
 * gradients), saving their writes when the consumer never reads pad rows
 * (combine and dispatch_bwd never do). The pages zero the pads of
 * combine_bwd's output only, and the review of "[PyTorch] Expert
 * Parallelism: PyTorch wrapper + autograd ops with symm-mem zero-copy"
 * weighs what the padded expert-major buffer costs (its buffer-sizing
 * thread); this flag makes the pad writes a choice. It does not change the
 * routing maps: one prepared handle serves both policies. */
enum {
  EP_LAYOUT_NO_PAD_FILL = 1u,
  EP_LAYOUT_ZERO_TAIL = 4u
};

/* EP_LAYOUT_ZERO_TAIL: the payload ops that write expert-major rows
 * (ep_dispatch's rows and weights, ep_combine_bwd's rows, and the weighted
 * backward's rows and weight gradients) also write +0 to every row at or past
 * min(total, recv_capacity), so that the whole [recv_capacity,...] buffer is
 * defined. This is the library's own addition: combine never reads those
 * rows, so their gradient is zero, and a caller that applies one function to
 * the whole receive buffer (a parameter shared by every row, a reduction
 * over it) then sees zeros there instead of stale memory. It costs one
 * zero write per tail row. */

/*
 * Per-layer sizes (the role of the layer configuration in the common C API,
 * passed by pointer as plain data). A zero-initialised dtype/flags pair
 * means bf16 payloads with zero-filled pads.
 *   num_tokens    T >= 0
 *   topk          K in [1, 64]
 *   num_experts   E in [1, 2048], local experts
 *   alignment     A >= 1 rows (the per-expert dispatch output alignment)
 *   dtype         EP_DTYPE_* of every payload row
 *   flags         EP_LAYOUT_* bits; other bits must be 0
 *   hidden        H >= 8, a multiple of 8 (elements per row)
 *   recv_capacity rows of every expert-major buffer, 0 <= cap < 2^31
 * T*K + E*(A-1) must be below 2^31 (every offset fits an int32). The handle
 * depends on num_tokens, topk, num_experts, alignment and recv_capacity
 * only; dtype, flags and hidden may differ between the ops that use it.
 */
typedef struct ep_layout {
  int64_t num_tokens;
  int32_t topk;
  int32_t num_experts;
  int32_t alignment;
  uint16_t dtype;
  uint16_t flags;
  int64_t hidden;
  int64_t recv_capacity;
} ep_layout_t;

/* Rows that can never overflow: every token sends min(K,E) distinct routes
 * and every expert adds at most A-1 pad rows: T*min(K,E) + E*(A-1). With
 * repeated ids in a token's top-k the bound is T*K + E*(A-1). Returns -1 for
 * out-of-range arguments. Host only. The library's own helper: the review of
 * "[PyTorch] Expert Parallelism: PyTorch wrapper + autograd ops with symm-mem
 * zero-copy" sizes the padded expert-major buffer for its worst case (the
 * thread on buffer sizing and recv_capacity_per_rank); this is that bound for
 * one GPU. */
int64_t ep_recv_capacity_worst(int64_t num_tokens, int32_t topk, int32_t num_experts,
                               int32_t alignment);

/* Bytes of device memory the caller must provide as `handle_mem` for this
 * layout. Returns 0 for an invalid layout. Host only. The handle-size query
 * of "Expert Parallelism: common C API + NCCL EP backend" (section "Public C
 * API", its "Lifecycle" list: layer registration reports the handle_mem size
 * the caller allocates); here it is a pure function of the layout, with no
 * registration step. */
size_t ep_handle_mem_size(const ep_layout_t* layout);

/* Byte offsets, inside handle_mem, of the routing maps that prepare writes,
 * so that callers can read them. The library's own addition: the handle of
 * the common C API is opaque caller memory. All int32 unless stated:
 *   status   uint32 status word (EP_STATUS_* bits)
 *   counts   [E]     valid routes per expert
 *   offsets  [E+1]   segment starts, offsets[E] = total
 *   slot     [T*K]   received row of route s, -1 if masked or dropped
 *   row_src  [recv_capacity]  route held by received row r, -1 for a pad row;
 *            entries at or past min(total, recv_capacity) are unspecified
 *   bytes    == ep_handle_mem_size(layout)
 *   maps_bytes  the size of the routing maps alone (<= bytes): the handle
 *            region every payload op reads. A handle of maps_bytes serves the
 *            payload ops; ep_prepare needs all `bytes` (its scratch closes the
 *            handle).
 *   runs     8 lists of run_list_entries (row, route) int32 pairs: the run
 *            entries that dispatch and combine_bwd copy by. The routes are
 *            cut into chunks of run_units * 512 consecutive routes; chunk c
 *            belongs to list c mod 8, and a list holds its chunks one after
 *            another, each as its routes that hold a row in ascending row
 *            order, then (-1, -1) for each of its valid routes dropped past
 *            the capacity.
 *   stream_live  int32 [8]: the number of entries in each list
 *   run_units    int32: units of 512 routes per chunk (1, 2 or 4), chosen
 *            by prepare from its layout's payload row size
 *   run_list_entries  (a count, not an offset) the entries each list can
 *            hold, 64 * ceil(T*K/512) + 2048
 * Every offset is a multiple of 256. Host only. */
typedef struct ep_handle_regions {
  size_t status;
  size_t counts;
  size_t offsets;
  size_t slot;
  size_t row_src;
  size_t bytes;
  size_t runs;
  size_t maps_bytes;
  size_t stream_live;
  size_t run_units;
  size_t run_list_entries;
} ep_handle_regions_t;

ep_status_t ep_handle_regions(const ep_layout_t* layout, ep_handle_regions_t* out);

/*
 * prepare: from the int64 routing table, write the per-expert token counts,
 * the aligned segment offsets and the slot map into the handle. The
 * per-step prepare of "Expert Parallelism: common C API + NCCL EP backend"
 * (section "Per-step (allocation-free, CUDA-graph capturable)"), with the
 * alignment taken from the layout.
 *   topk_idx        int64 [T,K]                  input
 *   token_counts    int32 [E]                    output: valid routes per expert
 *                                                (not padded)
 *   expert_offsets  int32 [E+1] or NULL          output: segment starts,
 *                                                expert_offsets[E] = total
 *   handle_mem      handle_bytes of device memory, fully (re)written here
 * After this call the handle holds, for the later ops, the received row of
 * every route (-1 if masked or dropped), the source route of every live
 * received row (-1 for pads) and the run entries (see ep_handle_regions),
 * whatever the layout's flags. Its status word is reset, then raises
 * BAD_EXPERT / OVERFLOW as described above.
 */
ep_status_t ep_prepare(const ep_layout_t* layout, const int64_t* topk_idx,
                       int32_t* token_counts, int32_t* expert_offsets, void* handle_mem,
                       size_t handle_bytes, hipStream_t stream);

/*
 * ep_prepare_static: ep_prepare for callers that cannot allocate (code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation)
 * and so cannot give the handle room for prepare's scratch. The same work and
 * the same routing maps, bit for bit, but the scratch (the expert
 * histograms and bad-id flags of the prepare kernels) lives in a static
 * device array of the library, EP_PREPARE_STATIC_SCRATCH_BYTES per device,
 * held until the process ends; so handle_mem needs only the routing maps,
 * `maps_bytes` of ep_handle_regions (ep_handle_mem_size also suffices).
 * Allocates nothing: the array's device address is looked up on the first
 * call on each device. Every call on one device shares that device's array,
 * so calls of ep_prepare_static that overlap on one device (several streams,
 * no ordering between them) race and must not be made; ep_prepare and the
 * payload ops do not touch the array. A layout whose scratch exceeds the
 * array returns EP_ERR_SCRATCH before any HIP call. With U = ceil(T*K/512)
 * units of routes the scratch is 4*E*(U + B + 1) bytes of histograms (one
 * row per unit, one per block of units, B = ceil(U/4) blocks of 4 units up
 * to 256 units and ceil(U/8) blocks of 8 past that, one row of totals) plus
 * 8*U bytes of per-unit words, each part rounded up to 256 bytes: at
 * E = 256, 3614 units (about 1.85 M routes) fit.
 */
#define EP_PREPARE_STATIC_SCRATCH_BYTES (4u << 20)

ep_status_t ep_prepare_static(const ep_layout_t* layout, const int64_t* topk_idx,
                              int32_t* token_counts, int32_t* expert_offsets, void* handle_mem,
                              size_t handle_bytes, hipStream_t stream);

/*
 * dispatch (the per-step dispatch of the same section):
 * recv_tokens[r,:] = tokens[s/K,:] and recv_topk_weights[r] =
 * topk_weights[s] for every live row r holding route s (bit copies); pad
 * rows get +0 in both (not written with EP_LAYOUT_NO_PAD_FILL). Rows at or
 * past min(total, recv_capacity) are not written (+0 with
 * EP_LAYOUT_ZERO_TAIL).
 *   tokens             payload [T,H]
 *   topk_weights       fp32 [T,K] or NULL
 *   recv_tokens        payload [recv_capacity,H]
 *   recv_topk_weights  fp32 [recv_capacity]; must be NULL iff topk_weights is
 *                      (when T > 0 and recv_capacity > 0)
 */
ep_status_t ep_dispatch(const ep_layout_t* layout, const void* handle_mem,
                        size_t handle_bytes, const void* tokens,
                        const float* topk_weights, void* recv_tokens,
                        float* recv_topk_weights, hipStream_t stream);

/*
 * combine (the per-step combine of the same section, unweighted there too):
 * result[t,:] = the sum over the valid routes of t, k ascending, of
 * expert_out[slot(t,k),:], accumulated in fp32 starting from the first valid
 * row and rounded once to the payload type (see the rounding convention
 * above). A token with no valid route gets +0. Unweighted.
 *   expert_out  payload [recv_capacity,H] (only the rows of valid routes are
 *               read)
 *   result      payload [T,H]
 */
ep_status_t ep_combine(const ep_layout_t* layout, const void* handle_mem,
                       size_t handle_bytes, const void* expert_out, void* result,
                       hipStream_t stream);

/*
 * dispatch_bwd (the per-step dispatch backward of the same section; the
 * adjoint of dispatch): grad_tokens = combine(grad) with the
 * same fp32 ascending-k rule; grad_topk_weights[s] = g_recv_topk_weights[r]
 * for the row r of a valid route s, else +0. A NULL g_recv_topk_weights
 * (no gradient flowed into the received weights) gives +0 everywhere; a NULL
 * grad_topk_weights skips the weight gradient.
 *   grad                 payload [recv_capacity,H]
 *   g_recv_topk_weights  fp32 [recv_capacity] or NULL
 *   grad_tokens          payload [T,H]
 *   grad_topk_weights    fp32 [T,K] or NULL
 */
ep_status_t ep_dispatch_bwd(const ep_layout_t* layout, const void* handle_mem,
                            size_t handle_bytes, const void* grad,
                            const float* g_recv_topk_weights, void* grad_tokens,
                            float* grad_topk_weights, hipStream_t stream);

/*
 * combine_bwd (the per-step combine backward of the same section; the
 * adjoint of combine): grad_expert_out[r,:] = grad[s/K,:] for
 * every live row r holding route s; pad rows are zeroed (not written with
 * EP_LAYOUT_NO_PAD_FILL). Rows at or past min(total, recv_capacity) are not
 * written (+0 with EP_LAYOUT_ZERO_TAIL).
 *   grad             payload [T,H]
 *   grad_expert_out  payload [recv_capacity,H]
 */
ep_status_t ep_combine_bwd(const ep_layout_t* layout, const void* handle_mem,
                           size_t handle_bytes, const void* grad, void* grad_expert_out,
                           hipStream_t stream);

/*
 * Weighted combine: the weight multiply folded into combine, which the review
 * of "[PyTorch] Expert Parallelism: PyTorch wrapper + autograd ops with
 * symm-mem zero-copy" (thread on the weight multiply) settles on as an
 * option, so that the caller's separate pre-multiply pass disappears. For
 * each token, over its valid routes in ascending k with received row r: the
 * first term is the fp32 product w[r] * y[r], each later term is a fused
 * multiply-add fma(w[r], y[r], acc); the fp32 sum is rounded once to the
 * payload type; a token with no valid route gets +0.
 *   expert_out         payload [recv_capacity,H] (y; only the rows of valid
 *                      routes are read)
 *   recv_topk_weights  fp32 [recv_capacity]   (w, e.g. dispatch's output)
 *   result             payload [T,H]
 */
ep_status_t ep_combine_weighted(const ep_layout_t* layout, const void* handle_mem,
                                size_t handle_bytes, const void* expert_out,
                                const float* recv_topk_weights, void* result,
                                hipStream_t stream);

/*
 * Backward of the weighted combine. For every live received row r holding
 * route s of token t = s/K:
 *   grad_expert_out[r,:]      = payload(fp32(w[r] * grad[t,:]))  (one fp32
 *                               product, then the payload rounding)
 *   grad_recv_topk_weights[r] = sum over h of grad[t,h] * expert_out[r,h]
 * Pad rows get +0 in both (not written with EP_LAYOUT_NO_PAD_FILL). The
 * weight gradient is an fp32 dot product over H accumulated in a fixed order,
 * bit-identical from run to run but not the sequential order: the row is cut
 * into P = ceil(H * elem / 1024) pieces of 64 16-byte vectors (N elements
 * each: 8 for bf16 and fp16, 4 for fp32); each lane chains N fused
 * multiply-adds over its vector, six butterfly adds combine a piece's lanes,
 * and the P partials are added in piece order. So every product passes
 * through at most n = N + P + 5 fp32 roundings and the result is within
 * gamma_n * sum_h |grad[t,h] * expert_out[r,h]| of the exact dot product,
 * gamma_n = n u / (1 - n u), u = 2^-24. (Rows of more than 1024 pieces, or
 * sizes whose piece indices pass 2^31, take a token-group form whose lanes
 * chain N * P multiply-adds: n = N * P + 6 there.) With
 * grad_recv_topk_weights NULL only the row gradient is computed and
 * expert_out may be NULL. Rows at or past min(total, recv_capacity) are not
 * written (+0, and +0 weight gradients, with EP_LAYOUT_ZERO_TAIL).
 *   grad                    payload [T,H]
 *   expert_out              payload [recv_capacity,H] or NULL
 *   recv_topk_weights       fp32 [recv_capacity]
 *   grad_expert_out         payload [recv_capacity,H]
 *   grad_recv_topk_weights  fp32 [recv_capacity] or NULL
 */
ep_status_t ep_combine_weighted_bwd(const ep_layout_t* layout, const void* handle_mem,
                                    size_t handle_bytes, const void* grad,
                                    const void* expert_out, const float* recv_topk_weights,
                                    void* grad_expert_out, float* grad_recv_topk_weights,
                                    hipStream_t stream);

/*
 * The experts' products and activation: what runs between dispatch and
 * combine, on the segments of a prepared handle. All five are the library's
 * own addition. They follow the conventions above: only the live rows of a
 * segment (its valid routes' rows below recv_capacity) are operands, so the
 * contents of pad rows and of the rows past the live total never matter,
 * whatever they hold; in an expert-major output the pad rows are zeroed (not
 * written with EP_LAYOUT_NO_PAD_FILL) and the rows at or past
 * min(total, recv_capacity) are not written (+0 with EP_LAYOUT_ZERO_TAIL).
 * The layout's hidden is the row length named at each call; feature counts
 * (H and N below) are multiples of 8 up to EP_MAX_FEATURES, else
 * EP_ERR_SHAPE. Sums are held in fp32 and rounded once to the payload type,
 * in an order that is fixed for given sizes and routing (results are
 * bit-identical from run to run) and otherwise unspecified. An infinity or
 * NaN in an operand reaches exactly the outputs whose sums contain it.
 * A product's kernel is chosen on the host for min(num_tokens * topk,
 * recv_capacity) / num_experts rows an expert: where most routes are masked (a
 * rank that holds a few of the experts), a capacity near the rows that can
 * come serves few rows best, and one for every route costs up to a tenth.
 */
#define EP_MAX_FEATURES (1 << 20)

/*
 * Grouped linear: out[r,:] = weight[e] x[r,:] for every live row r of every
 * expert e, one weight matrix per expert.
 *   x             payload [recv_capacity,H], H = layout->hidden
 *   weight        payload [E,N,H]
 *   out           payload [recv_capacity,N]
 *   out_features  N
 */
ep_status_t ep_grouped_linear(const ep_layout_t* layout, const void* handle_mem,
                              size_t handle_bytes, const void* x, const void* weight, void* out,
                              int64_t out_features, hipStream_t stream);

/*
 * Backward of the grouped linear, with H = layout->hidden (x's row length)
 * and N = out_features (grad's):
 *   grad_x[r,:]         = sum over n of grad[r,n] * weight[e,n,:]
 *   grad_weight[e,n,:]  = sum over the live rows r of e of grad[r,n] * x[r,:]
 * grad_weight is written whole: an expert without a live row gets +0. Either
 * output may be NULL and is then skipped, together with the operand only it
 * needs (weight for grad_x, x for grad_weight); both NULL is EP_ERR_NULL, but
 * with recv_capacity 0, where a grad_x of no rows may be NULL.
 *   grad         payload [recv_capacity,N]
 *   x            payload [recv_capacity,H] or NULL
 *   weight       payload [E,N,H] or NULL
 *   grad_x       payload [recv_capacity,H] or NULL
 *   grad_weight  payload [E,N,H] or NULL
 */
ep_status_t ep_grouped_linear_bwd(const ep_layout_t* layout, const void* handle_mem,
                                  size_t handle_bytes, const void* grad, const void* x,
                                  const void* weight, void* grad_x, void* grad_weight,
                                  int64_t out_features, hipStream_t stream);

/*
 * Grouped linear with 4-bit weights, for serving: out[r,:] = W[e] x[r,:] with
 *   W[e,n,h] = (q[e,n,h] - z[e,n,h/G]) * scales[e,n,h/G],
 * q in 0..15, G = group_size inputs to a group. Built for few rows per expert
 * (decoding), right for any number. bf16 and fp16 payloads (fp32 is
 * EP_ERR_SHAPE); G is 32, 64 or 128 and divides H. The dequantised weight is
 * never rounded: scale and zero point act on fp32 sums over a group. For fp16
 * these are sums of (q - z) x, of exact operands. For bf16 they are sums of
 * (16 + q) x that start at -(16 + z) times the sum of x, so an x that is
 * infinite, or beyond 2^112, may reach its row of out as NaN; other rows are not
 * touched by it.
 *   x             payload [recv_capacity,H], H = layout->hidden
 *   qweight       uint8 [E,N,H/2]; byte h/2 holds input h in its low four
 *                 bits for even h, in its high four bits for odd h
 *   scales        payload [E,N,H/G]
 *   zeros         uint8 [E,N,H/G] (any value is taken as that whole number),
 *                 or NULL for 8 everywhere
 *   out           payload [recv_capacity,N]
 *   out_features  N
 * qweight, scales and zeros are 16-byte aligned.
 */
ep_status_t ep_grouped_linear_quant(const ep_layout_t* layout, const void* handle_mem,
                                    size_t handle_bytes, const void* x, const uint8_t* qweight,
                                    const void* scales, const uint8_t* zeros, void* out,
                                    int64_t out_features, int32_t group_size,
                                    hipStream_t stream);

/*
 * Gated activation: out[r,i] = silu(gate_up[r,i]) * gate_up[r,I+i] for every
 * live row r, silu(g) = g / (1 + exp(-g)), I = layout->hidden. Computed in
 * fp32 up to the one rounding, for fp32 payloads with errors of the last bits
 * whatever the gate. 1 / (1 + exp(-g)) counts also where it is below fp32's
 * range; for g below -174, where it is under 2^-251, it may be 0.
 *   gate_up  payload [recv_capacity,2I]
 *   out      payload [recv_capacity,I]
 */
ep_status_t ep_swiglu(const ep_layout_t* layout, const void* handle_mem, size_t handle_bytes,
                      const void* gate_up, void* out, hipStream_t stream);

/*
 * Backward of the gated activation: with g, u the halves of a live row and
 * s = 1 / (1 + exp(-g)),
 *   grad_gate_up[r,i]   = grad[r,i] * u * s * (1 + g * (1 - s))
 *   grad_gate_up[r,I+i] = grad[r,i] * g * s
 *   grad          payload [recv_capacity,I], I = layout->hidden
 *   gate_up       payload [recv_capacity,2I]
 *   grad_gate_up  payload [recv_capacity,2I]
 */
ep_status_t ep_swiglu_bwd(const ep_layout_t* layout, const void* handle_mem,
                          size_t handle_bytes, const void* grad, const void* gate_up,
                          void* grad_gate_up, hipStream_t stream);

/*
 * The layer in 8 bits: rows and weights of e4m3 values (OCP 8-bit floating
 * point: four bits of exponent, three of mantissa, largest value 448, NaN 0x7F
 * and 0xFF, no infinity) with fp32 scales; a value stands for q * scale. A row
 * has one scale for every EP_SCALE_BLOCK of its values, the last block perhaps a
 * part, and room for EP_SCALE_COLUMNS of them: rows of scales are whole 16-byte
 * vectors this way, and ep_dispatch moves them as fp32 rows of that many values
 * (and 8-bit rows of H values as bf16 rows of H / 2), bit for bit. Weights
 * [E,N,H] have one scale for every 128 x 128: fp32 [E, ceil(N/128),
 * ceil(H/128)].
 *
 * Rounding to 8 bits (ep_rms_norm, ep_swiglu_scaled): with y a row's fp32
 * results and amax the largest magnitude among a block's finite ones,
 *   scale = max(amax, 448 * 2^-100) / 448,   q = e4m3(y / scale)
 * to nearest, ties to even (y / scale is taken as y times the fp32 reciprocal of
 * scale, so that a y within 2^-22 of the middle of two values may go either way).
 * An infinite or NaN y becomes NaN in its own place. Scale columns past a row's
 * blocks are +0.
 */
#define EP_SCALE_BLOCK 128
#define EP_SCALE_COLUMNS(H) (((H) + 1023) / 1024 * 8)

/*
 * Root-mean-square norm of the layout's T token rows, as it stands in front of
 * dispatch. With a residual,
 *   sum[t,:] = payload(x[t,:] + residual[t,:]),   s = sum[t,:]
 * and s = x[t,:] without one; then
 *   y = s / sqrt(mean(s^2) + eps) * weight
 * in fp32, given as out (rounded once), as out_q with out_scales, or as both.
 * The norm is that of the rounded sum, which the gradient is taken at. hidden up
 * to EP_MAX_NORM_FEATURES; with out_q a multiple of 16; eps 0 or more (with 0 a
 * row of zeros gives NaN). Uses the layout's num_tokens, hidden and dtype.
 *   x           payload [T,H]
 *   residual    payload [T,H] or NULL
 *   weight      payload [H]
 *   sum         payload [T,H]; NULL iff residual is; may be residual or x
 *               itself, which is then updated in place
 *   out         payload [T,H] or NULL
 *   out_q       e4m3 [T,H] or NULL; out and out_q are not both NULL
 *   out_scales  fp32 [T, EP_SCALE_COLUMNS(H)]; NULL iff out_q is
 */
#define EP_MAX_NORM_FEATURES 16384

ep_status_t ep_rms_norm(const ep_layout_t* layout, const void* x, const void* residual,
                        const void* weight, float eps, void* sum, void* out, uint8_t* out_q,
                        float* out_scales, hipStream_t stream);

/* Bytes of device memory that ep_rms_norm_bwd needs for its weight gradient, at
 * most 512 * H * 4; 0 for an invalid layout. Host only. */
size_t ep_rms_norm_bwd_workspace(const ep_layout_t* layout);

/*
 * Backward of the norm, with r = 1 / sqrt(mean(s^2) + eps) and n = s r:
 *   grad_x[t,:]     = r (g - n mean(g n)) + grad_sum[t,:],  g = grad[t,:] * weight
 *   grad_weight[:]  = sum over t of grad[t,:] * n
 * grad_x is the gradient of x and of the residual alike. grad_weight is summed in
 * fp32 in an order that the sizes fix, and written whole (+0 for T = 0).
 *   grad         payload [T,H]   of out
 *   grad_sum     payload [T,H]   of sum, or NULL
 *   x            payload [T,H]   what the norm was of: sum with a residual, else x
 *   weight       payload [H]
 *   grad_x       payload [T,H]
 *   grad_weight  payload [H] or NULL (skipped; workspace may be NULL then)
 *   workspace    workspace_bytes of device memory, rewritten here: calls that
 *                share one must be ordered on the GPU
 */
ep_status_t ep_rms_norm_bwd(const ep_layout_t* layout, const void* grad, const void* grad_sum,
                            const void* x, const void* weight, float eps, void* grad_x,
                            void* grad_weight, void* workspace, size_t workspace_bytes,
                            hipStream_t stream);

/*
 * ep_swiglu with its result in 8 bits. I = layout->hidden, a multiple of 16. Pad
 * and tail rows of out_q and out_scales follow the layout's flags as every
 * expert-major output does.
 *   gate_up     payload [recv_capacity,2I]
 *   out_q       e4m3 [recv_capacity,I]
 *   out_scales  fp32 [recv_capacity, EP_SCALE_COLUMNS(I)]
 */
ep_status_t ep_swiglu_scaled(const ep_layout_t* layout, const void* handle_mem,
                             size_t handle_bytes, const void* gate_up, uint8_t* out_q,
                             float* out_scales, hipStream_t stream);

/*
 * Grouped linear of 8-bit operands: ep_grouped_linear of the values that x and
 * weight stand for, the scales applied in fp32 to the sums over a block, out
 * rounded once to the payload type (bf16 or fp16; fp32 is EP_ERR_SHAPE). With up to
 * six rows an expert (the routes T*K, or the capacity if less, over E; 32 for one
 * expert alone), as when decoding, sums are fp32. With more, a block's sum is that of
 * the 8-bit matrix instruction, which cuts products off 13 bits below the largest of
 * the eight neighbours that it adds first, and fp32 from there on. For serving, with
 * no backward. H = layout->hidden is a multiple of 16, N = out_features of 8.
 *   x              e4m3 [recv_capacity,H]
 *   x_scales       fp32 [recv_capacity, EP_SCALE_COLUMNS(H)]
 *   weight         e4m3 [E,N,H]
 *   weight_scales  fp32 [E, ceil(N/128), ceil(H/128)]
 *   out            payload [recv_capacity,N]
 */
ep_status_t ep_grouped_linear_scaled(const ep_layout_t* layout, const void* handle_mem,
                                     size_t handle_bytes, const uint8_t* x,
                                     const float* x_scales, const uint8_t* weight,
                                     const float* weight_scales, void* out,
                                     int64_t out_features, hipStream_t stream);

/*
 * A whole expert layer for a few tokens, without a prepared handle: for every
 * token, over its valid routes k ascending, with e = topk_idx[t,k],
 *   a         = silu(gate_up[e,:I,:] x) * (gate_up[e,I:,:] x),  x = tokens[t,:]
 *   result[t] = payload(sum over k of topk_weights[t,k] * (down[e] a))
 * the products and the weighted sum in fp32 (the first term a product, each later
 * one a fused multiply-add); a is held as the sum of two values of the payload
 * type, to 16 bits in bf16, and in fp16 with an exponent for every 16 values, to 22
 * bits or 2^-36 of the largest among the 64 (8-bit weights: 128) that enter the
 * products together: neither range nor subnormals of the type take anything from
 * it. An infinite weight of down may reach its outputs as NaN. A route whose id is
 * outside [0,E), masked or not, counts nothing; a token with no valid route gets +0;
 * an expert may come more than once. T*K is at most EP_MAX_LAYER_ROUTES; uses the
 * layout's num_tokens, topk, num_experts, hidden and dtype (bf16 or fp16; fp32 is
 * EP_ERR_SHAPE). For serving, with no backward. The weights are of the payload type,
 * or, with both scales given, e4m3 with 128 x 128 scales (hidden and inner multiples
 * of 16 then); their values enter the products exactly and the scales the fp32 sums.
 *   topk_idx        int64 [T,K]
 *   topk_weights    fp32 [T,K]
 *   tokens          payload [T,H]
 *   gate_up         payload or e4m3 [E,2I,H], I = inner
 *   gate_up_scales  fp32 [E, ceil(2I/128), ceil(H/128)] or NULL
 *   down            payload or e4m3 [E,H,I]
 *   down_scales     fp32 [E, ceil(H/128), ceil(I/128)]; NULL iff the other is
 *   result          payload [T,H]
 *   workspace       ep_expert_layer_workspace bytes, rewritten here: calls that
 *                   share one must be ordered on the GPU
 */
#define EP_MAX_LAYER_ROUTES 1024

/* 0 for an invalid layout or size. Host only. */
size_t ep_expert_layer_workspace(const ep_layout_t* layout, int64_t inner);

ep_status_t ep_expert_layer(const ep_layout_t* layout, const int64_t* topk_idx,
                            const float* topk_weights, const void* tokens, const void* gate_up,
                            const float* gate_up_scales, const void* down,
                            const float* down_scales, void* result, int64_t inner,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Copy the handle's status word (EP_STATUS_* bits) to *host_out. Waits for
 * `stream`; not for the hot path. host_out is a host pointer. The library's
 * own addition: the review of "[PyTorch] Expert Parallelism: PyTorch wrapper
 * + autograd ops with symm-mem zero-copy" (thread on recv_capacity_per_rank)
 * has a sync-free mode drop what exceeds the static capacity and raise a
 * flag; this call reads that flag, and the bad-id and layout flags, back. */
ep_status_t ep_read_status(const void* handle_mem, uint32_t* host_out, hipStream_t stream);

/* Static description of an ep_status_t. Never NULL. Host only. The
 * library's own addition. */
const char* ep_status_str(ep_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* EP_MI355X_EP_H */
