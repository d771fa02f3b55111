/*
 * attn_jvp.h - C ABI of the B200 (sm_100a) custom-mask attention + JVP library.
 *
 * The operation (Causal-rCM summary page, App. B "FlashAttention-2 JVP Kernel
 * with Custom Masks"): for queries Q, keys K, values V and tangents tQ, tK,
 * tV, with softmax scale s and an additive mask M (0 where a query may attend
 * to a key, -inf elsewhere),
 *
 *     S  = s Q K^T + M,        P  = softmax(S) (row-wise),    O = P V
 *     tS = s (tQ K^T + Q tK^T)
 *     tP = P * (tS - rowsum(P * tS))                (elementwise *)
 *     tO = tP V + P tV
 *     LSE_i = log sum_j exp(S_ij)                   (natural log)
 *
 * Masked entries receive no tangent, because the discrete mask has none
 * (App. B); the tangent uses exactly the primal masked operator and the same
 * sparse schedule (App. B). The library returns the primal output, the
 * log-sum-exp values and the tangent output (App. B, last item).
 *
 * Masks are given as {mode, chunk_tokens c, n_chunks n}:
 *   ATTN_JVP_MASK_TEACHER_FORCING: the packed sequence [clean chunks | noisy
 *     chunks], L = 2 n c (Causal-rCM page, section 3 "Continuous-time
 *     consistency", TF-masked packed forward; Causal Forcing summary page,
 *     section 2, clean and noisy videos concatenated under a causal mask).
 *     A clean query in chunk j attends to clean chunks <= j. A noisy query in
 *     chunk i attends to clean chunks < i and to its own noisy chunk.
 *   ATTN_JVP_MASK_BLOCK_CAUSAL: L = n c; a query in chunk j attends to
 *     chunks <= j (Causal-rCM page, section 2 "Autoregressive video
 *     diffusion": causal across temporal blocks, full attention inside one).
 * Attention inside one chunk is full in both modes.
 *
 * Layout: q, k, v, tq, tk, tv, o, to are dense row-major [B, L, H, d] arrays
 * (d innermost) of the element type `dtype`; lse is a dense [B, H, L] float
 * array. All of them are DEVICE pointers of the current CUDA device unless a
 * function says otherwise.
 *
 * Ownership: the caller owns every buffer; the library never frees or keeps
 * a caller pointer after the call returns (work is stream-ordered: buffers
 * must stay valid until the stream reaches the launched work). The library
 * keeps, per device, a small status word and cached tensor-map descriptors;
 * it allocates nothing else. Outputs must not overlap inputs or each other.
 *
 * Errors: every function returns an int status (ATTN_JVP_OK = 0 on success)
 * and never throws. Argument errors are detected on the host before anything
 * is launched. attn_jvp_fwd does not synchronize; device-side faults of the
 * launched work (a bounded wait that ran out) are reported later by
 * attn_jvp_sync_status.
 *
 * Threading: functions may be called from several host threads; the cached
 * descriptors are protected by a lock.
 */
#ifndef ATTN_JVP_H_
#define ATTN_JVP_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------- */
enum {
  ATTN_JVP_OK = 0,
  ATTN_JVP_ERR_INVALID_ARGUMENT = 1, /* null pointer, bad size, L inconsistent with the mask */
  ATTN_JVP_ERR_UNSUPPORTED = 2,      /* dtype or head_dim the kernels do not implement */
  ATTN_JVP_ERR_MISALIGNED = 3,       /* a pointer is not 16-byte aligned */
  ATTN_JVP_ERR_CUDA = 4,             /* a CUDA runtime or driver call failed */
  ATTN_JVP_ERR_DEVICE_TIMEOUT = 5,   /* a kernel's bounded wait ran out; the outputs are invalid */
  ATTN_JVP_ERR_NO_DEVICE = 6,        /* no usable sm_100 device */
  ATTN_JVP_ERR_BAD_INDEX = 7         /* a position, length or page read on the device was out of range;
                                        what it pointed at was neither read nor written */
};

/* ---- mask ------------------------------------------------------------ */
typedef enum {
  ATTN_JVP_MASK_TEACHER_FORCING = 0,
  ATTN_JVP_MASK_BLOCK_CAUSAL = 1
} attn_jvp_mask_mode;

typedef struct {
  int32_t mode;         /* attn_jvp_mask_mode */
  int32_t chunk_tokens; /* c >= 1: tokens per chunk (one latent frame = 1560 in Wan2.1) */
  int32_t n_chunks;     /* n >= 1 */
} attn_jvp_mask;

/*
 * General masks (Causal-rCM summary page, App. B: the kernel takes masks as
 * query groups with admissible key ranges). Group g covers the query rows
 * [row_end of group g-1 (0 for g = 0), row_end of group g); each of those rows
 * may attend to keys [k0_begin, k0_end) and [k1_begin, k1_end). A table lists
 * 1 to ATTN_JVP_MAX_GROUPS groups in row order, the last ending at L, with
 * 0 <= k0_begin <= k0_end <= k1_begin <= k1_end <= L and at least one key per
 * group (either range may be empty). The teacher-forcing mask is such a table
 * with one group per chunk of rows (clean chunks, then noisy chunks).
 */
#define ATTN_JVP_MAX_GROUPS 512
typedef struct {
  int32_t row_end;
  int32_t k0_begin, k0_end;
  int32_t k1_begin, k1_end;
} attn_jvp_group;

/* ---- problem --------------------------------------------------------- */
typedef enum {
  ATTN_JVP_BF16 = 0, /* bf16 inputs/outputs, fp32 accumulation, tensor cores */
  ATTN_JVP_F32 = 1,  /* fp32 inputs/outputs, fp32 arithmetic on CUDA cores */
  ATTN_JVP_F16 = 2   /* fp16; only where a function below says so (the serving operators) */
} attn_jvp_dtype;

typedef struct {
  int64_t B;     /* batch >= 1 */
  int64_t L;     /* sequence length: 2 n c (teacher forcing) or n c (block causal) */
  int64_t H;     /* heads >= 1 */
  int64_t d;     /* head dim: 64 or 128 */
  int32_t dtype; /* attn_jvp_dtype */
  float scale;   /* softmax scale s; <= 0 selects 1/sqrt(d) */
} attn_jvp_shape;

/*
 * attn_jvp_fwd - O, tO and LSE of masked softmax attention and its JVP in one
 * fused pass (App. B: same online-softmax pass and shared rescaling for the
 * primal and tangent accumulators; fully masked key tiles are skipped).
 *
 *   shape   problem sizes and element type (host pointer, read during the call)
 *   q..tv   device inputs, [B, L, H, d] of `shape->dtype`, 16-byte aligned
 *   mask    mask mode and chunking; L must equal 2 n c or n c
 *   o, to   device outputs, [B, L, H, d] of `shape->dtype`, 16-byte aligned
 *   lse     device output, [B, H, L] float (natural-log log-sum-exp of the
 *           scaled, masked scores)
 *   stream  cudaStream_t to launch on (NULL = legacy default stream)
 *
 * Returns ATTN_JVP_OK after enqueueing the work, or an error code with
 * nothing launched. The call does not synchronize with the device.
 */
int attn_jvp_fwd(const attn_jvp_shape* shape,
                 const void* q, const void* k, const void* v,
                 const void* tq, const void* tk, const void* tv,
                 attn_jvp_mask mask,
                 void* o, void* to, float* lse,
                 void* stream);

/*
 * attn_jvp_fwd_groups - attn_jvp_fwd with a general mask given as a table of
 * row groups (see attn_jvp_group) instead of {mode, c, n}: same operation,
 * layouts, outputs and asynchronous behaviour.
 *
 *   groups    host array of n_groups groups; read during the call only (it is
 *             copied into the launch), the caller keeps ownership
 *   n_groups  1 .. ATTN_JVP_MAX_GROUPS
 *
 * Returns ATTN_JVP_ERR_INVALID_ARGUMENT for a table that breaks the rules
 * above (rows not increasing to L, ranges out of order or outside [0, L), a
 * group with no key) and ATTN_JVP_ERR_UNSUPPORTED for more than
 * ATTN_JVP_MAX_GROUPS groups; nothing is launched then. Each query block is
 * scheduled over the union of its rows' ranges, so key tiles in a gap of that
 * union are visited (and fully masked); tables whose neighbouring groups have
 * similar ranges waste little.
 */
int attn_jvp_fwd_groups(const attn_jvp_shape* shape,
                        const void* q, const void* k, const void* v,
                        const void* tq, const void* tk, const void* tv,
                        const attn_jvp_group* groups, int32_t n_groups,
                        void* o, void* to, float* lse,
                        void* stream);

/*
 * attn_jvp_fwd_host - the same operation on HOST buffers: copies the six
 * inputs host->device, runs attn_jvp_fwd, copies O, tO and LSE device->host
 * and waits for the stream. Host buffers should be pinned (page-locked) for
 * the copies to run at full speed (and to overlap with the kernel); pageable
 * memory also works.
 *
 * The heads go in up to 16 chunks (one head per chunk when H <= 16) through
 * two staging slots: the copies in
 * of chunk c+1 and the copies out of chunk c-1 run on two copy streams while
 * the kernel of chunk c runs on `stream`, ordered by events. The copy
 * streams and events are created on the first call on a device and kept
 * (like the status word); calls on one device are serialised by a lock.
 * Results are the same bits as attn_jvp_fwd on the same inputs.
 *
 *   h_q..h_tv  host inputs, [B, L, H, d]
 *   h_o, h_to  host outputs, [B, L, H, d];  h_lse host output [B, H, L]
 *   d_buf      caller-owned device staging buffer of at least
 *              attn_jvp_host_staging_bytes(shape) bytes, 256-byte aligned
 *   stream     stream for the copies and the kernel
 *
 * Returns the status of the whole sequence, including any device fault
 * (the call synchronizes on `stream`).
 */
int attn_jvp_fwd_host(const attn_jvp_shape* shape,
                      const void* h_q, const void* h_k, const void* h_v,
                      const void* h_tq, const void* h_tk, const void* h_tv,
                      attn_jvp_mask mask,
                      void* h_o, void* h_to, float* h_lse,
                      void* d_buf, void* stream);

/* Bytes of device staging attn_jvp_fwd_host needs for `shape` (0 on a bad shape):
 * two slots of one chunk of heads (8 tensors and the LSE of ceil(H / 16) heads,
 * each piece rounded up to 256 bytes), or one slot of the whole problem when H = 1. */
int64_t attn_jvp_host_staging_bytes(const attn_jvp_shape* shape);

/*
 * attn_jvp_sync_status - synchronizes `stream`, then reports and clears the
 * device status word of the current device: ATTN_JVP_ERR_DEVICE_TIMEOUT if a
 * kernel gave up on a bounded wait since the last call, else
 * ATTN_JVP_ERR_BAD_INDEX if a serving operator met a position, length or page out
 * of range (attn_jvp_fwd_host, which reports the first, leaves the second),
 * ATTN_JVP_ERR_CUDA if the stream reported an error, else ATTN_JVP_OK.
 */
int attn_jvp_sync_status(void* stream);

/* Static, NUL-terminated description of a status code. */
const char* attn_jvp_status_string(int status);

/*
 * attn_jvp_fwd_noalloc - attn_jvp_fwd for callers that cannot allocate device
 * memory (an allocator-free runtime, a plugin host that owns every device
 * buffer, code running where cudaMalloc is forbidden or would break a memory
 * budget). It allocates no device memory: not on the first call, not later.
 * (Its host-side work lists are built in fixed thread-local arrays, not on
 * the heap.) There is no counterpart in the pages; it is an addition of this
 * library.
 *
 * The bf16 kernel needs one word of scratch device memory besides its inputs
 * and outputs: the status word that a bounded wait sets when it runs out.
 * attn_jvp_fwd keeps that word in memory the library allocates once per
 * device. This entry point instead uses a fixed file-scope device array of
 * ATTN_JVP_NOALLOC_SCRATCH_BYTES bytes (ATTN_JVP_NOALLOC_SCRATCH_BYTES / 4
 * words, of which this version uses 1), which every GPU that loads the
 * library holds until the process exits. The scratch does not grow with the
 * problem; the entry point rejects any layout that would need more words than
 * the array holds with ATTN_JVP_ERR_UNSUPPORTED, and rejects problems the
 * kernels cannot run exactly as attn_jvp_fwd does.
 *
 * Only bf16 is accepted (the fp32 kernel needs no scratch; use attn_jvp_fwd).
 * Arguments, layout and outputs are those of attn_jvp_fwd. Unlike it, this
 * call is synchronous: it clears the scratch word on `stream`, launches,
 * copies the word back on `stream`, waits for `stream` and returns the
 * status of the launched work, so a bounded-wait timeout is reported here as
 * ATTN_JVP_ERR_DEVICE_TIMEOUT.
 *
 * The first call on a device (with that device current) looks up the array's
 * device address and the kernels' launch attributes; make that first call
 * before any stream capture. All calls share the one array: calls that
 * overlap on the GPU (other threads or streams) race on it.
 */
#define ATTN_JVP_NOALLOC_SCRATCH_BYTES 256
int attn_jvp_fwd_noalloc(const attn_jvp_shape* shape,
                         const void* q, const void* k, const void* v,
                         const void* tq, const void* tk, const void* tv,
                         attn_jvp_mask mask,
                         void* o, void* to, float* lse,
                         void* stream);

/* ---- backward of the primal attention --------------------------------- */

/*
 * attn_jvp_bwd - gradients dQ, dK, dV of the masked primal attention
 * O = softmax(s Q K^T + M) V, for training the network whose forward
 * attn_jvp_fwd computes. The fused forward returns LSE so that a backward
 * pass can rebuild P without a second softmax pass (Causal-rCM summary page,
 * App. B, last item); the pages say nothing more about the backward, and
 * this is the plain gradient under the same mask:
 *
 *     P_ij  = exp(s q_i . k_j - LSE_i) on admissible pairs, 0 elsewhere
 *     D_i   = dO_i . O_i - dLSE_i
 *     dS_ij = P_ij ((dO_i . v_j) - D_i)
 *     dV = P^T dO,    dK = s dS^T Q,    dQ = s dS K
 *
 * (dLSE is an optional cotangent of LSE; with it the result is the gradient
 * of a loss that also depends on LSE.)
 *
 *   shape      as for attn_jvp_fwd (same dtype, d and scale rules)
 *   q, k, v    device inputs of the forward, [B, L, H, d] of shape->dtype
 *   o          the forward's output O, [B, L, H, d] of shape->dtype
 *   dout       the cotangent dO of O, [B, L, H, d] of shape->dtype
 *   lse        the forward's LSE, [B, H, L] float (natural log)
 *   dlse       cotangent of LSE, [B, H, L] float, or NULL for none
 *   mask       the forward's mask
 *   dq, dk, dv device outputs, [B, L, H, d] of shape->dtype
 *   stream     cudaStream_t to launch on
 *
 * All pointers 16-byte aligned; outputs must not overlap inputs or each
 * other. Each output element has one writer, so results are the same bits
 * on every run. Keys that no row may attend to get zero gradients. lse must
 * be the forward's (finite) LSE of these inputs.
 *
 * bf16 (when 8 * 128 ceil(L/128) <= 2 d L, i.e. L >= 8 for d = 64 and
 * L >= 4 for d = 128): tensor cores, fp32 accumulation, P and dS rounded to
 * bf16 before the dV, dK and dQ products, outputs rounded to nearest even.
 * Three launches: per-row D_i = dO_i . O_i - dLSE_i and LSE_i log2(e) (fp32,
 * written into the dq buffer, which serves as scratch until the last launch
 * overwrites it with dQ), then dK and dV per block of 128 keys, then dQ per
 * block of 128 query rows. Its waits are bounded: a wait that runs out is
 * reported by attn_jvp_sync_status as ATTN_JVP_ERR_DEVICE_TIMEOUT.
 * fp32 (and bf16 below those lengths): fp32 arithmetic on CUDA cores, two
 * launches (dQ per block of 32 query rows, dK and dV per block of 32 keys).
 *
 * Returns ATTN_JVP_OK after enqueueing, or an error code with nothing
 * launched (argument errors are found on the host before any device call).
 * Does not synchronize.
 */
int attn_jvp_bwd(const attn_jvp_shape* shape,
                 const void* q, const void* k, const void* v,
                 const void* o, const void* dout,
                 const float* lse, const float* dlse,
                 attn_jvp_mask mask,
                 void* dq, void* dk, void* dv,
                 void* stream);

/* attn_jvp_bwd with a group-table mask (validated as for attn_jvp_fwd_groups). */
int attn_jvp_bwd_groups(const attn_jvp_shape* shape,
                        const void* q, const void* k, const void* v,
                        const void* o, const void* dout,
                        const float* lse, const float* dlse,
                        const attn_jvp_group* groups, int32_t n_groups,
                        void* dq, void* dk, void* dv,
                        void* stream);

/* ---- rotary position embedding ahead of the attention ------------------ */

/*
 * attn_jvp_rope - rotary position embedding of q, k and their tangents tq, tk
 * (Causal-rCM summary page, section 3, "KV Cache": RoPE is the positional
 * treatment of queries and keys, one of the attention's neighbours in the
 * layer-level JVP). The pages give no formula; this is the standard rotary
 * embedding on adjacent pairs, with per-token angles phi supplied as tables:
 *
 *     x'_2i   = x_2i cos(phi_ti) - x_2i+1 sin(phi_ti)
 *     x'_2i+1 = x_2i sin(phi_ti) + x_2i+1 cos(phi_ti)
 *
 * for every batch and head of token t. The rotation does not depend on its
 * input, so the tangents of the rotated queries and keys are the rotated
 * tangents; attn_jvp_fwd on the four outputs (with v and tv unchanged) is the
 * attention JVP with RoPE in front.
 *
 *   shape              as for attn_jvp_fwd (dtype, d; scale unused)
 *   q, k, tq, tk       device inputs, [B, L, H, d] of shape->dtype
 *   cos, sin           device tables, [L, d/2] float (token t, pair i)
 *   q_out .. tk_out    device outputs, [B, L, H, d] of shape->dtype; each may be
 *                      its own input (in place), and must not overlap any other
 *   stream             cudaStream_t to launch on
 *
 * All pointers 16-byte aligned. Arithmetic is fp32; bf16 outputs are rounded
 * to nearest even. One launch, one pass over HBM. Returns ATTN_JVP_OK after
 * enqueueing, or an error code with nothing launched; does not synchronize.
 */
int attn_jvp_rope(const attn_jvp_shape* shape,
                  const void* q, const void* k, const void* tq, const void* tk,
                  const float* cos, const float* sin,
                  void* q_out, void* k_out, void* tq_out, void* tk_out,
                  void* stream);

/*
 * attn_jvp_fwd_rope - attn_jvp_fwd with the rotary position embedding of
 * attn_jvp_rope applied to q, k and their tangents tq, tk first, in the same
 * launch for bf16 (Causal-rCM summary page, section 3, "KV Cache": RoPE on
 * queries and keys, the attention's neighbour in the layer-level JVP). The
 * operation is attn_jvp_fwd(R q, R k, v, R tq, R tk, tv) with R the rotation
 * by the cos/sin tables; the rotated tensors R q, R k, R tq, R tk are also
 * returned (the backward of the attention and a post-RoPE key cache need them).
 *
 *   q..tv       device inputs, [B, L, H, d] of shape->dtype
 *   cos, sin    device tables, [L, d/2] float (token t, pair i), as for attn_jvp_rope
 *   mask        as for attn_jvp_fwd
 *   q_rot..tk_rot  device outputs, [B, L, H, d]: the rotated q, k, tq, tk; each
 *               may be its own input (in place) and must not overlap any other
 *   o, to, lse  device outputs, as for attn_jvp_fwd
 *   stream      cudaStream_t to launch on
 *
 * bf16: one kernel launch. Its CTAs first rotate a share of q, k, tq, tk
 * each (one pass over HBM), meet at a bounded grid barrier and then run the
 * attention on the rotated tensors. The launch is cooperative (all its CTAs
 * resident at once, or it fails with ATTN_JVP_ERR_CUDA). The barrier uses
 * one of 1024 per-device words, tagged by a per-device launch count, so up
 * to 1024 such calls may be in flight on a device at once. fp32: the
 * rotation pass and then the CUDA-core kernel (two launches).
 *
 * All pointers 16-byte aligned; B * L * H * head_dim / 2 < 2^32 (else
 * ATTN_JVP_ERR_UNSUPPORTED).
 * Returns ATTN_JVP_OK after enqueueing, or an error code with nothing
 * launched. Does not synchronize; a bounded wait that runs out (the grid
 * barrier included) is reported by attn_jvp_sync_status.
 */
int attn_jvp_fwd_rope(const attn_jvp_shape* shape,
                      const void* q, const void* k, const void* v,
                      const void* tq, const void* tk, const void* tv,
                      const float* cos, const float* sin,
                      attn_jvp_mask mask,
                      void* q_rot, void* k_rot, void* tq_rot, void* tk_rot,
                      void* o, void* to, float* lse,
                      void* stream);

/* ---- host-side helpers (need no GPU) ---------------------------------- */

/* Number of admissible (query, key) pairs per (batch, head):
 * c^2 n (n+1) for teacher forcing, c^2 n (n+1) / 2 for block causal; -1 on a
 * bad mask. Effective FLOPs of one call are 12 d B H times this. */
int64_t attn_jvp_unmasked_pairs(attn_jvp_mask mask);

/*
 * attn_jvp_schedule_tiles - the key-tile schedule the bf16 kernel runs for one
 * query tile (App. B: masks as query groups with admissible key ranges; the
 * same sparse schedule drives primal and tangent scores).
 *
 *   mask, L       mask and sequence length (validated as for attn_jvp_fwd)
 *   block_m/_n    query / key tile sizes (rows / columns)
 *   q_tile        query tile index, 0 <= q_tile < ceil(L / block_m)
 *   tiles, full   caller arrays of `cap` entries: key tile indices in visit
 *                 order, and 1 where every (query, key) pair of the tile is
 *                 admissible (no element mask needed), 0 where it is partial
 *   cap           capacity of both arrays
 *
 * Returns the number of key tiles (>= 0; entries beyond `cap` are not
 * written) or -1 on a bad argument. Key tiles not listed are fully masked.
 */
int32_t attn_jvp_schedule_tiles(attn_jvp_mask mask, int64_t L, int32_t block_m,
                                int32_t block_n, int32_t q_tile,
                                int32_t* tiles, uint8_t* full, int32_t cap);

/*
 * attn_jvp_schedule_tiles_groups - the same for a group-table mask (the table
 * validated as for attn_jvp_fwd_groups, L = its last row_end). Returns the
 * number of key tiles or -1 on a bad argument.
 */
int32_t attn_jvp_schedule_tiles_groups(const attn_jvp_group* groups, int32_t n_groups, int64_t L,
                                       int32_t block_m, int32_t block_n, int32_t q_tile,
                                       int32_t* tiles, uint8_t* full, int32_t cap);

/*
 * attn_jvp_key_tile_query_bounds - the range of query tiles [*lo, *hi] that
 * the backward's dK/dV kernel scans for key tile k_tile (the transpose of
 * the schedule above: the query tiles whose schedule lists the key tile all
 * lie in the range). Exact for the closed-form masks (teacher forcing: clean
 * keys are seen from their chunk's clean rows on, noisy keys only by their
 * own chunk's noisy rows; block causal: from the key's chunk on).
 *
 *   mask, L       mask and sequence length (validated as for attn_jvp_fwd)
 *   block_m/_n    query / key tile sizes
 *   k_tile        key tile index, 0 <= k_tile < ceil(L / block_n)
 *
 * Returns 0, or -1 on a bad argument (nothing written).
 */
int32_t attn_jvp_key_tile_query_bounds(attn_jvp_mask mask, int64_t L, int32_t block_m,
                                       int32_t block_n, int32_t k_tile, int32_t* lo, int32_t* hi);

/*
 * attn_jvp_debug_wait - TEST ONLY: drives the bf16 forward kernels' bounded
 * waits to run out without a device fault (a wait on a barrier that nothing
 * completes), so that the timeout path can be tested. Not part of the
 * operation (the pages have no counterpart); it exists for failure-detection
 * tests.
 *
 *   limit_ns    limit of every bounded wait of the bf16 forward kernels
 *               launched later from the calling host thread; 0 restores
 *               the default of 4 s (at most 60 s)
 *   stall_tile  -1: no stall. >= 0: in those launches the first work unit's
 *               MMA issuer, at its stall_tile-th key tile, waits on a barrier
 *               that nothing completes. The wait runs out after limit_ns, the
 *               kernel drains the copies and MMAs in flight, frees its tensor
 *               memory and returns; attn_jvp_sync_status (or
 *               attn_jvp_fwd_noalloc itself) reports
 *               ATTN_JVP_ERR_DEVICE_TIMEOUT and the outputs are invalid.
 *
 * The settings are per host thread and stay until changed; call
 * attn_jvp_debug_wait(0, -1) to restore normal operation. Returns
 * ATTN_JVP_ERR_INVALID_ARGUMENT for values out of range.
 */
int attn_jvp_debug_wait(int64_t limit_ns, int32_t stall_tile);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t attn_jvp_version(void);

/* ======================================================================
 * Serving operators: rotation at positions, a paged 8-bit key-value cache,
 * the attention over it, and the causal attention of packed prompts.
 *
 * Token rows are [T, heads, d] arrays with a stride per token and per head
 * (in elements; the d elements of a head are adjacent), so views of a fused
 * projection can be passed. Rows, codes and rotation tables are 16-byte
 * aligned, with strides of whole 16 bytes; integers, scales and lse as their
 * type is. Query heads are grouped: query head h reads
 * key head h / (H / Hkv); H is a multiple of Hkv.
 *
 * Positions, lengths and page numbers are device data, which the host cannot
 * check without waiting for it. The kernels check each before they use it;
 * one that is out of range is not used (each function says what becomes of
 * its outputs: by default they are left as they were), and
 * attn_jvp_sync_status reports ATTN_JVP_ERR_BAD_INDEX later.
 *
 * Outputs do not overlap inputs unless the function says that they may.
 * No function here synchronizes, allocates device memory or keeps state
 * between calls, so each can be captured in a CUDA graph, and calls on
 * several streams may overlap as long as their outputs do not.
 * ====================================================================== */

/* Packed token rows. */
typedef struct {
  int64_t T;     /* tokens >= 0 (T = 0: nothing is done) */
  int64_t H;     /* query heads >= 1 (cache_append: ignored) */
  int64_t Hkv;   /* key/value heads >= 1; H is a multiple of it */
  int64_t d;     /* head dim: 64 or 128 */
  int32_t dtype; /* attn_jvp_dtype */
  float scale;   /* softmax scale s < 2.35e38; <= 0 selects 1/sqrt(d) (attention only) */
} attn_jvp_tokens;

/* Strides of a [T, heads, d] array, in elements. */
typedef struct {
  int64_t token, head;
} attn_jvp_strides;

/* Which columns of a head form a pair in a rotation of its first `rot` columns. */
typedef enum {
  ATTN_JVP_ROPE_INTERLEAVED = 0, /* (2i, 2i + 1) */
  ATTN_JVP_ROPE_HALF = 1         /* (i, i + rot/2) */
} attn_jvp_rope_layout;

/* Rotation tables: cos and sin [n_positions, rot/2] float, dense. */
typedef struct {
  const float* cos;
  const float* sin;
  int64_t n_positions;
  int64_t rot;    /* columns rotated: a multiple of 16, <= d; the others are copied */
  int32_t layout; /* attn_jvp_rope_layout */
} attn_jvp_rope_tables;

/*
 * attn_jvp_rope_at - rotary embedding of queries and keys at given positions:
 * for token t, p = positions[t] and each pair (a, b) of its columns,
 *     a' = a cos[p] - b sin[p],   b' = a sin[p] + b cos[p]
 * in fp32, rounded once. With transpose != 0 the transposed matrix (sin
 * negated) is applied: the gradient with respect to q and k, given the
 * gradients of the rotated ones. Scaled positions and a magnitude live in the
 * tables.
 *
 *   shape      T, H (heads of q), Hkv (heads of k), d, dtype (all three types)
 *   q, k       inputs with their strides; k may be NULL (then k_out too)
 *   positions  T integers of position_bytes (4 or 8) each, 0 <= p < n_positions;
 *              a token whose position is outside keeps its output rows as they were
 *   q_out, k_out  outputs with their strides; each may be its own input
 */
int attn_jvp_rope_at(const attn_jvp_tokens* shape, const void* q, attn_jvp_strides q_strides,
                     const void* k, attn_jvp_strides k_strides, const void* positions,
                     int32_t position_bytes, const attn_jvp_rope_tables* tables, int32_t transpose,
                     void* q_out, attn_jvp_strides q_out_strides, void* k_out,
                     attn_jvp_strides k_out_strides, void* stream);

/*
 * A paged key-value cache in 8 bits. A page holds page_tokens tokens of every
 * key head: e4m3 codes, and one fp32 scale per page and head; the value of a
 * code c is c * scale. Strides are in elements (bytes for the codes), the
 * same for k and v; the d codes of a token's head are adjacent.
 */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t pages;       /* pages in the pool, >= 1 */
  int64_t page_tokens; /* 16, 32, 64 or 128 */
  int64_t page_stride, head_stride, token_stride;  /* of k and v; multiples of 16; the first and last below 2^32 */
  int64_t scale_page_stride, scale_head_stride;       /* of k_scale and v_scale */
} attn_jvp_cache;

/*
 * attn_jvp_cache_append - append tokens to the cache, the keys rotated on the
 * way if tables are given. Token starts[b] + i of the packed rows becomes
 * token p = cached[b] + i of sequence b: its key (rotated by position p) and
 * value go to row p % page_tokens of page table[b][p / page_tokens].
 *
 * The scale of a page and head is a power of two: the smallest 2^e with
 * |x| <= 448 * 2^e over the finite values x of the new tokens in the page,
 * -32 <= e <= 32, and not below the page's scale before the call (read as the
 * attention reads it, between 2^-40 and 2^40) where the page keeps earlier
 * tokens of the sequence. Where it grows, those tokens'
 * codes are rounded anew to it (exact but for the smallest, subnormal codes).
 * A value is rounded once, from fp32 to e4m3 (to nearest even; behind a scale of
 * the caller's own that is no power of two, its quotient in fp32 is); values beyond
 * 448 * 2^e, infinities among them, become the largest code, NaN stays NaN.
 * Rows of a page behind the last appended token are left as they were. Calling
 * it twice with the same arguments gives the same cache.
 *
 *   shape    T = tokens in k and v, <= 2^30; Hkv <= 32767, d, dtype (all three types);
 *            B <= 2^20
 *   starts   [B + 1] int32, non-decreasing, starts[0] >= 0, starts[B] <= T;
 *            rows outside them are ignored
 *   cached   [B] int32, tokens of each sequence in the cache before the call
 *   cache    its pages, heads and tokens (and its scales) nested in any order:
 *            each stride covers all that smaller ones span
 *   table    [B, table_width] int32 page numbers, table_stride apart; the pages
 *            written belong to one sequence each, once
 *   rope     NULL for no rotation; else n_positions must exceed every p
 */
int attn_jvp_cache_append(const attn_jvp_tokens* shape, const void* k, attn_jvp_strides k_strides,
                          const void* v, attn_jvp_strides v_strides, const attn_jvp_cache* cache,
                          int64_t B, const int32_t* starts, const int32_t* cached,
                          const int32_t* table, int64_t table_width, int64_t table_stride,
                          const attn_jvp_rope_tables* rope, void* stream);

/*
 * attn_jvp_cache_attn - attention of the newest n tokens of each sequence over
 * its cached keys and values:
 *     O = softmax(s Q K^T) V,   LSE = log sum exp(s Q K^T)   (natural log)
 * over the keys j < lens[b] (causal == 0), or j < lens[b] - n + i + 1 for query
 * i of n (causal != 0: the n queries are the sequence's last n tokens). A row
 * that sees no key gets O = 0, LSE = -infinity.
 *
 *   shape   B = sequences <= 65535, L = n <= 2^24, H, d, dtype (bf16 or fp16), scale < 2.35e38
 *   Hkv     key/value heads
 *   q       [B, n, H, d]: q_strides[0..2] in elements for B, n, H
 *   lens    [B] int32, tokens of each sequence in the cache, the new ones
 *           included; <= table_width * page_tokens
 *   table   as for attn_jvp_cache_append
 *   max_len an upper bound of lens known on the host, or 0 for
 *           table_width * page_tokens; it sets how the work is split, and longer
 *           sequences are still computed whole
 *   workspace  at least attn_jvp_cache_attn_workspace_bytes(shape, Hkv, m) bytes,
 *           m being max_len, or table_width * page_tokens if that is smaller or
 *           max_len is 0; 16-byte aligned; NULL if that is 0. Its contents
 *           before and after the call mean nothing; calls that may overlap need
 *           one each
 *   o       [B, n, H, d] dense, of dtype;  lse [B, H, n] float dense
 *
 * Sums, maxima and LSE are in 32 bits; e^(x_j) b_j, b_j being the value scale of
 * key j's page, is held in fp16, the row's largest at 2^7 or more: each is off by
 * at most 2^-11 of itself, or by 2^-32 of the row's largest, and counts as 0 from
 * there down. Value scales of a head that differ by more than some 2^20 reach that
 * limit if the values that count lie on the pages of small scale.
 *
 * Scales in the cache are read as at least 2^-40 and at most 2^40. A sequence
 * whose length is out of range gets the empty row's result, and the tokens of
 * a page whose number is out of range count as hidden.
 */
int attn_jvp_cache_attn(const attn_jvp_shape* shape, int64_t Hkv, const void* q,
                        const int64_t* q_strides, const attn_jvp_cache* cache,
                        const int32_t* lens, const int32_t* table, int64_t table_width,
                        int64_t table_stride, int64_t max_len, int32_t causal, void* workspace,
                        int64_t workspace_bytes, void* o, float* lse, void* stream);

/* Bytes of workspace for sequences of up to max_len tokens on the current
 * device (0 where none is needed), or -1 on a bad argument or no device. */
int64_t attn_jvp_cache_attn_workspace_bytes(const attn_jvp_shape* shape, int64_t Hkv,
                                            int64_t max_len);

/*
 * attn_jvp_prompt_attn - causal attention inside each of B packed sequences:
 * rows starts[b] <= t < starts[b + 1] of q, k and v, query t seeing keys
 * starts[b] <= j <= t. Nothing outside a row's keys reaches it, infinities
 * and NaN in masked rows included. Rows outside the sequences are left as
 * they were. Sums, maxima and LSE are in 32 bits; the probabilities are rounded to
 * dtype, fp16 ones by at most 2^-11 of themselves or 2^-32 of the row's largest.
 *
 *   shape   T, H, Hkv, d, dtype (bf16 or fp16), scale
 *   q, k, v  with strides of at least d (of 0 nowhere: give Hkv the number of
 *           key heads that there are)
 *   starts  [B + 1] int32, as for attn_jvp_cache_append; B <= 2^20
 *   o       [T, H, d] dense, of dtype;  lse [H, T] float dense
 */
int attn_jvp_prompt_attn(const attn_jvp_tokens* shape, const void* q, attn_jvp_strides q_strides,
                         const void* k, attn_jvp_strides k_strides, const void* v,
                         attn_jvp_strides v_strides, int64_t B, const int32_t* starts, void* o,
                         float* lse, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_JVP_H_ */
