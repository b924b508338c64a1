/*
 * sdm.h -- C ABI of the GB300 (sm_103a) hot path of the chunked sparse-delta-memory (SDM)
 * recurrence: the forward's Phase 1 and Phase-2 decay-and-write (DW), the saving forward's dense
 * snapshot, and the deterministic backward's step kernels (Phase A, GWR, GDS); and of the operators a model
 * needs around that layer (gated linear recurrence, norm and rotation of queries and keys, token log
 * probabilities, gated delta rule, norms around a block, embedding; from their own section on).
 *
 * Definitions followed (sparse-delta-memory 2.0.0):
 *   phase1_cuda.py, module docstring ........ the Phase-1 outputs and the determinism contract
 *   phase1_cuda.py, p1_keys_zw_kernel ........ entry order and payload bits, invalid tokens
 *   phase1_cuda.py, p1_scan_kernel ........... gates, log-cumsums, rex, cpe, flags, pos pack,
 *                                              sorted-row elements
 *   phase1_cuda.py, p1_pairs_kernel comment .. the A / QK pair triangles
 *   mover_da2_cuda.py, module docstring ...... DW: bank[s] = fma(base, cpe_last, acc),
 *                                              acc = fma(sc_m, dv[tok_m], acc) in sorted order
 *   mover_fx_cuda.py, module docstring ....... the bank-direct DW contract (base read from the
 *                                              bank row itself; one writer per row and launch)
 *   pa_dc_cuda.py, module docstring .......... the backward step: Phase A (the backward of DW)
 *                                              and GWR (the write side's token gather)
 *   mover_da2_cuda.py, "GDS, split by data need" the backward's read side (dots and scatter)
 *
 * Conventions shared by every entry point
 *   - Every data pointer is a DEVICE pointer owned by the caller. The library never allocates
 *     device or host memory. It launches on `stream` and never synchronizes it (except
 *     sdm_device_status, which reads a word back).
 *   - Layout is chunk-major: chunk c = ti * P + p holds tokens [ti*C, (ti+1)*C) of stream p,
 *     for ti in [0, steps). N = steps * P chunks.
 *       k_idx [N, C, W] int32, q_idx [N, C, R] int32: stream-local slot ids in [0, S). Ids of
 *         invalid tokens (t >= valid_last in the last step's chunks) are ignored.
 *       k_val [N, C, W], q_val [N, C, R]: val_dtype (float32 or bfloat16).
 *       g: float32 [N, C] one gate per token (gate_per_entry = 0) or [N, C, W] per write entry (1).
 *       dv [N * C, hd]: dv_dtype; row c * C + t is token t of chunk c.
 *       bank [P * S, hd]: bank_dtype; stream p owns rows [p*S, (p+1)*S). Updated in place.
 *   - Alignment: bank, dv and every output array 16-byte aligned; hd a multiple of 4.
 *   - Limits: 1 <= C <= 256, 1 <= W, R <= 256, C * (W + R) <= 8192 (one chunk sorts on chip),
 *     1 <= S <= 2^31 - 1, P * S * hd fits in int64.
 *   - Shape, dtype, alignment and workspace errors are returned BEFORE any launch. Errors the
 *     device finds (a valid slot id outside [0, S)) are OR-ed into a status word inside the
 *     workspace (read it with sdm_device_status), or, for the backward entry points, into the
 *     caller's optional status word. No kernel traps, and no kernel waits on another thread block.
 *   - Determinism: for fixed inputs, shapes and GPU type every output is bitwise reproducible.
 *     The sort is stable, scans combine in a fixed tree, every A/QK cell and every bank row has
 *     one writer that adds its terms in an input-determined order, and no atomics touch a sum.
 */
#ifndef SDM_H
#define SDM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* sdm_stream_t;

typedef enum {
    SDM_OK = 0,
    SDM_ERR_ARG = -1,       /* a required pointer is NULL, or a step range is reversed / out of range */
    SDM_ERR_SHAPE = -2,     /* a size is outside the limits above */
    SDM_ERR_DTYPE = -3,     /* an unknown dtype code */
    SDM_ERR_ALIGN = -4,     /* a pointer is not 16-byte aligned, or hd % 4 != 0 */
    SDM_ERR_WORKSPACE = -5, /* ws is NULL, misaligned or smaller than sdm_workspace_bytes */
    SDM_ERR_SMEM = -6,      /* the chunk does not fit the device's shared memory */
    SDM_ERR_CUDA = -7,      /* a CUDA runtime call failed (launch, attribute, memset) */
    SDM_ERR_DEVICE = -8     /* sdm_device_status found a nonzero device status word */
} sdm_status;

typedef enum { SDM_F32 = 0, SDM_BF16 = 1 } sdm_dtype;

/* Bits of the device status word (sdm_device_status). */
#define SDM_DEV_BAD_SLOT 0x1u /* a valid entry's slot id was outside [0, S): the entry is dropped */
#define SDM_DEV_BAD_OFFSET 0x2u   /* sequence offsets not ascending within [0, rows]: cut to it */
#define SDM_DEV_BAD_POSITION 0x4u /* a position at or above max_pos: treated as padding */
#define SDM_DEV_BAD_TARGET 0x8u   /* a target at or above V: treated as ignored */
#define SDM_DEV_BAD_TOKEN 0x10u   /* a token id at or above V: treated as padding */
#define SDM_DEV_STALLED 0x20u     /* a wait inside a kernel ran out: the call's outputs are not valid */

typedef struct {
    int32_t P;              /* streams */
    int32_t C;              /* tokens per chunk */
    int32_t W;              /* write (K) entries per token */
    int32_t R;              /* read (Q) entries per token */
    int32_t hd;             /* bank / dv row width */
    int32_t valid_last;     /* valid tokens of the last step's chunks, 1..C */
    int64_t steps;          /* chunks per stream */
    int64_t S;              /* slots per stream */
    int32_t val_dtype;      /* sdm_dtype of k_val, q_val and of cpe / k_eff / q_w */
    int32_t dv_dtype;       /* sdm_dtype of dv */
    int32_t bank_dtype;     /* sdm_dtype of the bank */
    int32_t gate_per_entry; /* 0: g [N, C]; 1: g [N, C, W] */
    /* Launch geometry of the forward's kernels, 0 = chosen from the shape (the backward's entry
     * points ignore both). Neither changes any output bit (every sum is taken in an order fixed by
     * the input), only how the work is split:
     *   dw_log_buckets 1..11 (<= ceil(log2 S)): the DW walk's hashed slot buckets per stream, 2^k
     *                  (changes sdm_workspace_bytes and Phase 1's shared memory per block: 8 bytes a
     *                  bucket); 0 = about 32768 / ceil(hd / 128) DW work items per launch, at most 2^10
     *                  buckets;
     *   p1_warps       the automatic count .. 32: warps of a Phase-1 block (extra warps hold
     *                  padding entries; more shared memory per block). */
    int32_t dw_log_buckets;
    int32_t p1_warps;
} sdm_shape;

/*
 * Phase-1 outputs, entry order (phase1_cuda.py module docstring and p1_scan_kernel). Any field
 * may be NULL: it is not written.
 *   [N, C, W]: log_k f32 (log-cumsum of the slot's gates at the entry, own token included),
 *              rex f32 (gates of the slot's later writes in the chunk), cpe val_dtype
 *              (exp of the slot's total gate in the chunk), k_eff val_dtype (k * exp(log_k)),
 *              is_last / is_only int8, pos_k int32 (position pack below).
 *   [N, C, R]: log_q f32, q_w val_dtype (q * exp(log_q)), pos_q int32, q_last / q_only int8.
 *   A, QK [N, C, C] f32: A[i][j] = sum over shared slots of k_i k_j exp(log_k_i - log_k_j),
 *              j < i; QK[i][j] = sum of q_i k_j exp(log_q_i - log_k_j), j <= i; zero elsewhere.
 *   sorted_k [N, C*W], sorted_q [N, C*R] int32: each kind's entries in sorted order as
 *              (entry bits: lane | isQ << 8 | token << 9 | invalid << 17)
 *              | min(peers before, 4095) << 18 | LAST << 30 | FIRST << 31; invalid: | 3 << 30.
 *   repeats: one int64 to which the count of repeated write entries (a token's write entry on
 *            a slot its previous write entry of the group already holds) is ADDED.
 *   ngroups [N] int32: the chunk's valid write groups (slots with at least one valid write
 *            entry), i.e. the rows of its dense compact snapshot; written only by the saving
 *            forward's Phase 1 (sdm_phase1_saving, sdm_forward_chunks_saving).
 *   stats [4] int64: counters of the call's chunks, ADDED to (the caller zeroes them): [0] valid
 *            write groups (slot groups with at least one valid write entry: the DW's base-row reads
 *            and row writes), [1] slot groups whose pair terms took the dense rank-1 path, [2] pair
 *            terms summed one by one (an entry and an earlier write entry of its group, into A or
 *            QK), [3] A / QK rows the pair phase writes (a token's row in a triangle where one of its
 *            entries has an earlier valid write entry in its group, or that a dense group
 *            reaches). [1..3] are counted only when A or QK is requested. Diagnostic counters in the manner of phase1_cuda.py's repeats counter.
 * Position pack: r | min(after, 127) << 17 | min(before + 1 + min(after, 127), 127) << 24 for a
 * valid entry (r = position in the chunk's sorted row, before / after = valid entries of the
 * same kind and slot before / after it), r alone for an invalid entry. Invalid entries:
 * log 0, rex 0, cpe 1, k_eff / q_w 0, flags 0.
 */
typedef struct {
    float* log_k;
    float* rex;
    void* cpe;
    void* k_eff;
    int8_t* is_last;
    int8_t* is_only;
    int32_t* pos_k;
    float* log_q;
    void* q_w;
    int32_t* pos_q;
    int8_t* q_last;
    int8_t* q_only;
    float* A;
    float* QK;
    int32_t* sorted_k;
    int32_t* sorted_q;
    int64_t* repeats;
    int32_t* ngroups;
    int64_t* stats;
} sdm_p1_out;

/*
 * Bytes of the caller-allocated device workspace for this shape: a 256-byte header (status word,
 * DW work counter), the DW records of every chunk (16 bytes per write entry) and the per-chunk
 * slot-bucket bounds of the DW work split. The workspace must be 256-byte aligned and, before its
 * first use, initialised with sdm_workspace_init. One workspace serves one stream of calls at a
 * time. Returns 0 for an invalid shape.
 */
size_t sdm_workspace_bytes(const sdm_shape* shape);

/* Zeroes the workspace's header (status word and work counter) on `stream`. */
sdm_status sdm_workspace_init(void* ws, size_t ws_bytes, sdm_stream_t stream);

/*
 * Phase 1 of the chunks of steps [step_begin, step_end) (all P streams): the outputs in `out`
 * and, in `ws`, the DW records of those chunks. Inputs are the full [N, ...] arrays; only the
 * range's chunks are read and written. Launches one kernel (one CTA per chunk).
 */
sdm_status sdm_phase1(const sdm_shape* shape, const int32_t* k_idx, const int32_t* q_idx,
                      const void* k_val, const void* q_val, const float* g, const sdm_p1_out* out,
                      int64_t step_begin, int64_t step_end, void* ws, size_t ws_bytes,
                      sdm_stream_t stream);

/*
 * DW of steps [step_begin, step_end), in step order, from the records sdm_phase1 left in `ws`
 * for those steps: per slot group of each chunk, bank[p*S + s] = fma(base, cpe_last, acc),
 * acc = fma(sc_m, dv[tok_m], acc) over the group's write entries in sorted order starting at 0,
 * sc = f32(k) * expf(rex), base = the row before this step (stored RN in bfloat16, or as the f32
 * result). One launch runs every step: each warp owns a range of slots of one stream and applies
 * the range's groups of all steps in order, so no warp ever waits for another.
 */
sdm_status sdm_dw(const sdm_shape* shape, const void* dv, void* bank, int64_t step_begin,
                  int64_t step_end, void* ws, size_t ws_bytes, sdm_stream_t stream);

/*
 * The forward over steps [step_begin, step_end): sdm_phase1 then sdm_dw on `stream`.
 * `out` may be NULL (no Phase-1 outputs written; records still go to ws). Running [0, k) then
 * [k, steps) gives the same bits as [0, steps).
 */
sdm_status sdm_forward_chunks(const sdm_shape* shape, const int32_t* k_idx, const int32_t* q_idx,
                              const void* k_val, const void* q_val, const float* g, const void* dv,
                              void* bank, const sdm_p1_out* out, int64_t step_begin,
                              int64_t step_end, void* ws, size_t ws_bytes, sdm_stream_t stream);

/*
 * Phase 1 of the saving forward: sdm_phase1, and in addition each group's FIRST DW record carries
 * the group's dense ordinal (below) and out->ngroups is written. Its records serve sdm_dw_saving
 * (and sdm_dw); the records of sdm_phase1 serve sdm_dw only. Errors: those of sdm_phase1.
 */
sdm_status sdm_phase1_saving(const sdm_shape* shape, const int32_t* k_idx, const int32_t* q_idx,
                             const void* k_val, const void* q_val, const float* g,
                             const sdm_p1_out* out, int64_t step_begin, int64_t step_end, void* ws,
                             size_t ws_bytes, sdm_stream_t stream);

/*
 * The saving forward's DW (mover_fx_cuda.py, module docstring; mover_da2_cuda.py, the WR mode of the
 * DW walk): sdm_dw, and in addition every valid write group's base row -- the bank row before this
 * step's write, as raw bytes of the bank type -- goes to the dense compact snapshot
 *   snap [N, C*W, hd] (bank dtype, 16-byte aligned, caller-owned), row c * (C*W) + g,
 * g = the group's dense ordinal in chunk c: the number of the chunk's valid write groups (slots with
 * at least one valid write entry) before it in sorted order, i.e. slots ascending. Rows g >=
 * ngroups[c] (sdm_p1_out.ngroups) are not written. The records must come from sdm_phase1_saving
 * (they carry the ordinals). Bank results are those of sdm_dw, bit for bit.
 * Errors: those of sdm_dw; snap NULL -> SDM_ERR_ARG, misaligned -> SDM_ERR_ALIGN.
 */
sdm_status sdm_dw_saving(const sdm_shape* shape, const void* dv, void* bank, void* snap,
                         int64_t step_begin, int64_t step_end, void* ws, size_t ws_bytes,
                         sdm_stream_t stream);

/* sdm_phase1_saving then sdm_dw_saving on `stream` (arguments as sdm_forward_chunks, plus snap). */
sdm_status sdm_forward_chunks_saving(const sdm_shape* shape, const int32_t* k_idx,
                                     const int32_t* q_idx, const void* k_val, const void* q_val,
                                     const float* g, const void* dv, void* bank, void* snap,
                                     const sdm_p1_out* out, int64_t step_begin, int64_t step_end,
                                     void* ws, size_t ws_bytes, sdm_stream_t stream);

/* Bytes of the library-owned scratch used by sdm_forward_chunks_noalloc (16 MiB). */
#define SDM_NOALLOC_SCRATCH_BYTES (16u << 20)

/*
 * The forward of sdm_forward_chunks for callers that cannot allocate device memory -- for example
 * code inside a host framework that owns every device allocation, or a plugin interface that is
 * handed only its input and output buffers. It takes no workspace: it uses a scratch array of
 * SDM_NOALLOC_SCRATCH_BYTES compiled into the library (every GPU that loads the library holds it
 * until the process exits). It calls no cudaMalloc / cudaFree and no allocating library routine.
 * The pages (sparse-delta-memory 2.0.0) have no counterpart of this entry point.
 *   - Arguments and results are those of sdm_forward_chunks, without ws / ws_bytes.
 *   - Shapes whose workspace (sdm_workspace_bytes) exceeds SDM_NOALLOC_SCRATCH_BYTES are rejected
 *     with SDM_ERR_WORKSPACE before any launch; use sdm_forward_chunks with a caller workspace.
 *   - status_out (nullable): one device int32 that receives the call's device status word
 *     (SDM_DEV_* bits, 0 = fine), copied on `stream` after the kernels.
 *   - A call outside stream capture looks up the scratch's device address (with the calling
 *     thread's current device), so a device context created again (after cudaDeviceReset) is
 *     picked up; a call inside a stream capture reuses the address of the last call on that device
 *     outside capture: make at least one call before any capture, and again after a device reset.
 *   - Every call shares the one scratch and clears its header first. Calls whose kernels overlap
 *     on the GPU (different streams, or concurrent host threads) race on it: serialize them.
 */
sdm_status sdm_forward_chunks_noalloc(const sdm_shape* shape, const int32_t* k_idx,
                                      const int32_t* q_idx, const void* k_val, const void* q_val,
                                      const float* g, const void* dv, void* bank,
                                      const sdm_p1_out* out, int64_t step_begin, int64_t step_end,
                                      int32_t* status_out, sdm_stream_t stream);

/*
 * The forward's read-side token gather (mover_fx_cuda.py: fx_fwd_steps, each step's gather before its
 * dual matmul and DW; the weighted read whose vector-Jacobian product in q_w is the GDS dot
 * d_q_w[t, r] = <gr[t], bank[slot]> of mover_da2_cuda.py's module docstring; the token_gather form of
 * GWR's d_delta_v, pa_dc_cuda.py's module docstring), for every chunk c = ti * P + p of steps
 * [step_begin, step_end):
 *   y[c, t] = acc, acc = 0; acc = fmaf(q_w[c, t, r], bank[p*S + q_idx[c, t, r]], acc) over the read
 *   lanes r = 0 .. R-1 in order (float32; a lane whose id lies outside [0, S) adds nothing) for valid
 *   tokens t; padding tokens (t >= valid_last in the last step) get zeros.
 *   q_idx [N, C, R] int32, q_w [N, C, R] val_dtype (Phase 1's q_w output, or any weights),
 *   bank [P*S, hd] bank_dtype, read only: the rows as they are when the kernel runs, so a range of
 *   several steps reads one bank state (the forward's order is the caller's: the read of step t, then
 *   the DW of step t); y [N, C, hd] float32, only the range's chunks written. The pages' "dual matmul"
 *   (the chunk-internal part of the read, from A / QK) is not printed there and is not provided.
 *   status (nullable): SDM_DEV_BAD_SLOT is OR-ed when a valid token reads an id outside [0, S).
 * Errors: the shape's (SDM_ERR_SHAPE / DTYPE / ALIGN for hd % 4), SDM_ERR_ARG (step range, null
 * q_idx / q_w / bank / y), SDM_ERR_ALIGN (bank or y not 16-byte aligned), before any launch.
 * One launch (resident warps looping over (token, 128-column slice) units).
 */
sdm_status sdm_read(const sdm_shape* shape, const int32_t* q_idx, const void* q_w, const void* bank, float* y,
                    int64_t step_begin, int64_t step_end, uint32_t* status, sdm_stream_t stream);

/*
 * Phase A of the backward (pa_dc_cuda.py, module docstring: "PA per write group"; records kernel):
 * the backward of DW for the steps [step_begin, step_end), LAST step first (one launch per step;
 * step ti reads the grad rows step ti + 1 wrote). Per valid write group of chunk c = ti * P + p
 * (slot s, members m in sorted order, as sorted_k lists them):
 *   sc_m = -beta[c, tok_m] * (f32(k_m) * expf(log_k_m))
 *   acc = 0; acc = fmaf(sc_m, dva[c, tok_m], acc) over the members in order
 *   grad[p*S + s] = RN(fmaf(gdw, cpe_last, acc))    gdw = the row before this step, cpe_last = cpe of
 *                                                    the group's last member (f32 grad: the fmaf itself)
 *   bank[p*S + s] = the group's snapshot row        (raw bytes: the row before the forward's write)
 *   grad_g[e] = cpe_e * <gdw, snap>,  d_k_eff[e] = -beta[c, tok_e] * <dva[c, tok_e], snap>
 * Dots are f32: per lane an fmaf chain over 4 columns of a 128-column slice, an xor butterfly over
 * the 32 lanes, slices added in order, so results do not depend on the launch geometry.
 * Arguments (device pointers, 16-byte aligned, caller-owned; shapes use `shape`'s N = steps * P):
 *   grad_dtype: sdm_dtype of grad (SDM_F32, or SDM_BF16 for grad rows in the bank's format).
 *   sorted_k [N, C*W] int32: as sdm_phase1 writes it (entries whose slot is outside [0, S) are
 *            invalid there). log_k f32 / cpe val_dtype [N, C, W]: sdm_phase1's outputs.
 *   k_idx int32 / k_val val_dtype [N, C, W]: the forward's inputs. beta f32 [N, C].
 *   dva f32 [N, C, hd]: the gradient of the forward's token rows (dv) for these steps.
 *   grad [P*S, hd] grad_dtype, bank [P*S, hd] bank_dtype: updated in place.
 *   snap: the dense compact snapshot rows of the steps in range, [step_end - step_begin, P, C*W, hd]
 *         in the bank dtype: row ((ti - step_begin) * P + p) * C*W + g for the group of dense ordinal g
 *         (sdm_dw_saving's layout; a caller holding all N chunks passes its row step_begin * P * C*W).
 *   d_k_eff, grad_g [N, C, W] f32: written for every entry of the range's chunks (0 for invalid
 *         entries).
 *   status (nullable): device word OR-ed with SDM_DEV_BAD_SLOT when a group's slot (k_idx of its
 *         first member) lies outside [0, S); the group is then skipped.
 * Errors: SDM_ERR_SHAPE / SDM_ERR_DTYPE / SDM_ERR_ALIGN for the shape (as sdm_phase1), grad_dtype
 * not 0 or 1 -> SDM_ERR_DTYPE, a NULL array -> SDM_ERR_ARG, a misaligned array -> SDM_ERR_ALIGN, a
 * bad step range -> SDM_ERR_ARG, a failed launch -> SDM_ERR_CUDA. No launch happens on an error
 * found before the first launch.
 */
sdm_status sdm_pa(const sdm_shape* shape, int32_t grad_dtype, const int32_t* sorted_k, const int32_t* k_idx,
                  const void* k_val, const float* log_k, const void* cpe, const float* beta, const float* dva,
                  void* grad, void* bank, const void* snap, float* d_k_eff, float* grad_g, int64_t step_begin,
                  int64_t step_end, uint32_t* status, sdm_stream_t stream);

/*
 * GWR, the token gather of the write side of the backward (pa_dc_cuda.py: module docstring, "GWR",
 * and its GWR kernel), for the steps [step_begin, step_end), LAST step first (one launch per step).
 * Per chunk c = ti * P + p and valid token t (t < valid_last in the last step's chunks, else t < C):
 *   d_delta_v[c, t] = acc, acc = 0; acc = fmaf(write_w[c, t, n], grad[p*S + k_idx[c, t, n]], acc)
 *                     over the write lanes n = 0 .. W-1 in order;
 *   d_k_pd[c, t, n] = <dv[c*C + t], grad[p*S + k_idx[c, t, n]]>  (f32 dots as sdm_pa's);
 * padding tokens get zero rows and zero dots.
 * Arguments (device pointers, 16-byte aligned, caller-owned; N = steps * P):
 *   grad_dtype: sdm_dtype of grad. k_idx int32 [N, C, W]: the forward's write ids. write_w f32
 *   [N, C, W]: the write weights. dv [N*C, hd] dv_dtype: the forward's token rows. grad [P*S, hd]
 *   grad_dtype: read only. d_delta_v f32 [N, C, hd], d_k_pd f32 [N, C, W]: written for the range.
 *   status (nullable): device word OR-ed with SDM_DEV_BAD_SLOT when a valid token's write id lies
 *   outside [0, S) (that lane adds nothing and its dot is 0).
 * Errors: as sdm_pa.
 */
sdm_status sdm_gwr(const sdm_shape* shape, int32_t grad_dtype, const int32_t* k_idx, const float* write_w,
                   const void* dv, const void* grad, float* d_delta_v, float* d_k_pd, int64_t step_begin,
                   int64_t step_end, uint32_t* status, sdm_stream_t stream);

/*
 * GDS, the read side of the backward (mover_da2_cuda.py: module docstring, the "GDS, split by data
 * need" comment, its read-records kernel), for the steps [step_begin, step_end), LAST step first
 * (two launches per step: the dots, then the scatter). Per chunk c = ti * P + p:
 *   d_q_w[c, t, r] = <gr[c, t], bank[p*S + q_idx[c, t, r]]> for the valid tokens t (t < valid_last
 *                   in the last step's chunks, else t < C); 0 for padding tokens;
 *   per read group (slot s with valid read entries; members m in sorted order as sorted_q lists them)
 *   acc = 0; acc = fmaf(sc_m, gr[c, tok_m], acc), sc = f32(q_m) * expf(log_q_m);
 *   grad[p*S + s] = RN(grad[p*S + s] + acc)          (one rounding per element; f32 grad: the sum)
 * Dots are f32 like sdm_pa's (per-lane fmaf chain over 4 columns, a fixed lane tree, slices in
 * order), so results do not depend on the launch geometry; every grad row has one writer per launch.
 * Arguments (device pointers, 16-byte aligned, caller-owned; N = steps * P):
 *   grad_dtype: sdm_dtype of grad (SDM_F32, or SDM_BF16 for grad rows in the bank's format).
 *   sorted_q [N, C*R] int32: as sdm_phase1 writes it. log_q f32 [N, C, R]: sdm_phase1's output.
 *   q_idx int32 / q_val val_dtype [N, C, R]: the forward's inputs. gr f32 [N, C, hd]: the gradient of
 *   the read results. bank [P*S, hd] bank_dtype: read only. grad [P*S, hd] grad_dtype: updated in
 *   place (must not alias bank). d_q_w [N, C, R] f32: written for every read entry of the range.
 *   status (nullable): device word OR-ed with SDM_DEV_BAD_SLOT when a valid token's read id lies
 *   outside [0, S) (its dot is 0 and it adds nothing).
 * Errors: as sdm_pa.
 */
sdm_status sdm_gds(const sdm_shape* shape, int32_t grad_dtype, const int32_t* sorted_q, const int32_t* q_idx,
                   const void* q_val, const float* log_q, const float* gr, const void* bank, void* grad, float* d_q_w,
                   int64_t step_begin, int64_t step_end, uint32_t* status, sdm_stream_t stream);

/* ================================================================================================
 * The operators around the memory: the gated linear recurrence, the norm and rotation of query and
 * key heads, log probabilities of tokens, the gated delta rule, the norms around a block, and the embedding. They share the conventions above (caller-owned device
 * pointers, no allocation, no synchronization, checks before any launch, every output bitwise
 * reproducible) and differ in these:
 *   - Row arrays take the distance between rows in elements (`*_ld`), so that a slice of a wider row
 *     can be passed. Inputs may repeat a row (ld 0). A base and its ld are aligned to 4 elements of the
 *     array's type unless said otherwise; states, tables and head weights to 16 bytes; the other small arrays to
 *     their elements.
 *   - An output overlaps no input unless said otherwise.
 *   - Row counts may be 0: nothing is read or written but what is said to be.
 *   - status (nullable): a device word to which SDM_DEV_* bits are OR-ed.
 *   - Errors: SDM_ERR_DTYPE / SHAPE / ALIGN for the shape, SDM_ERR_ARG for a NULL array or an ld below
 *     the row's length, SDM_ERR_ALIGN for a misaligned array or ld, SDM_ERR_WORKSPACE, SDM_ERR_CUDA.
 * ================================================================================================ */

/* Rows between two saved states of the recurrence. */
#define SDM_GLR_CHUNK 64

typedef struct {
    int32_t P;          /* sequences */
    int32_t D;          /* channels of a row, a multiple of 4, up to 2^20 */
    int32_t gate_width; /* channels that share a gate: 1 (a gate per channel), or a multiple of 4 that
                         * divides D (a gate per head of that many channels; D: one per row) */
    int32_t x_dtype;    /* sdm_dtype of x, y and their gradients */
    int32_t g_dtype;    /* sdm_dtype of g and dg */
    int64_t rows;       /* rows of all sequences together */
} sdm_glr_shape;

/*
 * The gated linear recurrence (the dense, per-channel counterpart of the memory's decay and write):
 *   h_t = exp(g_t) h_{t-1} + x_t,   y_t = h_t rounded to x_dtype,
 * for the rows of each sequence in order, in float32.
 *   x, y [rows, D]; g [rows, D / gate_width]: log gates, at most 0 (a gate of -inf starts anew; with gates
 *   above 0 the product of a span's gates may overflow). A row of per-head gates has no alignment rule.
 *   A product of gates below float32's range counts as 0: an infinite state may be NaN behind such a span.
 *   offsets: int64 [P + 1] on the device, sequence p owns rows [offsets[p], offsets[p+1]), empty ones
 *   allowed; or NULL: P sequences of rows / P rows each (rows a multiple of P). Rows before offsets[0] and from
 *   offsets[P] on belong to none: they are not read, and what y, dx and dg hold there stays.
 *   h0 (nullable: zeros) and hT (nullable) float32 [P, D]: the states before and after; hT may be h0; an
 *   empty sequence hands its state on.
 *   states (nullable) float32, sdm_glr_states_bytes: the state before every SDM_GLR_CHUNK-th row of each
 *   sequence, for the backward (row offsets[p] / SDM_GLR_CHUNK + p + j holds sequence p's j-th).
 *   y may be x (same ld); long sequences of few channels take longer then.
 * Spans of rows are computed apart and joined in a fixed order, so a sequence cut in two calls agrees with one
 * call to rounding, not bit for bit.
 */
size_t sdm_glr_states_bytes(const sdm_glr_shape* shape);
sdm_status sdm_glr_forward(const sdm_glr_shape* shape, const void* x, int64_t x_ld, const void* g, int64_t g_ld,
                           const int64_t* offsets, const float* h0, void* y, int64_t y_ld, float* hT, float* states,
                           uint32_t* status, sdm_stream_t stream);

/*
 * Its backward: with l_t = dy_t + exp(g_{t+1}) l_{t+1} (past a sequence's end: dhT, or 0 where NULL),
 *   dx_t = l_t,   dg_t = exp(g_t) l_t h_{t-1} (summed over the gate's channels),   dh0 = exp(g_1) l_1
 * (dhT for an empty sequence). h_{t-1} is computed again from x and the forward's states, so the rounding of
 * y enters no gradient. x, g, offsets as the forward had them; dy, dx [rows, D]; dg [rows, D / gate_width];
 * dhT, dh0 (nullable) float32 [P, D]; dh0 may be dhT; dx may be dy or x (same ld; as for y above). ws:
 * sdm_glr_workspace_bytes, 16-byte aligned (used where gate_width > 128; may be NULL otherwise).
 */
size_t sdm_glr_workspace_bytes(const sdm_glr_shape* shape);
sdm_status sdm_glr_backward(const sdm_glr_shape* shape, const void* x, int64_t x_ld, const void* g, int64_t g_ld,
                            const void* dy, int64_t dy_ld, const int64_t* offsets, const float* states,
                            const float* dhT, void* dx, int64_t dx_ld, void* dg, int64_t dg_ld, float* dh0, void* ws,
                            size_t ws_bytes, uint32_t* status, sdm_stream_t stream);

/*
 * One token of each of `rows` requests (P is not used): state[s] = exp(g_i) state[s] + x_i, y_i = state[s], with
 * s = slots[i] (int32 [rows], distinct), or i where slots is NULL. state float32 [states, D] with rows state_ld
 * apart. A row with a slot below 0 is padding: y_i = 0 and no state changes; so too one at or above `states`,
 * which sets SDM_DEV_BAD_SLOT.
 */
sdm_status sdm_glr_step(const sdm_glr_shape* shape, const void* x, int64_t x_ld, const void* g, int64_t g_ld,
                        const int32_t* slots, float* state, int64_t state_ld, int64_t states, void* y, int64_t y_ld,
                        uint32_t* status, sdm_stream_t stream);

typedef struct {
    int64_t tokens;     /* tokens times heads: below about 2^31 */
    int32_t q_heads;    /* heads of q and of k (either may be 0, not both) */
    int32_t k_heads;
    int32_t hd;         /* columns of a head, a multiple of 8, up to 1024 */
    int32_t rot_dim;    /* the first columns that turn, a multiple of 8, 0 .. hd */
    int32_t max_pos;    /* positions of the table */
    int32_t layout;     /* pairs that turn together: 0 half (i, i + rot_dim / 2), 1 interleaved (2i, 2i + 1) */
    int32_t dtype;      /* sdm_dtype of q, k, their outputs and gradients */
    int32_t norm;       /* 1: RMS norm of each head first; 0: the rotation alone (weights unused) */
    float eps;
} sdm_rope_shape;

/*
 * table [max_pos, rot_dim] float32: row m holds scale cos(m f_i) for i < rot_dim / 2, then scale sin(m f_i).
 * inv_freq: the rot_dim / 2 angles f_i of one position in radians, a HOST array read during the call. Angles are
 * reduced exactly for every position.
 */
sdm_status sdm_rope_table(const sdm_rope_shape* shape, const double* inv_freq, float scale, float* table,
                          sdm_stream_t stream);

/*
 * Per token t and head, x its row of hd columns and w the weights of its kind (float32 [hd], NULL: ones):
 *   n = x rsqrt(mean x^2 + eps) w   (norm 0: n = x),
 *   out_a = n_a c_i - n_b s_i, out_b = n_b c_i + n_a s_i for pair i = (a, b), c, s from the table's row
 * positions[t]; columns from rot_dim on are n. float32 throughout, rounded once. q, q_out [tokens, q_heads, hd],
 * k, k_out [tokens, k_heads, hd], a token's heads contiguous, tokens `*_ld` apart. positions int32 [tokens]: below 0
 * is a padding token (its outputs are 0); at or above max_pos likewise, and sets SDM_DEV_BAD_POSITION. q_out
 * may be q and k_out may be k (same ld).
 */
sdm_status sdm_qk_norm_rope(const sdm_rope_shape* shape, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                            const int32_t* positions, const float* table, const float* wq, const float* wk, void* q_out,
                            int64_t qo_ld, void* k_out, int64_t ko_ld, uint32_t* status, sdm_stream_t stream);

/*
 * Its backward, from the outputs' gradients and the forward's inputs: e = the gradient turned back by the angle,
 * dw += e x r over tokens and heads (r the row's rsqrt), and with u = e w: dx = r (u - x r^2 mean(u x)). Padding
 * tokens get zeros and add nothing. dwq, dwk float32 [hd] (nullable), written (with zeros for norm 0); ws:
 * sdm_rope_workspace_bytes, 16-byte aligned (may be NULL with norm 0 or where neither is asked for). dq may be dq_out,
 * dk may be dk_out (same ld).
 */
size_t sdm_rope_workspace_bytes(const sdm_rope_shape* shape);
sdm_status sdm_qk_norm_rope_backward(const sdm_rope_shape* shape, const void* dq_out, int64_t dqo_ld,
                                     const void* dk_out, int64_t dko_ld, const void* q, int64_t q_ld, const void* k,
                                     int64_t k_ld, const int32_t* positions, const float* table, const float* wq,
                                     const float* wk, void* dq, int64_t dq_ld, void* dk, int64_t dk_ld, float* dwq,
                                     float* dwk, void* ws, size_t ws_bytes, uint32_t* status, sdm_stream_t stream);

typedef struct {
    int64_t rows;       /* tokens, below 2^31 */
    int32_t V;          /* logits of a row, up to 2^28 */
    int32_t K;          /* top alternatives of a row, 0 .. min(32, V) */
    int32_t dtype;      /* sdm_dtype of logits and dlogits */
    float scale;        /* logits are multiplied by it first (1 / temperature), 1e-3 .. 1e3 */
} sdm_logprob_shape;

/*
 * Per row x [V] of logits (rows ld apart, no alignment rule but the element's), z = scale x:
 *   lse = log sum exp z, logp = z_target - lse, entropy = -sum p log p with p = exp(z - lse) (0 log 0 = 0),
 *   top_vals, top_idx [rows, K]: log probabilities and ids of the K largest logits, descending, the lower id first
 *   among equal logits.
 * targets int32 [rows]: below 0 is ignored (logp 0); at or above V likewise, and sets SDM_DEV_BAD_TARGET. logp
 * float32 [rows]; entropy, lse, top_vals, top_idx nullable. A row whose logits are all -inf has lse = -inf, log
 * probabilities -inf and entropy 0. Finite logits of any size have the probabilities of their differences (a row of a
 * type's lowest value is uniform); where lse lies past float32's range it is the largest or lowest finite value, and a
 * log probability below it is -inf. A row that holds NaN or +inf has NaN for its float outputs; NaN counts as the
 * largest logit in top_idx.
 */
sdm_status sdm_token_logprobs(const sdm_logprob_shape* shape, const void* logits, int64_t ld, const int32_t* targets,
                              float* logp, float* entropy, float* lse, float* top_vals, int32_t* top_idx,
                              uint32_t* status, sdm_stream_t stream);

/*
 * The gradient of the logits, from the forward's lse and entropy:
 *   dlogits_v = scale (d_logp (1[v = target] - p_v) - d_entropy p_v (log p_v + entropy)),
 * d_logp float32 [rows] (taken as 0 where the target is ignored), d_entropy float32 [rows] (nullable: zeros, and
 * entropy may be NULL then). In a row whose logits are all -inf every p is 0. dlogits may be logits (same ld). K is not
 * used.
 */
sdm_status sdm_token_logprobs_backward(const sdm_logprob_shape* shape, const void* logits, int64_t ld,
                                       const int32_t* targets, const float* lse, const float* entropy,
                                       const float* d_logp, const float* d_entropy, void* dlogits, int64_t d_ld,
                                       uint32_t* status, sdm_stream_t stream);

/* Rows between two saved states of the delta rule, and rows of a block of its walk. */
#define SDM_GDR_CHUNK 64

typedef struct {
    int32_t P;          /* sequences */
    int32_t k_heads;    /* heads of q and k */
    int32_t v_heads;    /* heads of v, g, beta and y, a multiple of k_heads: value head h goes with key head
                         * h / (v_heads / k_heads) */
    int32_t dk;         /* channels of a key head, a multiple of 8, up to 128 */
    int32_t dv;         /* channels of a value head, a multiple of 8, up to 128 */
    int32_t x_dtype;    /* sdm_dtype of q, k, v, y and their gradients */
    int32_t g_dtype;    /* sdm_dtype of g, beta and their gradients */
    float scale;        /* of the answers */
    int64_t rows;       /* rows of all sequences together */
} sdm_gdr_shape;

/*
 * The gated delta rule (the dense counterpart of the memory's decay, read and write): per sequence and value head, with
 * a state S [dk, dv] of slots addressed by every key at once,
 *   S_t = exp(g_t) S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t),   y_t = scale S_t^T q_t.
 *   q, k [rows, k_heads * dk], v, y [rows, v_heads * dv], aligned to 16 bytes like their ld; g, beta [rows, v_heads], no alignment
 *   rule: log decays, at most 0 (-inf starts anew; a product of decays below float32's range counts as 0), and write
 *   strengths (below 2^-80 they count as 2^-80). Keys of length 1 and beta in [0, 2] keep the state bounded.
 *   offsets: as in sdm_glr_forward (ragged sequences, rows of no sequence).
 *   h0 (nullable: zeros) and hT (nullable) float32 [P, v_heads, dk, dv]: the states before and after; hT may be h0; an
 *   empty sequence hands its state on. No other output overlaps an input.
 *   states (nullable), sdm_gdr_states_bytes, 16-byte aligned: the state before every SDM_GDR_CHUNK-th row of each sequence,
 *   what every row writes and what its block gives without the state, for the backward, in a form of its own.
 *   ws: sdm_gdr_workspace_bytes(shape, 0), 16-byte aligned. It holds nothing from one call to the next.
 * Few and long sequences (of bfloat16 rows) are walked in segments, as the shape alone decides, so the same sequence in calls of
 * different shapes agrees to rounding. A segment's matrix stays as small as a state does for keys no longer than 1; where longer keys take
 * it or a state out of float32's range, the segment walks on to the sequence's end for that head.
 * Blocks of 64 rows are solved together on the tensor cores; sums are float32, and float32 values enter the products as sums of
 * two bfloat16 (within 2^-17) beside bfloat16 rows, of three (2^-25) beside float32 rows. A value that is not finite spoils its sequence and head from the start of its block on (as NaN).
 */
size_t sdm_gdr_states_bytes(const sdm_gdr_shape* shape);
size_t sdm_gdr_workspace_bytes(const sdm_gdr_shape* shape, int32_t backward);
sdm_status sdm_gdr_forward(const sdm_gdr_shape* shape, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                           const void* v, int64_t v_ld, const void* g, int64_t g_ld, const void* beta, int64_t beta_ld,
                           const int64_t* offsets, const float* h0, void* y, int64_t y_ld, float* hT, void* states,
                           void* ws, size_t ws_bytes, uint32_t* status, sdm_stream_t stream);

/*
 * Its backward: the gradients dq, dk [rows, k_heads * dk] (summed over the value heads of a key head), dv [rows, v_heads * dv], dg,
 * dbeta [rows, v_heads] and dh0 (nullable, float32 [P, v_heads, dk, dv]) from dy and dhT (nullable: zeros; the gradient of the states
 * after). q, k, v, g, beta and offsets as the forward had them, states as it saved them; dh0 may be dhT. ws:
 * sdm_gdr_workspace_bytes(shape, 1), 16-byte aligned; it serves the forward too. Alignments as for the forward. No output overlaps an input.
 */
sdm_status sdm_gdr_backward(const sdm_gdr_shape* shape, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                            const void* v, int64_t v_ld, const void* g, int64_t g_ld, const void* beta, int64_t beta_ld,
                            const void* dy, int64_t dy_ld, const int64_t* offsets, const void* states, const float* dhT,
                            void* dq, int64_t dq_ld, void* dk, int64_t dk_ld, void* dv, int64_t dv_ld, void* dg,
                            int64_t dg_ld, void* dbeta, int64_t dbeta_ld, float* dh0, void* ws, size_t ws_bytes,
                            uint32_t* status, sdm_stream_t stream);

/*
 * One token of each of `rows` requests (P is not used), in float32: state[s] as above, with s = slots[i] (int32 [rows], distinct),
 * or i where slots is NULL. state float32 [states, v_heads * dk * dv] with rows state_ld apart, aligned to 16 bytes. A row with
 * a slot below 0 is padding: y_i = 0 and no state changes; so too one at or above `states`, which sets SDM_DEV_BAD_SLOT.
 */
sdm_status sdm_gdr_step(const sdm_gdr_shape* shape, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                        const void* v, int64_t v_ld, const void* g, int64_t g_ld, const void* beta, int64_t beta_ld,
                        const int32_t* slots, float* state, int64_t state_ld, int64_t states, void* y, int64_t y_ld,
                        uint32_t* status, sdm_stream_t stream);

typedef struct {
    int64_t rows;
    int32_t D;          /* columns of a row, a multiple of 4, up to 16384 */
    int32_t group;      /* columns that the norm behind the block takes together: a multiple of 4 that divides D (D: whole
                         * rows); with very many narrow groups a row does not fit (SDM_ERR_SHAPE): always up to D = 2048 */
    int32_t post;       /* 1: the block's output is normed; 0: taken as it is (w_post unused) */
    int32_t gate;       /* of the block's output: 0 none, 1 sigmoid(z), 2 z sigmoid(z) */
    int32_t residual;   /* 1: x is added */
    int32_t pre;        /* 1: the sum is normed for the next block; 0: not (y, w_pre unused) */
    int32_t dtype;      /* sdm_dtype of all rows */
    float eps;
    float scale;        /* of the gated output */
} sdm_norm_shape;

/*
 * The norms behind and before a block, with its gate and the residual. Per row, in float32:
 *   m = o rsqrt(mean o^2 + eps) w_post over each group (post 0: m = o),   n = m act(z),
 *   r = x + scale channel_scale n, rounded,   y = r rsqrt(mean r^2 + eps) w_pre over the row, of r as it is stored.
 * o, z, x, r, y [rows, D]; w_post float32 [group], the same for every group; w_pre, channel_scale float32 [D] (each nullable: ones). r may
 * be x or o, and y may be o, z or x (same ld).
 */
sdm_status sdm_block_norm(const sdm_norm_shape* shape, const void* o, int64_t o_ld, const void* z, int64_t z_ld, const void* x,
                          int64_t x_ld, const float* w_post, const float* w_pre, const float* channel_scale, void* r,
                          int64_t r_ld, void* y, int64_t y_ld, sdm_stream_t stream);

/*
 * Its backward, from the forward's inputs and its r (which the norm before the next block needs; unused where pre is 0): dr is the
 * gradient of r (nullable where pre is 1: zeros), dy that of y. d_o, dz (gate), dx (nullable: the gradient of the sum, x's and
 * all that came before) [rows, D]; dw_post [group], dw_pre, d_channel_scale [D] float32 (nullable), written, with zeros for what the
 * shape does not have. dx may be dr, dz may be z and d_o may be o (same ld). ws: sdm_block_norm_workspace_bytes, 16-byte aligned
 * (may be NULL where no gradient of a weight that the shape has is asked for).
 */
size_t sdm_block_norm_workspace_bytes(const sdm_norm_shape* shape);
sdm_status sdm_block_norm_backward(const sdm_norm_shape* shape, const void* o, int64_t o_ld, const void* z, int64_t z_ld,
                                   const void* r, int64_t r_ld, const void* dr, int64_t dr_ld, const void* dy, int64_t dy_ld,
                                   const float* w_post, const float* w_pre, const float* channel_scale, void* d_o, int64_t do_ld,
                                   void* dz, int64_t dz_ld, void* dx, int64_t dx_ld, float* dw_post, float* dw_pre,
                                   float* d_channel_scale, void* ws, size_t ws_bytes, sdm_stream_t stream);

typedef struct {
    int64_t tokens;      /* below 2^31 - 2^20 */
    int32_t V;           /* rows of the table, up to 2^28 */
    int32_t D;           /* columns of a row, a multiple of 4, up to 2^20 */
    int32_t table_dtype; /* sdm_dtype of table and dtable */
    int32_t dtype;       /* sdm_dtype of y and dy */
    float scale;
} sdm_embed_shape;

/*
 * y_i = scale table[ids_i], in float32, rounded. ids int32 [tokens]: below 0 is padding (y_i = 0); at or above V likewise, and sets
 * SDM_DEV_BAD_TOKEN. table [V, D], y [tokens, D].
 */
sdm_status sdm_embed(const sdm_embed_shape* shape, const int32_t* ids, const void* table, int64_t table_ld, void* y, int64_t y_ld,
                     uint32_t* status, sdm_stream_t stream);

/*
 * The table's gradient: row v of dtable [V, D] is scale times the sum of dy_i over the tokens with ids_i = v, added in float32 in an order
 * that the ids alone fix, and rounded once. accumulate 0: every row is written (zeros where there is no token); 1: the sum
 * is added to rows that have tokens, the others are not touched. ws: sdm_embed_workspace_bytes, 16-byte aligned.
 */
size_t sdm_embed_workspace_bytes(const sdm_embed_shape* shape);
sdm_status sdm_embed_backward(const sdm_embed_shape* shape, const int32_t* ids, const void* dy, int64_t dy_ld, void* dtable,
                              int64_t dtable_ld, int32_t accumulate, void* ws, size_t ws_bytes, uint32_t* status,
                              sdm_stream_t stream);

/*
 * Synchronizes `stream`, reads the workspace's device status word into *code_out (0 = fine,
 * else SDM_DEV_* bits) and, if `clear`, zeroes it. Returns SDM_ERR_DEVICE when the word is
 * nonzero, SDM_ERR_CUDA when the copy fails.
 */
sdm_status sdm_device_status(const void* ws, int32_t* code_out, int32_t clear, sdm_stream_t stream);

/* A static string naming a status code. */
const char* sdm_status_string(sdm_status status);

#ifdef __cplusplus
}
#endif

#endif /* SDM_H */
