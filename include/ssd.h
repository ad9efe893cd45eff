/*
 * ssd.h -- C ABI of the GB300 (sm_103a) Mamba-2 chunked SSD forward library.
 *
 * The operation (source: "Jane Street ML Engineers Map Mamba-2 Recurrent State
 * Computation to Tensor Cores with cuTile", paragraphs on the fixed-size
 * recurrent state, the jump formula and the three-kernel decomposition): for
 * every batch b and head h, with head h reading group g = h / (nheads/ngroups)
 * of Bm and Cm and the state h_t a headdim x dstate matrix,
 *
 *     h_t = exp(dt_t * A_h) * h_{t-1} + dt_t * x_t b_t^T        (h_{-1} = init_state or 0)
 *     y_t = h_t c_t + D_h * x_t                                  final_state = h_{L-1}
 *
 * computed chunk by chunk (chunk_size tokens) in four kernels: a log-space
 * cumsum of dt*A per chunk, each chunk's state contribution on the tensor
 * cores, a sequential pass over chunks that carries the state (the jump
 * formula with decay), and a fused output kernel (carried-state term, causally
 * masked decayed interaction matrix, D*x skip).
 *
 * Conventions shared by every entry point below:
 *  - Pointers are caller-owned DEVICE memory (CUDA global memory of the current
 *    device), row-major and contiguous, never freed or kept by the library.
 *  - Layouts: x, y [batch][seqlen][nheads][headdim]; dt [batch][seqlen][nheads];
 *    A, D [nheads]; Bm, Cm [batch][seqlen][ngroups][dstate];
 *    init_state, final_state [batch][nheads][headdim][dstate].
 *  - dtype: x, Bm, Cm and y are fp32 (SSD_F32: TF32 tensor-core products with
 *    fp32 accumulation) or bf16 (SSD_BF16: bf16 products, fp32 accumulation,
 *    y rounded to nearest even).  dt, A, D, init_state and final_state are
 *    always fp32.  dt is used as given (post-activation, positive).
 *  - Work is enqueued on `stream` (0 = legacy default stream) and is
 *    asynchronous: no call synchronises.  Calls that share a workspace must be
 *    ordered on one stream.
 *  - Argument errors are reported before anything is enqueued.  CUDA launch
 *    errors return SSD_ERR_CUDA.  Waits inside the kernels are bounded; a wait
 *    that runs out records SSD_ERR_DEVICE_TIMEOUT in the workspace status word,
 *    which ssd_fwd_check() reads after the caller synchronises.  The library
 *    never aborts the process.
 *  - Supported shapes: headdim == 64; dstate in {64, 128, 256};
 *    chunk_size in {64, 128, 256}; nheads % ngroups == 0 and (nheads/ngroups)
 *    even; x, Bm, Cm, y and the workspace 16-byte aligned.  Anything else
 *    returns SSD_ERR_UNSUPPORTED (shape) or SSD_ERR_INVALID_ARG (pointer,
 *    negative size).  batch == 0 or seqlen == 0 is valid (empty input).
 */
#ifndef SSD_GB300_H_
#define SSD_GB300_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* ssd_stream_t; /* same handle as cudaStream_t */

typedef enum {
  SSD_OK = 0,
  SSD_ERR_INVALID_ARG = 1,
  SSD_ERR_UNSUPPORTED = 2,
  SSD_ERR_WORKSPACE = 3,
  SSD_ERR_CUDA = 4,
  SSD_ERR_DEVICE_TIMEOUT = 5
} ssd_status;

typedef enum { SSD_F32 = 0, SSD_BF16 = 1 } ssd_dtype;

typedef struct {
  int64_t batch;      /* B >= 0 */
  int64_t seqlen;     /* L >= 0; need not be a multiple of chunk_size */
  int32_t nheads;     /* H */
  int32_t headdim;    /* P (64) */
  int32_t ngroups;    /* G, divides H */
  int32_t dstate;     /* N */
  int32_t chunk_size; /* Q */
  int32_t dtype;      /* ssd_dtype of x, Bm, Cm, y */
} ssd_shape;

/* Byte offsets of the workspace regions (each 1024-byte aligned).  The
 * workspace is caller-owned scratch; its contents between calls are
 * intermediate results exposed for testing:
 *   status      int32 device status word (0 = OK)
 *   cumsum      fp32 [B][H][nc*Q]  inclusive cumsum of dt*A within each chunk
 *   dt_t        fp32 [B][H][nc*Q]  dt transposed to head-major order (0 past L)
 *   states      [B][nc][H][P][N] chunk states S_c, fp32 for SSD_F32 and bf16
 *               for SSD_BF16; after the state pass, for SSD_F32 the state
 *               entering each chunk (in place)
 *   states_bf16 bf16 [B][nc][H][P][N]  (SSD_BF16 only) state entering each
 *               chunk, rounded to bf16 for the output kernel's tensor cores
 *   chain       int32 [1 + B*H/2]  one-pass kernel: tile counter, then per
 *               (batch, head pair) the number of windows whose state is
 *               published (cleared by the call's first kernel)
 *   hslot       fp32, B*H*P*N values  one-pass kernel: the state handed from
 *               one run of windows to the next, per head pair in a layout of
 *               its own ([N/32][8][2*P rows][4]: a warp's 16-byte accesses are
 *               consecutive)
 *   cbm         (SSD_BF16 only) bf16 [B][nw][G][128][128], nw = ceil(seqlen/128):
 *               for every 128-token window and group the causal select of
 *               C B^T, M[i][j] = c_i . b_j for j <= i and 0 above the
 *               diagonal (one-pass schedule, written by its first step)
 * nc = ceil(seqlen / chunk_size), Lp = nc * chunk_size. */
typedef struct {
  size_t status;
  size_t cumsum;
  size_t dt_t;
  size_t states;
  size_t states_bf16;
  size_t chain;
  size_t hslot;
  size_t cbm;
  size_t total;
} ssd_workspace_layout;

/* Human-readable name of a status code (static storage; never NULL). */
const char* ssd_status_string(ssd_status s);

/* Checks the shape (see "Supported shapes") without touching memory. */
ssd_status ssd_validate_shape(const ssd_shape* shape);

/* Workspace regions for `shape`; returns SSD_OK or the shape error. */
ssd_status ssd_fwd_workspace_layout(const ssd_shape* shape, ssd_workspace_layout* out);

/* Bytes of device workspace ssd_fwd needs for `shape` (0 if the shape is
 * invalid or unsupported). */
size_t ssd_fwd_workspace_size(const ssd_shape* shape);

/* The whole forward pass, enqueued on `stream`.  Three schedules give the
 * recurrence's result (see the steps below for the formulas):
 *  - one-pass (ssd_fwd_fused; SSD_BF16 only): ssd_causal_cb, then one
 *    persistent kernel (ssd_fused_pass) that runs every 128-token window of a
 *    (batch, head pair): the window's cumulative decay, its state product on
 *    the tensor core accumulated onto the running state, the carried-state
 *    and intra-window products and y; the state moves between windows in
 *    tensor memory and between runs of windows through the workspace (or
 *    final_state).  x is read once and the states never reach HBM.
 *  - staged: chunk_state (which forms each chunk's cumsum itself, exactly as
 *    chunk_cumsum does, and writes the cumsum and dt_t rows), state_passing and
 *    compute_out.
 *  - segmented one-pass (SSD_BF16 only): chunk_cumsum, chunk_state and
 *    state_passing with segments of 2048 (or 1024) tokens as their chunk,
 *    which leaves every segment's entering state (fp32) in the workspace and
 *    writes final_state, then the one-pass pair on the sequences' segments
 *    taken as a batch of one-segment sequences, each from its entering state.
 * ssd_fwd takes the one-pass schedule for SSD_BF16 when there are at least as
 * many (batch, head pair) sequences as multiprocessors (below that the chain
 * of windows, not bandwidth, bounds the one-pass kernel); below that, the
 * segmented one when the segments divide the sequence and give at least two
 * per multiprocessor over all pairs; otherwise the staged one (always for
 * SSD_F32).  The one-pass schedules work in windows of 128
 * tokens whatever chunk_size is; the result is the recurrence's either way.
 * init_state may be NULL (zero initial state); final_state
 * may be NULL (not written; the workspace holds the running state instead).
 * When given, final_state is also the running state's storage during the
 * call, so it must not overlap the inputs (it may equal init_state).  The
 * workspace must hold ssd_fwd_workspace_size(shape) bytes. */
ssd_status ssd_fwd(const ssd_shape* shape, const void* x, const float* dt, const float* A,
                   const void* Bm, const void* Cm, const float* D, const float* init_state, void* y,
                   float* final_state, void* workspace, size_t workspace_bytes, ssd_stream_t stream);

/* ssd_fwd forced onto the one-pass schedule (same arguments and contract).
 * SSD_ERR_UNSUPPORTED unless shape->dtype is SSD_BF16. */
ssd_status ssd_fwd_fused(const ssd_shape* shape, const void* x, const float* dt, const float* A,
                         const void* Bm, const void* Cm, const float* D, const float* init_state, void* y,
                         float* final_state, void* workspace, size_t workspace_bytes, ssd_stream_t stream);

/* Step 1 of the one-pass schedule alone ("Jane Street ML Engineers Map Mamba-2
 * Recurrent State Computation to Tensor Cores with cuTile", compute_out
 * paragraph: C B^T by one matrix product, causal mask made in registers):
 * writes the workspace's cbm region, the causal select of C B^T in bf16 for
 * every (batch, 128-token window, group), shared by every head of the group;
 * also clears the status word and the one-pass run counter and flags.
 * SSD_BF16 only (SSD_ERR_UNSUPPORTED otherwise). */
ssd_status ssd_causal_cb(const ssd_shape* shape, const void* Bm, const void* Cm, void* workspace,
                         size_t workspace_bytes, ssd_stream_t stream);

/* Step 2 of the one-pass schedule alone (ssd_fwd_fused is ssd_causal_cb
 * followed by this call): the persistent kernel described under ssd_fwd.
 * Needs step 1.  SSD_BF16 only (SSD_ERR_UNSUPPORTED otherwise); arguments as
 * for ssd_fwd. */
ssd_status ssd_fused_pass(const ssd_shape* shape, const void* x, const float* dt, const float* A, const void* Bm,
                          const void* Cm, const float* D, const float* init_state, void* y, float* final_state,
                          void* workspace, size_t workspace_bytes, ssd_stream_t stream);

/* The launches ssd_fwd makes for `shape`, numbered 0 .. ssd_fwd_kernel_count()-1
 * in the order ssd_fwd enqueues them, restricted to those with index in
 * [first_launch, end_launch): the same kernels with the same arguments, so
 * that calls covering consecutive ranges on one stream compute exactly what
 * one ssd_fwd call computes.  Inside one call a launch overlaps the tail of
 * the launch before it as in ssd_fwd; the first launch of a call waits for
 * the work already on the stream.  Used to time the schedule's kernels one by
 * one with events between the calls.  Arguments as for ssd_fwd;
 * SSD_ERR_INVALID_ARG if first_launch < 0 or end_launch < first_launch. */
ssd_status ssd_fwd_range(const ssd_shape* shape, const void* x, const float* dt, const float* A,
                         const void* Bm, const void* Cm, const float* D, const float* init_state, void* y,
                         float* final_state, void* workspace, size_t workspace_bytes, int first_launch,
                         int end_launch, ssd_stream_t stream);

/* After the caller has synchronised the stream of a call that used
 * `workspace`: SSD_OK, or SSD_ERR_DEVICE_TIMEOUT if a bounded wait inside a
 * kernel ran out (its outputs are then invalid).  Blocking 4-byte read. */
ssd_status ssd_fwd_check(const void* workspace);

/* --- The four steps, callable one by one (for SSD_F32, ssd_fwd computes
 * exactly what these four calls in order compute -- its chunk_state launch
 * forms the step-1 rows itself; for SSD_BF16 the four calls in order give the
 * same result as ssd_fwd through the staged path).  Each reads and writes the
 * workspace regions named. ---- */

/* Step 1 (page 1, chunk_cumsum): cumsum[b][h][cQ+i] = sum_{k<=i} dt*A over the
 * chunk, dt_t = dt transposed; tokens past seqlen contribute 0.  Also clears
 * the status word. */
ssd_status ssd_chunk_cumsum(const ssd_shape* shape, const float* dt, const float* A, void* workspace,
                            size_t workspace_bytes, ssd_stream_t stream);

/* Step 2 (page 1, jump formula with decay; fwd_pass_state's per-chunk MMA):
 * states[b][c][h][p][n] = sum_{j in chunk c} exp(G_last - G_j) dt_j x_j[p] b_j[n]
 * on the tensor cores (tcgen05, accumulator in tensor memory, operands staged
 * by TMA).  Needs step 1. */
ssd_status ssd_chunk_state(const ssd_shape* shape, const void* x, const void* Bm, void* workspace,
                           size_t workspace_bytes, ssd_stream_t stream);

/* Step 3 (page 1, fwd_pass_state's sequential loop over chunks): with
 * h = init_state (or 0), for c = 0..nc-1: entering_c = h;
 * h = exp(G_last_c) h + S_c.  Writes the entering states (see the layout) and
 * final_state = h (if not NULL).  Needs steps 1-2. */
ssd_status ssd_state_passing(const ssd_shape* shape, const float* init_state, float* final_state,
                             void* workspace, size_t workspace_bytes, ssd_stream_t stream);

/* Step 4 (page 1, compute_out): y_i = exp(G_i) C_i h_entering^T
 *   + sum_{j<=i in chunk} (C_i . B_j) exp(G_i - G_j) dt_j x_j + D_h x_i,
 * one fused tile kernel on the tensor cores; the causal mask is made in
 * registers and the chunk_size x chunk_size matrix never reaches global
 * memory.  Needs steps 1-3. */
ssd_status ssd_compute_out(const ssd_shape* shape, const void* x, const void* Bm, const void* Cm,
                           const float* D, void* y, void* workspace, size_t workspace_bytes,
                           ssd_stream_t stream);

/* Test hook for the failure path: enqueues one block that waits, for at most
 * `limit_us` microseconds, on a barrier nothing arrives at, then records
 * SSD_ERR_DEVICE_TIMEOUT in the workspace status word and exits (no trap, no
 * hang).  The workspace needs at least 4 bytes. */
ssd_status ssd_debug_timeout_probe(void* workspace, uint32_t limit_us, ssd_stream_t stream);

/* Number of kernels ssd_fwd enqueues for `shape` (0 for an empty input): 2
 * on the one-pass schedule, 5 on the segmented one and 3 on the staged one. */
int ssd_fwd_kernel_count(const ssd_shape* shape);

/* Bytes of the device array that ssd_fwd_static_scratch uses as its workspace. */
#define SSD_STATIC_SCRATCH_BYTES ((size_t)32 << 20)

/* ssd_fwd for callers that may not allocate device memory.  The pages describe
 * no counterpart: this is a service of the library, not a step of the method.
 *
 * Who needs it: code that runs inside a host which owns all device memory
 * (a plugin of another runtime with its own pool), serving processes that
 * allow no allocation after start-up, and any caller for whom a cudaMalloc
 * on the hot path is not allowed or too risky (it can stall the device and
 * can fail under memory pressure).  Such a caller passes only the inputs and
 * outputs of ssd_fwd; the workspace is a fixed array of
 * SSD_STATIC_SCRATCH_BYTES in the library's own device data, which every GPU
 * that loads the library holds until the process exits.  The call itself
 * allocates nothing.  Under lazy module loading (the CUDA default) the
 * array's memory is committed when the library's device code first loads on
 * a device, which is at the latest this entry point's first call there; make
 * that first call at start-up (where an out-of-memory error can still be
 * handled) and before any stream capture.
 *
 * Arguments, layouts, dtypes and supported shapes are those of ssd_fwd.
 * Returns SSD_ERR_WORKSPACE, before enqueuing anything, when
 * ssd_fwd_workspace_size(shape) is larger than SSD_STATIC_SCRATCH_BYTES.
 * The first call on a device also looks up the array's device address
 * (cudaGetSymbolAddress) for that device; this set-up is one more reason to
 * make it before any stream capture.  Argument errors are returned before
 * anything is enqueued.
 * A non-empty call's first kernel clears the status word and the one-pass
 * counters before the rest of the array is overwritten; the array keeps the
 * last call's intermediate results.
 * All calls share the one array: calls whose GPU work can overlap in time
 * (different streams, or threads without ordering between them) race and
 * give wrong results.  A device-timeout status (see ssd_fwd_check) is left in
 * the array and cannot be read through this entry point. */
ssd_status ssd_fwd_static_scratch(const ssd_shape* shape, const void* x, const float* dt, const float* A,
                                  const void* Bm, const void* Cm, const float* D, const float* init_state,
                                  void* y, float* final_state, ssd_stream_t stream);

/* ===========================================================================
 * The layer around ssd_fwd, for serving: the short causal convolution in front
 * of it, the selective scan (a decay per channel and state instead of one per
 * head), the single-token form of both recurrences, the gated delta rule,
 * products of a few tokens with 4-bit weights, beam search's selection and
 * reordering of states, and the verification of drafted tokens.
 * The pages describe none of these; the formulas are stated with each call.
 *
 * Each call takes one argument struct.  Its first field is the struct's own
 * size (a caller compiled against another layout gets SSD_ERR_INVALID_ARG).
 * Strides are in elements.  "rows" are tensors whose innermost dimension is
 * contiguous and whose other strides are free (a slice of a projection's
 * output); every other tensor is contiguous.  Tensors are aligned to their
 * element; 16-byte alignment of data and strides is faster, never required
 * (except where a call says so).  The conventions above hold otherwise:
 * device pointers, work enqueued on `stream`, argument errors before anything
 * is enqueued, nothing allocated or kept.
 *
 * State caches hold `nslots` rows; sequence b uses row slots[b] (row b where
 * slots is NULL).  The rows of one call must differ.  A sequence whose row
 * lies outside [0, nslots) is idle: its outputs are 0 and no cache row is
 * read or written for it.
 *
 * A convolution's cache is a ring of `width` tokens: [nslots][width][channels],
 * where slot q holds the input of the sequence's newest token t with
 * t mod width == q.  Tokens before a sequence's first are 0 whatever the ring
 * holds, so a ring needs no clearing. */

typedef enum { SSD_ACT_NONE = 0, SSD_ACT_SILU = 1 } ssd_activation;

/* y[b][t][c] = act(bias[c] + sum_{j < width} weight[c][j] * u[b][t - width + 1 + j][c])
 * for the tokens t < lengths[b], 0 for those after them; inputs before the
 * call's first token come from the ring.  The output is split by channel over
 * up to three tensors, so that x, Bm and Cm land where ssd_fwd reads them. */
typedef struct {
  int64_t size;              /* sizeof(ssd_conv_args) */
  int64_t batch, seqlen;     /* >= 0; batch <= 65535, seqlen <= 2^30 */
  int64_t nslots;            /* rows of the ring; >= batch where slots is NULL */
  int32_t channels, width;   /* width 2, 3 or 4 */
  int32_t dtype, activation; /* of u, ring and out; ssd_activation */
  int32_t nout;              /* 1..3 */
  int32_t out_channels[3];   /* channels of each output; they add up to `channels` */
  const void* u;             /* rows [batch][seqlen][channels] */
  int64_t u_batch, u_token;  /* strides */
  const float* weight;       /* [channels][width] */
  const float* bias;         /* [channels] or NULL */
  const void* ring;          /* or NULL: nothing came before, nothing is kept */
  void* new_ring;            /* the ring after the call, written in the rows of this call's sequences alone;
                              * NULL: `ring` is updated in place */
  const int32_t* positions;  /* [batch] tokens before this call; NULL: 0 */
  const int32_t* lengths;    /* [batch] tokens of this call, taken into [0, seqlen]; NULL: seqlen */
  const int32_t* slots;      /* [batch] or NULL */
  void* out[3];              /* [batch][seqlen][out_channels[i]] */
} ssd_conv_args;

ssd_status ssd_conv_fwd(const ssd_conv_args* args, ssd_stream_t stream);

/* The selective scan.  With d = delta + delta_bias, put through softplus where
 * `softplus` is set, and channel c in group g = c / (channels / ngroups):
 *     h_t[c][n] = exp(d_t[c] * A[c][n]) * h_{t-1}[c][n] + d_t[c] * u_t[c] * Bm_t[g][n]
 *     y_t[c] = (sum_n h_t[c][n] * Cm_t[g][n] + D[c] * u_t[c]) * silu(z_t[c])
 * for t < lengths[b]; y is 0 after that and the state stays.  State, decay and
 * sums are 32 bits.  seqlen 1 is the single-token form; final_state may be
 * init_state (updated in place).  Long sequences with few channels are cut
 * into segments that run side by side, which takes the workspace. */
typedef struct {
  int64_t size;
  int64_t batch, seqlen; /* batch <= 65535 */
  int32_t channels, dstate, ngroups, dtype; /* dstate 1..64; ngroups divides channels */
  int32_t softplus, reserved;
  const void *u, *delta, *z, *Bm, *Cm; /* rows [batch][seqlen][...]; z may be NULL */
  int64_t u_batch, u_token, delta_batch, delta_token, z_batch, z_token;
  int64_t B_batch, B_token, C_batch, C_token; /* Bm, Cm [..][ngroups][dstate], the last two contiguous */
  const float* A;          /* [channels][dstate] */
  const float* D;          /* [channels] or NULL (0) */
  const float* delta_bias; /* [channels] or NULL (0) */
  const float* init_state; /* [batch][channels][dstate] or NULL (0) */
  float* final_state;      /* the same shape, or NULL */
  void* y;                 /* [batch][seqlen][channels] */
  const int32_t* lengths;  /* [batch] or NULL */
  void* workspace;         /* 16-byte aligned */
  size_t workspace_bytes;
} ssd_selective_scan_args;

/* Bytes of workspace on the current device (0 where none is needed or the sizes
 * are refused); only batch, seqlen, channels, dstate and ngroups are read. */
size_t ssd_selective_scan_workspace_size(const ssd_selective_scan_args* args);
ssd_status ssd_selective_scan(const ssd_selective_scan_args* args, ssd_stream_t stream);

/* Test hook: ssd_selective_scan, but where a sequence is shared by two blocks
 * the state that one hands to the other does not arrive (`taken` not 0: the
 * first is also told that the second has taken the sequence over).  After a
 * bounded wait the second computes the sequence alone: the results are
 * ssd_selective_scan's, bit for bit. */
ssd_status ssd_debug_scan_handover(const ssd_selective_scan_args* args, int32_t taken, ssd_stream_t stream);

/* One token of a Mamba-2 layer's convolution and recurrence, for every
 * sequence of a batch: x, Bm, Cm = silu(convolution of u and the ring), the
 * ring takes u, and with d = dt + dt_bias (through softplus where set)
 *     h = exp(d * A_h) * h + d * x b^T,   y = (h c + D_h * x) * silu(z).
 * The continuation of ssd_conv_fwd and ssd_fwd: state is ssd_fwd's final_state. */
typedef struct {
  int64_t size;
  int64_t batch, nslots; /* batch <= 65535 */
  int32_t nheads, headdim, ngroups, dstate; /* headdim 64; dstate 64, 128 or 256 */
  int32_t width, dtype;  /* of u, z, ring and y */
  int32_t dt_dtype, softplus;
  const void *u, *z, *dt; /* rows [batch][nheads*headdim + 2*ngroups*dstate], [batch][nheads*headdim] or NULL, [batch][nheads] */
  int64_t u_batch, z_batch, dt_batch;
  const float* weight;  /* [nheads*headdim + 2*ngroups*dstate][width] */
  const float* bias;    /* or NULL */
  const float* A;       /* [nheads] */
  const float* D;       /* [nheads] */
  const float* dt_bias; /* [nheads] or NULL */
  void* ring;           /* [nslots][width][...], updated in place; a row has fewer than 2^31 elements */
  const float* state;   /* [nslots][nheads][headdim][dstate], 16-byte aligned */
  float* new_state;     /* the state after the token; NULL: updated in place */
  const int32_t* positions; /* [batch] tokens before this one */
  const int32_t* slots;     /* [batch] or NULL */
  void* y;                  /* [batch][nheads][headdim] */
} ssd_step_args;

ssd_status ssd_step(const ssd_step_args* args, ssd_stream_t stream);

/* y[m][n] = sum_k x[m][k] * (q[n][k] - 8) * scales[n][k / group] (+ add[m][n]),
 * q the 4-bit codes, for a few tokens m.  Codes are packed in tiles of 16 rows
 * and 64 columns, [ceil(n/16)][ceil(k/64)][32 lanes][4 words], codes outside
 * the matrix 8: lane 4 r + c, word 2 h + i holds, at bit 4 (a + 2 e) + 16 p,
 * row 8 a + r and column 32 h + 8 c + 4 i + 2 e + p of its tile
 * (r < 8, c < 4, h, i, a, e, p < 2).  Products and sums are 32 bits: bf16 x
 * enters exactly, fp32 x as the exact sum of three bf16 parts. */
typedef struct {
  int64_t size;
  int64_t tokens; /* 0..65535 */
  int32_t n, k, group, dtype; /* n, k <= 2^30; group 32, 64 or 128; dtype of x, add and y */
  const void* x;  /* rows [tokens][k] */
  int64_t x_token;
  const void* packed; /* 16-byte aligned */
  const float* scales; /* [n][ceil(k/group)] */
  const void* add;     /* rows [tokens][n] or NULL */
  int64_t add_token;
  void* y; /* [tokens][n] */
  void* workspace; /* 16-byte aligned */
  size_t workspace_bytes;
} ssd_w4_matvec_args;

/* Bytes of workspace: for 32-bit x and for rows of x that are not 16-byte
 * vectors (0 otherwise, or where the sizes are refused); tokens, k, n, group,
 * dtype, x and x_token are read. */
size_t ssd_w4_matvec_workspace_size(const ssd_w4_matvec_args* args);
ssd_status ssd_w4_matvec(const ssd_w4_matvec_args* args, ssd_stream_t stream);

/* Beam search's choice.  Candidate (w, v) has the score
 *     scores[b][w] + (logits[b][w][v] - log sum_v' exp(logits[b][w][v'])),
 * a NaN counting as -infinity; a finished beam has one candidate that is not
 * -infinity, (w, eos), at scores[b][w].  Writes the k best per b in falling
 * order, equal scores by rising w * vocab + v: their scores, beams and tokens.
 * k in 1..64, k <= beams * vocab, beams in 1..64, beams * vocab < 2^31. */
typedef struct {
  int64_t size;
  int64_t batch; /* <= 65535 */
  int32_t beams, vocab, k, dtype; /* of logits */
  int32_t eos, reserved;
  const void* logits; /* rows [batch][beams][vocab] */
  int64_t logits_batch, logits_beam;
  const float* scores;     /* [batch][beams] */
  const uint8_t* finished; /* [batch][beams], not 0: finished; or NULL */
  float* out_scores;       /* [batch][k] */
  int32_t *parents, *tokens;
  void* workspace; /* 16-byte aligned */
  size_t workspace_bytes;
} ssd_beam_select_args;

/* Bytes of workspace on the current device; only batch, beams, vocab, k are read. */
size_t ssd_beam_select_workspace_size(const ssd_beam_select_args* args);
ssd_status ssd_beam_select(const ssd_beam_select_args* args, ssd_stream_t stream);

/* new row (b, i) = old row (b, parents[b][i]) of every tensor: dst[j] is
 * [batch][k][row_bytes[j]], src[j] [batch][beams][row_bytes[j]].  dst[j] may
 * be src[j] (then k == beams, and rows that stay are not moved); they must not
 * overlap otherwise.  A parent outside [0, beams) leaves its row unwritten. */
#define SSD_REORDER_MAX 16
typedef struct {
  int64_t size;
  int64_t batch;
  int32_t beams, k, count, reserved; /* k, beams in 1..64; count <= SSD_REORDER_MAX */
  const int32_t* parents; /* [batch][k] */
  const void* src[SSD_REORDER_MAX];
  void* dst[SSD_REORDER_MAX];
  int64_t row_bytes[SSD_REORDER_MAX];
} ssd_beam_reorder_args;

ssd_status ssd_beam_reorder(const ssd_beam_reorder_args* args, ssd_stream_t stream);

/* The gated delta rule: the recurrence of ssd_fwd, but what the state already
 * returns for the key b_t = Bm_t is taken off the value before it is written:
 *     h' = exp(dt_t * A_h) * h_{t-1}
 *     h_t = h' + beta_t * (x_t - h' b_t) b_t^T,      y_t = scale * h_t c_t
 * for t < lengths[b]; y is 0 after that and the state stays.  Head h reads group
 * h / (nheads/ngroups) of Bm and Cm.  dt is dt + dt_bias, through softplus where
 * set; beta goes through a sigmoid where set; with norm_eps >= 0 every row v of
 * Bm and Cm counts as v / sqrt(|v|^2 + norm_eps) (a row of zeros as zeros).
 * State, decay and sums are 32 bits.  Any seqlen: whole prompts, a few drafted
 * tokens, single tokens.  Sequence b's state is row slots[b] (as for the caches
 * above) of init_state and final_state, which may be one tensor, updated in
 * place, and must not overlap otherwise; a sequence at position 0 starts from 0
 * whatever its row holds.  Rows of final_state that no sequence of the call has
 * stay as they are; outputs must not overlap the inputs otherwise.
 * Calls of 32 tokens or more with a dstate of 64 or 128 run in chunks of 64
 * tokens on the tensor cores.  Their products keep 22 bits of every factor (11
 * where only a bf16 y takes them), or 2^-38 of the largest of a chunk's tokens in
 * 32 channels: the state is off by 5e-7 of its norm.  There a value of x or
 * init_state that is not finite makes its own channel NaN, from the first of its
 * 64 tokens on, and no other; one of Bm, Cm, dt or beta may do so to all of a
 * head that reads it; and with dt A above 0 its sums over 64 tokens must not pass
 * 88, where exp leaves 32 bits.  Fewer tokens, and a dstate of 256, go one by one. */
typedef struct {
  int64_t size;
  int64_t batch, seqlen;    /* batch <= 65535, seqlen <= 2^30 */
  int64_t nslots;           /* rows of the states; >= batch where slots is NULL */
  int32_t nheads, headdim, ngroups, dstate; /* headdim a multiple of 16, <= 1024; dstate 64, 128 or 256 */
  int32_t dtype, gate_dtype; /* of x, Bm, Cm, y; of dt and beta (dtype or SSD_F32) */
  int32_t dt_softplus, beta_sigmoid;
  float scale, norm_eps;    /* finite; norm_eps < 0: Bm and Cm as they are */
  const void *x, *Bm, *Cm;  /* [batch][seqlen][nheads][headdim], [..][ngroups][dstate], the last two dimensions contiguous */
  int64_t x_batch, x_token, B_batch, B_token, C_batch, C_token;
  const void *dt, *beta;    /* rows [batch][seqlen][nheads] */
  int64_t dt_batch, dt_token, beta_batch, beta_token;
  const float* A;           /* [nheads] */
  const float* dt_bias;     /* [nheads] or NULL (0) */
  const float* init_state;  /* [nslots][nheads][headdim][dstate] or NULL (0), 16-byte aligned */
  float* final_state;       /* the same shape, or NULL, 16-byte aligned */
  const int32_t* slots;     /* [batch] or NULL */
  const int32_t* positions; /* [batch] tokens before this call; NULL: every sequence has a state */
  const int32_t* lengths;   /* [batch] tokens of this call, taken into [0, seqlen]; NULL: seqlen */
  void* y;                  /* [batch][seqlen][nheads][headdim] */
  void* workspace;          /* 16-byte aligned */
  size_t workspace_bytes;
} ssd_delta_args;

/* Bytes of workspace on the current device: for calls that run in chunks (0
 * otherwise, or where the sizes are refused); the sizes and dtype are read, no
 * tensor.  1 GiB at most, and the states of the sequences that fit in that (with
 * thousands of heads two chunks of all of one sequence's, some 50 KB a head each
 * in bf16, 115 in fp32).  A wait in these calls' kernels that runs out (see above) leaves NaN
 * in the outputs of its head. */
size_t ssd_delta_workspace_size(const ssd_delta_args* args);
ssd_status ssd_delta_fwd(const ssd_delta_args* args, ssd_stream_t stream);

/* Verification of drafted tokens (speculative decoding).  With p_i and q_i the
 * softmax of scale[b] * logits[b][i] and scale[b] * draft_logits[b][i] (without
 * draft_logits, all of q_i is at the drafted token: a draft that was looked up),
 * draft i is accepted while uniforms[b][i] * q_i(draft_i) < p_i(draft_i).  Let n
 * be the first that is not, or lengths[b].  Then one token is drawn from
 * max(p_n - q_n, 0) (from p_n where n is lengths[b], or where nothing is left of
 * the difference): the first v whose sum up to v is above uniforms[b][drafts]
 * times the sum of all.  tokens[b] = the n accepted drafts, that token, then -1;
 * accepted[b] = n; logprobs = log p of each token, 0 beside a -1.  n + 1 is the
 * number of tokens to commit where the model has run on the last token and the
 * drafts: the `lengths` of ssd_conv_fwd, ssd_selective_scan and ssd_delta_fwd.
 * The drawn token is that of 64-bit arithmetic, up to numbers within 2^-34 of a
 * token's border.  Drafts are accepted in 32 bits: a number within 2^-20 of the
 * border p_i / q_i, relatively (and 2^-24 of the scaled logits' distances from
 * their rows' largest, if that is more), may fall either way, and what is left of
 * p_n - q_n counts as nothing where it may be below 2^-20 in all.  Log-probabilities
 * are off by 2^-20, relatively or absolutely.
 * A NaN logit counts as -infinity; a row with +infinity is shared by its
 * infinities.  A drafted token outside the vocabulary is not accepted, and
 * nothing is taken off p for it.  Where the target's row allows no token, or
 * scale[b] is not above 0 and at most 1e37 (then n is 0), -1 is drawn. */
typedef struct {
  int64_t size;
  int64_t batch; /* <= 65535 */
  int32_t drafts, vocab, dtype, reserved; /* drafts 0..64; vocab <= 2^19; dtype of both logits */
  const void* logits;       /* rows [batch][drafts + 1][vocab] */
  int64_t logits_batch, logits_row;
  const void* draft_logits; /* rows [batch][drafts][vocab] or NULL */
  int64_t draft_logits_batch, draft_logits_row;
  const int32_t* draft;     /* [batch][drafts] */
  const float* uniforms;    /* [batch][drafts + 1], in [0, 1) */
  const float* scale;       /* [batch] or NULL (1): the inverse of the temperature */
  const int32_t* lengths;   /* [batch] drafts of each sequence, taken into [0, drafts]; NULL: drafts */
  int32_t* tokens;          /* [batch][drafts + 1] */
  int32_t* accepted;        /* [batch] */
  float* logprobs;          /* [batch][drafts + 1] */
  void* workspace;          /* 16-byte aligned */
  size_t workspace_bytes;
} ssd_draft_verify_args;

/* Bytes of workspace on the current device; batch, drafts, vocab, dtype and whether draft_logits is NULL are read. */
size_t ssd_draft_verify_workspace_size(const ssd_draft_verify_args* args);
ssd_status ssd_draft_verify(const ssd_draft_verify_args* args, ssd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_GB300_H_ */
