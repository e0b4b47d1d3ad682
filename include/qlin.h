/*
 * qlin -- skinny W4A8 / W6A8 quantized linear for GB300 (sm_103a).
 *
 *   y[M, N] = s_m * sum_g sw[n, g] * sum_{k in group g} q[m, k] * level[n, k]
 *
 * for M = 1..8 rows (one decoded token plus up to seven multi-token-prediction
 * drafts), with level = code - 2^(b-1) from b = 4 or 6 bit weight codes, fp32
 * group scales sw, and q = per-row int8 quantisation of the activation, which
 * is x itself, RMSNorm(x) or silu(gate) * up.
 *
 * Sources (page title, section):
 *  [LIN]  "Doubling the LLM token rate in ComfyUI", section "Optimising the
 *         linear kernel": skinny GEMV for M = 1 and thin MTP verification M;
 *         weights and per-group scales interleaved in the order the kernel
 *         reads them, rearranged once per model load in place in VRAM; the M
 *         rows mapped onto the 8-wide side of a tensor-core MMA so that up to
 *         eight rows cost about what one row costs; the activation
 *         quantisation absorbs the RMSNorm or SwiGLU in front of it.
 *  [BOT]  same page, section "What is the bottleneck?": every token reads
 *         every weight once, so decode speed is VRAM read speed.
 *  [MTP]  same page, section "Adaptive-tree MTP": verification carries at
 *         most eight rows (one committed token plus seven drafts).
 *  [FMT]  "Comfy Quantization Formats", section "Weight formats": N output
 *         width, K input width, G group size, FP32 scales.
 *  [OPT]  same page, section "Format options": asym_w4a8_int8 (uniform levels
 *         without a codebook) and w6a8_int8; symmetric weights; grouped W4A8
 *         needs K % 16 == 0, K % G == 0, G >= 4 and (16 % G == 0 or
 *         G % 16 == 0); W6A8 needs K % 32 == 0 and G % 16 == 0; backends may
 *         restrict shapes further.
 *  [ACT]  same page, section "Activations and smoothing": integer formats take
 *         float activations and quantise them inside the kernel; no stored
 *         input scale.
 *
 * Conventions for every entry point:
 *  - All buffer pointers are DEVICE pointers owned by the caller; the library
 *    never allocates, frees or synchronises (except qlin_read_device_status).
 *  - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is the
 *    legacy default stream) on the current device.
 *  - Argument and shape errors are returned before anything is enqueued.
 *    Launch failures return QLIN_ERR_CUDA.  A device-side bounded wait that
 *    expires writes QLIN_ERR_DEVICE_TIMEOUT into the workspace status word,
 *    read back by qlin_read_device_status; the kernel returns instead of
 *    hanging.
 *  - fmt is QLIN_W4A8 or QLIN_W6A8; b = 4 or 6 bits per code.
 *  - Backend limits beyond [OPT] (QLIN_ERR_UNSUPPORTED): G in {4, 8, 16, 32,
 *    64, 128, 256} (4 and 8 for 4-bit codes, as the format allows),
 *    K % 32 == 0, N % 16 == 0, K <= 65536 (K <= 57344 for G = 4, whose
 *    per-group start values fill the shared memory of 16 CTAs first), M <= 8.
 */
#ifndef QLIN_H_
#define QLIN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QLIN_OK = 0,
  QLIN_ERR_INVALID_ARG = 1,    /* bad pointer, alignment, size, or a shape [OPT] forbids */
  QLIN_ERR_UNSUPPORTED = 2,    /* legal per [OPT] but outside this backend's limits */
  QLIN_ERR_CUDA = 3,           /* a CUDA runtime call or launch failed */
  QLIN_ERR_DEVICE_TIMEOUT = 4, /* a device-side bounded wait expired (status word) */
  QLIN_ERR_WORKSPACE = 5,      /* workspace smaller than the size query returned */
  QLIN_ERR_BAD_INDEX = 6       /* a device-side index (page, kept row) was out of range (status word) */
} qlin_status;

typedef enum { QLIN_W4A8 = 0, QLIN_W6A8 = 1 } qlin_format;

typedef enum {
  QLIN_PROLOGUE_NONE = 0,    /* a = x */
  QLIN_PROLOGUE_RMSNORM = 1, /* a = x * gamma / sqrt(mean(x^2) + eps) */
  QLIN_PROLOGUE_SWIGLU = 2   /* a = gate / (1 + exp(-gate)) * up */
} qlin_prologue;

/* qlin_forward flags. */
#define QLIN_FLAG_PDL 1u /* Launch with programmatic dependent launch: the kernel may start
                            streaming `packed` and reading `gamma` while earlier kernels in
                            `stream` still run.  The caller asserts that neither was written
                            by any kernel still in flight in `stream` (true for model
                            weights repacked at load time and for norm weights).
                            Activations, y and the workspace are still touched only after
                            earlier kernels complete. */

/* Library version string. */
const char* qlin_version(void);

/* Human-readable name of a status code (static storage). */
const char* qlin_status_string(qlin_status s);

/* Validate a weight shape against [OPT] and the backend limits.  Host only.
 * Returns QLIN_OK, QLIN_ERR_INVALID_ARG or QLIN_ERR_UNSUPPORTED. */
qlin_status qlin_check_shape(int fmt, int64_t N, int64_t K, int64_t G);

/* Bytes of one quantized weight, in either layout: N*K*b/8 code bytes plus
 * N*(K/G)*4 scale bytes [FMT].  0 when qlin_check_shape fails. */
size_t qlin_packed_bytes(int fmt, int64_t N, int64_t K, int64_t G);

/*
 * In-place repack [LIN]: rewrites `buf` from the checkpoint layout into the
 * kernel-order stream that qlin_forward reads.  Same size in and out
 * (qlin_packed_bytes).  One call per weight, once per load; calling it twice
 * does not give the same bytes as calling it once.
 *
 * Checkpoint layout (input): codes, then scales.
 *   4-bit: uint8 [N, K/2], low nibble = even k.  6-bit: uint8 [N, 3K/4], each 3
 *   bytes a little-endian 24-bit word holding 4 codes, code i at bits 6i..6i+5.
 *   Scales: fp32 [N, K/G] row-major, little-endian, right after the codes.
 * Stream layout (output), KB = max(128, G):
 *   tiles of 128 output rows (the last may hold fewer, a multiple of 16), in
 *   order; inside a tile, units of KB input columns (the last may be
 *   narrower), in order; a unit of R rows and W columns is
 *     scale block  R*(W/G) fp32: for each group of the unit, for each 16-row
 *                  slab, for p = 0..7: sw[row p], sw[row p + 8];
 *     code block   for each slab, for each pair of 16-wide k-steps:
 *                  4-bit plane: 32 lanes x {word for step A, word for step B};
 *                  6-bit codes only, then the 2-bit plane: 32 lanes x 1 word.
 *   A lane (g, t) = (lane / 4, lane % 4) holds the A operand of a 16x16 fp16
 *   tensor-core tile: register i in 0..3 holds (row g, k 2t..2t+1),
 *   (row g+8, k 2t..2t+1), (row g, k 2t+8..2t+9), (row g+8, k 2t+8..2t+9).  In
 *   a 4-bit plane word, register i's two elements sit at bits 4i..4i+3 and
 *   16+4i..16+4i+3 (the low 4 bits of the code).  In the 2-bit plane word the
 *   top 2 bits of register i of step s (0 = A, 1 = B) sit at bits
 *   8s + 2*(i / 2) + 4*(i % 2) and 16 above that (odd k).  So a row-g field
 *   and its row-g+8 partner are 4 bits apart in both planes, and one shift of
 *   the 2-bit word lines a pair up with its nibbles.  Codes are stored
 *   unsigned (not offset).
 *
 * buf: device, 16-byte aligned, qlin_packed_bytes(fmt, N, K, G) bytes.
 * ws : device scratch, 256-byte aligned, at least *min_bytes from
 *      qlin_repack_workspace_bytes; larger means fewer, bigger copy waves.
 *      Strictly zero extra memory is not possible because codes and scales sit
 *      in separate regions of the input; the scratch holds all scales plus one
 *      wave of 128-row code tiles.
 */
qlin_status qlin_repack_workspace_bytes(int fmt, int64_t N, int64_t K, int64_t G,
                                        size_t* min_bytes, size_t* recommended_bytes);
qlin_status qlin_repack(int fmt, int64_t N, int64_t K, int64_t G, void* buf,
                        void* ws, size_t ws_bytes, void* stream);

/*
 * Forward workspace: one status word (plus reserved bytes) that a device-side
 * wait which expires sets to QLIN_ERR_DEVICE_TIMEOUT.  Zero it once with
 * qlin_workspace_init; one workspace may serve every call of a model.  The
 * forward keeps everything else (the quantised activations, the split-K
 * partial sums) in on-chip shared memory.
 */
/*
 * qlin_repack for a W4A8 weight whose levels come from a codebook
 * (qlin_forward_codebook): the same stream, except that in a 4-bit plane
 * word A-register i's two codes sit in byte i (even k at bits 8i..8i+3, odd
 * k at 8i+4..8i+7), so that one table lookup yields one register.  Same
 * arguments, sizes and errors as qlin_repack with fmt = QLIN_W4A8.  A buffer
 * repacked this way is for qlin_forward_codebook only.
 */
qlin_status qlin_repack_codebook(int64_t N, int64_t K, int64_t G, void* buf, void* ws, size_t ws_bytes,
                                 void* stream);

qlin_status qlin_forward_workspace_bytes(int fmt, int64_t N, int64_t K, int64_t G, size_t* bytes);
qlin_status qlin_workspace_init(void* ws, size_t ws_bytes, void* stream);

/*
 * y = packed-weight x quantised activation [LIN], [ACT], [MTP].
 *   fmt, prologue : qlin_format, qlin_prologue.
 *   M             : rows, 1..8 (M = 0 or N = 0 enqueues nothing; with M = 0
 *                   the activation and output pointers are not read and may
 *                   be null).
 *   packed        : device, repacked stream (qlin_repack), 16-byte aligned.
 *   x             : bf16 [M, K] row-major, 16-byte aligned (NONE, RMSNORM).
 *   gate, up      : bf16 [M, K] row-major, 16-byte aligned (SWIGLU).
 *   gamma         : fp32 [K], 16-byte aligned (RMSNORM); eps >= 0 (RMSNORM).
 *   y             : fp32 [M, N] row-major, 4-byte aligned; fully overwritten.
 *   ws, ws_bytes  : forward workspace (see above), 256-byte aligned.
 *   flags         : 0 or QLIN_FLAG_PDL.
 * Numerics: the prologue and the scale s_m = amax/127 are computed in fp32,
 * q = clamp(round-half-even(a / s_m), -127, 127) (s_m = 0, q = 0 for an
 * all-zero row; with no prologue a / s_m is the IEEE fp32 quotient, with a
 * prologue a * c, c = rstd * 127 / amax from fast fp32 reciprocals, which the
 * method's tolerance allows); group sums are exact integers; y is accumulated
 * in fp32 in a fixed order that depends on (N, K, G) and the device, never on
 * M or on the other rows, so row m of an 8-row call equals the same row run
 * alone: the split of K over the CTAs of a cluster is planned for 8 rows
 * whatever M is, and M changes only how deep the weight ring is.  One kernel
 * is enqueued: a cluster of CTAs per 256 output rows
 * splits K, computes the prologue and the row statistics in shared memory,
 * streams the weights through the tensor cores and reduces its split-K
 * partial sums through distributed shared memory.
 */
qlin_status qlin_forward(int fmt, int prologue, int M, int64_t N, int64_t K, int64_t G,
                         const void* packed, const void* x, const void* gate, const void* up,
                         const float* gamma, float eps, float* y,
                         void* ws, size_t ws_bytes, unsigned flags, void* stream);

/*
 * Several weights that read the same activation, in one launch [LIN], [ACT]:
 * y[l] = packed[l] x quantised activation for l = 0..n-1, e.g. the q, k and v
 * projections after one RMSNorm, or gate and up.  The prologue and the
 * activation quantisation are computed for the shared input only; fusing the
 * steps that share an input follows "Doubling the LLM token rate in
 * ComfyUI", section "Optimising the linear kernel" (the prologue is absorbed
 * into the quantisation and the launches between them disappear).
 *   n             : 1..QLIN_MAX_MULTI weights.
 *   N             : host array [n] of output rows (each N[l] obeys the rules
 *                   of qlin_forward; N[l] = 0 skips weight l).
 *   packed        : host array [n] of device pointers, each a repacked stream
 *                   of shape (N[l], K, G), 16-byte aligned.
 *   y             : host array [n] of device pointers, fp32 [M, N[l]]
 *                   row-major, 4-byte aligned; fully overwritten.
 *   bias          : NULL, or a host array [n] of device pointers (each NULL or
 *                   fp32 [N[l]], 4-byte aligned): y[l][m][n] gets bias[l][n]
 *                   added once, unscaled ("Comfy Quantization Formats",
 *                   sections "Checkpoint layout" and "Activations and
 *                   smoothing": a layer's bias stays floating point).
 *   All other arguments, the numerics and the errors are those of
 *   qlin_forward; the host arrays are read during the call only.  Each y[l]
 *   equals qlin_forward on weight l within the output tolerance; the
 *   split-K order may differ because the cluster size is chosen for the
 *   whole launch.
 */
#define QLIN_MAX_MULTI 8

/*
 * Expert bank (MoE) [MOE]: y[m][j][:] = expert ids[m][j] applied to the
 * quantised activation of token m.  "Comfy Quantization Formats", section
 * "Embeddings and MoE": a grouped W4A8 / W6A8 bank stores its experts with
 * the expert and output rows flattened to E * N, and an optional [E, N] bias.
 *   bank   : device, the bank repacked as one weight of E * N rows
 *            (qlin_repack with N = E * N), 16-byte aligned.
 *   E, N   : experts (1..4096) and rows per expert (a multiple of 128 here,
 *            so that every expert starts on a stream tile).  G >= 32 here.
 *   ids    : device int32 [M, topk], topk in 1..8: the expert of each token
 *            and slot.  It may be written by the previous kernel in the
 *            stream: it is read after the dependency wait.  An id outside
 *            [0, E) routes nowhere and its output row is not written; a token
 *            may name one expert in several slots.
 *   bias   : device fp32 [E, N], or NULL.
 *   y      : device fp32 [M, topk, N] row-major; every routed (m, j) row is
 *            fully overwritten.  No routing weights are applied.
 *   Other arguments, numerics and errors as qlin_forward.  One launch is
 *   sized for min(E, M * topk) experts; the experts actually routed take its
 *   row blocks in increasing id order, the remaining blocks return at once.
 *   The split of K is planned for min(E, 8 * topk) experts, so for a given
 *   bank (E, N, K, G) and topk, token m's output does not depend on M or on
 *   the other tokens' routing.
 *   Under QLIN_FLAG_PDL the weights are not streamed before the previous
 *   kernel completes (the routing decides which weights).
 */
#define QLIN_MOE_MAX_E 4096
#define QLIN_MOE_MAX_TOPK 8
qlin_status qlin_forward_moe(int fmt, int prologue, int M, int E, int64_t N, int64_t K, int64_t G, const void* bank,
                             const int32_t* ids, int topk, const void* x, const void* gate, const void* up,
                             const float* gamma, float eps, const float* bias, float* y, void* ws, size_t ws_bytes,
                             unsigned flags, void* stream);
/*
 * 4-bit codes with a codebook [FMT]: "Comfy Quantization Formats", section
 * "Format options" -- a W4A8 weight may carry a float [16] codebook that
 * replaces the uniform levels (code - 8); W6A8 has none.  Here the level of
 * code c is codebook[c], scaled per group by the weight scale as usual:
 *   y[m][n] = s_m * sum_g sw[n][g] * sum_{k in g} q[m][k] * codebook[code[n][k]]
 *             (+ bias[n]).
 *   fmt      : QLIN_W4A8 only (else QLIN_ERR_INVALID_ARG); G >= 32 here.
 *   packed   : the stream written by qlin_repack_codebook (the codebook
 *              layout of the 4-bit plane), 16-byte aligned.
 *   codebook : device fp32 [16], 4-byte aligned.  It is read like `packed`
 *              (before the dependency wait under QLIN_FLAG_PDL).
 *   bias     : device fp32 [N], or NULL.
 *   Other arguments, numerics and errors as qlin_forward, except that the
 *   group sums are not exact integers: the table is scaled by the power of
 *   two that puts its largest magnitude in [2^14, 2^15) and rounded to fp16
 *   (11 significant bits, relative error <= 2^-12 per level), products and
 *   sums in fp32, the power of two removed exactly afterwards.
 */
qlin_status qlin_forward_codebook(int fmt, int prologue, int M, int64_t N, int64_t K, int64_t G, const void* packed,
                                  const float* codebook, const void* x, const void* gate, const void* up,
                                  const float* gamma, float eps, const float* bias, float* y, void* ws,
                                  size_t ws_bytes, unsigned flags, void* stream);
qlin_status qlin_forward_multi(int fmt, int prologue, int M, int n, const int64_t* N, int64_t K, int64_t G,
                               const void* const* packed, const void* x, const void* gate, const void* up,
                               const float* gamma, float eps, float* const* y, const float* const* bias, void* ws,
                               size_t ws_bytes, unsigned flags, void* stream);

/* Launch shape of qlin_forward's GEMV on the current device: CTAs, stream
 * units (128 rows x KB columns) and bytes of `packed` read per call.  The
 * CTAs are the same for every M (the split of K does not depend on M). */
qlin_status qlin_forward_launch_info(int fmt, int64_t N, int64_t K, int64_t G,
                                     int64_t* ctas, int64_t* units, int64_t* stream_bytes);

/* Synchronises `stream`, then returns the workspace status word (QLIN_OK when
 * no device-side wait has expired since qlin_workspace_init).  For tests. */
qlin_status qlin_read_device_status(const void* ws, void* stream);

/*
 * Test export: qlin_forward with extra outputs (device pointers, each may be
 * NULL): y fp32 [M, N]; acc int32 [M, N, K/G], the exact per-group integer
 * sums sum_k q[m,k] * level[n,k]; q int8 [M, K], the activation codes; s fp32
 * [M], the row scales.  It runs a build of the forward kernel that carries
 * these exports (the production kernels do not), with the same arithmetic:
 * its y equals qlin_forward's bit for bit.
 */
qlin_status qlin_debug_forward(int fmt, int prologue, int M, int64_t N, int64_t K, int64_t G,
                               const void* packed, const void* x, const void* gate, const void* up,
                               const float* gamma, float eps, float* y, int32_t* acc, int8_t* q, float* s,
                               void* ws, size_t ws_bytes, void* stream);

/*
 * Test export for failure detection: qlin_forward, except that the first CTA
 * of the launch never issues the weight copy of its local unit `unit` (0 is
 * its first unit and always exists).  Its consumers' bounded wait on that
 * unit expires after about a second; the kernel writes
 * QLIN_ERR_DEVICE_TIMEOUT into the workspace status word, waits (bounded) for
 * the copies it did issue, and returns, leaving the context usable.  y is
 * unspecified afterwards.  Nothing faults.
 */
qlin_status qlin_debug_forward_fault(int fmt, int prologue, int M, int64_t N, int64_t K, int64_t G,
                                     const void* packed, const void* x, const void* gate, const void* up,
                                     const float* gamma, float eps, float* y, void* ws, size_t ws_bytes,
                                     int64_t unit, void* stream);

/*
 * Test export: the plan qlin_forward uses on the current device for a weight
 * of N rows, K columns and group size G at M rows: *cluster = CTAs that split
 * K for one 256-row block (the same for every M), *stages = ring stages per
 * CTA (more for fewer rows, whose activation operand is smaller).
 */
qlin_status qlin_debug_plan(int fmt, int M, int64_t N, int64_t K, int64_t G, int* cluster, int* stages);

/*
 * Test exports of the second main loop, on the 5th-generation tensor cores
 * (tcgen05.mma with the fp16 weight operand in tensor memory, accumulators in
 * tensor memory), kept to measure it against qlin_forward's warp-level MMA
 * loop; it computes the same results ("Doubling the LLM token rate in
 * ComfyUI", section "Optimising the linear kernel": the M <= 8 activation
 * rows on the narrow side of the tensor-core product).  It is slower on this
 * path: every 4-bit code is unpacked on the CUDA cores either way, and the
 * tensor-memory stores, the hand-offs between warps and the MMA issue (one
 * 128 x 16 step per instruction) cost more than the warp-level MMAs they
 * replace.
 *
 * qlin_debug_repack_tcgen05: qlin_repack into the row layout this loop reads
 *   (G >= 32): per unit of R rows and W columns,
 *     scale block  R*(W/G) fp32, [group][row];
 *     4-bit plane  for each 32-wide k chunk c, for each row: 4 words, word j
 *                  holding the low 4 bits of the codes of k = 32c + 8j + i at
 *                  bits 4i (i = 0..7);
 *     6-bit codes only, then the 2-bit plane: for each chunk, for each row: 2
 *                  words; word h holds the top 2 bits of the codes of words
 *                  2h (at offset 0) and 2h+1 (at offset 2), code i of a word
 *                  at bit P(i) + offset, P = (4, 8, 0, 12, 20, 24, 16, 28).
 *   Arguments and errors as qlin_repack; QLIN_ERR_UNSUPPORTED for G < 32.
 * qlin_debug_forward_tcgen05: qlin_debug_forward on a weight repacked by
 *   qlin_debug_repack_tcgen05 (y required; acc, q, s may be NULL), with
 *   qlin_forward's flags.  Its split of K is planned for its own shared-memory
 *   operand, so y may differ from qlin_forward's in the last bits (the order
 *   of the fp32 partial sums); the group sums are the same exact integers.
 */
qlin_status qlin_debug_repack_tcgen05(int fmt, int64_t N, int64_t K, int64_t G, void* buf, void* ws,
                                      size_t ws_bytes, void* stream);
qlin_status qlin_debug_forward_tcgen05(int fmt, int prologue, int M, int64_t N, int64_t K, int64_t G,
                                       const void* packed, const void* x, const void* gate, const void* up,
                                       const float* gamma, float eps, float* y, int32_t* acc, int8_t* q, float* s,
                                       void* ws, size_t ws_bytes, unsigned flags, void* stream);

/*
 * qlin_forward without a caller workspace.  The method has no counterpart: this
 * is for callers that cannot allocate device memory where they run the layer
 * (a host whose memory pool owns the whole device and forbids cudaMalloc, code
 * that must avoid cudaMalloc's implicit synchronisation, a fixed-footprint
 * deployment).  The call allocates nothing; it uses a 64 KiB device array
 * inside the library instead, which every GPU that loads the library holds
 * until the process exits.
 *  - Arguments are those of qlin_forward without ws/ws_bytes.
 *  - Returns QLIN_ERR_WORKSPACE when the shape's workspace
 *    (qlin_forward_workspace_bytes) exceeds 64 KiB; nothing is enqueued then.
 *  - The first call on a device looks up the array's device address (once per
 *    device, with that device current); make that first call before any CUDA
 *    stream capture.
 *  - All calls share the one array, which keeps the previous call's contents.
 *    The forward kernel keeps nothing there that must start at zero: the
 *    array holds only the status word, written only when a wait expires.
 *    Calls that overlap on the GPU (different streams, or unordered work)
 *    race on it: order them on one stream.
 *  - A device-side wait that expires is recorded in the array's status word,
 *    which this entry point does not read back; the kernel still returns
 *    instead of hanging.
 */
qlin_status qlin_forward_noalloc(int fmt, int prologue, int M, int64_t N, int64_t K, int64_t G,
                                 const void* packed, const void* x, const void* gate, const void* up,
                                 const float* gamma, float eps, float* y, unsigned flags, void* stream);

/* ---------------------------------------------------------------------------
 * The rest of a decode / verification step: what stands between and behind the
 * linears ("Doubling the LLM token rate in ComfyUI", section "Adaptive-tree
 * MTP": one committed token and a tree of drafted ones are verified in one
 * pass).  q/k/v (qlin_forward_multi) -> qlin_kv_append -> qlin_tree_attention
 * -> o (qlin_forward) ... -> qlin_sample -> qlin_kv_keep.  With images or videos,
 * a cache kept within its room, or rules on the logits: qlin_kv_append_at ->
 * qlin_tree_attention_stats ... -> qlin_adjust_logits -> qlin_sample ->
 * qlin_kv_weigh -> qlin_kv_keep -> qlin_kv_evict.
 *
 * The conventions above hold: device pointers, nothing allocated or
 * synchronised, errors of arguments returned before anything is enqueued.  The
 * structs themselves are host memory, read during the call only.  A step of no
 * sequences or no rows enqueues nothing and writes nothing.
 * ------------------------------------------------------------------------ */
typedef enum { QLIN_BF16 = 0, QLIN_F16 = 1, QLIN_F32 = 2 } qlin_dtype;

/*
 * A paged cache of keys and values.  Token row i of head h on page p starts at
 * element p * page_stride + h * head_stride + i * token_stride of k and of v
 * and holds `width` contiguous elements, so [pages, heads, page_size, width]
 * and [pages, page_size, heads, width] are both caches, and so are slices of
 * a larger pool.
 *   dtype      : QLIN_BF16 or QLIN_F16.
 *   width      : 64, 128 or 256.     heads : 1..1024.
 *   page_size  : 16, 32, 64, 128 or 256 tokens.    pages : 1..2^31-1.
 *   k, v       : 16-byte aligned; the strides multiples of 8 elements, each
 *                in 1..2^36 and token_stride >= width.
 */
typedef struct {
  void* k;
  void* v;
  int64_t pages, page_stride, head_stride, token_stride;
  int32_t dtype, heads, width, page_size;
} qlin_kv_cache;

/*
 * One step: B sequences, T rows each (row b * T + t of q, k, v and the
 * output).  Token i of sequence b lies on page page_table[b][i / page_size],
 * row i % page_size.  Rows are stored behind the sequence's committed tokens:
 * row t is token len[b] + t.
 *   page_table : int32 [B, max_pages], rows table_stride entries apart.
 *                Entries behind the last page in use are not read.
 *   len        : int32 [B], committed tokens (0: none yet).  len[b] < 0: no
 *                sequence in this place; its rows have no effect and nothing of
 *                it is written.
 *   count      : int32 [B] or NULL (T rows in every sequence): rows in use;
 *                the rows behind them have no effect, whatever they hold, and
 *                what they would have written is left as it was.
 *   depth      : int32, row t's distance from the committed tokens, so its
 *                rotation position is len[b] + depth[t]; NULL: t.
 *   mask       : int32 bits, bit j of row t: row t sees row j of its own
 *                sequence (its own bit too); NULL: the rows up to its own.
 *                T <= 32.  Bits of rows not in use are ignored.
 *   tree_stride: entries between the sequences' rows of depth and mask; 0 for
 *                one tree shared by all sequences.
 * A page index outside [0, pages), or a token behind the table's last page, is
 * never followed: what it would have read or written is left out, the
 * sequence's results are unspecified, and QLIN_ERR_BAD_INDEX goes to the
 * workspace's status word (where the call has a workspace).
 */
typedef struct {
  const int32_t* page_table;
  const int32_t* len;
  const int32_t* count;
  const int32_t* depth;
  const int32_t* mask;
  int64_t table_stride, tree_stride;
  int32_t B, T, max_pages;
} qlin_kv_step;

/* Rotation frequencies for qlin_kv_append: turns[i] = radians[i] / (2 pi)
 * modulo 1, as a 64-bit fraction of a turn, so that the angle of any position
 * is an exact integer product.  Host memory on both sides; copy the result to
 * the device once.  radians[i] finite, n in 0..128. */
qlin_status qlin_rope_turns(const double* radians, int n, uint64_t* turns);

/*
 * The projected rows of a step into the cache: q' = R(q * q_gamma / rms(q))
 * head by head, k' likewise, and k' and v stored behind the sequences'
 * committed tokens.  rms(x)^2 = mean(x^2) + eps over one head; R rotates the
 * first 2 * n_turns elements of a head by the row's position.
 *   Hq            : query heads (0 with q = NULL).
 *   src           : type of q, k, v: QLIN_F32 (what qlin_forward writes) or
 *                   QLIN_BF16.
 *   q, k, v       : [B * T, heads * width], rows *_stride elements apart,
 *                   16-byte aligned rows.  q may be NULL (nothing is written
 *                   to q_out); k and v may both be NULL (nothing is stored).
 *   q_out         : [B * T, Hq * width] in the cache's type, rows
 *                   q_out_stride elements apart, 16-byte aligned rows.  Its
 *                   rows share no memory with those of q, k and v
 *                   (QLIN_ERR_INVALID_ARG), but a bf16 q of the same rows may
 *                   be q_out itself.
 *   q_gamma, k_gamma : fp32 [width], 16-byte aligned, or NULL: no norm.
 *   turns, n_turns   : device, from qlin_rope_turns, 8-byte aligned;
 *                   n_turns in 0..width / 2 (0: no rotation).
 *   pairs         : 0: element i turns with i + n_turns; 1: 2i with 2i + 1.
 *   ws            : a workspace (256 bytes) for the status word, or NULL (a bad
 *                   index is then not followed either, but not reported).
 *   flags         : 0 or QLIN_FLAG_PDL (nothing is read before earlier kernels
 *                   complete).
 * T is not limited: a prompt's rows are appended the same way.  Computed in
 * fp32 (the angle exactly, see above) and rounded once.
 */
qlin_status qlin_kv_append(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, int src, const void* q,
                           int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const float* q_gamma, const float* k_gamma, float eps, const uint64_t* turns, int n_turns,
                           int pairs, void* q_out, int64_t q_out_stride, void* ws, size_t ws_bytes, unsigned flags,
                           void* stream);

/*
 * qlin_kv_append with the rows' positions given, on up to four axes: pair i of
 * a head turns by position[row][axis[i]] * turns[i].  For the rows of an image
 * or a video (time, height and width each turn pairs of their own), and for
 * rows whose place in the cache is not their position (after qlin_kv_evict).
 * Rows are stored behind the committed tokens as by qlin_kv_append; depth is
 * not read.
 *   position : int32, row b * T + t of it position_stride entries behind the
 *              one before, `axes` entries each; any values (negative too).
 *              Shares no memory with q_out.  Rows not in use are read, but
 *              have no effect.
 *   axes     : 1..QLIN_MAX_AXES.
 *   axis     : host memory, read during the call: n_turns values below axes.
 *              NULL: axis 0 everywhere (axes = 1 only).
 */
#define QLIN_MAX_AXES 4
qlin_status qlin_kv_append_at(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, int src, const void* q,
                              int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const float* q_gamma, const float* k_gamma, float eps, const uint64_t* turns,
                              int n_turns, int pairs, const int32_t* position, int64_t position_stride, int axes,
                              const uint8_t* axis, void* q_out, int64_t q_out_stride, void* ws, size_t ws_bytes,
                              unsigned flags, void* stream);

/*
 * Attention of a step's rows over the cache: every row sees all committed
 * tokens of its sequence, and of the step's own rows (already appended) those
 * that its mask names.  out = sum_j softmax_j(scale * q . k_j) v_j; a row that
 * sees nothing gives zeros.  Query head h reads cache head h / (Hq / heads).
 * Masked rows of the step contribute nothing whatever they hold (NaN too); a
 * committed token that is not finite makes the columns of the results that it
 * reaches not finite either.
 *   T         : 1..32 rows per sequence, T * Hq / heads <= 128.
 *   Hq        : a multiple of the cache's heads.
 *   q         : [B * T, Hq * width], the cache's type, rows q_stride elements
 *               apart, 16-byte aligned rows (q_out of qlin_kv_append).
 *   out       : bf16 [B * T, Hq * width], rows out_stride elements apart,
 *               16-byte aligned rows (the o projection's activation) that
 *               share no memory with those of q (QLIN_ERR_INVALID_ARG).
 *   scale     : finite.
 *   ws        : 256-byte aligned, at least
 *               qlin_tree_attention_workspace_bytes; its first word is the
 *               status word.  Calls that overlap on the GPU need workspaces
 *               of their own.
 *   flags     : 0 or QLIN_FLAG_PDL.
 * Scores, softmax statistics and sums are fp32; the weights are rounded to the
 * cache's type for the product with v.  The result does not depend on the
 * other sequences' values, only (in the order of its sums) on all lengths.
 */
#define QLIN_MAX_TREE 32
qlin_status qlin_tree_attention_workspace_bytes(const qlin_kv_cache* cache, int B, int T, int Hq, size_t* bytes);
qlin_status qlin_tree_attention(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q,
                                int64_t q_stride, float scale, void* out, int64_t out_stride, void* ws,
                                size_t ws_bytes, unsigned flags, void* stream);

/*
 * qlin_tree_attention, and the rows' softmax statistics beside it: stats, fp32
 * [B * T, Hq, 2], contiguous, 8-byte aligned, gets each row's reference r and sum
 * l: the weight of token j is 2^(scale log2(e) q . k_j - r) / l.  (-inf, 0): the
 * row saw nothing.  r is near the row's largest score, not always equal to it.
 * Rows not in use are left as they were.  Shares no memory with q and out.
 */
qlin_status qlin_tree_attention_stats(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q,
                                      int64_t q_stride, float scale, void* out, int64_t out_stride, float* stats,
                                      void* ws, size_t ws_bytes, unsigned flags, void* stream);

/*
 * Test export for failure detection: qlin_tree_attention without flags, except
 * that the launch's first CTA never issues its `copy`-th copy of a tile (0: the
 * keys of its first tile, 1: their values, 2: the next tile's keys ...).  The
 * bounded waits on it expire after about a second; the kernel writes
 * QLIN_ERR_DEVICE_TIMEOUT into the status word, waits (bounded) for the copies
 * and products that it did issue, frees its tensor memory and returns, leaving
 * the context and the workspace usable.  out is unspecified afterwards.
 * Nothing faults.  bf16 caches of width 128 and T * Hq / heads <= 32 only
 * (else QLIN_ERR_UNSUPPORTED).
 */
qlin_status qlin_debug_tree_attention_fault(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq,
                                            const void* q, int64_t q_stride, float scale, void* out,
                                            int64_t out_stride, void* ws, size_t ws_bytes, int64_t copy,
                                            void* stream);

/*
 * Keeps an accepted path of a verified tree: row keep[b][i] of sequence b
 * moves to token len[b] + i, for i < n_keep[b], and len_out[b] = len[b] +
 * n_keep[b].  The kept rows are given in increasing order (a row's parent
 * stands before it); a list that is not, or that names a row outside
 * 0..count[b] - 1, moves nothing, len_out[b] = len[b], and the status word gets
 * QLIN_ERR_BAD_INDEX.
 *   keep    : int32 [B, T], rows keep_stride entries apart.
 *   n_keep  : int32 [B], 0..count[b].
 *   len_out : int32 [B], or NULL; may be step->len itself.  Not written where
 *             len[b] < 0.
 *   ws      : a workspace (256 bytes) for the status word, or NULL (a bad list
 *             or index then moves nothing either, but is not reported).
 * T <= 32.  depth and mask are not read.
 */
qlin_status qlin_kv_keep(const qlin_kv_cache* cache, const qlin_kv_step* step, const int32_t* keep,
                         int64_t keep_stride, const int32_t* n_keep, int32_t* len_out, void* ws, size_t ws_bytes,
                         unsigned flags, void* stream);

#define QLIN_MAX_ROOM 1048576
/*
 * The attention weight that the cache's tokens got from a step's rows, added to
 * what they got before: for cache head h and each committed token j
 *   score_out[b][h][j] = decay * score[b][h][j] + sum of the weights of j
 * over the kept rows and the query heads that read h.  The step's own tokens of
 * kept rows get their weights alone, at the places len[b] + i that qlin_kv_keep
 * gives them (call this before it), and position_out their positions there.
 *   Hq, q, scale : as qlin_tree_attention was given them.
 *   stats        : from qlin_tree_attention_stats.
 *   keep, n_keep : as for qlin_kv_keep: the accepted path, of which each row sees
 *                  those before it and itself.  Both NULL: the rows in use are
 *                  all kept, and see one another as the step's mask says.  A bad
 *                  list keeps nothing, and the status word gets QLIN_ERR_BAD_INDEX.
 *   decay        : finite; 1: nothing fades.
 *   score, score_out, position_out, the strides, room : as for qlin_kv_evict
 *                  (score_out may be score); position_out may be NULL.  Neither
 *                  shares memory with q, stats and at (QLIN_ERR_INVALID_ARG).
 *                  What would lie at room or behind is left out and reported,
 *                  as are committed tokens and kept rows behind the page table.
 *   at           : int32 [B * T]: the rows' positions, as given to
 *                  qlin_kv_append_at; NULL: len + depth.
 *   T            : 1..32 rows per sequence, T * Hq / heads <= 128.
 *   ws           : a workspace (256 bytes) for the status word, or NULL.
 *   flags        : 0 or QLIN_FLAG_PDL.
 * Scores and sums are fp32.  A row whose statistics are not finite (a key that it
 * sees, or its own query, is not) weighs nothing in that cache head, as one that
 * saw nothing does; a key that is not finite may make its own token's score not
 * finite, and no other's.  Places of tokens that are not there, or lie
 * on a page out of range, and whole sequences with len[b] < 0, are left as they
 * were.  Where scores pass 2^23 (log2 units), and fp32 holds them a unit or more
 * apart, a weight is no more than 1.
 */
qlin_status qlin_kv_weigh(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q, int64_t q_stride,
                          const float* stats, float scale, const int32_t* keep, int64_t keep_stride,
                          const int32_t* n_keep, float decay, const float* score, int64_t seq_stride,
                          int64_t head_stride, float* score_out, int32_t* position_out, int64_t out_seq_stride,
                          int64_t out_head_stride, int64_t room, const int32_t* at, void* ws, size_t ws_bytes,
                          unsigned flags, void* stream);

/*
 * Test export for failure detection: qlin_kv_weigh of all rows in place or with
 * the strides of score, except that the launch's first CTA never issues its
 * `copy`-th copy of a panel of keys.  The bounded waits on it expire after about
 * a second; the kernel writes QLIN_ERR_DEVICE_TIMEOUT into the status word, waits
 * (bounded) for the copies and products that it did issue, frees its tensor memory
 * and returns.  score_out is unspecified afterwards.  Nothing faults.  bf16 caches
 * of width 128 only (else QLIN_ERR_UNSUPPORTED).
 */
qlin_status qlin_debug_kv_weigh_fault(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q,
                                      int64_t q_stride, const float* stats, float scale, const float* score,
                                      int64_t seq_stride, int64_t head_stride, float* score_out, int64_t room, void* ws,
                                      size_t ws_bytes, int64_t copy, void* stream);

/*
 * Eviction by accumulated weight (qlin_kv_weigh): of each sequence's committed
 * tokens, head by head, the n_keep[b] of the highest score stay (all, where there
 * are no more); equal scores by index, the lowest first, NaN behind all others.
 * A token whose position is below `first`, or at least since[b], counts as the
 * highest.  Kept tokens before place n_keep[b] stay where they are; those
 * behind it move, in order, into the places that empty before it: keys, values,
 * scores and positions.  len_out[b] = the tokens left, the same for all heads.
 * The order of a head's tokens is then no longer that of their positions
 * (attention does not depend on it; rows appended later need qlin_kv_append_at,
 * and what is kept by position needs `position`).
 *   score        : fp32 [B, heads, room], sequences seq_stride and heads
 *                  head_stride elements apart, the tokens' contiguous.
 *   position     : int32 in the same layout, the tokens' positions; NULL: a
 *                  token's place is its position.
 *   score_out    : of the same shape, strides of its own: the tokens left.  May
 *                  be score itself (of the same strides); else the ranges that
 *                  these four lie in do not overlap (QLIN_ERR_INVALID_ARG).
 *   position_out : the same for position, or NULL.  (position NULL and
 *                  position_out given: where the tokens left have been.)
 *   room         : 0..QLIN_MAX_ROOM.  A sequence of more tokens than that, or
 *                  than its page table names, is left alone, and the status word gets
 *                  QLIN_ERR_BAD_INDEX; so are rows on a page out of range.
 *   n_keep       : int32 [B] (below 0: as 0).
 *   first        : 0 or more.     since : int32 [B], or NULL: none.
 *   len_out      : int32 [B], or NULL; may be step->len itself.  Not written where
 *                  len[b] < 0.
 *   ws           : 256-byte aligned, at least qlin_kv_evict_workspace_bytes; its
 *                  first word is the status word.  Calls that overlap on the GPU
 *                  need workspaces of their own.
 *   flags        : 0 or QLIN_FLAG_PDL.
 * count, depth and mask are not read.  The places of two sequences' committed
 * tokens must not lie on one page: the rows of one would move under the other.
 * Scores and positions behind the tokens left are not written.
 */
qlin_status qlin_kv_evict_workspace_bytes(const qlin_kv_cache* cache, int B, int64_t room, size_t* bytes);
qlin_status qlin_kv_evict(const qlin_kv_cache* cache, const qlin_kv_step* step, const float* score,
                          const int32_t* position, int64_t seq_stride, int64_t head_stride, float* score_out,
                          int32_t* position_out, int64_t out_seq_stride, int64_t out_head_stride, int64_t room,
                          const int32_t* n_keep, int first, const int32_t* since, int32_t* len_out, void* ws,
                          size_t ws_bytes, unsigned flags, void* stream);

/*
 * One token per row of logits, from a given uniform number.  The row's tokens
 * stand in order of their logits, equal ones by index.  Kept are the first
 * top_k; of those the shortest beginning whose mass is at least top_p of
 * theirs; of those the ones with w >= min_p, where w = exp((x - max) /
 * temperature).  The token is the first kept one, in order of the vocabulary,
 * at which the running sum of the kept w exceeds u times their sum.
 *   logits      : [M, V] of type dtype (QLIN_F32 or QLIN_BF16), rows ld
 *                 elements apart, aligned to the element.  -inf: a forbidden
 *                 token, never chosen; +inf: only those tokens are left, alike.
 *   M >= 0, V   : 1..524288.
 *   u           : fp32 [M], in [0, 1); values outside are clamped.
 *   temperature : fp32 [M] or NULL (1).  Not above 0 (or NaN): the row's
 *                 largest logit, the lowest index of equal ones, prob = 1.
 *   top_k       : int32 [M] or NULL; below 1 or above V - 1: all tokens.
 *   top_p       : fp32 [M] or NULL; 1 and above, or NaN: all; 0 and below:
 *                 the first token alone.
 *   min_p       : fp32 [M] or NULL; 0 and below, or NaN: all; above 1: as 1.
 *   token       : int32 [M].  -1 for a row of -inf alone or with a NaN.
 *   prob        : fp32 [M] or NULL: the token's share of the kept mass (0 with
 *                 token -1).
 * The weights are 42-bit fractions and every sum of them is an exact integer,
 * so the token does not depend on an order of summation.  A weight above 2^-10
 * is within 2.5 * 2^-31 of itself at temperatures up to 2^100, a lower one
 * within half of 2^-42 besides; a token with w below 2^-43 has none and is
 * never chosen.
 */
#define QLIN_SAMPLE_MAX_V 524288
qlin_status qlin_sample(int M, int64_t V, int dtype, const void* logits, int64_t ld, const float* u,
                        const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                        int32_t* token, float* prob, unsigned flags, void* stream);

/*
 * Logits before qlin_sample: penalties for repeated tokens, biases, a grammar's
 * mask.  Row b * T + t belongs to sequence b.  A token v stands n times in the
 * row's generated text: in the history from prompt_len on, and on the row's
 * path of drafted tokens.  Then, in fp32, rounded once at the end,
 *   x' = x / r if x > 0, else x * r   where v stands in the history or the path
 *   x' = x' - frequency * n - presence            where n > 0
 *   x' = x' + bias                 of v; several of them are first added to one
 *                                  another, in the list's order, in fp32
 *   x' = -inf                                     where v is not allowed.
 * A logit that none of these concerns is copied as it is.  Any pointer may be
 * NULL: what it would give is left out.  The struct is host memory, read during
 * the call only.
 *   history     : int32 [B, L], rows history_stride apart; the sequence's tokens
 *                 but for the step's.  Entries outside [0, V) count for nothing.
 *   history_len : int32 [B]: entries in use (NULL: L).
 *   prompt_len  : int32 [B]: of these, the first ones that are the prompt's
 *                 (NULL: none).
 *   draft       : int32 [B, T], contiguous: the step's tokens; row t's path are
 *                 those that its mask names, its own token among them.  T <= 32.
 *   mask        : as in qlin_kv_step, tree_stride too (NULL: the rows up to its own).
 *   repetition  : fp32 [B]; not above 0, or NaN: 1.   presence, frequency: fp32 [B].
 *   bias_token, bias : int32, fp32 [B, n_bias], rows bias_stride apart (0: one
 *                 list for all).  Tokens outside [0, V) are left out.
 *   allowed     : int32, rows allowed_stride apart (0: one for all), token v the
 *                 bit v % 32 of word v / 32: 1 where it is allowed.
 *   L           : 0..QLIN_MAX_HISTORY.      n_bias : 0..QLIN_MAX_BIAS.
 */
#define QLIN_MAX_HISTORY 1000000
#define QLIN_MAX_BIAS 1024
#define QLIN_MAX_SEQUENCES 65535
typedef struct {
  const int32_t *history, *history_len, *prompt_len, *draft, *mask;
  const float *repetition, *presence, *frequency;
  const int32_t* bias_token;
  const float* bias;
  const int32_t* allowed;
  int64_t history_stride, tree_stride, bias_stride, allowed_stride;
  int32_t L, n_bias;
} qlin_adjustments;

/*
 *   B           : 0..QLIN_MAX_SEQUENCES, B * T at most 2^24.
 *   V           : 1..524288.   dtype : QLIN_F32 or QLIN_BF16, of logits and out.
 *   logits, out : [B * T, V], rows ld and out_ld elements apart, aligned to the
 *                 element.  out may be the logits themselves (same rows; then
 *                 only what changes is read and written); else they share no
 *                 memory (QLIN_ERR_INVALID_ARG).  Nor does out with what the
 *                 struct names.
 */
qlin_status qlin_adjust_logits(int B, int T, int64_t V, int dtype, const void* logits, int64_t ld, void* out,
                               int64_t out_ld, const qlin_adjustments* adjustments, unsigned flags, void* stream);

/*
 * Test export: the weights that qlin_sample gives to logits x under their row's
 * largest (finite, x <= max) and a temperature above 0, as multiples of 2^-42.
 * Host memory, computed on the host by the kernel's own source; nothing is
 * enqueued.
 */
qlin_status qlin_debug_sample_weight(int n, const float* x, const float* max, const float* temperature,
                                     uint64_t* weight);

/*
 * Test export: the plan that qlin_sample uses for M rows of V logits of type
 * dtype, with top_k given (1) or not (0), on a device whose clusters hold at
 * most `most` CTAs (8 or 16): *ctas = CTAs per row, *in_place = 1 where they
 * read the row where it is (up to 65536 tokens each) and 0 where from shared
 * memory (up to 32768 each).  Host only.
 */
qlin_status qlin_debug_sample_plan(int64_t M, int64_t V, int dtype, int top_k, int most, int* ctas, int* in_place);

#ifdef __cplusplus
}
#endif
#endif /* QLIN_H_ */
