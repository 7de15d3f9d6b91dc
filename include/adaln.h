/*
 * libadaln -- operators of video diffusion transformer blocks for GB300
 * (sm_103a): the fused AdaLN LayerNorm-Modulate, described here, and, further
 * down, rotary positions with the norm of queries and keys (adaln_qk_rope_*),
 * the gated feed-forward block (adaln_ffn_*), dropout with the gate and the
 * residual of a branch (adaln_dropout_*), tokens sorted by expert and back
 * (adaln_route, adaln_expert_*) and the experts' feed-forward blocks on them
 * (adaln_experts_ffn_*), which share its conventions on ownership, streams, errors
 * and the status word.
 *
 * The AdaLN is the fused adaptive LayerNorm of video / MMDiT diffusion
 * transformers described in "AdaptiveLoad: Towards Efficient Video Diffusion
 * Transformer Training", Technical summary, section 2.B ("Fused
 * LayerNorm-Modulate CUDA kernels"): normalisation and modulation in a single
 * kernel launch (forward), and a backward whose modulation-gradient reduction
 * along the sequence dimension is laid out so that each thread owns a feature
 * column d and accumulates down the sequence (the "D-tile coalesced
 * reduction").  The pages give no formula; this library computes, for every
 * token row t of a packed variable-length batch with b = seg_id[t]:
 *
 *   mean[t] = (1/D) sum_d x[t,d]
 *   var[t]  = (1/D) sum_d (x[t,d] - mean[t])^2         (biased)
 *   rstd[t] = 1 / sqrt(var[t] + eps)
 *   xhat    = (x - mean[t]) * rstd[t]
 *   y       = xhat * (1 + scale[b,d]) + shift[b,d]
 *   g       = dy * (1 + scale[b,d])
 *   dx      = rstd[t] * (g - mean_d(g) - xhat * mean_d(g * xhat))
 *   dscale[b,d] = sum_{t: seg_id[t]=b} dy[t,d] * xhat[t,d]
 *   dshift[b,d] = sum_{t: seg_id[t]=b} dy[t,d]
 *
 * Layout: all tensors row-major and contiguous.  x, y, dy, dx are [T, D];
 * shift, scale are [nseg, D]; all of these have the element type `dtype`.
 * seg_id is int32 [T]; mean, rstd are fp32 [T]; dshift, dscale are fp32
 * [nseg, D].  Arithmetic is fp32; bf16 outputs are rounded once (to nearest
 * even) at the store.
 *
 * Ownership: every pointer is owned by the caller and must point to device
 * memory of the current CUDA device (except host_* arguments).  The library
 * never allocates, frees or retains caller memory.
 *
 * Asynchrony: work is enqueued on `stream` (a cudaStream_t; NULL = the legacy
 * default stream) and the calls return without synchronising.  The kernels
 * are launched as programmatic dependents of the stream's previous kernel:
 * they may be scheduled while it ends, but read nothing before it has
 * completed.  They also let the stream's next kernel be scheduled before they
 * complete; a kernel launched after them with programmatic stream
 * serialization must wait (cudaGridDependencySynchronize) before reading
 * their outputs, as that launch mode requires anyway.  Ordinary launches,
 * copies and events see the usual stream order.  Return codes
 * report errors detectable on the host before launch, and launch failures.
 * Data errors found on the device (a seg_id outside [0, nseg) or decreasing
 * along the rows) are clamped so that every access stays in bounds, and are
 * recorded in a status word read by adaln_get_status() (per device, or one the
 * calling thread bound with adaln_status_bind()); outputs of such a call are
 * unspecified.
 *
 * Preconditions (checked, ADALN_ERR_* on violation):
 *   - T >= 0 (T = 0 does nothing, except that adaln_bwd zeroes dshift/dscale);
 *   - D >= 1, D * sizeof(element) a multiple of 16 bytes (D % 8 == 0 for bf16,
 *     D % 4 == 0 for fp32), D <= ADALN_MAX_D_BF16 / ADALN_MAX_D_F32;
 *   - 1 <= nseg <= ADALN_MAX_NSEG;
 *   - x, y, dy, dx, shift, scale, dshift, dscale and the workspace 16-byte
 *     aligned; seg_id, mean, rstd 4-byte aligned;
 *   - eps finite and >= 0;
 *   - seg_id non-decreasing along rows (segments packed contiguously), values
 *     in [0, nseg).  Segments may be empty.
 */
#ifndef ADALN_H
#define ADALN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Symbol visibility of the exported entry points. */
#if defined(__GNUC__)
#define ADALN_API __attribute__((visibility("default")))
#else
#define ADALN_API
#endif

#define ADALN_MAX_D_BF16 8192
#define ADALN_MAX_D_F32 4096
#define ADALN_MAX_NSEG (1 << 24)
#define ADALN_MAX_HEADS 4096
#define ADALN_MAX_HEAD_DIM 512
#define ADALN_MAX_ROPE_AXES 4
#define ADALN_FFN_MAX_T (1 << 24)
#define ADALN_FFN_MAX_DIM (1 << 18)
#define ADALN_DROPOUT_MAX_D (1 << 18)
#define ADALN_MAX_EXPERTS 256
#define ADALN_MAX_TOPK 32
#define ADALN_MAX_ROUTE_ALIGN 4096

typedef enum {
  ADALN_F32 = 0,  /* IEEE binary32 */
  ADALN_BF16 = 1  /* bfloat16 */
} adaln_dtype_t;

typedef enum {
  ADALN_OK = 0,
  ADALN_ERR_NULL = 1,      /* a required pointer is NULL */
  ADALN_ERR_DIM = 2,       /* T, D or nseg outside the supported range */
  ADALN_ERR_ALIGN = 3,     /* a pointer is not aligned as required */
  ADALN_ERR_DTYPE = 4,     /* unknown dtype */
  ADALN_ERR_SEG = 5,       /* device status: seg_id out of range or decreasing */
  ADALN_ERR_WORKSPACE = 6, /* workspace smaller than required */
  ADALN_ERR_CUDA = 7,      /* a CUDA runtime call or launch failed */
  ADALN_ERR_ARG = 8,       /* eps negative or not finite; bad trace argument */
  ADALN_ERR_TIMEOUT = 9,   /* device status: an internal pipeline wait gave up */
  ADALN_ERR_POS = 10,      /* device status: a rotary position outside the table */
  ADALN_ERR_EXPERT = 11    /* device status: an expert, or a sorted row, out of range */
} adaln_status_t;

/* Bits of the device status word (adaln_get_status). */
#define ADALN_DEV_SEG_RANGE 1u   /* a seg_id was outside [0, nseg) */
#define ADALN_DEV_SEG_ORDER 2u   /* seg_id decreased from one row to the next */
#define ADALN_DEV_TIMEOUT 4u     /* a bounded wait on a copy pipeline expired */
#define ADALN_DEV_POS_RANGE 8u   /* a rotary position was outside [-1, rows) */
#define ADALN_DEV_EXPERT_RANGE 16u /* an expert was outside [-1, E), or a sorted row or
                                      an expert's start outside what the call was given */

/*
 * Forward (section 2.B, forward pass): per-row statistics reduced on chip and
 * the modulation applied in the same launch.  Reads x once, writes y, mean,
 * rstd.  One kernel launch on `stream`.
 */
ADALN_API int adaln_fwd(const void* x, const void* shift, const void* scale,
              const int32_t* seg_id, int64_t T, int32_t D, int32_t nseg,
              adaln_dtype_t dtype, float eps, void* y, float* mean,
              float* rstd, void* stream);

/*
 * Bytes of device workspace adaln_bwd needs for these sizes on the current
 * device (it depends on the device's SM count).  Written to *bytes.
 */
ADALN_API int adaln_bwd_workspace_size(int64_t T, int32_t D, int32_t nseg,
                             adaln_dtype_t dtype, size_t* bytes);

/*
 * Backward (section 2.B, backward pass with the D-tile coalesced reduction).
 * Reads dy and x once (plus the saved mean/rstd), writes dx [T, D] and the
 * fp32 sequence reductions dshift, dscale [nseg, D].  Two kernel launches on
 * `stream`: a row pass that also accumulates per-(CTA, segment) column
 * partials into `workspace`, then a fixed-order reduction of those partials.
 * No floating-point atomics: for a given device and sizes the results of
 * valid input are bitwise reproducible.  (With an invalid seg_id the outputs
 * are unspecified and may differ between runs: teams whose clamped segment
 * paths cross can share a partial slot.)  `workspace` (at least
 * adaln_bwd_workspace_size bytes, 16-byte aligned) is scratch owned by the
 * caller; its contents on entry do not matter.  Calls sharing one workspace
 * must not overlap on the device.  A NULL workspace is ADALN_ERR_NULL
 * (adaln_bwd_noalloc serves callers without one); a short one is
 * ADALN_ERR_WORKSPACE.
 */
ADALN_API int adaln_bwd(const void* dy, const void* x, const float* mean,
              const float* rstd, const void* scale, const int32_t* seg_id,
              int64_t T, int32_t D, int32_t nseg, adaln_dtype_t dtype,
              void* dx, float* dshift, float* dscale, void* workspace,
              size_t workspace_bytes, void* stream);

/*
 * Backward that allocates nothing, for callers that cannot call cudaMalloc
 * (for example code inside a host framework whose allocator owns all device
 * memory, or code on a latency-critical path where allocating would
 * synchronise the device).  The paper has no counterpart: this is a
 * deployment variant of adaln_bwd.  Same arguments, results and launches as
 * adaln_bwd, minus the workspace: the scratch is a fixed file-scope device
 * array of ADALN_NOALLOC_SCRATCH_BYTES.  A device holds it from the first
 * adaln_bwd_noalloc call on it (under CUDA's default lazy module loading;
 * from the library's first use there under eager loading) until the process
 * exits.  The partials grow with the SM count (G = SMs x teams per SM):
 * 3072-wide bf16 rows with 822 segments fit up to 181 SMs.  Sizes whose
 * adaln_bwd_workspace_size exceeds it are rejected with ADALN_ERR_WORKSPACE
 * before anything is launched.  The first call on a device looks up the
 * array's device address (cudaGetSymbolAddress) with that device current;
 * make that first call before any stream capture.  All calls on a device share the array and it
 * keeps the last call's contents (nothing in it needs to start at zero);
 * calls that overlap on the GPU race on it.  No cudaMalloc, cudaFree or other
 * allocating routine is called.
 */
#define ADALN_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
ADALN_API int adaln_bwd_noalloc(const void* dy, const void* x, const float* mean,
              const float* rstd, const void* scale, const int32_t* seg_id,
              int64_t T, int32_t D, int32_t nseg, adaln_dtype_t dtype,
              void* dx, float* dshift, float* dscale, void* stream);

/*
 * One forward + backward step on HOST-resident tensors: the operator of
 * section 2.B of the AdaptiveLoad technical summary, as adaln_fwd followed by
 * adaln_bwd (the formulas at the top of this file), for training steps whose
 * tensors live in host memory.  The pages describe no host pipeline; this
 * entry point is this library's own.
 *
 * Rows are processed in chunks of at most `chunk_rows` (0 = about 32 MB per
 * [rows, D] tensor and chunk; shorter chunks at both ends shorten the time
 * the link carries one direction only): the copies of chunk i + 1 in and of
 * chunk i - 1 out overlap the kernels of chunk i, on three internal streams
 * of the current device.  The step starts after the work already queued on
 * `stream` and after the previous call of this function on the device;
 * `stream` waits for the whole step (the host buffers may be read once it
 * has drained).
 *
 * Arguments: x, dy, shift, scale, seg_id are HOST pointers read by the step;
 * y, mean, rstd, dx, dshift, dscale are HOST pointers it writes; shapes and
 * element types as above.  Page-locked (pinned) host memory lets the copies
 * run asynchronously; pageable memory works but serialises them.  `scratch`
 * is DEVICE memory of at least adaln_fwd_bwd_host_scratch_size(T, D, nseg,
 * dtype, chunk_rows) bytes, 256-byte aligned, owned by the caller; calls on
 * different scratch buffers may share none of them while in flight.
 *
 * Results: y, mean, rstd, dx equal those of the device calls bit for bit;
 * dshift, dscale add the chunks' per-segment sums in chunk order (a fixed
 * association, deterministic for a given chunk size).
 *
 * Errors: ADALN_ERR_DIM, _DTYPE as for adaln_fwd; ADALN_ERR_NULL for a NULL
 * pointer (row pointers may be NULL when T = 0); ADALN_ERR_ARG for a bad eps
 * or a negative chunk_rows; ADALN_ERR_ALIGN when scratch is not 256-byte
 * aligned; ADALN_ERR_WORKSPACE when scratch_bytes is too small;
 * ADALN_ERR_CUDA when a copy or launch fails
 * (work enqueued before the failure may still run).  Device data errors go
 * to the status word as for the device calls.
 */
ADALN_API int adaln_fwd_bwd_host_scratch_size(int64_t T, int32_t D, int32_t nseg,
              adaln_dtype_t dtype, int64_t chunk_rows, size_t* bytes);
ADALN_API int adaln_fwd_bwd_host(const void* x, const void* dy, const void* shift,
              const void* scale, const int32_t* seg_id, int64_t T, int32_t D,
              int32_t nseg, adaln_dtype_t dtype, float eps, void* y, float* mean,
              float* rstd, void* dx, float* dshift, float* dscale,
              int64_t chunk_rows, void* scratch, size_t scratch_bytes, void* stream);

/*
 * Queries and keys of the attention that a DiT block runs on modulated
 * tokens: rotary positions over up to four axes (time, height, width, ...),
 * with an optional RMS norm of every head in the same pass.  For one head x
 * of token t, R = 2P rotated elements, pair p on axis a(p) (the axes own
 * pairs[0], pairs[1], ... consecutive pairs, P in all), and
 * (c, s) = table[pos[t, a(p)], p]:
 *
 *   n  = x * w / sqrt(mean(x^2) + eps)                (n = x when norm = 0)
 *   y1 = n1 c - n2 s,   y2 = n2 c + n1 s              (y = n from element R on)
 *
 * where a pair's elements are (2p, 2p+1) (interleaved) or (p, p+P) (halves).
 * A position of -1 leaves that axis's pairs of the token unrotated (text
 * tokens of a joint stream).  A pair whose sine is zero takes nothing from
 * its partner.  Arithmetic is fp32, each output rounded once.
 */
typedef struct {
  void* ptr;            /* token 0, head 0, element 0 */
  int64_t token_stride; /* elements from a token to the next, >= 0 */
  int64_t head_stride;  /* elements from a head to the next, >= 0 */
} adaln_heads_t;        /* [T, heads, dh]; a head's elements are contiguous */

typedef struct {
  const float* table;   /* device, fp32 [rows, P, 2]: cosine, sine; 8-byte aligned */
  const int32_t* pos;   /* device, int32 [T, axes]: a row of the table, or -1 */
  int32_t rows;         /* >= 1 */
  int32_t axes;         /* 1 .. ADALN_MAX_ROPE_AXES */
  int32_t pairs[ADALN_MAX_ROPE_AXES]; /* pairs of each axis; 1 <= P, 2P <= dh */
  int32_t interleaved;  /* pairs of neighbours, else of the two halves */
} adaln_rope_t;

/*
 * Forward, one launch.  q [T, hq, dh] and k [T, hk, dh] (hk or hq may be 0,
 * its pointers NULL) may be views of a packed projection; q_out, k_out may be
 * the inputs themselves (in place), but may not overlap them otherwise, nor
 * themselves or each other.  wq, wk [dh] have the element type `dtype`; NULL
 * means ones.  Heads of at most 64 whole 16-byte vectors at 16-byte aligned
 * addresses take a vector path (for halves, P elements are then whole vectors
 * too, of 16, 8 or 4 bytes, aligned as such), everything else a scalar one with
 * the same results up to fp32 rounding.
 * A position outside [-1, rows) is treated as -1 and recorded in the status
 * word (ADALN_DEV_POS_RANGE).
 *
 * Errors: ADALN_ERR_DTYPE; ADALN_ERR_DIM for T outside [0, 2^31), dh outside
 * [1, ADALN_MAX_HEAD_DIM], head counts outside [0, ADALN_MAX_HEADS] or both 0,
 * axes, rows or pairs out of range, a negative stride, or an output two of whose
 * heads (of one token or of two) overlap; ADALN_ERR_NULL;
 * ADALN_ERR_ALIGN for a pointer below its element's alignment; ADALN_ERR_ARG
 * for a bad eps (with norm).
 */
ADALN_API int adaln_qk_rope_fwd(const adaln_heads_t* q, const adaln_heads_t* k, int64_t T,
              int32_t hq, int32_t hk, int32_t dh, adaln_dtype_t dtype,
              const adaln_rope_t* rope, int32_t norm, const void* wq, const void* wk,
              float eps, const adaln_heads_t* q_out, const adaln_heads_t* k_out,
              void* stream);

/*
 * Backward.  Without norm: dq, dk are dq_out, dk_out turned back (one launch;
 * q, k, workspace unused; dwq and dwk must be NULL).  With norm: also reads q
 * and k, the forward's inputs (it saves nothing), and, where dwq / dwk are not
 * NULL, writes the fp32 gradients [dh] of the weights, summed over tokens and
 * heads in a fixed order (a second launch; bitwise reproducible for a given
 * device and sizes).  dq, dk may be dq_out, dk_out or q, k themselves.
 * `workspace` holds the partial sums: at least
 * adaln_qk_rope_bwd_workspace_size bytes, 16-byte aligned, the caller's;
 * needed only with dwq or dwk.  T = 0 zeroes dwq and dwk.
 * Errors as for the forward; ADALN_ERR_WORKSPACE for a short workspace,
 * ADALN_ERR_ARG for a dwq or dwk without norm.
 */
ADALN_API int adaln_qk_rope_bwd_workspace_size(int64_t T, int32_t hq, int32_t hk, int32_t dh,
              adaln_dtype_t dtype, size_t* bytes);
ADALN_API int adaln_qk_rope_bwd(const adaln_heads_t* dq_out, const adaln_heads_t* dk_out,
              const adaln_heads_t* q, const adaln_heads_t* k, int64_t T, int32_t hq,
              int32_t hk, int32_t dh, adaln_dtype_t dtype, const adaln_rope_t* rope,
              int32_t norm, const void* wq, const void* wk, float eps,
              const adaln_heads_t* dq, const adaln_heads_t* dk, float* dwq, float* dwk,
              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gated feed-forward block of a transformer layer, on the tensor cores:
 *
 *   y = (act(x Wg') * (x Wu')) Wd'
 *
 * x, y, dy, dx [T, D]; Wg, Wu and their gradients [F, D]; Wd and its gradient
 * [D, F]; all bf16 (dtype must be ADALN_BF16), row-major and contiguous,
 * 16-byte aligned.  D and F are multiples of 8 up to ADALN_FFN_MAX_DIM, T is
 * at most ADALN_FFN_MAX_T.  Outputs, saved values and workspace may not overlap
 * each other or an input.  Sums are fp32; the hidden product h and, in the
 * backward, the gradients of the two projections are rounded to bf16 once,
 * like the outputs.
 */
typedef enum {
  ADALN_ACT_SILU = 0,      /* g / (1 + exp(-g)) */
  ADALN_ACT_GELU_TANH = 1, /* the tanh approximation of GELU */
  ADALN_ACT_GELU = 2       /* g Phi(g) */
} adaln_act_t;

/*
 * Device bytes: of what a forward saves for its backward (x Wg' and x Wu' at
 * 24 bits a value, in blocks of 32 tokens: 6 F bytes
 * a token), and of each call's workspace on the current
 * device (either pointer of the second may be NULL).
 */
ADALN_API int adaln_ffn_saved_size(int64_t T, int32_t D, int32_t F, adaln_dtype_t dtype,
              size_t* bytes);
ADALN_API int adaln_ffn_workspace_size(int64_t T, int32_t D, int32_t F, adaln_dtype_t dtype,
              size_t* fwd_bytes, size_t* bwd_bytes);

/*
 * Forward: two launches (a third where few rows make it worth splitting the
 * sum over F).  `saved` receives what the backward needs, adaln_ffn_saved_size
 * bytes; NULL for inference.  `workspace` is scratch of
 * adaln_ffn_workspace_size bytes.  T = 0 does nothing.
 *
 * Errors: ADALN_ERR_DTYPE, ADALN_ERR_DIM, ADALN_ERR_ARG (unknown act),
 * ADALN_ERR_NULL, ADALN_ERR_ALIGN (16 bytes), ADALN_ERR_WORKSPACE (short),
 * ADALN_ERR_CUDA.
 */
ADALN_API int adaln_ffn_fwd(const void* x, const void* wg, const void* wu, const void* wd,
              int64_t T, int32_t D, int32_t F, adaln_dtype_t dtype, adaln_act_t act,
              void* y, void* saved, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward, from dy, the forward's inputs and what it saved: dx and the three
 * weight gradients, in the weights' type.  No atomics: bitwise reproducible
 * for a given device and sizes.  T = 0 zeroes the weight gradients.  Errors
 * as for the forward.
 */
ADALN_API int adaln_ffn_bwd(const void* dy, const void* x, const void* wg, const void* wu,
              const void* wd, const void* saved, int64_t T, int32_t D, int32_t F,
              adaln_dtype_t dtype, adaln_act_t act, void* dx, void* dwg, void* dwu,
              void* dwd, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Dropout whose mask is never stored, with what stands around it where a branch
 * of a block meets the residual stream:
 *
 *   y = [x +] [gate[b] *] m s h                        b = seg_id[t]
 *
 * The mask m comes from a counter-based generator (Philox-4x32, ten rounds; key =
 * seed, counter = (t ceil(D / 8) + c, offset), 64 bits each, lowest word first):
 * elements 8c .. 8c + 7 of token t take the eight 16-bit parts of its output,
 * lowest first, and one is dropped (m = 0) where its part is below
 * n = floor(65536 p + 1/2).  s = 65536 / (65536 - n).  So the same seed and
 * offset give the same mask, in a backward too, whatever the element type and
 * the device; p = 0 (or below 2^-17) drops nothing and p = 1 everything, and
 * neither reads the generator's state.
 */
typedef struct {
  uint64_t seed, offset;
  const int64_t* state; /* device: (seed, offset) read from here when the call runs,
                           instead of the two above (for captured graphs, whose
                           replays then draw other masks); or NULL.  8-byte aligned */
} adaln_rng_t;

/*
 * Forward, one launch.  h, x, y [T, D] and gate [nseg, D] have the element type
 * `dtype`; x (the residual) and gate may be NULL, seg_id and nseg are used with a
 * gate only.  y may be h or x itself, but may not overlap them otherwise.
 * Arithmetic is fp32, y rounded once; a dropped element takes nothing from h or
 * the gate, whatever they hold.  A bad seg_id is clamped and recorded
 * (ADALN_DEV_SEG_RANGE, ADALN_DEV_SEG_ORDER).
 *
 * Errors: ADALN_ERR_DTYPE; ADALN_ERR_DIM for T outside [0, 2^31), D outside [1,
 * ADALN_DROPOUT_MAX_D] or not of whole 16-byte vectors, T ceil(D / 8) of 2^32 - 256
 * or more, or (with a gate) a bad nseg; ADALN_ERR_ARG for p outside [0, 1]; ADALN_ERR_NULL (rng too, where the
 * mask is drawn); ADALN_ERR_ALIGN (16 bytes, seg_id 4).
 */
ADALN_API int adaln_dropout_fwd(const void* h, const void* x, const void* gate,
              const int32_t* seg_id, int64_t T, int32_t D, int32_t nseg, adaln_dtype_t dtype,
              double p, const adaln_rng_t* rng, void* y, void* stream);

/*
 * Backward (dx is dy itself):
 *
 *   dh = [gate[b] *] m s dy,     dgate[b] = sum_{t: seg_id[t] = b} m s dy h
 *
 * Without dgate (NULL) one launch, and h and workspace are unused; with it (fp32
 * [nseg, D], needs gate and the forward's h) a second one adds partial sums in a
 * fixed order: bitwise reproducible for a given device and sizes.  dh may be dy or
 * h itself.  `workspace`: at least adaln_dropout_bwd_workspace_size bytes, 16-byte
 * aligned, the caller's.  T = 0 zeroes dgate.  Errors as for the forward;
 * ADALN_ERR_WORKSPACE for a short workspace.
 */
ADALN_API int adaln_dropout_bwd_workspace_size(int64_t T, int32_t D, int32_t nseg,
              adaln_dtype_t dtype, size_t* bytes);
ADALN_API int adaln_dropout_bwd(const void* dy, const void* h, const void* gate,
              const int32_t* seg_id, int64_t T, int32_t D, int32_t nseg, adaln_dtype_t dtype,
              double p, const adaln_rng_t* rng, void* dh, float* dgate, void* workspace,
              size_t workspace_bytes, void* stream);

/*
 * Tokens sorted by expert, and back, for a feed-forward block that is a mixture of
 * experts.  expert [T, k] holds each token's choices (-1: none, a padded token's
 * say; a token may name an expert twice).  A sorted array [rows, D] has expert 0's
 * pairs (t, j) first, in the order t k + j, then expert 1's, each expert's start
 * rounded up to a multiple of `align` rows; its rows between an expert's last and
 * the next one's start are zeros, and rows from starts[E] on are left as they were.
 *
 *   row [T, k]    each pair's row, -1 for expert -1
 *   starts [E+1]  each expert's first row, and the end of the last one's
 *   counts [E]    each expert's pairs
 *
 * all int32, in device memory: nothing here waits for the host.  `rows` is at least
 * adaln_route_rows: T k + min(E, T k) (align - 1), rounded down to whole `align`.
 * One launch; two above 131072 pairs, which need the workspace
 * (adaln_route_workspace_size bytes, 0 otherwise, 16-byte aligned).  An expert
 * outside [-1, E) counts as -1 and is recorded (ADALN_DEV_EXPERT_RANGE).  T = 0
 * writes starts and counts.
 *
 * Errors: ADALN_ERR_DIM for T outside [0, 2^31), k outside [1, ADALN_MAX_TOPK], E
 * outside [1, ADALN_MAX_EXPERTS], align outside [1, ADALN_MAX_ROUTE_ALIGN] or rows
 * above 2^31 - 1; ADALN_ERR_NULL, ADALN_ERR_ALIGN, ADALN_ERR_WORKSPACE.
 */
ADALN_API int adaln_route_rows(int64_t T, int32_t k, int32_t E, int32_t align, int64_t* rows);
ADALN_API int adaln_route_workspace_size(int64_t T, int32_t k, int32_t E, size_t* bytes);
ADALN_API int adaln_route(const int32_t* expert, int64_t T, int32_t k, int32_t E, int32_t align,
              int32_t* row, int32_t* starts, int32_t* counts, void* workspace,
              size_t workspace_bytes, void* stream);

/*
 * xs[row[t, j]] = x[t], and the gradient dx[t] = sum_j dxs[row[t, j]] (fp32 sums, j
 * in order).  x, dx [T, D] and xs, dxs [rows, D] have the element type `dtype`, D as
 * for the dropout.  A row outside [-1, rows) is skipped and recorded
 * (ADALN_DEV_EXPERT_RANGE).  T = 0 does nothing.  Outputs may not overlap inputs.
 * Errors as above and ADALN_ERR_DTYPE.
 */
ADALN_API int adaln_expert_sort_fwd(const void* x, const int32_t* row, const int32_t* starts,
              const int32_t* counts, int64_t T, int32_t k, int32_t E, int32_t align, int32_t D,
              adaln_dtype_t dtype, int64_t rows, void* xs, void* stream);
ADALN_API int adaln_expert_sort_bwd(const void* dxs, const int32_t* row, int64_t T, int32_t k,
              int32_t D, adaln_dtype_t dtype, int64_t rows, void* dx, void* stream);

/*
 * y[t] = sum_j weight[t, j] ys[row[t, j]] with weight fp32 [T, k], and its gradients
 * dys[row[t, j]] = weight[t, j] dy[t] (zeros between the experts, as in xs) and, fp32
 * [T, k], dweight[t, j] = <dy[t], ys[row[t, j]]> (0 for expert -1).  No atomics:
 * bitwise reproducible.  Otherwise as the sort.
 */
ADALN_API int adaln_expert_combine_fwd(const void* ys, const float* weight, const int32_t* row,
              int64_t T, int32_t k, int32_t D, adaln_dtype_t dtype, int64_t rows, void* y,
              void* stream);
ADALN_API int adaln_expert_combine_bwd(const void* dy, const void* ys, const float* weight,
              const int32_t* row, const int32_t* starts, const int32_t* counts, int64_t T,
              int32_t k, int32_t E, int32_t align, int32_t D, adaln_dtype_t dtype, int64_t rows,
              void* dys, float* dweight, void* stream);

/*
 * The gated feed-forward block of each expert on its rows of a sorted array (a
 * route's with `align` a multiple of 64):
 *
 *   y = (act(x Wg[e]') * (x Wu[e]')) Wd[e]'            for expert e's rows x
 *
 * xs, ys, dys, dxs [rows, D]; Wg, Wu and their gradients [E, F, D]; Wd and its
 * gradient [E, D, F], all bf16, contiguous, 16-byte aligned; starts int32 [E + 1] in
 * device memory, multiples of 64 from 0 on that do not decrease, up to rows.  Expert e's
 * rows are those from starts[e] on to starts[e + 1], zero rows between the tokens'
 * and the next expert's among them: xs and dys have zeros there (as the sort and the
 * combination's backward write them), and ys and dxs get zeros.  Rows from starts[E]
 * on are neither read into a result nor written.  Sums, roundings and what is saved
 * are the feed-forward block's: h, dg and du are rounded to bf16 before the products that
 * take them, so results are off by two roundings where one is the least (of normally
 * distributed values 2.35e-3 in the 2-norm, 1.66e-3 with none in between).  So are D and
 * F; rows is at most ADALN_FFN_MAX_T.
 * Starts that break these rules are recorded (ADALN_DEV_EXPERT_RANGE); no access leaves
 * the arrays, and the outputs of such a call are unspecified.
 *
 * Forward: two launches (a third where few rows make it worth splitting the sum over
 * F).  Backward: two launches (three with few rows, or where dx's sum is split); the
 * gradient of an expert without rows is zeros.  No atomics: bitwise reproducible for a
 * given device and sizes.  Errors as for the feed-forward block.
 */
ADALN_API int adaln_experts_ffn_saved_size(int64_t rows, int32_t E, int32_t D, int32_t F,
              adaln_dtype_t dtype, size_t* bytes);
ADALN_API int adaln_experts_ffn_workspace_size(int64_t rows, int32_t E, int32_t D, int32_t F,
              adaln_dtype_t dtype, size_t* fwd_bytes, size_t* bwd_bytes);
ADALN_API int adaln_experts_ffn_fwd(const void* xs, const void* wg, const void* wu, const void* wd,
              const int32_t* starts, int64_t rows, int32_t E, int32_t D, int32_t F,
              adaln_dtype_t dtype, adaln_act_t act, void* ys, void* saved, void* workspace,
              size_t workspace_bytes, void* stream);
ADALN_API int adaln_experts_ffn_bwd(const void* dys, const void* xs, const void* wg, const void* wu,
              const void* wd, const int32_t* starts, const void* saved, int64_t rows, int32_t E,
              int32_t D, int32_t F, adaln_dtype_t dtype, adaln_act_t act, void* dxs, void* dwg,
              void* dwu, void* dwd, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Synchronise `stream`, then read and clear the status word: the one the
 * calling thread bound (adaln_status_bind), else the current device's.
 * *host_bits (if non-NULL) receives the ADALN_DEV_* bits.  Returns ADALN_OK,
 * ADALN_ERR_SEG, ADALN_ERR_POS, ADALN_ERR_EXPERT, ADALN_ERR_TIMEOUT or ADALN_ERR_CUDA.  The device's word is
 * shared by all calls on the device that use it since it was last cleared.
 */
ADALN_API int adaln_get_status(uint32_t* host_bits, void* stream);

/*
 * Bind a caller-owned device status word for the calls the calling host
 * thread makes from now on (its kernels OR ADALN_DEV_* bits into it, and
 * adaln_get_status() reads and clears it), instead of the device's shared
 * word; NULL returns to the shared word.  For callers that drive several
 * streams: with one word per stream (bound by the thread issuing that
 * stream's calls), a data error is reported to the caller whose call caused
 * it.  `device_word` is a 4-byte aligned uint32 in device memory of the
 * device the calls run on, owned by the caller, zeroed by the caller before
 * first use, and left bound until unbound or the thread exits (the library
 * keeps only the pointer).  Returns ADALN_OK or ADALN_ERR_ALIGN.  The paper
 * describes no status reporting; this is the library's own.
 */
ADALN_API int adaln_status_bind(uint32_t* device_word);

/* Static description of a status code. */
ADALN_API const char* adaln_strerror(int code);

/*
 * Kernel timing trace.  Between adaln_trace_begin(capacity) and
 * adaln_trace_end(), every kernel launch made by this library (from any
 * thread) is bracketed by a pair of CUDA events recorded on its stream, up to
 * `capacity` launches.  adaln_trace_end() synchronises those events and sums
 * the elapsed time per kernel; adaln_trace_get() reads the sums.
 * Kernel ids: ADALN_KERNEL_FWD, ADALN_KERNEL_BWD_ROWS, ADALN_KERNEL_BWD_FINALIZE;
 * ADALN_KERNEL_QK_ROPE, ADALN_KERNEL_FFN, ADALN_KERNEL_DROPOUT and
 * ADALN_KERNEL_EXPERTS count every launch of the rotary, the feed-forward, the
 * dropout and the experts' calls (5 is no id).
 */
#define ADALN_KERNEL_FWD 0
#define ADALN_KERNEL_BWD_ROWS 1
#define ADALN_KERNEL_BWD_FINALIZE 2
#define ADALN_KERNEL_QK_ROPE 3
#define ADALN_KERNEL_FFN 4
#define ADALN_KERNEL_DROPOUT 6
#define ADALN_KERNEL_EXPERTS 7
#define ADALN_NUM_KERNELS 8
ADALN_API int adaln_trace_begin(int capacity);
ADALN_API int adaln_trace_end(void);
ADALN_API int adaln_trace_get(int kernel_id, int64_t* launches, double* total_ms);

/*
 * Self-test of failure detection: launches one thread that waits, through the
 * bounded wait the staging pipelines use, on an mbarrier that nothing ever
 * completes, giving up after limit_us microseconds (1..100000).  On return of
 * the next adaln_get_status() the device status word must hold
 * ADALN_DEV_TIMEOUT (ADALN_ERR_TIMEOUT), and the device must remain usable.
 * The pipelines' own limit is 2 s; the staging kernels never wait unbounded.
 */
ADALN_API int adaln_selftest_wait_timeout(uint32_t limit_us, void* stream);

/*
 * Launch shape chosen for these sizes on the current device: grid (CTAs),
 * threads per CTA, ring stages, dynamic shared memory bytes.  `which` is
 * ADALN_KERNEL_FWD or ADALN_KERNEL_BWD_ROWS.  For reports and tests.
 */
ADALN_API int adaln_launch_shape(int which, int64_t T, int32_t D, int32_t nseg,
                       adaln_dtype_t dtype, int32_t* grid, int32_t* threads,
                       int32_t* stages, int32_t* smem_bytes);

#ifdef __cplusplus
}
#endif
#endif /* ADALN_H */
