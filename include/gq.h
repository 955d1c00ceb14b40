/*
 * gq.h -- C ABI of the B200 library for bucketed gradient quantization (libgq.so).
 *
 * The library implements the data-parallel step that the page "gradient quantization for
 * communication" (glossary) describes in its section "How Gradient Quantization Works":
 * Quantize -> Transmit -> Dequantize -> Aggregate, with the error feedback of its section
 * "Quantization Schemes".  Quantize is bucketed (buckets of d elements, the review
 * "[Paper Review] Optimal Gradient Quantization Condition for Communication-Efficient
 * Distributed Training", section "Proposed method") with one of five level fits:
 *   QSGD-s and TernGrad (max-abs scaling; "Gradient Quantization" glossary),
 *   BinGrad-b, BinGrad-pb and ORQ-s (the review's proposed schemes).
 * W workers are W separate buffers on one GPU; "Transmit" is the message each worker writes to
 * device memory, and Dequantize + Aggregate read it back (or, in gq_fused_step, never leave
 * the chip).
 *
 * Conventions for every call:
 *   - Pointers named "device" are CUDA device (or managed) memory owned by the caller, 16-byte
 *     aligned.  Arrays of pointers (grads[], residuals[], msgs[]) are HOST arrays of W device
 *     pointers.  The library keeps no pointer after a call returns.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls only enqueue
 *     work; results are ready when the stream is.  Calls on one plan must not overlap on the
 *     GPU (the plan's status word is shared).
 *   - Argument errors are reported synchronously (GQ_ERR_INVALID / GQ_ERR_UNSUPPORTED) and
 *     nothing is enqueued.  A launch failure returns GQ_ERR_CUDA.  Non-finite input does not
 *     fail the call: it raises a flag on the plan that gq_plan_status reports; the outputs of
 *     the affected bucket are then unspecified (but every access stays in bounds).
 *   - The library never allocates inside a call except gq_plan_create.
 *   - With n = 0 every call is a no-op that returns GQ_OK; data pointers may then be NULL.
 */
#ifndef GQ_H
#define GQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define GQ_API __attribute__((visibility("default")))
#else
#define GQ_API
#endif

#define GQ_MAX_WORKERS 64
#define GQ_MIN_BUCKET 128
#define GQ_MAX_BUCKET 32768
#define GQ_MAX_LEVELS 16
/* Largest level count of the QSGD family (QSGD, QSGD-nearest, QSGD-l2): 129 .. 256 levels take
 * 8-bit codes (255 levels with nearest rounding is symmetric INT8). */
#define GQ_MAX_QSGD_LEVELS 256

typedef enum {
    GQ_QSGD = 0,       /* s uniform levels on [-m, m], m = max|u| of the bucket, stochastic rounding */
    GQ_TERNGRAD = 1,   /* QSGD with s = 3: levels {-m, 0, m} */
    GQ_BINGRAD_B = 2,  /* two levels at the side means of the SSE-optimal split, deterministic */
    GQ_BINGRAD_PB = 3, /* two grid levels at least as far apart as BinGrad-b's, minimising the expected squared
                        * error among such pairs; stochastic inside, clamped outside */
    GQ_ORQ = 4,        /* s levels: {min, max} plus s-2 greedy picks from a 64-point grid, stochastic rounding */
    /* Biased baselines ("Gradient Quantization" glossary, "Deterministic vs stochastic rounding"
     * and "Ternary and binary quantization"); buckets of d <= 512 only: */
    GQ_QSGD_NEAREST = 5, /* the QSGD-s levels and message, each value rounded to its nearest level (ties to the
                          * upper one), no randomness; s = 3 is deterministic TernGrad, s = 15 symmetric INT4 */
    GQ_SIGNSGD = 6,      /* scaled sign: levels -m1 and +m1, m1 = mean |u| of the bucket (exact fixed-point
                          * sum), code 1 for u >= 0; 1 bit per element */
    /* QSGD as published (l2 scaling; the glossary's QSGD, whose codes are Elias-coded), d <= 512: */
    GQ_QSGD_L2 = 7,      /* the QSGD-s levels and stochastic rounding with m = ||u||_2 of the bucket (exact
                          * fixed-point sum of squares) in place of max |u|; sparse codes for gq_elias_pack */
    /* TernGrad with one scale per parameter tensor (the glossary's "single scaling factor per
     * layer"); needs the tensors' offsets (gq_plan_set_segments); no clipping: */
    GQ_TERNGRAD_LAYER = 8
} gq_scheme_t;

typedef enum {
    GQ_OK = 0,
    GQ_ERR_INVALID = 1,     /* an argument is out of range, NULL where required, or misaligned */
    GQ_ERR_UNSUPPORTED = 2, /* a valid combination this build does not implement */
    GQ_ERR_CUDA = 3,        /* a CUDA call failed (launch, allocation of the plan's status word) */
    GQ_ERR_NONFINITE = 4,   /* gq_plan_status: some input value was NaN or infinite */
    GQ_ERR_NOMEM = 5,       /* host allocation failed */
    GQ_ERR_TIMEOUT = 6      /* gq_plan_status: a kernel's bounded wait for a bulk copy gave up */
} gq_status_t;

/*
 * Configuration of a plan.
 *   scheme         gq_scheme_t.
 *   levels         s.  QSGD: 2..16.  TernGrad: 3 (0 means 3).  BinGrad-b/pb: 2 (0 means 2).
 *                  ORQ: 2..16.  QSGD-nearest, QSGD-l2: 2..16.  SignSGD: 2 (0 means 2).  Codes take
 *                  b = ceil(log2 s) bits (1..4).
 *   bucket         d, elements per bucket: a power of two in [128, 32768] (at most 512 for
 *                  QSGD-nearest, SignSGD and QSGD-l2: GQ_ERR_UNSUPPORTED above).  The vector is cut
 *                  into ceil(n/d) buckets; the last one may hold fewer than d elements.
 *   workers        W in [1, 64] for gq_fused_step (gq_encode ignores it).
 *   error_feedback 1: v = g + r is quantized and r <- v - Q(v); 0: v = g, no residual.
 *   clip_sigma     c >= 0.  c > 0 clips each bucket to [-c*sigma, c*sigma] before the fit
 *                  (sigma: the bucket's population standard deviation); the residual keeps the
 *                  clipped part.  0 disables clipping.
 *   seed           key of the Philox4x32-10 stream used for stochastic rounding.
 *   n              elements per worker, 0 <= n < 2^40.
 */
typedef struct {
    int32_t scheme;
    int32_t levels;
    int32_t bucket;
    int32_t workers;
    int32_t error_feedback;
    float clip_sigma;
    uint64_t seed;
    int64_t n;
} gq_config_t;

typedef struct gq_plan *gq_plan_t; /* opaque; owned by the library */

/* Validate a configuration without touching any device.  GQ_OK if a plan can be made. */
GQ_API gq_status_t gq_config_check(const gq_config_t *cfg);

/*
 * Layout of one worker's message, the bytes a worker would transmit (host computation, no
 * device needed).  *bytes: total size.  *codes_off: offset of the packed codes, ceil(n/d)
 * buckets of d*b/32 uint32 words each.  *levels_off: offset (16-byte aligned) of the level
 * tables, ceil(n/d) tables of L float32 each (L = 1 for the QSGD family: the scale m;
 * 2 for BinGrad-b/pb and SignSGD: the two levels; s for ORQ: the ascending levels).
 * Packing inside a bucket: dense, in element order, least significant bit first: bit j of the
 * code (the index of its level) of element e is bit (b*e + j) % 32 of word (b*e + j) / 32 of
 * the bucket's words.  Padding elements of the last bucket have code 0.
 * Any output pointer may be NULL.
 */
GQ_API gq_status_t gq_message_layout(const gq_config_t *cfg, size_t *bytes, size_t *codes_off, size_t *levels_off);

/* Create a plan: validates cfg, selects kernels and allocates on the current device the plan's
 * 4-byte status word and the scratch of gq_quant_error (the only device allocations the library
 * makes).  The plan must be used on that device only. */
GQ_API gq_status_t gq_plan_create(const gq_config_t *cfg, gq_plan_t *out);
/* Free the plan (synchronous; the caller must make sure no work of the plan is pending). */
GQ_API gq_status_t gq_plan_destroy(gq_plan_t plan);

/*
 * Quantize: one worker's gradient into its message (the "Quantize" step, with error feedback).
 *   worker    Philox worker index of this gradient (any 32-bit value; the draws for element i
 *             are keyed on (seed, step, worker, i)).
 *   step      training step; its low 32 bits key the draws.
 *   grad      device, n float32, read only.
 *   residual  device, n float32, read and overwritten with v - Q(v); must be NULL iff the
 *             plan's error_feedback is 0.
 *   msg       device, gq_message_layout bytes, written completely.
 */
GQ_API gq_status_t gq_encode(gq_plan_t plan, uint32_t worker, uint64_t step, const float *grad, float *residual,
                      void *msg, void *stream);

/*
 * Dequantize + Aggregate: avg[i] = (sum over w = 0..nmsgs-1, in that order, of the level of
 * element i in msgs[w]) * (1/nmsgs), in float32.
 *   msgs      host array of nmsgs (1..64) device pointers to messages written by gq_encode
 *             or gq_fused_step with this plan's configuration.
 *   avg       device, n float32, overwritten.
 */
GQ_API gq_status_t gq_decode_accumulate(gq_plan_t plan, const void *const *msgs, int nmsgs, float *avg, void *stream);

/*
 * The whole step for the plan's W workers: worker w (w = 0..W-1, Philox worker index w) is
 * quantized as by gq_encode and the mean of the W dequantized gradients is written to avg,
 * as by gq_decode_accumulate; the dequantized values never leave the chip (for d <= 512 they
 * are summed in registers; for larger buckets one CTA walks a bucket's W workers and keeps the
 * running sum in shared memory, or, above d = 8192, in avg's own slice while it stays in L2).
 *   grads      host array of W device pointers (n float32 each).
 *   residuals  host array of W device pointers (in/out), or NULL iff error_feedback is 0.
 *   msgs       host array of W device pointers receiving the messages, or NULL not to write
 *              messages.
 *   avg        device, n float32, overwritten.
 */
GQ_API gq_status_t gq_fused_step(gq_plan_t plan, uint64_t step, const float *const *grads, float *const *residuals,
                          void *const *msgs, float *avg, void *stream);

/*
 * Quantization error of one worker's gradient, for measuring how much a fit loses (the
 * expected quantization variance the review's ORQ minimises, section "Proposed method").  The
 * fit and the rounding are those of gq_encode (same worker, step and draws); nothing but `out`
 * is written and the residual is only read.
 *   out   device, 3 doubles: out[0] = sum over elements of the expected squared rounding error
 *         p (b - u)^2 + (1 - p) (a - u)^2 given the fitted levels (u the value quantized after
 *         clipping, [a, b] its bracket, p its probability of rounding up; (b - u)(u - a) for
 *         unbiased rounding), out[1] = sum of u^2, out[2] = sum of (Q(u) - u)^2 for this
 *         step's draws.  Binary64; each bucket's sums are reduced in a fixed order, so the
 *         result does not depend on the launch shape.
 * Uses the plan's error scratch of 24 * (ceil(n/d) + ceil(ceil(n/d) / 4096)) bytes.
 */
GQ_API gq_status_t gq_quant_error(gq_plan_t plan, uint32_t worker, uint64_t step, const float *grad,
                                  const float *residual, double *out, void *stream);

/*
 * Allocation-free variant of gq_quant_error.  There is no counterpart in the paper: this entry
 * point exists for callers that cannot call cudaMalloc -- code running inside a framework's
 * caching allocator or memory pool (which must not be re-entered), processes whose device
 * memory is reserved up front, plugins that are handed buffers but no allocator.  Such callers
 * cannot create a plan (gq_plan_create allocates), so this call takes the configuration and
 * computes exactly what gq_quant_error computes for it, bit for bit (cfg->workers is ignored:
 * any value is accepted, the call covers one worker's gradient).
 * Its scratch is a file-scope device array of the library, GQ_NOALLOC_SCRATCH_BYTES (about
 * 384 KB), held on every device that loads the library until the process exits.  Hence:
 *   - the input may span at most GQ_NOALLOC_MAX_BUCKETS buckets (ceil(n/d) <= 16384); larger
 *     inputs return GQ_ERR_UNSUPPORTED before anything is enqueued;
 *   - every call on a device shares that scratch and leaves its contents behind; calls whose
 *     work overlaps on the GPU (different streams or host threads) race;
 *   - there is no plan status word to query: when a kernel of the call sees a non-finite value,
 *     or a bounded wait of its kernels gives up (the kernel then stops early), all three
 *     outputs are NaN;
 *   - the first call on each device looks up the scratch's device address
 *     (cudaGetSymbolAddress) and caches it with the identity of the device's current context;
 *     make that first call, and the first call after the context was replaced (for instance by
 *     cudaDeviceReset), before any stream capture.
 * Allocates nothing, on the device or on the host.
 */
#define GQ_NOALLOC_MAX_BUCKETS 16384
#define GQ_NOALLOC_SCRATCH_BYTES (256 + 24 * (GQ_NOALLOC_MAX_BUCKETS + (GQ_NOALLOC_MAX_BUCKETS + 4095) / 4096))
GQ_API gq_status_t gq_quant_error_noalloc(const gq_config_t *cfg, uint32_t worker, uint64_t step, const float *grad,
                                          const float *residual, double *out, void *stream);

/*
 * Base-s packing of a message's codes.  The review "[Paper Review] Optimal Gradient Quantization
 * Condition for Communication-Efficient Distributed Training" ("Key findings") quotes
 * compression ratios of 20.2 for 3 levels and 10.1 for 9 levels, which are 32 / log2(s) bits:
 * codes of s levels carry log2(s) bits each, and b = ceil(log2 s) bits waste the rest.  These
 * calls convert between the dense message of gq_message_layout and a base-s message in which,
 * per bucket, g consecutive codes form one number V = sum_k code[g*i + k] * s^k (codes past the
 * bucket's d-th count as 0) of B bits:
 *     s = 3: g = 5, B = 8   (1.6 bits per code)
 *     s = 5: g = 3, B = 7   (2.33 bits per code)
 *     s = 9: g = 5, B = 16  (3.2 bits per code)
 * Other level counts return GQ_ERR_UNSUPPORTED.  Group i of a bucket is bits B*i .. B*i + B - 1,
 * least significant bit first, of the bucket's ceil(ceil(d/g) * B / 32) uint32 words (the bits
 * above the last group are 0).
 *
 * gq_entropy_layout: *bytes total; *codes_off = 0: the ceil(n/d) buckets' words, one after the
 * other; *levels_off (16-byte aligned): the level tables, exactly as in the dense message.  Host
 * computation, any output pointer may be NULL.
 */
GQ_API gq_status_t gq_entropy_layout(const gq_config_t *cfg, size_t *bytes, size_t *codes_off, size_t *levels_off);

/*
 * gq_entropy_pack: dense message -> base-s message.  gq_entropy_unpack: the inverse.
 *   cfg   the configuration the message was written with (cfg->workers is ignored).
 *   msg   device, the dense message (gq_message_layout bytes); read by pack, written completely
 *         by unpack (its padding bytes 0).
 *   emsg  device, the base-s message (gq_entropy_layout bytes); written completely by pack (its
 *         padding bytes 0), read by unpack.
 * Both 16-byte aligned and not overlapping (GQ_ERR_INVALID otherwise).  A dense message with a
 * code >= s packs to unspecified group values below 2^B, and a base-s message with a group value
 * >= s^g unpacks to unspecified codes below 2^b (accesses stay in bounds either way).
 * Stateless: no plan, no status word, no allocation; one kernel launch on `stream`.
 */
GQ_API gq_status_t gq_entropy_pack(const gq_config_t *cfg, const void *msg, void *emsg, void *stream);
GQ_API gq_status_t gq_entropy_unpack(const gq_config_t *cfg, const void *emsg, void *msg, void *stream);

/*
 * Elias-gamma coding of a message's codes.  The glossary "Gradient Quantization" (section QSGD)
 * says QSGD encodes its quantized values with Elias integer coding for further lossless
 * compression.  Elias gamma (Elias, 1975) writes x >= 1 with N = floor(log2 x) as N zero bits
 * followed by x's N + 1 bits, most significant first.  Supported: the QSGD family (QSGD,
 * TernGrad, QSGD-nearest, QSGD-l2) with an odd number of levels s and d <= 512; anything else
 * returns GQ_ERR_UNSUPPORTED.  Code c is sent as the signed level z = c - (s-1)/2, zigzag-mapped
 * to x = 2z + 1 (z >= 0) or -2z (z < 0): the zero level costs one bit.
 *
 * Message, little-endian: [uint64 T: the stream's bit count][8 zero bytes][ceil(n/d) uint64:
 * each bucket's first stream bit, padded to 16 bytes][the level tables, as in the dense message,
 * padded to 16 bytes][the stream: every bucket's valid codes in element order, stream bit k is
 * bit k % 32 of word k / 32, zero bits after T up to the next 16 bytes].  Its size depends on
 * the data: gq_elias_used_bytes(T) of the gq_elias_layout capacity are written.
 *
 * gq_elias_layout: *cap_bytes the largest message (buffers are sized for it), and the offsets of
 * the offsets region, the tables region and the stream.  Host computation; outputs may be NULL.
 * gq_elias_used_bytes: bytes of a message whose stream holds `stream_bits` bits (T, read by the
 * caller from the message's first 8 bytes).  GQ_ERR_INVALID if T exceeds the capacity.
 */
GQ_API gq_status_t gq_elias_layout(const gq_config_t *cfg, size_t *cap_bytes, size_t *offsets_off, size_t *tables_off,
                                   size_t *stream_off);
GQ_API gq_status_t gq_elias_used_bytes(const gq_config_t *cfg, uint64_t stream_bits, size_t *bytes);

/*
 * gq_elias_pack: dense message -> Elias message (five launches on `stream`; its level-table
 * region serves as the scan's scratch before the tables are written).  gq_elias_unpack: the
 * inverse (one launch).
 *   msg   device, the dense message (gq_message_layout bytes): read by pack, written completely
 *         by unpack.
 *   emsg  device, gq_elias_layout capacity bytes: its first gq_elias_used_bytes(T) bytes are
 *         written by pack (the rest is left as it was) and read by unpack.
 * Both 16-byte aligned and not overlapping (GQ_ERR_INVALID otherwise).  Codes >= s in a dense
 * message are encoded as s - 1; a damaged stream decodes to unspecified codes below 2^b, every
 * read inside the capacity.  Stateless: no plan, no allocation.
 */
GQ_API gq_status_t gq_elias_pack(const gq_config_t *cfg, const void *msg, void *emsg, void *stream);
GQ_API gq_status_t gq_elias_unpack(const gq_config_t *cfg, const void *emsg, void *msg, void *stream);

/*
 * TernGrad with one scale per parameter tensor (scheme GQ_TERNGRAD_LAYER, 3 levels).  The
 * glossary "Gradient Quantization" (section Ternary and binary quantization) gives TernGrad a
 * single scaling factor per layer; here the gradient is the concatenation of nseg tensors,
 * tensor t holding elements [offsets[t], offsets[t+1]).  Per worker m_t = max |v| over tensor t
 * (v = g + r), and each element is rounded between the two of {-m_t, 0, +m_t} around it exactly
 * as GQ_TERNGRAD rounds it (same position, probability and Philox draw).
 * Message: the 2-bit codes in the layout of the dense message (bucket after bucket), then the
 * nseg scales (float32); both regions 16-byte aligned.  gq_message_layout cannot size it (it
 * depends on nseg): use gq_plan_message_layout.
 *
 * gq_plan_set_segments: offsets is a HOST array of nseg + 1 non-decreasing offsets with
 * offsets[0] = 0 and offsets[nseg] = n (empty tensors allowed); the plan copies it to device
 * memory it owns (this call allocates, like gq_plan_create; a second call replaces the first).
 * GQ_ERR_INVALID for another scheme or bad offsets.  gq_encode, gq_decode_accumulate and
 * gq_fused_step on such a plan return GQ_ERR_INVALID until the segments are set; gq_quant_error
 * returns GQ_ERR_UNSUPPORTED.
 * gq_plan_message_layout: the plan's message size and region offsets (any scheme; for
 * GQ_TERNGRAD_LAYER once the segments are set).
 */
GQ_API gq_status_t gq_plan_set_segments(gq_plan_t plan, const int64_t *offsets, int nseg);
GQ_API gq_status_t gq_plan_message_layout(gq_plan_t plan, size_t *bytes, size_t *codes_off, size_t *levels_off);

/*
 * The format of a plan's messages.  The review "[Paper Review] Optimal Gradient Quantization
 * Condition for Communication-Efficient Distributed Training" ("Key findings") quotes compression
 * ratios of 32 / log2(s); GQ_FORMAT_BASE_S is the message of gq_entropy_pack (g codes per B-bit
 * base-s number, the level tables unchanged), written by gq_encode / gq_fused_step and read by
 * gq_decode_accumulate directly, so that no dense message exists.  s = 3, 5 or 9 levels; ORQ and
 * the QSGD family (QSGD, TernGrad, QSGD-nearest, QSGD-l2); d <= 512.
 * gq_plan_set_format: GQ_FORMAT_DENSE (the default) or GQ_FORMAT_BASE_S; afterwards
 * gq_plan_message_layout gives the message size and offsets (gq_entropy_layout's for base-s).
 * GQ_ERR_UNSUPPORTED for a plan base-s does not cover, GQ_ERR_INVALID for an unknown format.
 * Host only; no allocation.  gq_message_layout keeps describing the dense message.
 */
#define GQ_FORMAT_DENSE 0
#define GQ_FORMAT_BASE_S 1
GQ_API gq_status_t gq_plan_set_format(gq_plan_t plan, int format);

/* Synchronize `stream`, then report and clear the plan's status flags: GQ_ERR_TIMEOUT if a
 * kernel's bounded wait for a bulk copy gave up (the kernel then stopped early; its outputs are
 * incomplete), else GQ_ERR_NONFINITE if a non-finite input was seen since the last call;
 * GQ_ERR_CUDA if the stream failed. */
GQ_API gq_status_t gq_plan_status(gq_plan_t plan, void *stream);

/* Self-test of the failure path, no counterpart in the pages: every wait of the kernels for a
 * bulk copy is bounded in time and, when it gives up, raises the plan's timeout flag instead of
 * hanging; the waits inside gq_act_weight_grad are bounded in cycles.  This call enqueues three
 * warps that wait, with those same bounded waits, on barriers that nothing completes; after
 * limit_ns nanoseconds (clamped to [1e6, 1e9]) and twice as many cycles they give up, and once
 * all have, the flag is raised.  gq_plan_status then returns GQ_ERR_TIMEOUT, and the plan and the
 * context stay usable.  Returns GQ_ERR_INVALID for a NULL plan, GQ_ERR_CUDA if the launch fails. */
GQ_API gq_status_t gq_selftest_bounded_wait(gq_plan_t plan, int64_t limit_ns, void *stream);

/*
 * Activations kept in 8 bits, and the backward pass that reads them.
 *
 * The gradient that gq_encode takes is made by a backward pass, which needs every layer's input of
 * the forward pass.  These calls keep such an input in 8 bits (a "checkpoint", 33/32 bytes per
 * element) and compute from it the slices of the flat float32 gradient vector: a linear layer's
 * weight and bias gradient, a layer norm's, and the gradients passed on through activation
 * functions and norms.  There is no counterpart in the pages; the bucketed codes and the table of
 * scales are the message's idea (gq_message_layout) on groups of 32.
 *
 * Conventions, besides those above:
 *   - Stateless: no plan, no status word, no allocation.  Calls that may overlap on the GPU (other
 *     streams, other captured graphs) need outputs and workspaces of their own.  The first call of a
 *     kind in a process loads its kernels: make it before any stream capture.
 *   - A matrix is rows of cols elements of type `dtype`, its rows `stride` elements apart; a column
 *     step other than 1 is not supported.  Rows of an input may repeat (stride 0) or overlap; those
 *     of an output may not (stride >= cols).  With one row the stride is not used.  The first row
 *     starts on 16 bytes, as every device pointer; the others may start anywhere, and take the faster
 *     loads where they too start on 16 bytes.
 *   - 0 <= rows < 2^31, 1 <= cols <= GQ_ACT_MAX_COLS.  With rows = 0 nothing is read; gradients that
 *     sum over the rows are then written as 0 (or left as they are when accumulating).
 *   - float32 outputs (gradients, mean, rstd) and mean/rstd inputs need 4-byte alignment only, so
 *     that they may be any slice of a flat vector; gamma and beta their type's.
 *   - No output may share memory with an input or another output (GQ_ERR_INVALID); columns of one
 *     wider buffer with the same stride do not share any.
 *   - Non-finite values pass through as in the formulas; a group with one in a checkpoint reads as
 *     NaN throughout.  Sums are binary32 and their order is fixed: equal calls give equal bits.  The
 *     order may depend on the call's sizes: a row may get other last bits among another number of rows.
 *   - Should a kernel's bounded wait give up (a fault: no wait is expected to last a second), the
 *     outputs it was computing are NaN; there is no status word to ask.
 */
#define GQ_ACT_MAX_COLS (1 << 24)

typedef enum { GQ_FLOAT32 = 0, GQ_BFLOAT16 = 1, GQ_FLOAT16 = 2 } gq_dtype_t;

/*
 * Layout of the checkpoint of rows x cols values (host computation; outputs may be NULL).
 * codes_off = 0: rows of int8 codes, each row padded with 0 to a whole number of groups of 32
 * columns (pitch 32 * ceil(cols / 32) bytes).  exps_off (16-byte aligned): rows of exponent bytes,
 * one per group, each row padded with 0 to a multiple of four (pitch 4 * ceil(cols / 128) bytes).
 * Value of code q under exponent E: q * 2^(E - 133); E = 255: NaN.
 * E is chosen per group from m = max |x|: the smallest for which every code rint(x * 2^(133 - E)),
 * ties to even, stays within +-127, at least 0 and at most 254 (where codes saturate at +-127).
 * Every value is exact in bfloat16 and float32.
 */
GQ_API gq_status_t gq_act_layout(int64_t rows, int64_t cols, size_t *bytes, size_t *codes_off, size_t *exps_off);

/* x -> checkpoint (device, gq_act_layout bytes, 16-byte aligned; the up to 15 bytes that round a
 * region up to 16 are left as they were). */
GQ_API gq_status_t gq_act_pack(int dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride, void *ckpt,
                               void *stream);
/* Checkpoint -> x.  In float16 values are rounded and saturate at +-65504 (the largest value of a
 * group may round up to 65536).  The type need not be the one packed. */
GQ_API gq_status_t gq_act_unpack(int dtype, int64_t rows, int64_t cols, const void *ckpt, void *x, int64_t x_stride,
                                 void *stream);

/*
 * Activation functions.  forward: y = f(x), and, unless ckpt is NULL, the checkpoint of x in the
 * same pass.  backward: dx = dy * f'(xh), xh the checkpoint's values.
 *   GQ_FN_GELU       x Phi(x), Phi the normal distribution function;
 *   GQ_FN_GELU_TANH  x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2;
 *   GQ_FN_SILU       x / (1 + exp(-x)).
 */
typedef enum { GQ_FN_GELU = 0, GQ_FN_GELU_TANH = 1, GQ_FN_SILU = 2 } gq_fn_t;
GQ_API gq_status_t gq_act_fn_forward(int kind, int dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride,
                                     void *y, int64_t y_stride, void *ckpt, void *stream);
GQ_API gq_status_t gq_act_fn_backward(int kind, int dtype, int64_t rows, int64_t cols, const void *ckpt, const void *dy,
                                      int64_t dy_stride, void *dx, int64_t dx_stride, void *stream);

/*
 * A linear layer's gradients (y = x W^T + b, W of out x in) from the checkpoint of its input:
 *   dw[n][k] = sum over t of dy[t][n] * xh[t][k]    (out x in float32, rows dw_stride apart)
 *   db[n]    = sum over t of dy[t][n]               (NULL: not wanted)
 * accumulate = 1 adds to dw and db (micro-batches), 0 overwrites them.
 *   ckpt       checkpoint of tokens x in values; xh is decoded to dy's type, as by gq_act_unpack:
 *              exact for bfloat16 and float32.
 *   dy         tokens x out values of type dtype (float32: bits below 2^-133 may be cut off).
 *   workspace  device, at least gq_act_weight_grad_workspace bytes (given the same arguments; bias
 *              is db != NULL), 16-byte aligned; NULL if that is 0.  Its contents do not outlive the call.
 */
GQ_API gq_status_t gq_act_weight_grad_workspace(int dtype, int64_t tokens, int64_t in, int64_t out, int64_t dy_stride,
                                                int bias, size_t *bytes);
GQ_API gq_status_t gq_act_weight_grad(int dtype, int64_t tokens, int64_t in, int64_t out, const void *ckpt, const void *dy,
                                      int64_t dy_stride, float *dw, int64_t dw_stride, float *db, int accumulate,
                                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * Layer norm over each row: y = (x - mean) * rstd * gamma + beta, rstd = 1 / sqrt(var + eps), var the
 * population variance around the mean.  The squares and their sums are binary32 too: rows whose spread is
 * above some 1e17, or, with eps = 0, below some 1e-19, leave its range, and rstd is then 0, inexact or infinite.
 *   gamma, beta  cols values of type param_dtype (dtype or GQ_FLOAT32); NULL: 1 and 0.
 *   mean, rstd   device, rows float32, written for the backward pass.
 *   ckpt         receives the checkpoint of x, in the same pass (NULL: none).
 */
GQ_API gq_status_t gq_layer_norm_forward(int dtype, int param_dtype, int64_t rows, int64_t cols, const void *x,
                                         int64_t x_stride, const void *gamma, const void *beta, float eps, void *y,
                                         int64_t y_stride, float *mean, float *rstd, void *ckpt, void *stream);

/*
 * Its backward pass, with xh = (x - mean) * rstd and g = dy * gamma:
 *   dx     = rstd * (g - sum(g) / cols - xh * sum(g xh) / cols)
 *   dgamma = sum over rows of dy * xh,  dbeta = sum over rows of dy   (cols float32 each; NULL: not
 *            wanted).  accumulate = 1 adds to them, 0 overwrites them.
 *   x, ckpt    the input, or its checkpoint: exactly one of the two.
 *   workspace  device, at least gq_layer_norm_workspace bytes, 16-byte aligned (may be NULL if neither
 *              dgamma nor dbeta is wanted).  Its contents do not outlive the call.
 */
GQ_API gq_status_t gq_layer_norm_workspace(int64_t rows, int64_t cols, size_t *bytes);
GQ_API gq_status_t gq_layer_norm_backward(int dtype, int param_dtype, int64_t rows, int64_t cols, const void *dy,
                                          int64_t dy_stride, const void *x, int64_t x_stride, const void *ckpt,
                                          const void *gamma, const float *mean, const float *rstd, void *dx,
                                          int64_t dx_stride, float *dgamma, float *dbeta, int accumulate, void *workspace,
                                          size_t workspace_bytes, void *stream);

/*
 * Matrices in 8-bit floating point, and a linear layer's products from them.
 *
 * With y = x W^T + b the forward pass, the input's gradient dx = dy W and the weight's gradient
 * dW = dy^T x are products of two matrices along their rows, when each operand is packed along the
 * axis that the product sums over.  gq_fp8_pack packs a matrix along its rows, along its columns, or
 * both in one pass; gq_fp8_matmul multiplies.  (gq_act_weight_grad computes dW from the checkpoint
 * instead, whose 7 bits and groups of 32 keep more.)  There is no counterpart in the pages.
 *
 * The conventions of the section on activations hold (stateless; matrices, strides, alignment, overlap;
 * fixed order of sums; NaN where a bounded wait gives up).
 */

/*
 * Layout of the packed form of rows x cols values (host computation; outputs may be NULL).
 * A block is 128 columns of a row (tile = 0), or of 128 rows (tile = 1); the last ones may be cut.
 * codes_off = 0: rows of code bytes, each padded with 0 to whole blocks (pitch 128 * ceil(cols / 128)
 * bytes).  exps_off (16-byte aligned): rows of exponent bytes, one a block, for every row (tile = 0) or
 * every 128 rows (tile = 1), each padded with 0 to a multiple of four (pitch 4 * ceil(cols / 512)).
 * Value of code c under exponent E: c * 2^(E - 127), c in the format's own value; E = 255: NaN.
 *   GQ_FP8_E4M3  4 exponent and 3 mantissa bits, largest 448, smallest 2^-9, NaN 0x7f and 0xff;
 *   GQ_FP8_E5M2  5 and 2, largest finite 57344, smallest 2^-16, infinities and NaN.
 * E is the smallest with max |x| <= 1.75 * 2^(8 or 15) * 2^(E - 127) over the block, at least 10; codes
 * are rounded to nearest, ties to even.  Every value under such an E is exact in bfloat16 and float32.  (Packed forms
 * of other origin may have any E; what passes binary32 is infinite when unpacked.)  A block with a NaN
 * or an infinity has E = 255 and all its codes 0x7f, what pads a cut block among them.
 */
typedef enum { GQ_FP8_E4M3 = 0, GQ_FP8_E5M2 = 1 } gq_fp8_t;
GQ_API gq_status_t gq_fp8_layout(int tile, int64_t rows, int64_t cols, size_t *bytes, size_t *codes_off,
                                 size_t *exps_off);

/*
 * x (rows x cols) -> its packed form, and the packed form of its transpose (cols x rows).
 *   packed    device, gq_fp8_layout(tile, rows, cols) bytes, 16-byte aligned (NULL: not wanted);
 *   packed_t  device, gq_fp8_layout(tile, cols, rows) bytes (NULL: not wanted; not both NULL);
 *             rows <= GQ_ACT_MAX_COLS, and with rows = 0 packed_t must be NULL.
 * The up to 15 bytes that round a region up to 16 are left as they were.
 */
GQ_API gq_status_t gq_fp8_pack(int dtype, int format, int tile, int64_t rows, int64_t cols, const void *x,
                               int64_t x_stride, void *packed, void *packed_t, void *stream);
/* Packed form -> x.  In float16 values are rounded and saturate at +-65504. */
GQ_API gq_status_t gq_fp8_unpack(int dtype, int format, int tile, int64_t rows, int64_t cols, const void *packed, void *x,
                                 int64_t x_stride, void *stream);

/*
 * y[i][j] = sum over c < k of a[i][c] * b[j][c]  + bias[j], i < m, j < n.
 *   a, b       packed forms of m x k and n x k values, each with its own format and tile.
 *   bias       n float32 values, 4-byte aligned (NULL: none).
 *   y          m x n values of type dtype, rows y_stride apart; its element type's alignment is enough.
 *   accumulate 1 adds to y (float32 only: GQ_ERR_UNSUPPORTED otherwise), 0 overwrites it.
 *   workspace  device, at least gq_fp8_matmul_workspace bytes, 16-byte aligned; NULL if that is 0.  Its
 *              contents do not outlive the call.
 * m = 0 is a no-op; 1 <= n < 2^31, 1 <= k <= GQ_ACT_MAX_COLS.  Products are exact; sums are binary32, and the tensor
 * cores cut them off instead of rounding: of every 32 products and the sum so far what lies below 2^-25 of the
 * largest one's power of two, then of their sum what lies below 2^-23.  Float32 results are summed so over runs of up
 * to 4096 columns, which are added rounded: a run is off by at most 1.4e-4 of its largest partial sum (where one product
 * outweighs all others; by less than 1e-6 where they are of about one size).  Where y has 16 bits runs have up to 16384
 * columns, and four times that: beside half a step of y, 3.9e-3 in bfloat16, 4.9e-4 in float16.  Sums below 2^-126
 * may read as 0.  A row of y with a NaN block in its operands is NaN where the formula is.
 */
GQ_API gq_status_t gq_fp8_matmul_workspace(int64_t m, int64_t n, int64_t k, size_t *bytes);
GQ_API gq_status_t gq_fp8_matmul(int dtype, int64_t m, int64_t n, int64_t k, int format_a, int tile_a, const void *a,
                                 int format_b, int tile_b, const void *b, const float *bias, void *y, int64_t y_stride,
                                 int accumulate, void *workspace, size_t workspace_bytes, void *stream);

/*
 * AdamW over many tensors at once: the step that takes the averaged gradient.
 *
 *   g = grad * scale                                      (scale: the clipping factor; 1 without one)
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr lr_scale weight_decay) - lr lr_scale / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in binary32, each operation rounded on its own (with moments in 8 bits the square root and the quotient may be off
 * by 2 units in the last place); (1 - beta1), 1 / (1 - beta1^t) and 1 / sqrt(1 - beta2^t) are computed in binary64 and
 * rounded once.
 *
 * Moments in 32 bits (state_bits = 32) are n float32 values each.  In 8 bits (state_bits = 8) each is
 * gq_adamw_layout bytes, 16-byte aligned: a code byte an element, padded to whole blocks of 128, then one
 * exponent byte a block, padded to a multiple of 16.  The step uses the moments as it computes them and
 * keeps them as follows:
 *   m  GQ_FP8_E4M3 codes and exponents as gq_fp8_pack's blocks (a caller's own have E from 10 to 247, or all codes
 *      0).  For beta1 <= 17/18 it is rounded to nearest, exactly as there: a gradient's change by less than half a
 *      code's step over 1 - beta1 may then not be seen by m where the gradients have no noise.  For beta1 above 17/18
 *      nearest values would keep m where it is for good (a step without a gradient takes less off it than half a
 *      code's step, which is up to 1/18), and it is rounded stochastically: away from 0 with the probability that its
 *      remainder has, sign kept;
 *   v  code 0: 0; code c > 0 under exponent E: (8 + c mod 8) * 2^(floor(c / 8) - 34 + E - 127).  E is the
 *      smallest with max v <= 1.875 * 2^(E - 127) over the block, in [32, 254]; E = 255: NaN (codes 0).
 *      v is rounded stochastically: up with the probability that its remainder has, from 16 random bits of
 *      Philox4x32-10 (nearest values would keep v where it is for good: it decays by 0.1 % a step, a
 *      code's step is 6 to 12 %).  v > 0 keeps a code of at least 1.
 *   Random bits: key: the seed.  Counter: (i / 8 low, high word; t; tensor's number in the list + 2^31, for m
 *   + 2^31 + 2^30) for element i of its tensor; element i takes bits 16 (i mod 2) .. of word (i mod 8) / 2, as a
 *   fraction of 2^16 of its code's step; a remainder counts in whole 2^-16 of the step, cut off.
 * Zero bytes are moments of 0, as for a first step.
 *
 * The list of tensors is fixed by gq_adamw_create, which copies it to device memory that the optimizer owns
 * (the only allocation); the tensors' memory stays the caller's and must outlive the optimizer.
 *   param    n values of type param_dtype; grad: n values of grad_dtype, e.g. a slice of gq_fused_step's avg;
 *   master   n float32 values that are updated in the parameters' place, param receiving them rounded;
 *            NULL: none.  All tensors of a 16-bit type have one, or none has.
 *   These, and moments in 32 bits, need their type's alignment only.  Fastest are arrays that all begin equally far
 *   behind 16-byte boundaries, in elements (slices of flat vectors at the same offset); with moments in 8 bits, on them.
 *   Tensors may share gradients; what a step writes may overlap nothing else that it reads or writes
 *   (GQ_ERR_INVALID).  n = 0 is allowed; pointers may then be NULL.
 * Calls on one optimizer must not overlap on the GPU, and must be made with its device current
 * (GQ_ERR_INVALID).  Non-finite values pass through as in the formulas.
 */
typedef struct {
    int32_t param_dtype, grad_dtype; /* gq_dtype_t */
    int32_t state_bits;              /* 32 or 8 */
    uint64_t seed;                   /* key of the random bits (state_bits = 8) */
} gq_adamw_config_t;

typedef struct {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;
    int64_t n;          /* 0 <= n < 2^40 */
    float weight_decay; /* finite, >= 0 */
    float lr_scale;     /* finite, >= 0; 1 for the step's own lr */
} gq_adamw_tensor_t;

typedef struct gq_adamw *gq_adamw_t; /* opaque; owned by the library */

#define GQ_ADAMW_MAX_TENSORS (1 << 20)

/* Bytes of a moment of n elements in 8 bits, and the offset of its exponents (outputs may be NULL). */
GQ_API gq_status_t gq_adamw_layout(int64_t n, size_t *bytes, size_t *exps_off);

GQ_API gq_status_t gq_adamw_create(const gq_adamw_config_t *cfg, const gq_adamw_tensor_t *tensors, int count,
                                   gq_adamw_t *out);
/* Frees the optimizer's own memory; waits for the device. */
GQ_API gq_status_t gq_adamw_destroy(gq_adamw_t opt);

/*
 * out[0] = sqrt of the sum of grad^2 over all tensors, out[1] = min(1, max_norm / that) (1 for a norm of 0; NaN
 * if a gradient is not finite), both in binary64, in a fixed order, and rounded: a norm beyond float32's largest
 * value is infinite in out[0], while out[1] is still the quotient.  out: device, 2 floats, 4-byte aligned;
 * max_norm > 0 (infinity: only the check that the gradients are finite).
 */
GQ_API gq_status_t gq_adamw_norm(gq_adamw_t opt, double max_norm, float *out, void *stream);

/*
 * One step.  t = step >= 1 (below 2^32); lr >= 0, eps >= 0 finite; 0 <= beta1, beta2 < 1.
 *   scale    device, one float that multiplies the gradients, e.g. gq_adamw_norm's out + 1 (NULL: 1).  If it
 *            is NaN the step changes nothing.
 *   scalars  NULL, or device memory (16 bytes, 16-byte aligned) holding what gq_adamw_scalars gives, read when
 *            the step runs in the place of lr and step (for the same betas): a captured step is replayed with new ones.
 */
typedef struct {
    float lr;
    float inv1;    /* 1 / (1 - beta1^t) */
    float inv2;    /* 1 / sqrt(1 - beta2^t) */
    uint32_t step; /* t */
} gq_adamw_scalars_t;
GQ_API gq_status_t gq_adamw_scalars(double lr, double beta1, double beta2, int64_t step, gq_adamw_scalars_t *out);
GQ_API gq_status_t gq_adamw_step(gq_adamw_t opt, double lr, double beta1, double beta2, double eps, int64_t step,
                                 const float *scale, const void *scalars, void *stream);

/* The moments' values, all tensors one after another, in vectors of type dtype (device, 16-byte aligned; either
 * may be NULL).  Moments in 8 bits are exact in bfloat16 and float32; float16 saturates at +-65504. */
GQ_API gq_status_t gq_adamw_moments(gq_adamw_t opt, int dtype, void *m, void *v, void *stream);

/* Static description of a status code. */
GQ_API const char *gq_status_string(gq_status_t status);

/* Library version, "major.minor.patch". */
GQ_API const char *gq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GQ_H */
