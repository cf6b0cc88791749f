/*
 * lb.h -- C ABI of the LittleBit factorized binary linear forward on
 * AMD Instinct MI355X (gfx950).
 *
 * Sources (cited by short name throughout the library):
 *   [LB2 column] physicalainews.jp, "LittleBit-2: sub-1-bit LLM
 *                quantization (2026)".  Ch. 1: effective bit width of a
 *                layer, single path and residual.
 *   [LB news]    aifrontier.co.jp, "Samsung LittleBit: 13B to 0.84 GB".
 *                Sec. 2: W is approximated by two binarised (+-1) low-rank
 *                factors with FP16 row scale h, column scale g and latent
 *                scale l; a residual path is a second factorisation added
 *                at inference; inference is two small binary matrix
 *                products plus elementwise scaling.
 *
 * The layer computes, for every row x of an M x a input,
 *
 *     y = sum_p  h_p * ( S_U,p ( l_p * ( S_V,p^T ( g_p * x ) ) ) )
 *
 * with S_U,p in {+-1}^(b x s), S_V,p in {+-1}^(a x s), h_p (b), g_p (a),
 * l_p (s) in fp16, p = 0 only, or p = 0, 1 when residual.  a is the input
 * width and b the output width.  Accumulation is fp32; y is rounded once
 * to fp16 (round to nearest even).
 *
 * Conventions
 *   - Every call returns lb_status; the library never aborts or exits.
 *     lb_last_error() returns a thread-local text for the last failure.
 *   - Sign words ("canonical layout"): a factor with `rows` rows is given
 *     as rows x ceil(s/32) uint32 words, row-major; entry k of a row is
 *     bit (k % 32) of word (k / 32); bit 1 means +1 and bit 0 means -1.
 *     Bits past s are ignored.
 *   - fp16 values are passed as their IEEE binary16 bit patterns (uint16).
 *   - Host inputs are copied before the call returns; the caller may free
 *     them at once.  The library owns every device buffer it allocates.
 *   - Device pointers (x, y) are caller-owned, contiguous, row-major and
 *     16-byte aligned, and x must not overlap y.
 *   - Forward calls are asynchronous on the given hipStream_t (passed as
 *     void*, NULL = the null stream) and make no host synchronisation,
 *     with one exception each: the first call with M >= 64 on a layer
 *     builds the layer's matrix-core copy of the signs (allocates it and
 *     synchronises the device; lb_prepare does this ahead of time), and
 *     lb_stack_forward allocates (without synchronising) when M exceeds the
 *     rows reserved with lb_stack_reserve or by an earlier call, and sets
 *     up its one-launch M >= 64 path on the first call for a row count
 *     (allocates and synchronises; see lb_stack_forward).
 *   - Every buffer a forward call writes belongs to the layer or stack it
 *     runs (allocated by lb_create, lb_prepare or lb_stack_reserve) or to
 *     the caller: calls on different objects share nothing and may run on
 *     different streams at once.  Calls that use one layer or stack must be
 *     ordered on one stream: they share that object's workspace.  Nothing
 *     an object allocated is freed or moved before it is destroyed (a
 *     stack's outgrown scratch is retired, not freed).
 *   - Without a trace, lb_forward and lb_stack_forward (M within the rows
 *     already reserved, and for M >= 64 the matrix-core copies built) only
 *     launch kernels, so they can be captured into a HIP graph and
 *     replayed; such a call made under capture before that preparation
 *     returns LB_ENOTREADY instead of allocating.  The one-launch sweep
 *     carries its exchange generation from launch to launch on the device,
 *     so every replay is a fresh launch.
 */
#ifndef LB_H
#define LB_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct lb_layer lb_layer; /* opaque, library-owned */
typedef struct lb_stack lb_stack; /* opaque, library-owned */
typedef struct lb_bank lb_bank;   /* opaque, library-owned */
typedef struct lb_cache lb_cache; /* opaque, library-owned */

typedef enum {
  LB_OK = 0,
  LB_EINVAL = -1,        /* bad argument (null pointer, size, path, overlap) */
  LB_ENOMEM = -2,        /* device or host allocation failed */
  LB_EHIP = -3,          /* a HIP runtime call failed (text in lb_last_error) */
  LB_ENOTREADY = -4,     /* forward before signs and scales of every path */
  LB_EUNSUPPORTED = -5,  /* valid request the library cannot run here */
  LB_ETIMEOUT = -6       /* a device-side wait gave up (watchdog) */
} lb_status;

/* ---------------------------------------------------------------- layers */

/* Create a layer with input width a, output width b, rank s, and one
 * path (residual = 0) or two (residual = 1), on the current HIP device.
 * [LB2 column] Ch. 1 names a, b, s and residual; [LB news] Sec. 2 the
 * structure.  a, b, s >= 1, a, b <= 2^24 and s <= 4096.  Allocates the
 * layer's device storage: the signs once (in 16-row tile layouts that
 * every kernel for M < 64 reads: about P s (a + b) / 8 bytes), the scales
 * and their tile copies, and the layer's own forward workspace (chunk
 * partials and latent rows of up to 63 rows, the matrix-core latent and
 * split-K partials, the one-row launch's state).  The matrix-core copy of
 * the signs (the same count again) is added by lb_prepare or the first
 * forward with M >= 64.  *out is set on success only. */
lb_status lb_create(int64_t a, int64_t b, int64_t s, int residual, lb_layer **out);

/* Set the sign factors of one path (0, or 1 when residual) from host
 * canonical words: su is b x ceil(s/32), sv is a x ceil(s/32).  The words
 * are re-laid out for the device and copied synchronously (the device is
 * synchronised before return, so launches on any stream see them);
 * bit-exact.  A matrix-core copy already built is rebuilt too. */
lb_status lb_pack_signs(lb_layer *L, int path, const uint32_t *su, const uint32_t *sv);

/* Set the fp16 scales of one path from host arrays: h (b values, row /
 * output scale), g (a values, column / input scale), l (s values, latent
 * scale), [LB news] Sec. 2.  Copied synchronously (as lb_pack_signs). */
lb_status lb_set_scales(lb_layer *L, int path, const uint16_t *h, const uint16_t *g,
                        const uint16_t *l);

/* y[M x b] = layer(x[M x a]); x, y are device fp16.  M = 0 is a no-op.
 * M < 64 runs the wave-level binary GEMV path (sign-flip identity on
 * packed bits, fp32 throughout): one launch for M = 1 on small layers
 * (a <= 4096 and P s <= 256, e.g. the 4096^2 projections at 0.1 bits per
 * weight; workgroups take the first product, the reduction over input
 * chunks and the second product by an atomic ticket, each waiting only on
 * workgroups that started before it, so it needs no co-residency and may
 * share the device with other streams), three launches otherwise (faster
 * for larger layers); M >= 64 runs the fp16 matrix-core
 * path (two launches: the first product with split K, then the second), in
 * which the latent vector t is rounded once to fp16 before the second
 * product; the +-g and +-l operands are exact.  The first call with
 * M >= 64 on a layer builds its matrix-core copy of the signs (allocates,
 * synchronises the device; LB_ENOTREADY instead when `stream` is being
 * captured: call lb_prepare first).  Returns LB_ENOTREADY
 * unless every path has signs and scales; LB_ETIMEOUT (running nothing)
 * when an earlier one-row forward on the device gave up a bounded
 * device-side wait (which does not happen while the device runs its work;
 * the flag is then cleared). */
lb_status lb_forward(const lb_layer *L, const void *x, void *y, int64_t M, void *stream);

/* lb_forward for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * for M >= 2 the same kernels and the same result as lb_forward, bit for
 * bit (for M = 1 on a small layer the wave path's three launches, where
 * lb_forward takes one;
 * the two agree at the parity bar), but the scratch they need lives in one fixed 32 MB device array of the library
 * (16 KB of split-K tile counters plus 32 MB - 16 KB of workspace), held on
 * each device the library runs on until the process ends, instead of the
 * layer's own workspace.  Allocates nothing and makes no host
 * synchronisation.  The first call on a device looks the array's address
 * up (hipGetSymbolAddress) and clears its counters with a kernel on
 * `stream`; every launch leaves them zero.  All calls on one device share
 * the array, which keeps the last call's contents: calls that overlap on
 * one device (other streams, concurrent host threads) race, so order them.
 * M < 64 runs the wave path in row blocks that fit the array; M >= 64 the
 * matrix-core path, which needs its latent (256 rows of the padded latent
 * width) and split partials within the array, and the layer's matrix-core
 * copy of the signs built beforehand (lb_prepare, or an earlier lb_forward
 * with M >= 64; LB_ENOTREADY, nothing launched, otherwise).  LB_EUNSUPPORTED, with
 * nothing launched, when a layer needs more (not even one wave-path row, or
 * the matrix-core path, fits); the other errors as lb_forward. */
lb_status lb_forward_noalloc(const lb_layer *L, const void *x, void *y, int64_t M, void *stream);

/* Read the device signs of one path back into canonical words (padding
 * bits zero).  Bit-exact inverse of lb_pack_signs; synchronous. */
lb_status lb_unpack_signs(const lb_layer *L, int path, uint32_t *su, uint32_t *sv);

/* Read the fp16 scales of one path back (h: b values, g: a, l: s), the
 * bit patterns lb_set_scales or lb_init_from_factors stored; synchronous.
 * LB_ENOTREADY when that path's scales were never set. */
lb_status lb_get_scales(const lb_layer *L, int path, uint16_t *h, uint16_t *g, uint16_t *l);

/* Set the signs and scales of one path from real factors W ~= U V^T
 * (Dual-SVID, [LB news] Sec. 2): U is b x s and V is a x s, fp32,
 * row-major (row stride s), device memory on the layer's device, 4-byte
 * aligned, read on `stream` after the work already queued there and left
 * unchanged.  Readings of the one-line description, stated here:
 *   S_U = sign(U), S_V = sign(V), with sign(0) = sign(-0) = +1;
 *   |U| ~= h l_u^T and |V| ~= g l_v^T by the top singular pair of each
 *   (the best rank-1 fit in the Frobenius norm; both vectors >= 0), the
 *   singular value split evenly between the two vectors;
 *   l = l_u * l_v (elementwise), so that diag(h) S_U diag(l) S_V^T diag(g)
 *   approximates U V^T;
 *   h, g and l are rounded once to fp16 (nearest even).
 * The pair is found on the device by power iteration in fp64 with
 * fixed-order sums (deterministic), until successive unit iterates differ
 * by at most 1e-13 in every entry, within 2048 steps.  The truncated SVD
 * that gives U and V from W, and the residual W - W_1 for path 1, are the
 * caller's (e.g. a library SVD on the device).  Allocates device
 * temporaries of about 8 (s max(a, b) / 64 + a + b + 4 s) bytes plus the
 * sign words and scales, and synchronises `stream` several times; returns
 * when the layer holds the new path.  LB_EUNSUPPORTED,
 * with the layer unchanged, when the iteration has not settled (a top
 * singular value of |U| or |V| not separated from the next).
 * R, when not NULL, is an s x s fp64 row-major rotation on the device (8-byte
 * aligned, e.g. from lb_joint_itq): the path is then set from the fp64
 * factors U R and V R instead (one rocBLAS dgemm; about 16 (a + b) s more
 * bytes of device temporaries; (a + b) s < 2^31). */
lb_status lb_init_from_factors(lb_layer *L, int path, const float *U, const float *V,
                               const double *R, void *stream);

/* Joint-ITQ rotation ([LB2 column] Ch. 2): an orthogonal R between the
 * factors leaves U V^T unchanged, so LittleBit-2 rotates U <- U R and
 * V <- V R before binarising (pass R to lb_init_from_factors); R is found
 * by iterating on the stacked factors X = [U; V].  Readings, stated here:
 *   the iteration is iterative quantisation: one step sets B = sign(X R)
 *   (sign(0) = +1), then R = the orthogonal polar factor of X^T B (the
 *   orthogonal Procrustes solution, which minimises ||B - X R||_F), so the
 *   loss never increases; the pages' default is 50 steps;
 *   the start is R0 (device, s x s, fp64 row-major) or the identity when
 *   R0 is NULL.
 * U (b x s) and V (a x s) are fp32 row-major device arrays, read only; R
 * receives the s x s fp64 row-major rotation (device; may be R0).  All
 * arithmetic is fp64: the products are rocBLAS dgemm calls (atomics off,
 * reproducible), the polar factor a Newton-Schulz iteration run until
 * max |Z^T Z - I| <= 1e-12.  iters = 0 copies the start.  Needs
 * 1 <= a, b <= 2^24, 1 <= s <= 4096 and (a + b) s < 2^31.  Allocates
 * about 16 (a + b) s bytes of device temporaries, synchronises `stream`
 * and returns when R is written.  The library creates one rocBLAS handle
 * per device on first use and keeps it until the process ends; calls that
 * use it (this one and lb_init_from_factors with R) are serialised by a
 * library-wide lock.  LB_EUNSUPPORTED when X^T B is singular
 * or nearly so (the polar factor does not settle within 200 steps). */
lb_status lb_joint_itq(const float *U, const float *V, int64_t a, int64_t b, int64_t s, int iters,
                       const double *R0, double *R, void *stream);

/* Build now what forward calls of up to M rows read beyond the storage
 * lb_create made: for M >= 64 the matrix-core copy of the signs (bits
 * inverted and permuted for the fp16 operand sign flips; allocates and
 * synchronises the device).  Nothing for M < 64.  Call it before capturing
 * M >= 64 forwards into a graph or using lb_forward_noalloc with them.
 * The signs of every path must be set (LB_ENOTREADY otherwise). */
lb_status lb_prepare(lb_layer *L, int64_t M);

/* Device bytes the layer holds: *sign_bytes for its sign words (the tile
 * layouts, plus the matrix-core copy once built), *total_bytes for all of
 * its storage (signs, scales, workspace, one-row state).  Either pointer
 * may be NULL. */
lb_status lb_layer_device_bytes(const lb_layer *L, uint64_t *sign_bytes, uint64_t *total_bytes);

/* Shape queries. */
lb_status lb_layer_shape(const lb_layer *L, int64_t *a, int64_t *b, int64_t *s, int *residual);

lb_status lb_destroy(lb_layer *L);

/* ------------------------------------------------------- split stages */
/* The two halves of lb_forward, for callers that keep the latent vector
 * (the pages note that factorised K/V projections let a cache hold the
 * latent instead of the full width, [LB news] Sec. 4).
 * stage1: w[M x P*s] (fp32, device) = l_p * S_V,p^T (g_p * x), path-major
 *         (columns p*s .. p*s+s-1 belong to path p).
 * stage2: y[M x b] (fp16) = sum_p h_p * S_U,p w_p.  Any M >= 0. */
lb_status lb_forward_stage1(const lb_layer *L, const void *x, float *w, int64_t M, void *stream);
lb_status lb_forward_stage2(const lb_layer *L, const float *w, void *y, int64_t M, void *stream);

/* ---------------------------------------------------------- bit count */
/* Exact effective bits per weight of [LB2 column] Ch. 1:
 *   num_bits = P * (s*(a+b+16) + 16*(a+b)),  den = a*b,  P = 1 or 2.
 * Pure host arithmetic.  LB_EINVAL on overflow or a non-positive size. */
lb_status lb_eff_bits(int64_t a, int64_t b, int64_t s, int residual, uint64_t *num_bits,
                      uint64_t *den);

/* Largest rank s >= 0 with eff_bits(a, b, s, residual) <= bpw_num/bpw_den
 * (the same formula solved for s, floor).  LB_EINVAL when the scale
 * vectors alone exceed the budget. */
lb_status lb_rank_for_bpw(int64_t a, int64_t b, uint64_t bpw_num, uint64_t bpw_den, int residual,
                          int64_t *s);

/* -------------------------------------------------------------- stacks */
/* A stack is an ordered list of layers grouped into units: the layers of
 * one unit read the same input and have the same a and b; unit u+1 has
 * a = unit u's b.  Unit 0 reads the stack input x0.  Unit u+1 reads
 * fp16(kappa / sqrt(n_u) * sum of unit u's outputs), computed in fp32 from
 * the fp16 outputs, where n_u is unit u's layer count; the stack output
 * is the same combine of the last unit.  (The transformer parts between
 * LittleBit layers are not LittleBit layers; these linear stand-ins keep
 * the activations O(1).)  E.g. a Llama MLP stack has units [gate, up],
 * [down] per block.  Layers stay owned by the caller and must outlive the
 * stack; their signs and scales must be set before lb_stack_create.      */
lb_status lb_stack_create(lb_layer *const *layers, int n_layers, const int32_t *unit_sizes,
                          int n_units, float kappa, lb_stack **out);

/* Run the whole stack on device fp16 x0 [M x a_0] into y [M x b_last].
 * trace, when not NULL, receives every layer's fp16 output followed by
 * every unit's fp16 input, each M rows, in stack order (size from
 * lb_stack_trace_elems).  Automatic mode:
 *   M = 1       one launch for the whole sweep: one workgroup per compute
 *               unit, the latent vector of each unit summed across
 *               workgroups through device memory with bounded waits.  Its
 *               workgroups wait for one another, so all of them must be
 *               resident at once: run it while other streams' kernels do
 *               not hold the compute units.  A wait that gives up (e.g.
 *               when they do) sets a flag that lb_stack_check reports and
 *               that the next sweep returns as LB_ETIMEOUT;
 *   M = 2       without a trace: the one-launch sweep once per row (each
 *               row's output is exactly its M = 1 output);
 *   M >= 3      without a trace (M >= 2 when the device cannot hold the
 *               sweep): the whole stack in one launch per 256 rows on the
 *               matrix cores, its 32-row blocks pipelined through the units
 *               (as mode 3; measured faster than the per-layer kernels from
 *               3 rows, where the wave path has become ALU-bound).  The
 *               first such call builds the layers' matrix-core sign copies
 *               (lb_prepare, or lb_stack_reserve, does it ahead), and the
 *               first call for a row count sets up the launch's arguments
 *               (both allocate and synchronise the device).  While the
 *               stream is being captured before either exists, the
 *               per-layer kernels below run instead;
 *   otherwise   (a trace, a width that is not a multiple of 8, or that
 *               capture): for M < 64 the wave-path kernels of each layer,
 *               then a combine kernel per unit (fused into the unit's last
 *               layer up to 16 rows), or the sweep once per row for M <= 2
 *               (M <= 3 when the stack's mean matrix has at least 2^27
 *               weights) without a trace; for M >= 64 two matrix-core
 *               launches per unit, the combine fused into the second (the
 *               same tiles in the same order as the one launch, so the same
 *               output bit for bit).
 * x0, y and trace must be 16-byte aligned; y must not overlap x0. */
lb_status lb_stack_forward(lb_stack *S, const void *x0, void *y, void *trace, int64_t M,
                           void *stream);

/* Reserve the stack's scratch for up to M rows now (allocates; for
 * M >= 3, when the stack has a one-launch plan, or M >= 64, also builds
 * the layers' matrix-core sign copies, which synchronises the device), so
 * that later lb_stack_forward calls with at most M rows allocate nothing
 * except the one-launch setup of a new row count.  Scratch of an earlier, smaller
 * reservation is retired, not freed (launches already queued or captured
 * keep using it), until lb_stack_destroy. */
lb_status lb_stack_reserve(lb_stack *S, int64_t M);

/* Number of fp16 elements lb_stack_forward writes to trace for M rows. */
lb_status lb_stack_trace_elems(const lb_stack *S, int64_t M, int64_t *elems);

/* Synchronise the device and report whether any earlier persistent sweep
 * of this stack gave up a device-side wait (LB_ETIMEOUT; the stack resets
 * its synchronisation words before the next sweep).  LB_OK otherwise. */
lb_status lb_stack_check(lb_stack *S);

/* Diagnostics: record, in later persistent sweeps, eight device timestamps
 * (100 MHz counter) per phase and workgroup, taken by its first thread, into
 * the caller's device buffer buf (uint64, layout [workgroup][phase][8]:
 * phase start, second-product lookups done (first wave), second product
 * done (epilogue and combine), first-product tables built, first product done, exchange
 * level A done, level B done, exchange done).  *needed receives the element
 * count.  buf = NULL turns recording off.  The buffer must outlive its use. */
lb_status lb_stack_timeline(lb_stack *S, void *buf, int64_t capacity, int64_t *needed);

/* Diagnostics: test the failure path of the one-launch sweep.  With enable
 * != 0, later persistent sweeps of this stack wait for words nobody writes,
 * with a bound of 2048 polls, so every device-side wait gives up: the
 * kernel ends normally, its output is undefined, and lb_stack_check then
 * returns LB_ETIMEOUT.  enable = 0 restores normal sweeps.
 * LB_EUNSUPPORTED when the stack has no persistent sweep. */
lb_status lb_stack_test_wait_failure(lb_stack *S, int enable);

/* Diagnostics: stress the exchange of the one-launch sweep.  With
 * max_ticks > 0 (at most 100000), later persistent sweeps make each wave
 * wait, before each step of the cross-workgroup exchange (publishing its
 * partials, the intra-XCD sum, the cross-XCD store and poll, the final
 * poll), for a pseudo-random time drawn from seed, the sweep's generation,
 * the workgroup, the wave and the step: zero or up to max_ticks ticks of
 * 10 ns.  The output must not change (every sum has a fixed order), only
 * the time.  max_ticks = 0 turns it off.  LB_EUNSUPPORTED when the stack
 * has no persistent sweep. */
lb_status lb_stack_test_delay(lb_stack *S, uint32_t seed, uint32_t max_ticks);

/* Select the execution mode of lb_stack_forward: 0 = automatic (above),
 * 1 = every layer alone (as lb_forward) followed by a combine kernel per
 * unit, 2 = the one-launch sweep only (LB_EUNSUPPORTED unless M = 1 and
 * the device can hold one workgroup per compute unit), 3 = automatic
 * (where it takes the one launch, from 3 rows without a trace) without the
 * capture fallback.  The one launch runs the whole stack per 256 rows: the
 * matrix-core tiles of the two launches per unit, in the same order
 * (identical results), as work items dealt round robin to a grid of the
 * device's resident capacity, each waiting only for the previous step of
 * its own 32-row block, so row blocks pipeline through the units (kernels
 * on other streams that hold compute units delay it until they finish);
 * its bounded waits report a give-up as LB_ETIMEOUT from the next call, and
 * the first call for a row count sets up its launch arguments (allocates,
 * synchronises; LB_ENOTREADY under capture, where mode 0 falls back to
 * the per-layer kernels).  Mode 3 needs every width to be a multiple of 8
 * (LB_EUNSUPPORTED otherwise; mode 0 then keeps the per-layer kernels). */
lb_status lb_stack_set_mode(lb_stack *S, int mode);

lb_status lb_stack_destroy(lb_stack *S);

/* --------------------------------------------------------------- banks */
/* A bank is n layers of one shape (a, b, s, paths) on one device, each with
 * or without a gate layer of that shape.  It computes, for rows x of fp16,
 *
 *     y = act(L(x) + bias) + residual                      without gates
 *     y = act(G(x) + gate_bias) * (L(x) + bias) + residual     with gates
 *
 * for one of its layers (lb_bank_forward) or for rows sorted by layer, each
 * run of rows with its own (lb_bank_grouped: the experts of a mixture).
 * Accumulation is fp32 and the latent vector w = l t keeps 22 bits, at every
 * row count and size of h; y is rounded once.  That holds for |w_k| from
 * 2^-14 up; smaller ones are off by at most 2^-36.  Beyond 65504, fp16's
 * largest number, y is not finite (lb_forward, which keeps w in fp32 below 64
 * rows, has no such limit there).
 *
 * Layers stay owned by the caller and must outlive the bank; their signs
 * and scales must be set before lb_bank_create, which builds their
 * matrix-core sign copies (as lb_prepare), allocates and synchronises the
 * device.  Later lb_pack_signs and lb_set_scales calls on them are seen by
 * later forwards.  A layer may appear more than once.
 *
 * The bank's calls share its workspace (the latent rows, at most 256 MB or
 * one 64-row slot; longer calls run in windows): order them on one stream.
 * They launch kernels only, unless a call has more rows than were reserved
 * or used before: then the workspace grows (allocates without
 * synchronising; the old one is retired, not freed, until lb_bank_destroy),
 * or, under capture, the call returns LB_ENOTREADY.                      */

/* Element types of y, residual and logits. */
typedef enum { LB_F16 = 0, LB_F32 = 1 } lb_type;

/* Activations; GELU is v/2 (1 + erf(v / sqrt 2)), GELU_TANH its tanh form
 * v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))), SILU v / (1 + exp(-v)). */
typedef enum {
  LB_ACT_NONE = 0,
  LB_ACT_RELU = 1,
  LB_ACT_GELU = 2,
  LB_ACT_GELU_TANH = 3,
  LB_ACT_SILU = 4
} lb_act;

/* A bank of layers[0..n-1] (1 <= n <= 1024) with gates[0..n-1], or without
 * gates when gates is NULL. */
lb_status lb_bank_create(lb_layer *const *layers, lb_layer *const *gates, int n, lb_bank **out);

/* Workspace for calls of up to `rows` rows, now. */
lb_status lb_bank_reserve(lb_bank *B, int64_t rows);

/* M rows through layer `expert` (0 for a bank of one).
 *   x         device fp16, M x a, row stride ldx >= a elements
 *   y         device, M x b of y_type (lb_type), row stride ldy >= b
 *   bias, gate_bias   device fp16, n x b (row e belongs to layer e), or
 *             NULL; a gate_bias needs a bank with gates
 *   residual  device, M x b of y_type, row stride ldr >= b, or NULL; it may
 *             be y itself with the same stride (y is then added to)
 * Pointers need the alignment of their elements only; rows whose pointers,
 * strides and widths are multiples of 16 bytes are read and written in
 * 16-byte pieces (faster).  y must not overlap the other arrays: either
 * their spans, first to last element, are apart, or they are column blocks of
 * one buffer, with the same row stride in bytes and no column in common.
 * M = 0 is a no-op; M <= 2^30. */
lb_status lb_bank_forward(lb_bank *B, int expert, const void *x, int64_t ldx, void *y, int64_t ldy,
                          int y_type, int64_t M, int act, const void *bias, const void *gate_bias,
                          const void *residual, int64_t ldr, void *stream);

/* Rows offsets[e] .. offsets[e + 1] - 1 of y through layer e, for every e.
 *   offsets   device int32, n + 1 non-decreasing values in [0, rows]; an
 *             empty run is a layer without rows.  Read on the device only.
 *             Rows of y outside [offsets[0], offsets[n]) are left as they
 *             were.  (Values out of range are clamped to it; with decreasing
 *             ones the rows concerned are undefined.)
 *   index     device int32, `rows` values: row i reads x row index[i] (a
 *             row may be read any number of times), or NULL: row i of x.  An
 *             index outside [0, x_rows) reads a row of zeros.
 * The other arguments are as in lb_bank_forward, residual and y by row. */
lb_status lb_bank_grouped(lb_bank *B, const void *x, int64_t x_rows, int64_t ldx, const int32_t *index,
                          const int32_t *offsets, int64_t rows, void *y, int64_t ldy, int y_type,
                          int act, const void *bias, const void *gate_bias, const void *residual,
                          int64_t ldr, void *stream);

/* Layers of the bank, whether it has gates, widths, and the device that all
 * pointers and streams of its calls belong to.  Any pointer may be NULL. */
lb_status lb_bank_shape(const lb_bank *B, int *n, int *gated, int64_t *a, int64_t *b, int *device);

lb_status lb_bank_destroy(lb_bank *B);

/* ------------------------------------------------------------- routing */
/* Choose k of `experts` layers (1 <= k <= min(64, experts), experts <= 1024)
 * for every token and sort the chosen rows by expert, on the current device:
 *   logits    device fp16 or fp32 (logits_type), tokens x experts, row
 *             stride ld >= experts.  NaN counts as -inf.
 *   ids       tokens x k: the experts with the largest logits, largest
 *             first, equal ones by the lowest number.  Experts at -inf are
 *             never chosen: a choice without one has id -1, row -1, weight 0
 *   weights   tokens x k: softmax probabilities (fp32) of the choices, over
 *             all experts, or over the token's choices when renormalise
 *   offsets   experts + 1: where each expert's rows begin (for
 *             lb_bank_grouped); offsets[experts] rows in all
 *   token     tokens * k: the token of every row (lb_bank_grouped's index);
 *             an expert's rows are in the order of the tokens.  -1 behind
 *             the last row
 *   row       tokens x k: the row of every choice
 * No array may overlap another.  ws is device scratch of at least
 * lb_route_ws_bytes bytes (which never shrink as tokens grow; none for 32
 * tokens or fewer), not shared with calls that may run at the same time.  Only
 * launches kernels; with no tokens it writes offsets alone. */
lb_status lb_route_ws_bytes(int64_t tokens, int experts, int k, uint64_t *bytes);
lb_status lb_route(const void *logits, int logits_type, int64_t ld, int64_t tokens, int experts, int k,
                   int renormalise, int32_t *ids, float *weights, int32_t *offsets, int32_t *token,
                   int32_t *row, void *ws, uint64_t ws_bytes, void *stream);

/* out[t] = residual[t] + sum_j weights[t, j] * y[row[t, j]] (fp32, in the
 * order of j, rounded once), on the current device.  y is fp16, y_rows x
 * width; row and weights are tokens x k (k <= 64); residual (or NULL) and
 * out are of out_type; ldy, ldr and ldo are row strides.  Rows outside
 * [0, y_rows) add nothing.  residual may be out itself with the same
 * stride; out must not overlap the other arrays (column blocks of one buffer
 * with the same row stride in bytes do not). */
lb_status lb_route_combine(const void *y, int64_t y_rows, int64_t ldy, const int32_t *row,
                           const float *weights, int64_t tokens, int k, int64_t width,
                           const void *residual, int64_t ldr, void *out, int64_t ldo, int out_type,
                           void *stream);

/* --------------------------------------------------------------- norms */
/* The end of a block and the beginning of the next, on the current device:
 *
 *     u = y, or with post  N(y) * post_weight + post_bias
 *     r' = scale * r + gate * u
 *     x  = N(r') * weight + bias
 *
 * N(v) = v / sqrt(mean(v^2) + eps) (LB_NORM_RMS), or the same of v less its
 * mean (LB_NORM_LAYER).  fp32 throughout; x is the norm of r' before r' is
 * rounded, and out and x are rounded once.
 *   y         device, rows x width of y_type, row stride ldy, or NULL
 *   gate      device fp16, rows x width with row stride ldg, or with ldg = 0
 *             one row for all of them, or NULL
 *   r         device, rows x width of r_type, row stride ldr, or NULL (r' is
 *             gate * u then); y or r must be given
 *   out       r' of r_type, row stride ldo, or NULL
 *   x         fp16, row stride ldx, or NULL; out or x must be given
 *   post_weight, post_bias, weight, bias   device fp16, width, or NULL
 * out and x may be the same rows as y or r (same pointer, stride and type) and
 * must overlap nothing otherwise (column blocks of one buffer with the same
 * row stride in bytes do not).  1 <= width <= 32768. */
typedef enum { LB_NORM_RMS = 0, LB_NORM_LAYER = 1 } lb_norm_kind;
lb_status lb_norm(int kind, const void *y, int y_type, int64_t ldy, int post, const void *post_weight,
                  const void *post_bias, const void *gate, int64_t ldg, const void *r, int64_t ldr,
                  float scale, int r_type, const void *weight, const void *bias, float eps, void *out,
                  int64_t ldo, void *x, int64_t ldx, int64_t rows, int64_t width, void *stream);

/* -------------------------------------------------------------- caches */
/* A cache holds keys and values of attention in 8 bits, in pages of
 * page_tokens tokens (a power of two, 16 to 256) of kv_heads heads of
 * head_dim numbers (a multiple of 8, at most 256), with one fp32 scale for
 * the keys and one for the values of each page and head:
 * value = number * scale, numbers -127 .. 127, scale = largest / 127.
 * Which page belongs to whom is the caller's: a call gets its sequences as
 *   table     device int32, sequences x columns, row stride ldt: the pages
 *             of every sequence in the order of its tokens.  A page may stand
 *             in several places, but a call appends through one of them only
 *             (otherwise the page's numbers are undefined)
 *   lengths   device int32: tokens of every sequence, the call's included
 *   start     device int32, sequences + 1 non-decreasing values in
 *             [0, rows]: rows start[b] .. start[b + 1] - 1 are the last tokens
 *             of sequence b, at positions lengths[b] - count .. lengths[b] - 1;
 *             or NULL: row b is the last token of sequence b (rows =
 *             sequences)
 * These are read on the device only.  Rows outside [start[0],
 * start[sequences]) are left as they were; a page outside the cache is no
 * page (nothing is written there, nothing attended, zeros read), nor is what
 * lies past the table; rows at positions below 0 are dropped.
 *
 * The cache belongs to the device that is current at lb_cache_create; all
 * pointers and streams of its calls belong to it too.  lb_cache_attend uses
 * a workspace of the cache's own: order a cache's calls on one stream.  They
 * launch kernels only, unless lb_cache_attend needs more workspace than was
 * reserved or used before: then it grows (as a bank's), or, under capture,
 * the call returns LB_ENOTREADY. */
/* All numbers of a new cache are 0.  Allocates and synchronises the device. */
lb_status lb_cache_create(int64_t pages, int page_tokens, int kv_heads, int head_dim, lb_cache **out);

/* Any pointer may be NULL. */
lb_status lb_cache_shape(const lb_cache *C, int64_t *pages, int *page_tokens, int *kv_heads, int *head_dim,
                         int *device);

/* Append keys and values, turned by their positions, to the cache.
 *   k, v      device fp16, rows x (kv_heads * head_dim), row strides ldk, ldv
 *   q, q_out  device fp16, rows x (heads * head_dim): q turned as k is and
 *             rounded once; both NULL, or q_out may be q itself with the same
 *             stride
 *   rope      device fp32, positions x rot: of each position rot / 2 cosines,
 *             then rot / 2 sines, at least columns * page_tokens positions;
 *             rot even, at most head_dim, 0 for no rotation.  Pair i is dims
 *             (i, i + rot / 2), or (2i, 2i + 1) when interleaved:
 *             (a, b) -> (a cos - b sin, a sin + b cos), in fp32
 * A page whose first token is written starts a new scale; otherwise its scale
 * grows as needed and its earlier numbers are rounded again, by half a step
 * each time.  A page that receives a NaN or an infinity reads as NaN from then
 * on.  Appending the same rows twice leaves what appending them once does. */
lb_status lb_cache_append(lb_cache *C, const void *k, int64_t ldk, const void *v, int64_t ldv, const void *q,
                          int64_t ldq, void *q_out, int64_t ldqo, int heads, const float *rope,
                          int64_t positions, int rot, int interleaved, const int32_t *start,
                          const int32_t *lengths, const int32_t *table, int64_t ldt, int columns,
                          int sequences, int64_t rows, void *stream);

/* The values of the sequences' last tokens: k, v (device fp16, rows x
 * (kv_heads * head_dim), row strides ldk, ldv), each rounded once. */
lb_status lb_cache_read(const lb_cache *C, void *k, int64_t ldk, void *v, int64_t ldv, const int32_t *start,
                        const int32_t *lengths, const int32_t *table, int64_t ldt, int columns, int sequences,
                        int64_t rows, void *stream);

/* Workspace for lb_cache_attend calls of up to `rows` rows of `heads` heads,
 * `sequences` sequences and max_length tokens, now. */
lb_status lb_cache_reserve(lb_cache *C, int64_t rows, int heads, int64_t sequences, int64_t max_length);

/* out = softmax(scale * q K^T) V over the cache: exact products, scores,
 * softmax and sums in fp32, out rounded once.  A weight times its page's scale
 * of values enters the sum over V as two fp16 numbers (22 bits) where a
 * sequence has up to 32 rows of a key head (or one token) in the call, and as
 * one (11 bits) otherwise, lifted so that the largest is near 2^12.
 *   q, out    device fp16, rows x (heads * head_dim), row strides ldq, ldo;
 *             heads a multiple of kv_heads: head h reads key head
 *             h / (heads / kv_heads).  out must not overlap the inputs
 *   max_length  a bound on lengths that the call is cut up for (tokens past it
 *             are not seen), or 0: what the table can hold
 *   scale     0 to 1e6
 *   causal    a row sees its sequence's tokens up to its own position;
 *             otherwise all of them
 *   window    with causal: the last `window` of those only; 0 for all
 * A row that sees no token gets zeros; one that does, with an infinity or a
 * NaN in its q, NaN. */
lb_status lb_cache_attend(lb_cache *C, const void *q, int64_t ldq, int heads, void *out, int64_t ldo,
                          const int32_t *start, const int32_t *lengths, const int32_t *table, int64_t ldt,
                          int columns, int sequences, int64_t rows, int64_t max_length, float scale, int causal,
                          int window, void *stream);

lb_status lb_cache_destroy(lb_cache *C);

/* ---------------------------------------------------------- diagnostics */
const char *lb_status_str(lb_status st);
const char *lb_last_error(void);
/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int lb_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LB_H */
