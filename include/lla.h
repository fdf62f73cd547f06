/*
 * liblla: causal Local Linear Attention (LLA) forward on one NVIDIA GB300 (sm_103a).
 *
 * Definition (the operation every entry point below serves)
 * ---------------------------------------------------------
 * "Parallax" (Tilde Research blog), section 2 "Parallax & Local Linear Attention",
 * paragraph "Canonical Formulation"; the same definition in "Parallax: Parameterized Local
 * Linear Attention for Language Modeling" (arXiv 2605.29157), section 2, LLA paragraph.
 * For each query q_i (0-based position i) over its causal prefix j <= i (diagonal included),
 * LLA fits the local linear estimator b + W (x - q_i) to the pairs (k_j, v_j) by weighted
 * least squares with kernel weights w_ij = exp(q_i . k_j / h) and ridge penalty
 * lambda * ||W||_F^2, and outputs the intercept b. In closed form
 *     o_i = vbar_i + C_vk (C_kk + lambda I)^-1 (q_i - kbar_i),
 * with kbar, vbar the w-weighted means and C_kk, C_vk the (unnormalised) w-weighted centred
 * second moments. lambda is absolute against the raw weights exp(q.k/h); h divides the logit.
 *
 * Conventions shared by all entry points
 * --------------------------------------
 * - Layout: q, k are [B, H, T, d] and v, out are [B, H, T, dv], contiguous, row-major
 *   (innermost index = feature). Element type is given by `dtype` (lla_dtype) and is the same
 *   for q, k, v and out. Sums are accumulated in fp32 (in compensated fp32 pairs for the fp32
 *   element type). For bf16 inputs the forward runs on the tensor cores: the kernel weights enter
 *   the contraction rounded to bf16, the key products k_a*k_b exactly (as an exact pair of bf16
 *   values). With d < 64 it runs on zero-padded copies of q, k and v (d = dv = 64; zero features
 *   leave the intercept unchanged: their moments are exactly zero, so the ridge system is block-
 *   diagonal with a zero right-hand side on the padded block), at the cost of the padded work.
 * - Pointers named *_host are host memory; every other data pointer is device memory of the
 *   current CUDA device, 16-byte aligned. The caller owns every buffer; `out` must not overlap
 *   an input.
 * - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream). Calls are
 *   asynchronous on that stream unless stated otherwise; they return after validating the
 *   arguments and enqueueing work.
 * - Errors: every call returns an lla_status. Argument errors are detected on the host before
 *   any work is enqueued and leave all buffers untouched. Numerical failures inside a kernel
 *   (a non-positive pivot in a ridge solve, e.g. from non-finite inputs) are recorded in a
 *   per-device status word read by lla_stream_status(); the affected output rows are NaN. (The
 *   forward first retries such a row: in float64 from its moments on the tensor-core path, or,
 *   when its causal prefix holds at most 64 keys, exactly from q, k and v; only a row that still
 *   fails -- non-finite inputs, or a longer prefix with fewer than d + 1 affinely independent
 *   keys under a tiny effective ridge -- is reported.) No entry point aborts, traps or exits.
 * - Supported sizes: d, dv in {16, 32, 64}; B, H, T >= 0 with B*H*T < 2^31 (B*H*T == 0 is a
 *   no-op that returns LLA_OK); h > 0 and lambda > 0, both finite.
 */
#ifndef LLA_H
#define LLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LLA_VERSION_MAJOR 0
#define LLA_VERSION_MINOR 2
#define LLA_VERSION_PATCH 0

typedef enum {
  LLA_OK = 0,
  LLA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad h/lambda/dtype, negative size       */
  LLA_ERR_UNSUPPORTED = 2, /* d or dv outside {16, 32, 64}, or B*H*T >= 2^31; for the paged
                              operators, the limits listed with them                              */
  LLA_ERR_CUDA = 3,        /* a CUDA runtime call or kernel launch failed                         */
  LLA_ERR_NUMERICAL = 4,   /* a ridge solve met a non-positive pivot (rows set to NaN)            */
  LLA_ERR_TIMEOUT = 5      /* a bounded device-side wait gave up (kernel returned early)          */
} lla_status;

typedef enum { LLA_F32 = 0, LLA_BF16 = 1 } lla_dtype;

/* Implementation choices (lla_options.path). */
typedef enum {
  LLA_PATH_AUTO = 0,        /* tensor cores for bf16 (the forward: any d, zero-padded to 64 when
                               d < 64; the other ops: d = dv = 64; paged attention: every
                               head size), CUDA cores otherwise */
  LLA_PATH_CUDA_CORE = 1,   /* CUDA cores always */
  LLA_PATH_TENSOR_CORE = 2, /* tensor cores wherever supported (currently the same as AUTO) */
  LLA_PATH_CG = 3           /* lla_forward*_ex only: matrix-free conjugate gradients for the ridge
                               systems (bf16 with dv = 64 or d < 64; as AUTO elsewhere) */
} lla_path;

/* Closed form of the LLA intercept that a forward evaluates (lla_options.form). */
typedef enum { LLA_FORM_CENTRED = 0, LLA_FORM_PAGE = 1 } lla_form;

/* Test-only faults (lla_options.test_fault). */
typedef enum {
  LLA_FAULT_NONE = 0,
  LLA_FAULT_WITHHOLD_KEYS = 1 /* the tensor-core moments stage's key loader never stages its first
                                 key block, so the waits on it run out (see lla_forward_ex) */
} lla_test_fault;

/*
 * Per-call options of the *_ex entry points. An all-zero struct (or a NULL pointer) selects the
 * defaults, which are what the entry points without options use. Options belong to the one call
 * they are passed to: nothing is remembered between calls, so concurrent callers cannot change
 * each other's results.
 *   path         lla_path (the operations other than the forward accept AUTO, CUDA_CORE and
 *                TENSOR_CORE; CUDA_CORE selects their CUDA-core kernels).
 *   form         lla_form (forward only), see lla_forward_ex.
 *   cg_max_iters conjugate-gradient iteration cap, 1..1024 (0 = 1024), LLA_PATH_CG only.
 *   cg_rel_tol   CG stopping tolerance in (0, 1) (0 = 1e-3), LLA_PATH_CG only.
 *   test_fault   lla_test_fault (forward only; 0 in normal use).
 * Any other value of a field makes the call return LLA_ERR_INVALID_ARG before any work.
 */
typedef struct lla_options {
  int path;
  int form;
  int cg_max_iters;
  float cg_rel_tol;
  int test_fault;
  int reserved[3]; /* must be zero */
} lla_options;

/* Number of timed stages recorded per lla_forward call by the profiling hooks below:
 * 0 prep (per-head means, CUDA-core path; the tensor-core path's key frame runs beside stage 1
 * and is counted there), 1 weights (tensor-core path: row maxima, the weights and their sums),
 * 2 moments (the moment contraction; on the CUDA-core path also the weights), 3 solve,
 * 4 readout (with the exact pass over listed short prefixes beside it). A stage that a path does
 * not have records zero time. */
#define LLA_NUM_STAGES 5

/*
 * Causal LLA forward (the operation defined at the top of this header).
 * q, k: [B,H,T,d]; v: [B,H,T,dv]; out: [B,H,T,dv]; all device, element type `dtype`.
 * Scratch memory is taken from the CUDA stream-ordered allocator on `stream`
 * (cudaMallocAsync/cudaFreeAsync, released at the end of the call in stream order);
 * lla_workspace_size() tells how much. Use lla_forward_ws() to supply it yourself.
 * Rows whose causal prefix holds few keys may be recomputed exactly in float64 (the solve lists
 * them); that pass runs on a library-owned side stream of the current device, at its highest
 * priority, ordered after this call's solve and before the rest of the call by two events, so
 * that to the caller the whole call is still ordered on `stream`. The side stream and its events
 * are created on a device's first forward call (make that call before any stream capture); a
 * call captured into a CUDA graph forks to the side stream and joins back within the capture.
 */
int lla_forward(const void* q, const void* k, const void* v, void* out, int B, int H, int T,
                int d, int dv, float h, float lambda, int dtype, void* stream);

/* Bytes of device scratch lla_forward_ws needs for these sizes (0 for invalid sizes).
 * Host-only; touches no device. */
size_t lla_workspace_size(int B, int H, int T, int d, int dv, int dtype);

/*
 * lla_forward with caller-provided device scratch `workspace` (256-byte aligned, at least
 * lla_workspace_size(...) bytes, not used by anything else until the work on `stream` is done).
 * Allocates nothing. Returns LLA_ERR_INVALID_ARG if the workspace is missing or too small.
 */
int lla_forward_ws(const void* q, const void* k, const void* v, void* out, int B, int H, int T,
                   int d, int dv, float h, float lambda, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * lla_forward / lla_forward_ws with per-call options (opts may be NULL: the defaults). workspace
 * may be NULL (scratch from the stream-ordered allocator, as lla_forward) or caller-provided as
 * for lla_forward_ws (the size does not depend on the options).
 *
 * - opts->path: LLA_PATH_CUDA_CORE forces the CUDA-core moments, solve and readout for every
 *   shape; LLA_PATH_CG solves the per-query ridge systems by conjugate gradients instead of
 *   accumulating the d x d moments and factoring them: each product with C_kk is one streaming
 *   pass over the prefix, as the "Parallax" blog (s.2 "Difficulties in Scaling LLA") describes
 *   exact LLA being computed. Each query row iterates until ||r|| <= cg_rel_tol ||r_0|| (r the
 *   residual of (C_kk + lambda' I) y = q - kbar, r_0 = q - kbar) or cg_max_iters passes have run.
 *   A call on this path synchronises its stream every 8 iterations on the host to test whether any
 *   query tile is still iterating, so it blocks the calling thread and cannot be captured in a
 *   CUDA graph. Paths AUTO, CUDA_CORE and TENSOR_CORE compute the same moments; CG solves the
 *   same systems iteratively.
 * - opts->form ("Parallax" blog, s.2 Canonical Formulation and Appendix B; both forms equal the
 *   intercept of the weighted ridge regression):
 *     LLA_FORM_CENTRED (default) o = vbar + C_vk y,  (C_kk + lambda' I) y = q - kbar;
 *     LLA_FORM_PAGE  o = sum w (1 - z.rho*) v / sum w (1 - z.rho*),  z = k - q,
 *       (sum w z z^T + lambda' I) rho* = sum w z, evaluated as the exact-LLA two-branch epilogue
 *       (O1 - O2) / (d1 - d2). It runs on the tensor-core dense strategy only (bf16 with dv = 64
 *       or d < 64, path AUTO or TENSOR_CORE; otherwise LLA_ERR_UNSUPPORTED). Its system carries the rank-one
 *       term w (kbar - q)(kbar - q)^T on top of the centred one, so it is worse conditioned for
 *       queries far from the weighted key mean.
 * - opts->test_fault = LLA_FAULT_WITHHOLD_KEYS exercises the bounded device waits: the
 *   tensor-core moments stage (bf16; LLA_ERR_UNSUPPORTED on other paths) never stages
 *   its first key block, so every wait that needs it gives up after the wait limit (~2 s), the
 *   stage returns early without issuing the tensor-core work that depends on it, and
 *   LLA_ERR_TIMEOUT is recorded in the status word (lla_stream_status). The output of such a call
 *   is undefined; the stream and the device stay usable. For tests only.
 */
int lla_forward_ex(const void* q, const void* k, const void* v, void* out, int B, int H, int T,
                   int d, int dv, float h, float lambda, int dtype, const lla_options* opts,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Size of the fixed device scratch that lla_forward_noalloc uses: 64 MiB. */
#define LLA_NOALLOC_SCRATCH_BYTES (64ull << 20)

/*
 * lla_forward for callers that cannot allocate device memory. (The pages have no counterpart:
 * this is a deployment convenience, not part of the method.)
 *
 * Some callers are not allowed to allocate GPU memory themselves -- a plugin that its host
 * application only hands input and output buffers, or a latency-critical loop that must not call
 * the allocator while it runs, since an allocation can block on the device or fail under memory
 * pressure at an unpredictable moment. This entry point calls no allocator at all: its scratch is
 * one fixed array of LLA_NOALLOC_SCRATCH_BYTES in device memory owned by the library, which every
 * GPU that loads this part of the library keeps until the process exits. The caller still passes
 * q, k, v and out exactly as for lla_forward, and the result is the same.
 *
 * - Size limit: returns LLA_ERR_UNSUPPORTED, before touching the device, when
 *   lla_workspace_size(B, H, T, d, dv, dtype) exceeds LLA_NOALLOC_SCRATCH_BYTES (e.g. bf16
 *   d = dv = 64 fits T <= 4343 at B*H = 1 and T <= 704 at B*H = 8; the tensor-core path's weight
 *   scratch grows with B*H*T^2). Other argument errors are those of lla_forward.
 * - Set-up: the first call on each device looks up the scratch array's device address (with that
 *   device current) and caches it, and (as any first forward call) creates the side stream of the
 *   exact short-prefix pass; make that first call before any stream capture.
 * - Sharing: all calls on a device share the one array. Calls whose work overlaps on the GPU
 *   (other streams, other host threads, without ordering between them) race on it and corrupt
 *   each other's results; order them on one stream or synchronise between them. Each call
 *   overwrites whatever an earlier call left, and nothing from an earlier call is read.
 */
int lla_forward_noalloc(const void* q, const void* k, const void* v, void* out, int B, int H,
                        int T, int d, int dv, float h, float lambda, int dtype, void* stream);

/*
 * End-to-end variant on HOST buffers: copies q_host, k_host, v_host to the device on `stream`,
 * runs the forward, copies the result to out_host and synchronises `stream` before returning.
 * Host buffers may be pageable or pinned (pinned copies overlap better). Device buffers and
 * scratch come from the stream-ordered allocator and are released before the call returns.
 * Returns the forward's status, including any device status recorded by this call's kernels.
 */
int lla_forward_host(const void* q_host, const void* k_host, const void* v_host, void* out_host,
                     int B, int H, int T, int d, int dv, float h, float lambda, int dtype,
                     void* stream);

/*
 * Debug entry: raw max-shifted kernel-weighted moments for n selected queries (the sums from
 * which the pages' omega_i, mu_i and Sigma_i follow, "Parallax" blog s.2 Canonical
 * Formulation). idx[n] (device, int64) holds flat query indices (b*H + hh)*T + i.
 * For each selected query: m = max_{j<=i} q_i.k_j/h, w_j = exp(q_i.k_j/h - m) and
 *   m[n], omega[n] = sum w_j, sk[n,d] = sum w_j k_j, sv[n,dv] = sum w_j v_j,
 *   Skk[n,d,d] = sum w_j k_j k_j^T, Svk[n,dv,d] = sum w_j v_j k_j^T   (fp32, device, row-major).
 * Any output pointer may be NULL to skip it. Accumulation is in fp64 (not a fast path).
 * An out-of-range idx entry sets LLA_ERR_INVALID_ARG in the device status word and leaves that
 * query's outputs untouched.
 */
int lla_moments(const void* q, const void* k, const void* v, const int64_t* idx, int n,
                float* m, float* omega, float* sk, float* sv, float* Skk, float* Svk,
                int B, int H, int T, int d, int dv, float h, int dtype, void* stream);

/*
 * Causal Parallax forward with a given probe ("Parallax" blog, s.2 paragraph "Parallax" and
 * Appendix B with eta = 0; streaming form in s.3 "One extra branch, no extra I/O"; output
 * combination as printed in Appendix C): for each query i over its causal prefix j <= i,
 *     o_i = o_SA_i - Sigma_KV^(i) r_i = (1 + d2/d1) O1/d1 - O2/d1,
 * where p_ij = exp(q_i . k_j / h) / sum_l exp(q_i . k_l / h) are the softmax weights, o_SA_i =
 * sum_j p_ij v_j, Sigma_KV^(i) = sum_j p_ij (v_j - vbar_i)(k_j - kbar_i)^T (dv x d), and in the
 * streaming form P1 = exp(q.k/h), P2 = P1 * (r_i . k_j), O1 = P1 V, O2 = P2 V, d1 = sum P1,
 * d2 = sum P2. r = 0 gives causal softmax attention with scale 1/h.
 * q, k, r: [B,H,T,d]; v, out: [B,H,T,dv]; all device, element type `dtype`, 16-byte aligned; the
 * conventions at the top of this header apply (lambda plays no part). bf16 inputs with
 * d = dv = 64 run on the tensor cores (weights rounded to bf16, P2 as an exact hi/lo bf16 pair,
 * fp32 accumulation); everything else runs on the CUDA cores in fp32 (lla_parallax_forward_ex
 * with path LLA_PATH_CUDA_CORE forces them for every shape). Allocates nothing. Non-finite inputs
 * give non-finite outputs; no status is recorded.
 */
int lla_parallax_forward(const void* q, const void* k, const void* v, const void* r, void* out,
                         int B, int H, int T, int d, int dv, float h, int dtype, void* stream);
int lla_parallax_forward_ex(const void* q, const void* k, const void* v, const void* r, void* out,
                            int B, int H, int T, int d, int dv, float h, int dtype,
                            const lla_options* opts, void* stream);

/*
 * Rotary positions. A spec says how far a position turns each of rot/2 pairs of a head's first `rot`
 * features: pair i is (i, i + rot/2) (LLA_ROTARY_HALVES) or (2i, 2i + 1) (LLA_ROTARY_INTERLEAVED) and at
 * position pos becomes scale * (x0 cos a - x1 sin a, x0 sin a + x1 cos a), a = pos * freq[i]. The other
 * features are copied. (The probe of Parallax meets the keys like a query and is rotated like one.) Angles are exact: pos * freq[i] is
 * taken modulo a turn before it is rounded, so far positions lose nothing. rot is even, 2 .. d; |freq| <=
 * 2^20; specs are host memory, read during the call.
 */
typedef enum { LLA_ROTARY_HALVES = 0, LLA_ROTARY_INTERLEAVED = 1 } lla_rotary_layout;
typedef struct lla_rotary_spec {
  double freq[64];  /* radians per position of pair i */
  float scale;      /* on the rotated features */
  int rot;
  int layout;       /* lla_rotary_layout */
  int reserved[3];  /* must be zero */
} lla_rotary_spec;

/*
 * Fills a spec: freq[i] = base^(-2i/rot) (base >= 1), scale 1, stretched for contexts `factor` (>= 1) times longer by
 *   LLA_STRETCH_POSITIONS    freq / factor (positions interpolated),
 *   LLA_STRETCH_BASE         base * factor^(rot / (rot - 2)): the slowest pair as above, the fastest as it was,
 *   LLA_STRETCH_WAVELENGTHS  by the turns n that a pair makes over the `context` positions of training: with
 *                            keep = clamp((n - slow) / (fast - slow), 0, 1), freq * (keep + (1 - keep) / factor),
 *                            and scale = 0.1 ln(factor) + 1,
 * or not at all (LLA_STRETCH_NONE; factor is not used). Any other table of frequencies goes into the struct
 * directly. Host only; LLA_ERR_INVALID_ARG leaves the spec as it was.
 */
typedef enum {
  LLA_STRETCH_NONE = 0,
  LLA_STRETCH_POSITIONS = 1,
  LLA_STRETCH_BASE = 2,
  LLA_STRETCH_WAVELENGTHS = 3
} lla_rotary_stretch;
int lla_rotary_frequencies(lla_rotary_spec* spec, int rot, int layout, double base, int stretch, double factor,
                           int context, double slow, double fast);

/*
 * Rotates `count` (1 .. 3) tensors that share their positions, such as q, k and r of an attention: x[i] is
 * [B, heads[i], T, d], y[i] the same, 16-byte aligned (x[i] == y[i]: in place; otherwise none may overlap another), x,
 * y and heads host arrays. positions [B, T] (device) or NULL: 0 .. T-1. backward nonzero: the gradient with respect
 * to the input from that with respect to the output, which is the transposed rotation times scale. d in {16, 32, 64,
 * 128}; fewer than 2^31 rows, and at most 2^31 - 2^17 heads, in all (LLA_ERR_UNSUPPORTED). One launch, asynchronous,
 * allocates nothing; fp32 arithmetic, one rounding.
 */
int lla_rotary(const lla_rotary_spec* spec, const void* const* x, void* const* y, const int* heads, int count,
               const int* positions, int B, int T, int d, int backward, int dtype, void* stream);

/*
 * Decode: one query per head against a key/value cache of L positions that the query attends to
 * in full (it is the newest token; its own key and value are already appended). The output is
 * what lla_forward returns for its last row, o = vbar + C_vk (C_kk + lambda I)^-1 (q - kbar) with
 * w_j = exp(q . k_j / h) over all L positions ("Parallax" blog, s.2 Canonical Formulation).
 * q: [B,H,d]; k: [B,H,L,d]; v: [B,H,L,dv]; out: [B,H,dv]; device, element type `dtype`, 16-byte
 * aligned; d, dv in {16, 32, 64}; B*H*L < 2^31; h, lambda finite and positive. The cache of each
 * head is split over several CTAs that reduce their chunk to partial moments (float32, shifted by
 * a maximum logit of the chunk); the last CTA of the head to finish merges them and solves the
 * ridge system in float64 (split-KV with a last-arriver merge, as the blog's decode kernel,
 * Appendix C). For bf16 with d = dv = 64 the chunk's second moments run on the tensor cores
 * (weights rounded to bf16, exact products, float32 sums) unless lla_decode_ex is given path
 * LLA_PATH_CUDA_CORE; otherwise on the CUDA cores with float32 weights. Asynchronous on `stream`; scratch from the stream-ordered pool. B*H = 0 is a
 * no-op; L = 0 with B*H > 0 is LLA_ERR_INVALID_ARG. A non-positive pivot (non-finite inputs)
 * makes that head's output NaN and records LLA_ERR_NUMERICAL.
 */
int lla_decode(const void* q, const void* k, const void* v, void* out, int B, int H, int L, int d,
               int dv, float h, float lambda, int dtype, void* stream);
int lla_decode_ex(const void* q, const void* k, const void* v, void* out, int B, int H, int L,
                  int d, int dv, float h, float lambda, int dtype, const lla_options* opts,
                  void* stream);

/*
 * Parallax decode with probe r ([B,H,d], same dtype): o = vbar - Sigma_KV r over all L cached
 * positions, as lla_parallax_forward's last row, computed as the blog's streaming combination
 * (1 + d2/d1) O1/d1 - O2/d1 (Appendix C) with the same split-KV and last-arriver merge as
 * lla_decode (float32 partials, the merge in float64). Otherwise as lla_decode (lambda plays no
 * part; no status is recorded).
 */
int lla_parallax_decode(const void* q, const void* k, const void* v, const void* r, void* out,
                        int B, int H, int L, int d, int dv, float h, int dtype, void* stream);
int lla_parallax_decode_ex(const void* q, const void* k, const void* v, const void* r, void* out,
                           int B, int H, int L, int d, int dv, float h, int dtype,
                           const lla_options* opts, void* stream);

/*
 * Causal Parallax backward ("Parallax" blog, Appendix F "Parallax backward (closed form)": a
 * forward-like pass caches per-row scalars, then a row-tile pass and a column-tile pass). Given
 * the inputs of lla_parallax_forward (q, k, r: [B,H,T,d]; v: [B,H,T,dv]) and the upstream
 * gradient dout = dL/do ([B,H,T,dv]), writes dq = dL/dq, dk, dr ([B,H,T,d]) and dv ([B,H,T,dv]).
 * The appendix's formulas were lost in extraction; the gradients are those of the forward itself
 * (o_i = sum_j p_ij (1 + tbar_i - t_ij) v_j with p_i = softmax of q_i.k_j / h over j <= i,
 * t_ij = r_i . k_j, tbar_i = sum_j p_ij t_ij). All buffers are device pointers, contiguous
 * row-major, 16-byte aligned, of the dtype given (gradients in the inputs' dtype; fp32
 * arithmetic); the caller owns them; outputs must not alias inputs. d, dv in {16, 32, 64}
 * (else LLA_ERR_UNSUPPORTED); h > 0 and finite, B, H, T >= 0 (else LLA_ERR_INVALID_ARG). Three
 * launches, asynchronous on `stream`, with a scratch of 32 bytes per query row from the
 * stream-ordered pool: for bf16 with d = dv = 64, the tensor-core forward kernel caching the row
 * records, then tensor-core row-tile and column-tile passes (tcgen05; weights rounded to bf16,
 * fp32 accumulation); for every other shape (or with path LLA_PATH_CUDA_CORE through
 * lla_parallax_backward_ex), the same three passes on the CUDA cores in fp32. Returns LLA_OK,
 * LLA_ERR_* for invalid arguments, LLA_ERR_CUDA.
 */
int lla_parallax_backward(const void* q, const void* k, const void* v, const void* r,
                          const void* dout, void* dq, void* dk, void* dv, void* dr, int B, int H,
                          int T, int d, int dv_, float h, int dtype, void* stream);
int lla_parallax_backward_ex(const void* q, const void* k, const void* v, const void* r,
                             const void* dout, void* dq, void* dk, void* dv, void* dr, int B,
                             int H, int T, int d, int dv_, float h, int dtype,
                             const lla_options* opts, void* stream);

/*
 * Synchronises `stream`, then reads and clears the current device's status word.
 * Returns LLA_OK, LLA_ERR_NUMERICAL, LLA_ERR_TIMEOUT, LLA_ERR_INVALID_ARG (bad idx in
 * lla_moments) or LLA_ERR_CUDA (a sticky CUDA error or failed synchronisation).
 */
int lla_stream_status(void* stream);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* lla_status_string(int status);

/* LLA_VERSION_MAJOR*10000 + LLA_VERSION_MINOR*100 + LLA_VERSION_PATCH. */
int lla_version(void);

/* Number of kernels this library has launched in this process (all devices, all streams). */
unsigned long long lla_launch_count(void);

/*
 * Stage timing. lla_profile_enable(1) makes every later lla_forward/lla_forward_ws call record
 * CUDA events on its stream at the LLA_NUM_STAGES stage boundaries (no synchronisation is
 * added). lla_profile_collect() waits for the recorded events, writes the summed duration in
 * milliseconds of each stage over all recorded calls to stage_ms[0..min(max_stages,
 * LLA_NUM_STAGES)-1], stores the number of calls in *n_calls (if not NULL), and forgets them.
 * lla_profile_enable(0) stops recording. Returns LLA_OK or LLA_ERR_CUDA.
 */
int lla_profile_enable(int on);
int lla_profile_collect(float* stage_ms, int max_stages, int* n_calls);

/*
 * ---------------------------------------------------------------------------------------------
 * Paged caches: keys and values of many sequences in pages that a user's allocator hands out, the
 * append of new tokens, attention of those tokens over the cache (softmax, or Parallax with a
 * probe), and eviction of the positions that received the least attention.
 *
 * A cache holds num_pages pages of page_size slots per key/value head: k_pages is [num_pages,
 * kv_heads, page_size, d], v_pages [num_pages, kv_heads, page_size, dv], both of type `dtype`, and
 * mass (may be NULL where it is not used) [num_pages, kv_heads, page_size] fp32, the attention
 * weight that each slot has received so far. Position j of sequence b is slot j % page_size of page
 * page_table[b * max_pages + j / page_size]; lens[b] (0 .. max_pages * page_size) counts the
 * sequence's positions. Pages may come in any order and may be shared by sequences that only read
 * them. All pointers are device memory; k_pages, v_pages and mass 16-byte
 * aligned.
 *
 * New tokens of all sequences lie one after the other, as [tokens, heads, size] rows: sequence b's
 * are starts[b] .. starts[b+1]-1 (device memory, [num_seqs + 1], ascending, at most `tokens`), and
 * they are the sequence's last positions: lens already counts them. Rows that no sequence covers (before
 * starts[0], from starts[num_seqs] on) take no part, and their outputs are not written.
 *
 * Attention over these caches is softmax attention or Parallax; the local linear attention of lla_forward
 * and lla_decode reads contiguous keys and values only.
 *
 * Supported: d, dv in {16, 32, 64, 128}; page_size a power of two in 16 .. 1024; max_pages *
 * page_size < 2^30; tokens < 2^30, tokens * q_heads < 2^31, num_pages * kv_heads < 2^31, num_seqs and kv_heads
 * at most 65535, their product < 2^28 (LLA_ERR_UNSUPPORTED otherwise). What only the device can see is checked there: a
 * page index outside 0 .. num_pages-1, a length beyond the table, or starts that descend or pass
 * `tokens` are recorded in the status word (lla_stream_status: LLA_ERR_INVALID_ARG); nothing out of
 * range is read or written, and the outputs of that sequence are unspecified (with an impossible length or
 * starts it is left out: nothing is appended, no weight is added, nothing is kept of it). Slots that no row
 * sees may hold anything, infinities and NaN included.
 */
typedef struct lla_paged_cache {
  void* k_pages;
  void* v_pages;
  float* mass;
  const int* page_table; /* [num_seqs, max_pages] */
  int* lens;             /* [num_seqs] */
  int num_seqs, kv_heads, page_size, max_pages, num_pages, d, dv;
  int dtype;       /* lla_dtype */
  int reserved[2]; /* must be zero */
} lla_paged_cache;

/*
 * Writes the new tokens' keys k_new [tokens, kv_heads, d] and values v_new [tokens, kv_heads, dv]
 * into their slots and, when the cache has a mass, sets theirs to zero. Tokens beyond a sequence's
 * length (more new tokens than positions) are not written. Allocates nothing.
 */
int lla_paged_append(const lla_paged_cache* cache, const void* k_new, const void* v_new,
                     const int* starts, int tokens, void* stream);

/*
 * lla_paged_append with rotary positions: k_new is written rotated, and the same tokens' queries q and probe r
 * ([tokens, q_heads, d] or NULL; r needs q) come out rotated in q_out and r_out (which may be q and r; no other overlap). The
 * token's position is that of its sequence's first new token's slot plus offsets[token] (device memory,
 * [tokens]; NULL: its index among the sequence's new tokens, so its own slot's): the depth of a drafted
 * node, and, where eviction has dropped positions, their number besides. Rows of q_out and r_out that no sequence covers
 * are not written. At most 2^31 - 2^17 heads of k, q and r in all (LLA_ERR_UNSUPPORTED).
 */
int lla_paged_append_rotary(const lla_paged_cache* cache, const lla_rotary_spec* spec, const void* k_new,
                            const void* v_new, const void* q, const void* r, void* q_out, void* r_out, int q_heads,
                            const int* offsets, const int* starts, int tokens, void* stream);

/*
 * The queries of one lla_paged_attention call.
 *   q, r, out   [tokens, q_heads, d], the same (NULL: softmax attention), [tokens, q_heads, dv],
 *               of the cache's type. q_heads is a multiple of kv_heads: query heads hk*g ..
 *               hk*g + g-1 read key/value head hk, g = q_heads / kv_heads.
 *   lse         [tokens, q_heads] fp32 or NULL: log of the sum of exp(q.k/h) over the visible keys.
 *   max_new     at least the largest number of new tokens of a sequence (it sizes the launch; a
 *               sequence with more may be reported as a bad index, its rows unspecified).
 *   window      0, or how many last positions a token sees, its own included; sinks: the first
 *               positions that stay visible besides. The token at position i sees positions
 *               j <= i with window == 0, j > i - window or j < sinks.
 *   track_mass  nonzero: cache->mass of every visible slot grows by the softmax weights that the
 *               new tokens' rows give it, summed over the tokens and the g heads (with a probe too:
 *               its signed correction is not counted). The sums do not depend on scheduling.
 *               Sequences that track may not share pages (their sums would be lost).
 *   path        lla_path: AUTO, CUDA_CORE or TENSOR_CORE.
 */
typedef struct lla_paged_query {
  const void* q;
  const void* r;
  void* out;
  float* lse;
  const int* starts;
  int tokens, max_new, q_heads;
  float h;
  int window, sinks, track_mass, path;
  int reserved[2]; /* must be zero */
} lla_paged_query;

/*
 * Attention of the new tokens over the cache (append them first). Per row, over its visible keys:
 * p = softmax(q.k / h), o = sum p v, or with a probe the Parallax output
 * o = sum p (1 + tbar - t) v with t = r.k and tbar = sum p t, as lla_parallax_forward computes it.
 * A row that sees nothing (a position below zero, or only keys whose logit is -infinity) gives o = 0,
 * lse = -infinity and adds no weight. Sums are fp32.
 * `workspace` (256-byte aligned device memory of lla_paged_workspace_size bytes; its contents need
 * not be kept between calls) or NULL: scratch from the stream-ordered allocator.
 */
size_t lla_paged_workspace_size(const lla_paged_cache* cache, const lla_paged_query* query);
int lla_paged_attention(const lla_paged_cache* cache, const lla_paged_query* query, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Attention of trees of drafted tokens over the cache (append them first): a sequence's new tokens are the
 * nodes of a tree (or of several) that goes on where the sequence's other positions end. parents [tokens]
 * (device memory) holds of each node its parent's index among the sequence's new tokens, which comes before
 * the node's own, or -1: a child of the last position before the nodes. Node i lies in slot first + i,
 * first = lens - (number of nodes), and is at position first + depth(i), depth 0 being a child of -1. It sees
 * itself, its ancestors, and the positions before the nodes; with a window those of them whose position is
 * within the last `window` up to its own or among the first `sinks`. Otherwise as lla_paged_attention, for
 * the same caches and queries: parents[i] = i - 1 gives its results. Weights are not tracked: track_mass has to be 0,
 * and the positions that a node sees get nothing from it, not even when it is kept. After drafted steps the mass
 * that lla_paged_evict goes by holds the weights of the other tokens only.
 *
 * At most 1024 nodes to a sequence (LLA_ERR_UNSUPPORTED where max_new and tokens are both larger). Reported
 * in the status word, the sequence's outputs unspecified: a parent that does not come before its child,
 * more nodes than max_new or than positions.
 */
size_t lla_paged_tree_workspace_size(const lla_paged_cache* cache, const lla_paged_query* query);
int lla_paged_tree_attention(const lla_paged_cache* cache, const lla_paged_query* query, const int* parents,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * Eviction: for every sequence of `from` and key/value head, min(lens, budget) positions are kept:
 * the first `sinks`, the last `recent` (sinks + recent <= budget), and of the others those with the
 * largest mass (ties: the lower position; NaN counts as the lowest), in their order. Their keys,
 * values and mass are copied to slots 0, 1, .. of `to`, to->lens is set, and kept [num_seqs,
 * kv_heads, budget] gets their positions in `from` (-1 past the last). `to` has the same sequences,
 * heads, page size and types; it may use the same page arrays (another table, and pages that no
 * sequence of `from` holds), not the same table or lens.
 */
int lla_paged_evict(const lla_paged_cache* from, const lla_paged_cache* to, int budget, int sinks,
                    int recent, int* kept, void* stream);

/*
 * Sharing, growing and releasing pages. refs [num_pages] (device memory, 16-byte aligned, the caller's, zero at
 * first) counts the table entries that hold each page: sequence b holds the first ceil(lens[b] / page_size)
 * entries of its row, and a page is free while refs is 0. Sequences that fork share all their pages; one
 * that grows takes its own copy of a last page that it would write to while others hold it. Fork, free and
 * grow touch tables, lens and refs alone, which the caches of a model's layers share: they are called once,
 * lla_paged_copy and lla_paged_compact once per layer. lla_paged_evict neither reads nor changes refs: its `to`
 * gets the pages for the kept positions by lla_paged_grow. None of them allocates or synchronises, and all give
 * the same pages whatever the scheduling. Impossible lengths, page numbers, parents and paths are reported in the
 * status word (LLA_ERR_INVALID_ARG); unless it says otherwise below, that sequence or pair is left as it is.
 *
 * lla_paged_fork: sequence c of `to` becomes a copy of sequence parents[c] of `from` (-1: an empty one): its table
 * entries and length, the pages' refs one more each. `to` is another table and lens over the same pages (what
 * it held before is not released), with room for the lengths. A parent out of range, one that does not
 * fit, or one with a page number out of range, gives an empty sequence.
 */
int lla_paged_fork(const lla_paged_cache* from, const lla_paged_cache* to, const int* parents, int* refs, void* stream);

/*
 * Shortens each sequence to its first keep[b] positions (keep NULL or negative: to none; more than it has: as
 * it is) and gives up the pages behind them: refs one less each. A page that nobody held, or a number out of range,
 * is reported and passed over.
 */
int lla_paged_free(const lla_paged_cache* cache, const int* keep, int* refs, void* stream);

/*
 * Makes room for the new tokens of `starts` (as in lla_paged_append, which may follow): lens[b] grows by
 * starts[b+1] - starts[b], and the table gets the pages for that, the lowest free ones first, in the order of
 * the sequences. Where the first new position falls into a page that others hold too, the lowest free page
 * takes that page's place in the table before any other, and copies[b] = (old page, new page) is to be made by
 * lla_paged_copy for each layer; elsewhere copies[b] = (-1, -1). Among sequences that share such a page and
 * all grow, the last keeps it if nobody else holds it. copies: [num_seqs][2], 8-byte aligned.
 * *left (device memory): free pages afterwards. Negative: nothing has changed but copies, which is all -1. So many
 * free pages were missing, or entries in the rows of sequences that would outgrow the table (the sum of both); lens
 * then does not count the new tokens, so they may not be appended: lla_paged_append would take them for the
 * last positions that are there. The same holds for the tokens of a sequence with copies[b] = (-2, -2), which an
 * impossible length, descending starts or starts for more positions than a row holds leave out, reported, while the others
 * grow. A last page out of range is reported and stays in the table.
 * At most 4096 sequences (LLA_ERR_UNSUPPORTED).
 */
int lla_paged_grow(const lla_paged_cache* cache, const int* starts, int* refs, int* copies, int* left, void* stream);

/*
 * Copies whole pages, keys, values and (where both caches have it) mass: page pairs[i][0] of `from` to page
 * pairs[i][1] of `to`, count pairs in device memory, 8-byte aligned; a pair with a negative number is skipped. The caches (which may be
 * one) agree in kv_heads, page_size, d, dv and type; tables and lens are not used. No page may be written
 * twice, or written and read, in one call. A page's keys, values and mass: at most 32 GB less 32 KB; all pairs: fewer than
 * 2^31 pieces of 32 KB (LLA_ERR_UNSUPPORTED).
 */
int lla_paged_copy(const lla_paged_cache* from, const lla_paged_cache* to, const int* pairs, int count, void* stream);

/*
 * Keeps one path of each drafted tree (or any selection of new tokens): path[b][0 ..] are the indices, rising, of the
 * kept ones among sequence b's new tokens, ended by -1 where there are fewer than max_path. Their keys,
 * values and mass move to the slots first, first + 1, .. (first = lens[b] - number of new tokens), and keep[b] =
 * first + their number is what lla_paged_free is then given, once all layers are done: lens and table stay as
 * they are here. A path that does not rise, leaves the new tokens or moves one from or to a page out of range is
 * reported and nothing of it kept. The
 * moved positions' pages must be the sequence's own (as after lla_paged_grow). tokens: of the batch, as in
 * lla_paged_append. keep is not the cache's lens.
 */
int lla_paged_compact(const lla_paged_cache* cache, const int* starts, int tokens, const int* path, int max_path, int* keep,
                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LLA_H */
