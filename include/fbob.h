/*
 * fbob.h - C ABI of the GB300 (sm_103a) exact attention backward-over-backward
 * library (libfbob.so).
 *
 * The library computes, for softmax attention with scale tau,
 *   forward        O = softmax(tau Q K^T) V,  L = row logsumexp (natural log)
 *   first backward g(Q, K, V, dO) = (dQ, dK, dV) and D = rowsum(dO o O)
 *   BoB            J_g^T applied to (UQ, UK, UV) at (dQ, dK, dV), i.e. the
 *                  gradients gQ, gK, gV, gdO of
 *                  f = <UQ, dQ> + <UK, dK> + <UV, dV>
 *                  with respect to Q, K, V, dO.
 * Sources: "FlashBoB: I/O-Efficient Exact Backward-over-Backward for Softmax
 * Attention" - the abstract (aiqbench.com / arxivdaily.com pages) for the
 * forward / first backward / BoB chain, and the evolve.pub review: "Scope &
 * Claims" (BoB = J_g^T at (dQ, dK, dV), paper section 4.1), Summary and Key
 * claims (two-pass schedule, the row scalars alpha and E are the only length-N
 * vectors that cross the pass boundary, no N x N tensor in HBM; paper
 * Prop. 4.1 and Algorithm 1), FAQ "Is FlashBoB an approximation?" (exact
 * outputs, bf16 inputs with fp32 accumulation).
 *
 * Conventions shared by every call
 * --------------------------------
 * - All tensor arguments are DEVICE pointers owned by the caller.  The library
 *   never allocates device memory, frees or synchronises inside these calls;
 *   every launch is ordered on `stream` (fbob_attn_bwd and fbob_attn_bob may
 *   fork part of their work onto a stream of their own and join it back, see
 *   fbob_attn_bob) and the call
 *   returns before the GPU finishes.
 *   Outputs are overwritten, never accumulated into.
 * - Matrices are [B, H, N, d] row-major and contiguous (element (b, h, i, c)
 *   at ((b*H + h)*N + i)*d + c); row vectors (L, D) are [B, H, N]; the BoB
 *   workspace is [B, H, N, 2] floats (alpha, E interleaved per row).
 * - Inputs Q, K, V, dO, UQ, UK, UV have the element type `dtype` of the
 *   problem (bf16 or fp32); O, L, D, all gradients and the workspace are
 *   fp32.
 * - Every pointer must be 16-byte aligned and tensors must not overlap an
 *   output of the same call.
 * - Supported: d in {32, 64, 96, 128}; any N >= 1 (bf16 and fp32); causal or
 *   not.  (bf16 heads of 32 and 96 run on the 64- and 128-column tensor-core
 *   kernels with the missing columns zero-padded on chip.)
 *   B*H*N == 0 is a valid empty problem
 *   (returns FBOB_OK, launches nothing).
 * - Argument problems are reported BEFORE any launch (nothing is launched on
 *   error).  A failed launch returns FBOB_ERR_CUDA.  Kernels never trap: a
 *   device-side wait that exceeds its time limit makes the kernel give up and
 *   record FBOB_ERR_TIMEOUT in a device status word, read with
 *   fbob_device_status().
 * - No C++ exception crosses this interface.  Functions are thread-safe;
 *   fbob_last_error() is per host thread.
 */
#ifndef FBOB_H_
#define FBOB_H_

#include <stddef.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FBOB_ABI_VERSION 1

typedef enum {
  FBOB_OK = 0,
  FBOB_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad sizes or tau    */
  FBOB_ERR_UNSUPPORTED = 2,   /* valid problem outside the supported set      */
  FBOB_ERR_WORKSPACE = 3,     /* workspace pointer null or too small          */
  FBOB_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed         */
  FBOB_ERR_TIMEOUT = 5        /* a device-side wait ran out (device status)   */
} fbob_status;

typedef enum {
  FBOB_BF16 = 0,              /* inputs are IEEE bfloat16                     */
  FBOB_FP32 = 1               /* inputs are IEEE binary32                     */
} fbob_dtype;

/* One attention problem: B batches x H heads of N x d matrices. */
typedef struct {
  int B, H, N, d;
  float tau;                  /* score scale, S = tau Q K^T; finite, nonzero  */
  int dtype;                  /* fbob_dtype of Q, K, V, dO, UQ, UK, UV        */
  int causal;                 /* 0: full attention; nonzero: causal, query i  */
                              /* attends to keys j <= i                       */
} fbob_problem;

/*
 * Forward (FlashBoB abstract: FlashAttention-style forward).
 *   in : Q, K, V  [B,H,N,d] dtype
 *   out: O [B,H,N,d] fp32, L [B,H,N] fp32 (natural-log row logsumexp of
 *        tau Q K^T)
 */
fbob_status fbob_attn_fwd(const fbob_problem* p,
                          const void* Q, const void* K, const void* V,
                          float* O, float* L, cudaStream_t stream);

/*
 * First backward g (FlashBoB abstract; evolve.pub review FAQ "What is
 * backward-over-backward"):
 *   dV = P^T dO, dP = dO V^T, D = rowsum(dO o O), dS = P o (dP - D),
 *   dQ = tau dS K, dK = tau dS^T Q, with P = exp(tau Q K^T - L).
 *   in : Q, K, V, dO [B,H,N,d] dtype; O [B,H,N,d] fp32 and L [B,H,N] fp32
 *        from fbob_attn_fwd on the same Q, K, V
 *   out: dQ, dK, dV [B,H,N,d] fp32; D [B,H,N] fp32
 * Streams: like fbob_attn_bob (bf16), the heads may run as two groups, the
 * second on the library's forked stream; ordered on `stream` as one call.
 */
fbob_status fbob_attn_bwd(const fbob_problem* p,
                          const void* Q, const void* K, const void* V,
                          const float* O, const void* dO, const float* L,
                          float* dQ, float* dK, float* dV, float* D,
                          cudaStream_t stream);

/* Bytes of BoB workspace: 2 * B * H * N * sizeof(float) (alpha and E). */
size_t fbob_bob_workspace_bytes(const fbob_problem* p);

/*
 * Backward over backward (evolve.pub review, "Scope & Claims", Summary, Key
 * claims; paper section 4.1, Prop. 4.1, Algorithm 1).  Two passes on
 * `stream`:
 *   pass 1, per block of query rows, loops over all key tiles, reduces the
 *     row scalars alpha_i = sum_j P_ij B_ij and
 *     E_i = sum_j P_ij (C_ij + B_ij dP_ij)   (B = tau (UQ K^T + Q UK^T),
 *     C = dO UV^T) while accumulating alpha-free sums, applies the affine
 *     correction at the row end and writes gQ, gdO and (alpha, E);
 *   pass 2, per block of keys, loops over all query tiles and writes gK, gV.
 *   Only alpha and E (the workspace) cross between the passes; no N x N
 *   matrix is ever stored.
 *   in : Q, K, V, dO, UQ, UK, UV [B,H,N,d] dtype; O [B,H,N,d] fp32 and
 *        L [B,H,N] fp32 from fbob_attn_fwd; D [B,H,N] fp32 from fbob_attn_bwd
 *   out: gQ, gK, gV, gdO [B,H,N,d] fp32;
 *        workspace [B,H,N,2] fp32 = (alpha_i, E_i) per row, at least
 *        fbob_bob_workspace_bytes(p) bytes (FBOB_ERR_WORKSPACE otherwise)
 * Streams (bf16 inputs): when B*H >= 2 and each pass would end on a mostly
 * empty wave of thread blocks, the heads run as two groups, the second on a
 * library-owned stream forked from `stream` (it waits for the work already
 * queued there) and joined back (`stream` waits for it before any later
 * work).  Seen from `stream`, the call is ordered exactly as one launch
 * sequence; results do not depend on the grouping.  The first such call in
 * a CUDA context creates that stream and two events (kept until the process
 * exits); make it before any stream capture, like the first
 * fbob_attn_bob_noalloc call.
 */
fbob_status fbob_attn_bob(const fbob_problem* p,
                          const void* Q, const void* K, const void* V,
                          const float* O, const void* dO,
                          const float* L, const float* D,
                          const void* UQ, const void* UK, const void* UV,
                          float* gQ, float* gK, float* gV, float* gdO,
                          float* workspace, size_t workspace_bytes,
                          cudaStream_t stream);

/*
 * BoB on the four-pass schedule, an ablation of the two-pass fbob_attn_bob
 * ("FlashBoB", evolve.pub review - Strengths: the hierarchical affine
 * structure collapses a natural four-pass schedule to two).  The pages name
 * the four-pass schedule without spelling it out; this library's reading is
 * the order plain reverse mode imposes when the row scalars are not split
 * off affinely:
 *   1. row sweep: alpha_i = sum_j P tau B;
 *   2. row sweep: E in its natural form, which uses alpha (the cotangent of
 *      P carries - alpha dP from D = rowsum(dO o O));
 *   3. row sweep: gQ and gdO accumulated directly, alpha and E known;
 *   4. column pass: gK, gV (the same kernel as fbob_attn_bob's pass 2).
 * Same arguments, outputs (identical up to rounding order), workspace and
 * errors as fbob_attn_bob; bf16 inputs only (fp32 returns
 * FBOB_ERR_UNSUPPORTED).  It runs 25 GEMMs of 2 N^2 d per head against the
 * two-pass schedule's 19 counted (20 executed).
 */
fbob_status fbob_attn_bob_four_pass(const fbob_problem* p,
                                    const void* Q, const void* K, const void* V,
                                    const float* O, const void* dO,
                                    const float* L, const float* D,
                                    const void* UQ, const void* UK, const void* UV,
                                    float* gQ, float* gK, float* gV, float* gdO,
                                    float* workspace, size_t workspace_bytes,
                                    cudaStream_t stream);

/*
 * BoB without a caller workspace (the paper has no counterpart; this is a
 * convenience of this library).  Same inputs, outputs, passes and errors as
 * fbob_attn_bob, but the (alpha, E) workspace is a fixed device array inside
 * the library, so the caller passes only inputs and outputs and nothing is
 * allocated.  It serves callers that cannot obtain an extra device buffer:
 * hosts that hand over only their own tensors, or loops that must not call
 * cudaMalloc/cudaFree (they can synchronise the device).
 *   - Capacity: B*H*N <= 2097152 (2^21) query rows; larger problems return
 *     FBOB_ERR_UNSUPPORTED before any launch.  Every GPU that loads the
 *     library holds the array (16 MiB) until the process exits.
 *   - The array's device address belongs to the CUDA context the library's
 *     device code is loaded into.  The first call in a context (per device:
 *     its primary context, a non-primary context the caller made current, or
 *     the new context after cudaDeviceReset) looks the address up with that
 *     device current (cudaGetSymbolAddress, which may load the library's
 *     device code) and saves it for later calls in the same context; make
 *     that first call - on every device, and again after a cudaDeviceReset -
 *     before any stream capture.
 *   - All calls on a device share the array: calls whose kernels overlap on
 *     the GPU (e.g. on two unordered streams) race and give wrong results.
 *     Calls ordered on one stream are safe; no clearing is needed between
 *     them (pass 1 rewrites every element pass 2 reads).
 */
fbob_status fbob_attn_bob_noalloc(const fbob_problem* p,
                                  const void* Q, const void* K, const void* V,
                                  const float* O, const void* dO,
                                  const float* L, const float* D,
                                  const void* UQ, const void* UK, const void* UV,
                                  float* gQ, float* gK, float* gV, float* gdO,
                                  cudaStream_t stream);

/* ------------------------------------------------------------------------
 * The operators of a model around the attention.  Each has its forward, its
 * first backward and the vector-Jacobian product of that backward, so that a
 * Hessian-vector product passes through a whole model.  The pages have no
 * counterpart: the formulas stand at each call.
 *
 * Differences from the conventions above: tensors and gradients have the
 * descriptor's element types (row statistics, losses and workspaces are
 * fp32); a pointer needs the alignment of its elements only, unless a call
 * says otherwise (workspaces: 16 bytes), and rows that all start on 16 bytes
 * are read faster; an output that is marked optional is not computed when its
 * pointer is null.
 * ------------------------------------------------------------------------ */

/* Scaling of the rotary frequencies theta_i = base^(-2 i / rot). */
typedef enum {
  FBOB_ROTARY_NONE = 0,
  FBOB_ROTARY_LINEAR = 1,  /* theta / factor                                  */
  FBOB_ROTARY_BASE = 2,    /* base * factor^(rot / (rot - 2)) as the base     */
  FBOB_ROTARY_PARTS = 3    /* theta (w + (1 - w) / factor) with the turns     */
                           /* n = original theta / 2 pi and                   */
                           /* w = (n - slow) / (fast - slow) clamped to [0,1] */
} fbob_rotary_scaling;

typedef struct {
  int rot;          /* leading columns of a head that are rotated: even, 2..d */
  int interleaved;  /* 0: pairs (i, i + rot/2); else pairs (2i, 2i + 1)       */
  int scaling;      /* fbob_rotary_scaling                                    */
  double base;      /* > 1                                                    */
  double factor;    /* >= 1 (all scalings but NONE)                           */
  double original, slow, fast;  /* PARTS only: > 0 and 0 <= slow < fast       */
  double magnitude; /* multiplies the rotated columns; finite, nonzero        */
} fbob_rotary;

/* Heads of one tensor: x and y are [B, H, N, d] with element strides of
 * batch, head and position (not negative) and contiguous rows of d. */
typedef struct {
  const void* x;
  void* y;
  int H;
  long long x_stride[3], y_stride[3];
} fbob_rotary_heads;

/* theta_i, i < rot/2, into host memory. */
fbob_status fbob_rotary_frequencies(const fbob_rotary* r, double* theta);

/*
 * Rotary positions on one or two tensors (Q, K) in one launch:
 *   (y_a, y_b) = magnitude * (x_a cos - x_b sin, x_a sin + x_b cos) for each
 *   pair (a, b) = pair i and angle position * theta_i; columns from rot on
 *   are copied.  transpose != 0 turns the other way: the map's transpose, so
 *   the gradient of x from that of y (its own second order is the map again).
 *   positions: null (position of token n is offset + n) or integers of
 *   position_bytes (4 or 8), read at [b * position_stride + n] and added to
 *   offset (position_stride 0: shared by the batches); any sign.
 *   d <= 256.  Angles are reduced by whole turns exactly, whatever the
 *   position; what is left is theta's own rounding to 64 bits, position *
 *   2^-52 radians at most (5e-7 at 2^31, 2e-4 at 2^40).
 *   An output whose elements share addresses is refused.
 */
fbob_status fbob_rotary_apply(const fbob_rotary* r, int B, int N, int d, int dtype,
                              const fbob_rotary_heads* tensors, int count,
                              const void* positions, int position_bytes,
                              long long position_stride, long long offset,
                              int transpose, cudaStream_t stream);

/* Rows of D elements (1 <= D <= 16384), contiguous. */
typedef struct {
  long long rows;
  int D;
  int dtype;         /* x, y, dy, dx, ux, gx, gdy                             */
  int weight_dtype;  /* w, b, dw, db, uw, ub, gw: fp32, or bf16 with bf16 rows */
  float eps;         /* >= 0; the forward's only                              */
} fbob_norm;

/* Bytes of fp32 workspace of fbob_layer_norm_bwd with dw and db; half of it
 * serves one of them, or fbob_layer_norm_bob. */
size_t fbob_layer_norm_workspace_bytes(const fbob_norm* p);

/*
 * Layer norm: y = w xh + b, xh = (x - mean) rstd,
 * rstd = (mean((x - mean)^2) + eps)^(-1/2) over each row of D.
 * w and b are optional (null: ones, zeros).
 *   out: y [rows, D]; mean, rstd [rows] fp32
 */
fbob_status fbob_layer_norm_fwd(const fbob_norm* p, const void* x, const void* w, const void* b,
                                void* y, float* mean, float* rstd, cudaStream_t stream);

/*
 * Its backward: with a = w dy and m() the mean over a row,
 *   dx = rstd (a - m(a) - xh m(a xh)), dw = sum over rows of dy xh,
 *   db = sum over rows of dy; each optional.  dw and db are zero for no rows.
 * The sums over rows are taken in an order fixed by the sizes.
 */
fbob_status fbob_layer_norm_bwd(const fbob_norm* p, const void* x, const void* w,
                                const float* mean, const float* rstd, const void* dy,
                                void* dx, void* dw, void* db,
                                float* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * The vector-Jacobian product of (x, w, dy) -> (dx, dw, db) along
 * (ux, uw, ub): gradients of <ux, dx> + <uw, dw> + <ub, db>.  uw and ub are
 * optional (null: zeros).  With pu = ux - m(ux) - xh m(ux xh):
 *   gdy = rstd w pu + uw xh + ub;  gw = sum over rows of rstd pu dy;
 *   gx  = rstd (h - m(h) - xh m(h xh)) - rstd^2 xh m(pu a),
 *   h   = uw dy - rstd (a m(ux xh) + ux m(a xh));
 * each optional.
 */
fbob_status fbob_layer_norm_bob(const fbob_norm* p, const void* x, const void* w,
                                const float* mean, const float* rstd, const void* dy,
                                const void* ux, const void* uw, const void* ub,
                                void* gx, void* gw, void* gdy,
                                float* workspace, size_t workspace_bytes, cudaStream_t stream);

/* The cross entropy of a linear head: T tokens h of D columns, V classes. */
typedef struct {
  int T, D, V;             /* up to 2^24, 2^15, 2^24, and T V up to 2^45      */
  int dtype;               /* H, W, UH, UW and their gradients                */
  long long ignore_index;  /* target of the tokens that are not counted       */
  int piece;               /* classes whose gradient is held at once (rounded */
                           /* up to 256); 0: as many as 512 MiB hold, but at  */
                           /* least 2048, which take T x 4 KiB in bf16, T x   */
                           /* 12 KiB in fp32 and twice that in the second     */
                           /* order: above 512 MiB from 131,072 tokens (bf16, */
                           /* first order) on                                 */
} fbob_linear_ce;

/* Bytes of workspace of pass 0 (fwd), 1 (bwd) or 2 (bob); 0 for no tokens or
 * a descriptor that the calls refuse. */
size_t fbob_linear_ce_workspace_bytes(const fbob_linear_ce* p, int pass);

/*
 * Losses of the tokens under logits z = h W^T, which are never stored:
 *   lse_t = log sum_v exp z_tv, loss_t = lse_t - z_t,target; both 0 where
 *   target_t == ignore_index.  A target outside [0, V) that is not
 *   ignore_index makes loss_t NaN, counts as ignored in every gradient and is
 *   reported by fbob_device_status as FBOB_ERR_INVALID_ARG.
 *   in : H [T, D], W [V, D] (W 16-byte aligned when bf16 with D a multiple
 *        of 8), target [T] 64-bit
 *   out: loss, lse [T] fp32
 * Tokens that are not counted are never read into a sum, whatever H holds
 * there.  fp32 inputs are multiplied as three bf16 terms each and lose
 * nothing to about 2^-22.
 */
fbob_status fbob_linear_ce_fwd(const fbob_linear_ce* p, const void* H, const void* W,
                               const long long* target, float* loss, float* lse,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Gradients of sum_t g_t loss_t: with p = exp(z - lse) and
 * G = g (p - onehot(target)),
 *   dH = G W, dW = G^T H; each optional.  G is formed for one piece of the
 *   classes at a time, in bf16 for bf16 inputs (in two bf16 terms where up to
 *   16 tokens are counted, whatever T is).
 *   in : as fbob_linear_ce_fwd, its lse, and g [T] fp32
 */
fbob_status fbob_linear_ce_bwd(const fbob_linear_ce* p, const void* H, const void* W,
                               const long long* target, const float* lse, const float* g,
                               void* dH, void* dW, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/*
 * The vector-Jacobian product of (H, W, g) -> (dH, dW) along (UH, UW):
 * gradients of <UH, dH> + <UW, dW>.  With b = UH W^T + H UW^T,
 * alpha_t = sum_v p b and Z = g p (b - alpha),
 *   gH = Z W + G UW, gW = Z^T H + G^T UH, gg_t = alpha_t - b_t,target;
 * each optional; one of UH, UW may be null (zeros).
 */
fbob_status fbob_linear_ce_bob(const fbob_linear_ce* p, const void* H, const void* W,
                               const long long* target, const float* lse, const float* g,
                               const void* UH, const void* UW, void* gH, void* gW, float* gg,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Dropout: round(65536 p) of 65,536 elements are dropped (set to 0, whatever
 * they were), the others multiplied by m = 65536 / (65536 - that).  The element at
 * (row, column) is dropped by sixteen bits of a counter-based generator, so no
 * mask is stored and gradients draw the same one again: half column % 2 (low
 * first) of word column / 2 % 4 of Philox4x32 in ten rounds (Salmon, Moraes,
 * Dror, Shaw: Parallel Random Numbers: As Easy as 1, 2, 3, 2011) with key = seed
 * and counter words (column / 8, row, low and high half of the offset), being
 * below round(65536 p).  Calls with different offsets have independent masks. */
typedef struct {
  double p;                         /* 0 <= p <= 1                             */
  unsigned long long seed, offset;
} fbob_dropout;

/*
 * y = r + m x for rows of D elements, contiguous; r optional.  The map of x is
 * linear and its own transpose: the gradient of x is the same call on y's, that
 * of r is y's itself.
 *   counter: null, or a 64-bit integer on the device that is added to the
 *   offset modulo 2^64 when the call runs (a captured graph's steps advance it)
 *   rows < 2^32, D <= 2^30, rows D <= 2^40
 */
fbob_status fbob_dropout_apply(const fbob_dropout* d, const long long* counter,
                               long long rows, int D, int dtype, const void* x, const void* r,
                               void* y, cudaStream_t stream);

typedef enum {
  FBOB_ACT_NONE = 0,
  FBOB_ACT_RELU = 1,      /* max(z, 0); slope 0 at 0                          */
  FBOB_ACT_GELU = 2,      /* z F(z), F the normal distribution's integral     */
  FBOB_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2  */
  FBOB_ACT_SILU = 4       /* z / (1 + exp(-z))                                */
} fbob_activation;

/* A linear layer: T tokens of K columns, N outputs. */
typedef struct {
  int T, K, N;     /* up to 2^24, 2^20, 2^20; T K, T N and N K up to 2^40     */
  int dtype;       /* of every tensor but z: fp32, or fp16 beside bf16        */
  int activation;  /* fbob_activation                                         */
} fbob_linear;

/* Bytes of workspace of pass 0 (fwd), 1 (bwd) or 2 (bob); 0 if none is needed
 * or the calls refuse the descriptors.  dropout may be null. */
size_t fbob_linear_workspace_bytes(const fbob_linear* p, const fbob_dropout* dropout, int pass);

/*
 * y = r + m a(z), z = x W^T + b, with a the activation and m the dropout (null:
 * none) of element (token, output); counter as in fbob_dropout_apply.
 *   in : x [T, K], W [N, K]; b [N], r [T, N] optional
 *   out: y [T, N]; z [T, N] optional, which the calls below want unless the
 *        activation is NONE, where it is left as it was (fp16 beside bf16 tensors: clamped to
 *        its range, above which no slope changes; for RELU a positive value is kept as 2^-24 at
 *        least, so that its slope stays 1)
 * bf16 matrices whose rows are multiples of 16 bytes have to start on 16 bytes
 * where they are multiplied (x, W, dy, ux, uW).  Sums are fp32; fp32 inputs are
 * multiplied as three bf16 terms each and lose nothing to about 2^-22.  x W^T of few
 * tokens (one; up to 16 of fp32 or narrow layers) is summed outside the tensor cores.
 */
fbob_status fbob_linear_fwd(const fbob_linear* p, const fbob_dropout* dropout, const long long* counter,
                            const void* x, const void* W, const void* b, const void* r,
                            void* y, void* z, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/*
 * Gradients: with dz = m dy a'(z),
 *   dx = dz W, dW = dz^T x, db = sum over tokens of dz; each optional (that of
 *   r is dy).  dz is formed once, in bf16 for bf16 inputs (in two bf16 terms for
 *   up to 16 tokens); dW and db are zero for no tokens.
 */
fbob_status fbob_linear_bwd(const fbob_linear* p, const fbob_dropout* dropout, const long long* counter,
                            const void* x, const void* W, const void* z, const void* dy,
                            void* dx, void* dW, void* db, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/*
 * The vector-Jacobian product of (x, W, b, dy) -> (dx, dW, db) along
 * (ux, uW, ub): gradients of <ux, dx> + <uW, dW> + <ub, db>.  With
 * t = ux W^T + x uW^T + ub and q = m t dy a''(z),
 *   gdy = m t a'(z), gx = q W + dz uW, gW = q^T x + dz^T ux,
 *   gb = sum over tokens of q; each optional.  One of ux, uW may be null, ub too
 *   (zeros).  q is held as dz is.
 */
fbob_status fbob_linear_bob(const fbob_linear* p, const fbob_dropout* dropout, const long long* counter,
                            const void* x, const void* W, const void* z, const void* dy,
                            const void* ux, const void* uW, const void* ub,
                            void* gx, void* gW, void* gb, void* gdy,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Device status: waits for `stream` to finish (this call DOES synchronise),
 * then returns FBOB_ERR_TIMEOUT if any kernel of this library on the current
 * device gave up on a bounded wait since the last call, FBOB_ERR_INVALID_ARG
 * if fbob_linear_ce_* met a target outside its classes, else FBOB_OK (or
 * FBOB_ERR_CUDA if the synchronisation itself failed).  Clears the word.
 */
fbob_status fbob_device_status(cudaStream_t stream);

/*
 * Time limit, in nanoseconds, of every device-side wait of later launches
 * (default 2e9 = 2 s; 0 restores the default).  Meant for tests of the
 * give-up path; returns the previous limit.
 */
unsigned long long fbob_set_wait_limit_ns(unsigned long long ns);

/*
 * Per-kernel timing (measurement aid, off by default).  While enabled, every
 * kernel launch of the library is bracketed by two CUDA events recorded on
 * its stream.  fbob_profile_report waits for the recorded launches, adds
 * them to per-kernel totals and returns the length of the text
 * {"kernel": [launches, total_ms, min_ms, max_ms], ...}; if buf can hold the
 * whole text (len > length) it writes it NUL-terminated and clears the
 * totals, otherwise (e.g. buf == NULL) the totals are kept.
 * fbob_profile_enable returns the previous setting.
 */
int fbob_profile_enable(int on);
int fbob_profile_report(char* buf, size_t len);

/*
 * Test hook for the give-up path (off by default).  With stall = 1 the TMA
 * producer of every tensor-core kernel launched afterwards withholds its
 * first streamed tile, so the consumers' bounded waits run out: the kernels
 * give up, free their resources and return, and fbob_device_status reports
 * FBOB_ERR_TIMEOUT.  Returns the previous setting.
 */
int fbob_debug_stall_producer(int stall);

/* Static text for a status code. */
const char* fbob_status_string(fbob_status s);

/* Detail text of the last non-OK status returned on this host thread. */
const char* fbob_last_error(void);

/* FBOB_ABI_VERSION of the loaded library. */
int fbob_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FBOB_H_ */
