// C ABI of libfbob.so: the operators around the attention (rotary positions,
// layer norm, the linear head's cross entropy).  Argument validation and dispatch, as in api.cpp.
#include <cuda_runtime_api.h>
#include <math.h>
#include <string.h>

#include "api_check.h"
#include "fbob.h"
#include "internal.h"

namespace {

using fbob::aligned16;
using fbob::cuda_fail;
using fbob::fail;

fbob_status check_dtype(int dtype) {
  if (dtype != FBOB_BF16 && dtype != FBOB_FP32) return fail(FBOB_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  return FBOB_OK;
}

bool element_aligned(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == FBOB_BF16 ? 1u : 3u)) == 0;
}

fbob_status check_rotary(const fbob_rotary* r) {
  if (!r) return fail(FBOB_ERR_INVALID_ARG, "rotary descriptor is null");
  if (r->rot < 2 || r->rot % 2 != 0)
    return fail(FBOB_ERR_INVALID_ARG, "rot=%d must be an even number of columns, at least 2", r->rot);
  if (r->rot / 2 > fbob::kRotaryMaxPairs)
    return fail(FBOB_ERR_UNSUPPORTED, "rot=%d exceeds %d columns", r->rot, 2 * fbob::kRotaryMaxPairs);
  if (!isfinite(r->base) || r->base <= 1.0) return fail(FBOB_ERR_INVALID_ARG, "base must be above 1 (got %g)", r->base);
  if (!isfinite(r->magnitude) || r->magnitude == 0.0)
    return fail(FBOB_ERR_INVALID_ARG, "magnitude must be finite and nonzero (got %g)", r->magnitude);
  if (r->scaling < FBOB_ROTARY_NONE || r->scaling > FBOB_ROTARY_PARTS)
    return fail(FBOB_ERR_INVALID_ARG, "unknown scaling %d", r->scaling);
  if (r->scaling == FBOB_ROTARY_NONE) return FBOB_OK;
  if (!isfinite(r->factor) || r->factor < 1.0)
    return fail(FBOB_ERR_INVALID_ARG, "factor must be at least 1 (got %g)", r->factor);
  if (r->scaling == FBOB_ROTARY_BASE && r->rot == 2)
    return fail(FBOB_ERR_INVALID_ARG, "scaling the base needs rot above 2");
  if (r->scaling == FBOB_ROTARY_PARTS) {
    if (!isfinite(r->original) || r->original <= 0.0)
      return fail(FBOB_ERR_INVALID_ARG, "original length must be positive (got %g)", r->original);
    if (!isfinite(r->slow) || !isfinite(r->fast) || r->slow < 0.0 || r->fast <= r->slow)
      return fail(FBOB_ERR_INVALID_ARG, "0 <= slow < fast is needed (got %g, %g)", r->slow, r->fast);
  }
  return FBOB_OK;
}

// theta_i of a checked descriptor.
double theta(const fbob_rotary* r, int i) {
  double base = r->base;
  if (r->scaling == FBOB_ROTARY_BASE) base *= pow(r->factor, (double)r->rot / (r->rot - 2));
  double t = pow(base, -2.0 * i / r->rot);
  if (r->scaling == FBOB_ROTARY_LINEAR) t /= r->factor;
  if (r->scaling == FBOB_ROTARY_PARTS) {
    const double n = r->original * t / (2.0 * M_PI);
    const double w = fmin(fmax((n - r->slow) / (r->fast - r->slow), 0.0), 1.0);
    t *= w + (1.0 - w) / r->factor;
  }
  return t;
}

// Frequencies as 64-bit fractions of a turn.  The last description's are kept
// per host thread (a model rotates with one description; the powers would
// cost more than the launch).
const unsigned long long* fixed_frequencies(const fbob_rotary* r) {
  thread_local fbob_rotary last = {};
  thread_local unsigned long long freq[fbob::kRotaryMaxPairs];
  const bool same = last.rot == r->rot && last.scaling == r->scaling && last.base == r->base &&
                    last.factor == r->factor && last.original == r->original && last.slow == r->slow &&
                    last.fast == r->fast;
  if (!same) {
    for (int i = 0; i < r->rot / 2; ++i)  // a turn's fraction is below 2^-2, since theta <= 1
      freq[i] = (unsigned long long)ldexp(theta(r, i) / (2.0 * M_PI), 64);
    last = *r;
  }
  return freq;
}

// Whether no two elements of [B, H, N, d] with these strides (last one 1)
// share an address: each stride, from the smallest, steps over all that the
// smaller ones reach.
bool distinct(const long long* st, int B, int H, int N, int d) {
  const long long size[3] = {B, H, N};
  bool used[3] = {false, false, false};
  long long reach = d;  // elements spanned so far
  for (int k = 0; k < 3; ++k) {
    int best = -1;
    for (int i = 0; i < 3; ++i) {
      if (!used[i] && (best < 0 || (size[i] > 1 ? st[i] : -1) < (size[best] > 1 ? st[best] : -1))) best = i;
    }
    used[best] = true;
    if (size[best] <= 1) continue;
    if (st[best] < reach) return false;
    reach += (size[best] - 1) * st[best];
  }
  return true;
}

fbob_status check_norm(const fbob_norm* p) {
  if (!p) return fail(FBOB_ERR_INVALID_ARG, "norm descriptor is null");
  fbob_status st = check_dtype(p->dtype);
  if (st != FBOB_OK || (st = check_dtype(p->weight_dtype)) != FBOB_OK) return st;
  if (p->rows < 0 || p->D <= 0) return fail(FBOB_ERR_INVALID_ARG, "bad sizes rows=%lld D=%d", p->rows, p->D);
  if (p->D > 16384) return fail(FBOB_ERR_UNSUPPORTED, "D=%d exceeds 16384 columns", p->D);
  if (p->rows > (1ll << 40) / p->D) return fail(FBOB_ERR_UNSUPPORTED, "%lld rows of %d are too large", p->rows, p->D);
  if (!isfinite(p->eps) || p->eps < 0.f) return fail(FBOB_ERR_INVALID_ARG, "eps must be >= 0 (got %g)", (double)p->eps);
  if (p->dtype == FBOB_FP32 && p->weight_dtype == FBOB_BF16)
    return fail(FBOB_ERR_UNSUPPORTED, "fp32 rows with bf16 weights");
  return FBOB_OK;
}

struct Arg {
  const void* p;
  const char* name;
  int dtype;
  bool required;
};

fbob_status check_args(const Arg* a, int n) {
  for (int i = 0; i < n; ++i) {
    if (!a[i].p && a[i].required) return fail(FBOB_ERR_INVALID_ARG, "pointer %s is null", a[i].name);
    if (!element_aligned(a[i].p, a[i].dtype))
      return fail(FBOB_ERR_INVALID_ARG, "pointer %s is not aligned to its elements", a[i].name);
  }
  return FBOB_OK;
}

fbob_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return FBOB_OK;
  if (!ws) return fail(FBOB_ERR_WORKSPACE, "workspace pointer is null");
  if (!aligned16(ws)) return fail(FBOB_ERR_WORKSPACE, "workspace is not 16-byte aligned");
  if (have < need) return fail(FBOB_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", have, need);
  return FBOB_OK;
}

fbob::NormArgs norm_args(const fbob_norm* p) {
  fbob::NormArgs a;
  memset(&a, 0, sizeof(a));
  a.rows = p->rows, a.D = p->D, a.eps = p->eps;
  a.bf16 = p->dtype == FBOB_BF16, a.wbf16 = p->weight_dtype == FBOB_BF16;
  return a;
}

// Column sums over no rows are zero.
fbob_status zero_columns(const fbob_norm* p, void* const* outs, int n, cudaStream_t stream) {
  const size_t bytes = (size_t)p->D * (p->weight_dtype == FBOB_BF16 ? 2 : 4);
  for (int i = 0; i < n; ++i) {
    if (!outs[i]) continue;
    const cudaError_t e = cudaMemsetAsync(outs[i], 0, bytes, stream);
    if (e != cudaSuccess) return cuda_fail(e, "layer_norm memset");
  }
  return FBOB_OK;
}

fbob_status check_ce(const fbob_linear_ce* p) {
  if (!p) return fail(FBOB_ERR_INVALID_ARG, "linear_ce descriptor is null");
  const fbob_status st = check_dtype(p->dtype);
  if (st != FBOB_OK) return st;
  if (p->T < 0 || p->D <= 0 || p->V <= 0)
    return fail(FBOB_ERR_INVALID_ARG, "bad sizes T=%d D=%d V=%d", p->T, p->D, p->V);
  if (p->piece < 0) return fail(FBOB_ERR_INVALID_ARG, "piece is negative (%d)", p->piece);
  if (p->T > (1 << 24) || p->D > (1 << 15) || p->V > (1 << 24))
    return fail(FBOB_ERR_UNSUPPORTED, "T=%d D=%d V=%d exceed 2^24, 2^15, 2^24", p->T, p->D, p->V);
  // fewer than 2^31 tiles of 256 x 128 logits
  if ((long long)p->D * (p->T > p->V ? p->T : p->V) > (1ll << 40) || (long long)p->T * p->V > (1ll << 45))
    return fail(FBOB_ERR_UNSUPPORTED, "T=%d D=%d V=%d are too large", p->T, p->D, p->V);
  return FBOB_OK;
}

fbob::CeArgs ce_args(const fbob_linear_ce* p) {
  fbob::CeArgs a;
  memset(&a, 0, sizeof(a));
  a.T = p->T, a.D = p->D, a.V = p->V, a.bf16 = p->dtype == FBOB_BF16, a.piece = p->piece, a.ignore = p->ignore_index;
  return a;
}

fbob_status ce_run(const fbob::CeArgs& a, fbob::CePass pass, size_t have, const char* where, cudaStream_t stream) {
  fbob_status st = check_workspace(a.ws, have, fbob::linear_ce_workspace(a, pass));
  if (st != FBOB_OK) return st;
  fbob::DevCtx c;
  if ((st = fbob::make_ctx(&c)) != FBOB_OK) return st;
  const cudaError_t e = fbob::linear_ce(a, pass, c, stream);
  if (e != cudaSuccess) return cuda_fail(e, where);
  return FBOB_OK;
}

// The head is read in place by 16-byte copies when it is bf16 and its rows
// are 16-byte multiples.
fbob_status check_head(const fbob_linear_ce* p, const void* W, const char* name) {
  if (p->dtype == FBOB_BF16 && p->D % 8 == 0 && !aligned16(W))
    return fail(FBOB_ERR_INVALID_ARG, "pointer %s is not 16-byte aligned", name);
  return FBOB_OK;
}

fbob_status check_targets(const void* target) {
  if ((reinterpret_cast<uintptr_t>(target) & 7u) != 0)
    return fail(FBOB_ERR_INVALID_ARG, "pointer target is not aligned to its elements");
  return FBOB_OK;
}

// With no tokens the head's gradient is zero.
fbob_status zero_head(const fbob_linear_ce* p, void* dW, cudaStream_t stream) {
  if (!dW) return FBOB_OK;
  const cudaError_t e =
      cudaMemsetAsync(dW, 0, (size_t)p->V * p->D * (p->dtype == FBOB_BF16 ? 2 : 4), stream);
  return e == cudaSuccess ? FBOB_OK : cuda_fail(e, "linear_ce memset");
}

}  // namespace

extern "C" {

fbob_status fbob_rotary_frequencies(const fbob_rotary* r, double* out) {
  const fbob_status st = check_rotary(r);
  if (st != FBOB_OK) return st;
  if (!out) return fail(FBOB_ERR_INVALID_ARG, "pointer theta is null");
  for (int i = 0; i < r->rot / 2; ++i) out[i] = theta(r, i);
  return FBOB_OK;
}

fbob_status fbob_rotary_apply(const fbob_rotary* r, int B, int N, int d, int dtype, const fbob_rotary_heads* t,
                              int count, const void* positions, int position_bytes, long long position_stride,
                              long long offset, int transpose, cudaStream_t stream) {
  fbob_status st = check_rotary(r);
  if (st != FBOB_OK || (st = check_dtype(dtype)) != FBOB_OK) return st;
  if (B < 0 || N < 0 || d <= 0) return fail(FBOB_ERR_INVALID_ARG, "bad sizes B=%d N=%d d=%d", B, N, d);
  if (d > 2 * fbob::kRotaryMaxPairs) return fail(FBOB_ERR_UNSUPPORTED, "head size d=%d exceeds %d", d, 2 * fbob::kRotaryMaxPairs);
  if (r->rot > d) return fail(FBOB_ERR_INVALID_ARG, "rot=%d exceeds the head size d=%d", r->rot, d);
  if ((long long)B * N > 0x7fffffffll) return fail(FBOB_ERR_UNSUPPORTED, "B*N=%lld exceeds 2^31 - 1", (long long)B * N);
  if (!t || count < 1 || count > 2) return fail(FBOB_ERR_INVALID_ARG, "one or two tensors are needed (got %d)", count);
  if (positions && position_bytes != 4 && position_bytes != 8)
    return fail(FBOB_ERR_INVALID_ARG, "positions of %d bytes (4 or 8)", position_bytes);
  if (positions && (reinterpret_cast<uintptr_t>(positions) % position_bytes) != 0)
    return fail(FBOB_ERR_INVALID_ARG, "pointer positions is not aligned to its elements");
  if (positions && position_stride < 0) return fail(FBOB_ERR_INVALID_ARG, "position_stride is negative");
  long long heads = 0;
  for (int k = 0; k < count; ++k) {
    if (t[k].H < 0) return fail(FBOB_ERR_INVALID_ARG, "bad size H=%d", t[k].H);
    heads += t[k].H;
    for (int i = 0; i < 3; ++i) {
      if (t[k].x_stride[i] < 0 || t[k].y_stride[i] < 0) return fail(FBOB_ERR_INVALID_ARG, "a stride is negative");
    }
  }
  if (heads > 65535) return fail(FBOB_ERR_UNSUPPORTED, "%lld heads exceed 65535", heads);
  if (heads == 0 || B == 0 || N == 0) return FBOB_OK;
  fbob::RotaryArgs a;
  memset(&a, 0, sizeof(a));
  for (int k = 0, m = 0; k < count; ++k) {
    if (t[k].H == 0) continue;
    const Arg ps[] = {{t[k].x, "x", dtype, true}, {t[k].y, "y", dtype, true}};
    if ((st = check_args(ps, 2)) != FBOB_OK) return st;
    if (!distinct(t[k].y_stride, B, t[k].H, N, d))
      return fail(FBOB_ERR_INVALID_ARG, "elements of output %d share addresses", k);
    fbob::RotarySide& o = a.side[m++];
    o.x = t[k].x, o.y = t[k].y, o.H = t[k].H;
    const int size[3] = {B, t[k].H, N};
    for (int i = 0; i < 3; ++i) {  // the stride of a dimension of one is never stepped
      o.xs[i] = size[i] > 1 ? t[k].x_stride[i] : 0;
      o.ys[i] = size[i] > 1 ? t[k].y_stride[i] : 0;
    }
  }
  memcpy(a.freq, fixed_frequencies(r), sizeof(unsigned long long) * (r->rot / 2));
  a.positions = positions, a.pos_bytes = position_bytes, a.pos_stride = position_stride, a.offset = offset;
  a.B = B, a.N = N, a.d = d, a.rot = r->rot;
  a.interleaved = r->interleaved != 0, a.transpose = transpose != 0, a.bf16 = dtype == FBOB_BF16;
  a.magnitude = (float)r->magnitude;
  const cudaError_t e = fbob::rotary(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "rotary launch");
  return FBOB_OK;
}

size_t fbob_layer_norm_workspace_bytes(const fbob_norm* p) {
  if (!p || p->rows <= 0 || p->D <= 0) return 0;
  return sizeof(float) * fbob::layer_norm_workspace_floats(p->rows, p->D);
}

fbob_status fbob_layer_norm_fwd(const fbob_norm* p, const void* x, const void* w, const void* b, void* y, float* mean,
                                float* rstd, cudaStream_t stream) {
  fbob_status st = check_norm(p);
  if (st != FBOB_OK) return st;
  if (p->rows == 0) return FBOB_OK;
  const Arg ps[] = {{x, "x", p->dtype, true},         {w, "w", p->weight_dtype, false},
                    {b, "b", p->weight_dtype, false}, {y, "y", p->dtype, true},
                    {mean, "mean", FBOB_FP32, true},  {rstd, "rstd", FBOB_FP32, true}};
  if ((st = check_args(ps, 6)) != FBOB_OK) return st;
  fbob::NormArgs a = norm_args(p);
  a.x = x, a.w = w, a.b = b, a.y = y, a.mean = mean, a.rstd = rstd;
  fbob::DevCtx c;
  if ((st = fbob::make_ctx(&c)) != FBOB_OK) return st;
  const cudaError_t e = fbob::layer_norm_fwd(a, c, stream);
  if (e != cudaSuccess) return cuda_fail(e, "layer_norm_fwd launch");
  return FBOB_OK;
}

fbob_status fbob_layer_norm_bwd(const fbob_norm* p, const void* x, const void* w, const float* mean, const float* rstd,
                                const void* dy, void* dx, void* dw, void* db, float* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
  fbob_status st = check_norm(p);
  if (st != FBOB_OK) return st;
  const Arg ps[] = {{x, "x", p->dtype, p->rows > 0},         {w, "w", p->weight_dtype, false},
                    {mean, "mean", FBOB_FP32, p->rows > 0},  {rstd, "rstd", FBOB_FP32, p->rows > 0},
                    {dy, "dy", p->dtype, p->rows > 0},       {dx, "dx", p->dtype, false},
                    {dw, "dw", p->weight_dtype, false},      {db, "db", p->weight_dtype, false}};
  if ((st = check_args(ps, 8)) != FBOB_OK) return st;
  if (p->rows == 0) {
    void* const outs[] = {dw, db};
    return zero_columns(p, outs, 2, stream);
  }
  if (!dx && !dw && !db) return FBOB_OK;
  const size_t need = (dw || db) ? fbob_layer_norm_workspace_bytes(p) / ((dw && db) ? 1 : 2) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != FBOB_OK) return st;
  fbob::NormArgs a = norm_args(p);
  a.x = x, a.w = w, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd), a.dy = dy;
  a.dx = dx, a.dw = dw, a.db = db, a.ws = workspace;
  fbob::DevCtx c;
  if ((st = fbob::make_ctx(&c)) != FBOB_OK) return st;
  const cudaError_t e = fbob::layer_norm_bwd(a, c, stream);
  if (e != cudaSuccess) return cuda_fail(e, "layer_norm_bwd launch");
  return FBOB_OK;
}

fbob_status fbob_layer_norm_bob(const fbob_norm* p, const void* x, const void* w, const float* mean, const float* rstd,
                                const void* dy, const void* ux, const void* uw, const void* ub, void* gx, void* gw,
                                void* gdy, float* workspace, size_t workspace_bytes, cudaStream_t stream) {
  fbob_status st = check_norm(p);
  if (st != FBOB_OK) return st;
  const Arg ps[] = {{x, "x", p->dtype, p->rows > 0},        {w, "w", p->weight_dtype, false},
                    {mean, "mean", FBOB_FP32, p->rows > 0}, {rstd, "rstd", FBOB_FP32, p->rows > 0},
                    {dy, "dy", p->dtype, p->rows > 0},      {ux, "ux", p->dtype, p->rows > 0},
                    {uw, "uw", p->weight_dtype, false},     {ub, "ub", p->weight_dtype, false},
                    {gx, "gx", p->dtype, false},            {gw, "gw", p->weight_dtype, false},
                    {gdy, "gdy", p->dtype, false}};
  if ((st = check_args(ps, 11)) != FBOB_OK) return st;
  if (p->rows == 0) return zero_columns(p, &gw, 1, stream);
  if (!gx && !gw && !gdy) return FBOB_OK;
  const size_t need = gw ? fbob_layer_norm_workspace_bytes(p) / 2 : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != FBOB_OK) return st;
  fbob::NormArgs a = norm_args(p);
  a.x = x, a.w = w, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd), a.dy = dy;
  a.ux = ux, a.uw = uw, a.ub = ub, a.gx = gx, a.gw = gw, a.gdy = gdy, a.ws = workspace;
  fbob::DevCtx c;
  if ((st = fbob::make_ctx(&c)) != FBOB_OK) return st;
  const cudaError_t e = fbob::layer_norm_bob(a, c, stream);
  if (e != cudaSuccess) return cuda_fail(e, "layer_norm_bob launch");
  return FBOB_OK;
}

size_t fbob_linear_ce_workspace_bytes(const fbob_linear_ce* p, int pass) {
  if (check_ce(p) != FBOB_OK || p->T == 0 || pass < 0 || pass > 2) return 0;
  return fbob::linear_ce_workspace(ce_args(p), static_cast<fbob::CePass>(pass));
}

fbob_status fbob_linear_ce_fwd(const fbob_linear_ce* p, const void* H, const void* W, const long long* target,
                               float* loss, float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  fbob_status st = check_ce(p);
  if (st != FBOB_OK) return st;
  if (p->T == 0) return FBOB_OK;
  const Arg ps[] = {{H, "H", p->dtype, true},       {W, "W", p->dtype, true},     {target, "target", FBOB_FP32, true},
                    {loss, "loss", FBOB_FP32, true}, {lse, "lse", FBOB_FP32, true}};
  if ((st = check_args(ps, 5)) != FBOB_OK || (st = check_head(p, W, "W")) != FBOB_OK ||
      (st = check_targets(target)) != FBOB_OK)
    return st;
  fbob::CeArgs a = ce_args(p);
  a.H = H, a.W = W, a.target = target, a.loss = loss, a.lse_out = lse, a.ws = workspace;
  return ce_run(a, fbob::CePass::kFwd, workspace_bytes, "linear_ce_fwd launch", stream);
}

fbob_status fbob_linear_ce_bwd(const fbob_linear_ce* p, const void* H, const void* W, const long long* target,
                               const float* lse, const float* g, void* dH, void* dW, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
  fbob_status st = check_ce(p);
  if (st != FBOB_OK) return st;
  const bool some = p->T > 0;
  const Arg ps[] = {{H, "H", p->dtype, some},      {W, "W", p->dtype, some},  {target, "target", FBOB_FP32, some},
                    {lse, "lse", FBOB_FP32, some}, {g, "g", FBOB_FP32, some}, {dH, "dH", p->dtype, false},
                    {dW, "dW", p->dtype, false}};
  if ((st = check_args(ps, 7)) != FBOB_OK || (st = check_head(p, W, "W")) != FBOB_OK ||
      (st = check_targets(target)) != FBOB_OK)
    return st;
  if (!some) return zero_head(p, dW, stream);
  if (!dH && !dW) return FBOB_OK;
  fbob::CeArgs a = ce_args(p);
  a.H = H, a.W = W, a.target = target, a.lse = lse, a.g = g, a.dH = dH, a.dW = dW, a.ws = workspace;
  return ce_run(a, fbob::CePass::kBwd, workspace_bytes, "linear_ce_bwd launch", stream);
}

fbob_status fbob_linear_ce_bob(const fbob_linear_ce* p, const void* H, const void* W, const long long* target,
                               const float* lse, const float* g, const void* UH, const void* UW, void* gH, void* gW,
                               float* gg, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  fbob_status st = check_ce(p);
  if (st != FBOB_OK) return st;
  const bool some = p->T > 0;
  const Arg ps[] = {{H, "H", p->dtype, some},      {W, "W", p->dtype, some},  {target, "target", FBOB_FP32, some},
                    {lse, "lse", FBOB_FP32, some}, {g, "g", FBOB_FP32, some}, {UH, "UH", p->dtype, false},
                    {UW, "UW", p->dtype, false},   {gH, "gH", p->dtype, false}, {gW, "gW", p->dtype, false},
                    {gg, "gg", FBOB_FP32, false}};
  if ((st = check_args(ps, 10)) != FBOB_OK || (st = check_head(p, W, "W")) != FBOB_OK ||
      (st = check_head(p, UW, "UW")) != FBOB_OK || (st = check_targets(target)) != FBOB_OK)
    return st;
  if (!UH && !UW) return fail(FBOB_ERR_INVALID_ARG, "pointers UH and UW are both null");
  if (!some) return zero_head(p, gW, stream);
  if (!gH && !gW && !gg) return FBOB_OK;
  fbob::CeArgs a = ce_args(p);
  a.H = H, a.W = W, a.target = target, a.lse = lse, a.g = g, a.UH = UH, a.UW = UW;
  a.dH = gH, a.dW = gW, a.gg = gg, a.ws = workspace;
  return ce_run(a, fbob::CePass::kBob, workspace_bytes, "linear_ce_bob launch", stream);
}

}  // extern "C"
