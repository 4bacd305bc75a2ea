// encoder_api.cu -- C ABI of linear attention and group norm: argument checks,
// workspace layout, launches.
#include <math.h>
#include <string.h>

#include "encoder_internal.h"

using namespace semicrf;

namespace {

constexpr size_t kStatusBytes = 256;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

semicrf_status ws_ok(const void *ws, size_t have, size_t need)
{
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256) return SEMICRF_ERR_INVALID_ARG;
    return have < need ? SEMICRF_ERR_WORKSPACE_TOO_SMALL : SEMICRF_OK;
}

size_t type_size(int dtype) { return dtype == SEMICRF_F32 ? 4 : 2; }

semicrf_status attention_ok(const semicrf_attention_dims *d)
{
    if (!d || d->B < 1 || d->T < 1 || d->H < 1 || d->dk < 1 || d->dv < 1) return SEMICRF_ERR_INVALID_ARG;
    if (d->dtype < SEMICRF_F32 || d->dtype > SEMICRF_F16 || (d->reverse != 0 && d->reverse != 1) || !isfinite(d->scale))
        return SEMICRF_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if (d->q_stride[i] < 0 || d->k_stride[i] < 0 || d->v_stride[i] < 0 || d->o_stride[i] < 0)
            return SEMICRF_ERR_INVALID_ARG;
    if (d->dk > SEMICRF_MAX_HEAD || d->dv > SEMICRF_MAX_HEAD) return SEMICRF_ERR_UNSUPPORTED_SHAPE;
    // thread blocks of one launch (up to 8 slices of 32 columns and 2 segments an SM)
    if ((long long)d->B * d->H > (1LL << 27) || d->T > (1 << 30)) return SEMICRF_ERR_UNSUPPORTED_SHAPE;
    return SEMICRF_OK;
}

// Outputs that are written twice would race: no axis longer than one is repeated.
bool output_ok(const semicrf_attention_dims &d)
{
    const int length[3] = {d.B, d.T, d.H};
    for (int i = 0; i < 3; ++i)
        if (length[i] > 1 && d.o_stride[i] == 0) return false;
    return true;
}

size_t attention_ws(const semicrf_attention_dims &d, bool backward)
{
    return kStatusBytes + la_workspace(d.B, d.T, d.H, d.dk, d.dv, d.dtype, backward ? 3 : 1);
}

// Pieces of 8 values can be moved in 16-byte accesses: width, address and the strides of
// axes longer than one allow it.
int vectors(const void *p, const long long (&st)[3], const LaArgs &a, int width, int dtype)
{
    const size_t size = type_size(dtype);
    const int length[3] = {a.B, a.T, a.H};
    if (width % 8 || reinterpret_cast<uintptr_t>(p) % 16) return 0;
    for (int i = 0; i < 3; ++i)
        if (length[i] > 1 && st[i] * size % 16) return 0;
    return 1;
}

void strides(long long (&to)[3], const int64_t (&from)[3])
{
    for (int i = 0; i < 3; ++i) to[i] = from[i];
}

void dense(long long (&to)[3], const semicrf_attention_dims &d, int width)
{
    to[2] = width;
    to[1] = (long long)d.H * width;
    to[0] = d.T * to[1];
}

LaArgs attention_args(const semicrf_attention_dims &d, const float *log_decay, const int32_t *lengths, void *ws,
                      int nwalk)
{
    LaArgs a;
    memset(&a, 0, sizeof(a));
    a.nwalk = nwalk;
    a.B = d.B;
    a.T = d.T;
    a.H = d.H;
    a.log_decay = log_decay;
    a.lengths = lengths;
    a.status = static_cast<int32_t *>(ws);
    return a;
}

void finish_walk(LaWalk &w, const LaArgs &a, int dtype)
{
    w.q_vec = vectors(w.q, w.qs, a, w.dk, dtype);
    w.k_vec = vectors(w.k, w.ks, a, w.dk, dtype);
    w.v_vec = vectors(w.v, w.vs, a, w.dv, dtype);
    w.o_vec = vectors(w.o, w.os, a, w.dv, dtype);
}

// The walk of a forward call.
LaArgs forward_args(const semicrf_attention_dims &d, const void *q, const void *k, const void *v, const float *log_decay,
                    const int32_t *lengths, const float *state_in, void *o, float *state_out, void *ws)
{
    LaArgs a = attention_args(d, log_decay, lengths, ws, 1);
    LaWalk &w = a.w[0];
    w.q = q;
    w.k = k;
    w.v = v;
    w.o = o;
    strides(w.qs, d.q_stride);
    strides(w.ks, d.k_stride);
    strides(w.vs, d.v_stride);
    strides(w.os, d.o_stride);
    w.dk = d.dk;
    w.dv = d.dv;
    w.s_in = state_in;
    w.s_out = state_out;
    w.s_rs = d.dv;
    w.s_cs = 1;
    w.b = d.scale;
    w.c = 1.f;
    w.reverse = d.reverse;
    w.lead = 1;
    finish_walk(w, a, d.dtype);
    return a;
}

// The three walks of a backward call.
LaArgs backward_args(const semicrf_attention_dims &d, const void *q, const void *k, const void *v, const float *log_decay,
                     const int32_t *lengths, const float *state_in, const void *grad_o, const float *grad_state, void *dq,
                     void *dk, void *dv, float *grad_state_in, void *ws)
{
    LaArgs a = attention_args(d, log_decay, lengths, ws, 3);
    // dq_i = scale sum_j lam^{i-j} (do_i . v_j) k_j, and the given state transposed
    LaWalk &x = a.w[0];
    x.q = grad_o;
    strides(x.qs, d.o_stride);
    x.k = v;
    strides(x.ks, d.v_stride);
    x.v = k;
    strides(x.vs, d.k_stride);
    x.o = dq;
    dense(x.os, d, d.dk);
    x.dk = d.dv;
    x.dv = d.dk;
    x.s_in = state_in;
    x.s_rs = 1;
    x.s_cs = d.dv;
    x.b = d.scale;
    x.c = 1.f;
    x.reverse = d.reverse;
    x.lead = 1;
    // against the walk's direction the state is sum lam^{..} scale q do^T; the final
    // state's own gradient enters it one decay later than a position's would
    LaWalk &y = a.w[1];
    y.q = k;
    strides(y.qs, d.k_stride);
    y.k = q;
    strides(y.ks, d.q_stride);
    y.v = grad_o;
    strides(y.vs, d.o_stride);
    y.o = dv;
    dense(y.os, d, d.dv);
    y.dk = d.dk;
    y.dv = d.dv;
    y.s_in = grad_state;
    y.s_out = grad_state_in;
    y.s_rs = d.dv;
    y.s_cs = 1;
    y.b = 1.f;
    y.c = d.scale;
    y.reverse = !d.reverse;
    y.lead = 0;
    y.out_decay = 1;
    LaWalk &z = a.w[2];
    z.q = v;
    strides(z.qs, d.v_stride);
    z.k = grad_o;
    strides(z.ks, d.o_stride);
    z.v = q;
    strides(z.vs, d.q_stride);
    z.o = dk;
    dense(z.os, d, d.dk);
    z.dk = d.dv;
    z.dv = d.dk;
    z.s_in = grad_state;
    z.s_rs = 1;
    z.s_cs = d.dv;
    z.b = 1.f;
    z.c = d.scale;
    z.reverse = !d.reverse;
    z.lead = 0;
    for (LaWalk &w : a.w) finish_walk(w, a, d.dtype);
    return a;
}

semicrf_status run_walks(const LaArgs &a, int dtype, void *ws, size_t ws_bytes, void *stream)
{
    const semicrf_status s = ws_ok(ws, ws_bytes, kStatusBytes + la_need(a, dtype));
    if (s != SEMICRF_OK) return s;
    int n = 0;
    bool small;
    const cudaError_t e = launch_la(a, dtype, static_cast<unsigned char *>(ws) + kStatusBytes, ws_bytes - kStatusBytes,
                                    static_cast<cudaStream_t>(stream), &n, &small);
    return small ? SEMICRF_ERR_WORKSPACE_TOO_SMALL : ended(e, n);
}

semicrf_status norm_ok(const semicrf_norm_dims *d)
{
    if (!d || d->N < 1 || d->S < 1 || d->C < 1 || d->G < 1 || d->C % d->G) return SEMICRF_ERR_INVALID_ARG;
    if (d->dtype < SEMICRF_F32 || d->dtype > SEMICRF_F16 ||
        (d->weight_dtype != SEMICRF_F32 && d->weight_dtype != d->dtype) || d->activation < SEMICRF_ACT_NONE ||
        d->activation > SEMICRF_ACT_GELU || !(d->eps >= 0.f) || !isfinite(d->eps))
        return SEMICRF_ERR_INVALID_ARG;
    // thread blocks of one launch, and indices of one row block
    if (d->S > (1 << 30) || (long long)d->N * d->G > (1LL << 30) || d->C > (1 << 22)) return SEMICRF_ERR_UNSUPPORTED_SHAPE;
    return SEMICRF_OK;
}

NormArgs norm_args(const semicrf_norm_dims &d, const void *weight, const void *bias, const int32_t *lengths, void *ws)
{
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.N = d.N;
    a.S = d.S;
    a.C = d.C;
    a.G = d.G;
    a.act = d.activation;
    a.wdtype = d.weight_dtype;
    a.eps = d.eps;
    a.weight = weight;
    a.bias = bias;
    a.lengths = lengths;
    a.status = static_cast<int32_t *>(ws);
    a.part = reinterpret_cast<double *>(static_cast<unsigned char *>(ws) + kStatusBytes);
    return a;
}

}  // namespace

extern "C" {

size_t semicrf_linear_attention_workspace_bytes(const semicrf_attention_dims *dims, int32_t backward)
{
    if (attention_ok(dims) != SEMICRF_OK || (backward != 0 && backward != 1)) return 0;
    return attention_ws(*dims, backward);
}

size_t semicrf_linear_attention_workspace_bytes_at(const semicrf_attention_dims *dims, int32_t backward, const void *q,
                                                   const void *k, const void *v, const void *o)
{
    if (attention_ok(dims) != SEMICRF_OK || (backward != 0 && backward != 1)) return 0;
    const semicrf_attention_dims &d = *dims;
    const LaArgs a = backward ? backward_args(d, q, k, v, nullptr, nullptr, nullptr, o, nullptr, nullptr, nullptr, nullptr,
                                              nullptr, nullptr)
                              : forward_args(d, q, k, v, nullptr, nullptr, nullptr, const_cast<void *>(o), nullptr, nullptr);
    return kStatusBytes + la_need(a, d.dtype);
}

semicrf_status semicrf_linear_attention(const semicrf_attention_dims *dims, const void *q, const void *k,
                                        const void *v, const float *log_decay, const int32_t *lengths,
                                        const float *state_in, void *o, float *state_out, void *ws, size_t ws_bytes,
                                        void *stream)
{
    prof_reset();
    semicrf_status s = attention_ok(dims);
    if (s != SEMICRF_OK) return s;
    const semicrf_attention_dims &d = *dims;
    if (!q || !k || !v || !log_decay || !o || !output_ok(d)) return SEMICRF_ERR_INVALID_ARG;
    return run_walks(forward_args(d, q, k, v, log_decay, lengths, state_in, o, state_out, ws), d.dtype, ws, ws_bytes, stream);
}

semicrf_status semicrf_linear_attention_backward(const semicrf_attention_dims *dims, const void *q, const void *k,
                                                 const void *v, const float *log_decay, const int32_t *lengths,
                                                 const float *state_in, const void *grad_o, const float *grad_state,
                                                 void *dq, void *dk, void *dv, float *grad_state_in, void *ws,
                                                 size_t ws_bytes, void *stream)
{
    prof_reset();
    semicrf_status s = attention_ok(dims);
    if (s != SEMICRF_OK) return s;
    const semicrf_attention_dims &d = *dims;
    if (!q || !k || !v || !log_decay || !grad_o || !dq || !dk || !dv) return SEMICRF_ERR_INVALID_ARG;
    return run_walks(backward_args(d, q, k, v, log_decay, lengths, state_in, grad_o, grad_state, dq, dk, dv, grad_state_in, ws),
                     d.dtype, ws, ws_bytes, stream);
}

semicrf_status semicrf_linear_attention_step(const semicrf_attention_dims *dims, const void *q, const void *k,
                                             const void *v, const float *log_decay, float *state, void *o,
                                             void *stream)
{
    prof_reset();
    semicrf_status s = attention_ok(dims);
    if (s != SEMICRF_OK) return s;
    const semicrf_attention_dims &d = *dims;
    if (d.T != 1 || !q || !k || !v || !log_decay || !state || !o || !output_ok(d)) return SEMICRF_ERR_INVALID_ARG;
    LaStepArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    for (int i = 0; i < 2; ++i) {
        a.qs[i] = d.q_stride[2 * i];
        a.ks[i] = d.k_stride[2 * i];
        a.vs[i] = d.v_stride[2 * i];
        a.os[i] = d.o_stride[2 * i];
    }
    a.state = state;
    a.log_decay = log_decay;
    a.B = d.B;
    a.H = d.H;
    a.dk = d.dk;
    a.dv = d.dv;
    a.scale = d.scale;
    int n = 0;
    cudaError_t e = launch_la_step(a, d.dtype, static_cast<cudaStream_t>(stream), &n);
    return ended(e, n);
}

size_t semicrf_group_norm_workspace_bytes(const semicrf_norm_dims *dims, int32_t backward)
{
    if (norm_ok(dims) != SEMICRF_OK || (backward != 0 && backward != 1)) return 0;
    return kStatusBytes + up256(norm_scratch(dims->N, dims->S, dims->C, dims->G, dims->dtype, backward));
}

semicrf_status semicrf_group_norm(const semicrf_norm_dims *dims, const void *x, const void *weight, const void *bias,
                                  const int32_t *lengths, void *y, float *stats, void *ws, size_t ws_bytes,
                                  void *stream)
{
    prof_reset();
    semicrf_status s = norm_ok(dims);
    if (s != SEMICRF_OK) return s;
    if (!x || !y || !stats || reinterpret_cast<uintptr_t>(stats) % 8) return SEMICRF_ERR_INVALID_ARG;
    s = ws_ok(ws, ws_bytes, semicrf_group_norm_workspace_bytes(dims, 0));
    if (s != SEMICRF_OK) return s;
    NormArgs a = norm_args(*dims, weight, bias, lengths, ws);
    a.x = x;
    a.y = y;
    a.stats = stats;
    int n = 0;
    cudaError_t e = launch_norm(a, dims->dtype, false, static_cast<cudaStream_t>(stream), &n);
    return ended(e, n);
}

semicrf_status semicrf_group_norm_backward(const semicrf_norm_dims *dims, const void *dy, const void *x,
                                           const void *weight, const void *bias, const int32_t *lengths,
                                           const float *stats, void *dx, float *dweight, float *dbias, void *ws,
                                           size_t ws_bytes, void *stream)
{
    prof_reset();
    semicrf_status s = norm_ok(dims);
    if (s != SEMICRF_OK) return s;
    if (!dy || !x || !stats || !dx || reinterpret_cast<uintptr_t>(stats) % 8) return SEMICRF_ERR_INVALID_ARG;
    s = ws_ok(ws, ws_bytes, semicrf_group_norm_workspace_bytes(dims, 1));
    if (s != SEMICRF_OK) return s;
    NormArgs a = norm_args(*dims, weight, bias, lengths, ws);
    a.x = x;
    a.dy = dy;
    a.y = dx;
    a.stats = const_cast<float *>(stats);
    a.dw = dweight;
    a.db = dbias;
    int n = 0;
    cudaError_t e = launch_norm(a, dims->dtype, true, static_cast<cudaStream_t>(stream), &n);
    return ended(e, n);
}

semicrf_status semicrf_get_operators_status(void *stream)
{
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return SEMICRF_ERR_CUDA;
    int32_t found[3] = {0, 0, 0};
    if (la_found(found) != cudaSuccess || la_tma_found(found + 1) != cudaSuccess || norm_found(found + 2) != cudaSuccess)
        return SEMICRF_ERR_CUDA;
    for (int32_t f : found)
        if (f) return static_cast<semicrf_status>(f);
    return SEMICRF_OK;
}

semicrf_status semicrf_clear_operators_status(void *stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool ok = la_clear_found(st) == cudaSuccess && la_tma_clear_found(st) == cudaSuccess &&
                    norm_clear_found(st) == cudaSuccess;
    return ok ? SEMICRF_OK : SEMICRF_ERR_CUDA;
}

}  // extern "C"
