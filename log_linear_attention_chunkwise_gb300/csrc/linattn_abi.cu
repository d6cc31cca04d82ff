// C ABI of linear attention with per-head decays and of layer norm: argument
// validation and dispatch.  Declarations, layouts and error behaviour:
// include/lla.h.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "layer_norm.cuh"
#include "linattn.cuh"
#include "padding.cuh"

using namespace lla;

namespace {

bool is_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool is_dtype(lla_dtype dt) { return dt == LLA_F32 || dt == LLA_BF16; }

// every pointer is there and 16-byte aligned
template <typename... P> bool good(P... p)
{
    return ((p != nullptr && ((uintptr_t)p & 15u) == 0) && ...);
}
// nullable pointers: 16-byte aligned
template <typename... P> bool aligned(P... p) { return ((((uintptr_t)p & 15u) == 0) && ...); }

size_t elt(lla_dtype dt) { return dt == LLA_BF16 ? 2 : 4; }

// A buffer of a call.  An output that overlaps what other CTAs still read (or write) would be a race: refused.
struct Span {
    const void *p;
    size_t bytes;
};

bool overlap(const Span &a, const Span &b)
{
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x != 0 && y != 0 && x < y + b.bytes && y < x + a.bytes;
}

// no output overlaps another one or an input
bool apart(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs)
{
    for (const Span *o = outputs.begin(); o != outputs.end(); o++) {
        for (const Span *p = outputs.begin(); p != o; p++)
            if (overlap(*o, *p)) return false;
        for (const Span &i : inputs)
            if (overlap(*o, i)) return false;
    }
    return true;
}

// the same buffer, or no common byte
bool same_or_apart(const Span &a, const Span &b) { return a.p == b.p || !overlap(a, b); }

// the outputs of lla_linattn_fwd
bool fwd_apart(const void *q, const void *k, const void *v, const float *state_in, const void *out,
               const float *state_out, int B, int H, int T, int dk, int dv, lla_dtype dt)
{
    const size_t rows = (size_t)B * H * T, bk = rows * dk * elt(dt), bv = rows * dv * elt(dt);
    const size_t bs = (size_t)B * H * dk * dv * 4;
    return apart({{out, bv}, {state_out, bs}}, {{q, bk}, {k, bk}, {v, bv}}) && !overlap({out, bv}, {state_in, bs}) &&
           same_or_apart({state_out, bs}, {state_in, bs});
}

// the outputs of lla_layer_norm_fwd
bool norm_fwd_apart(const void *x, const float *weight, const float *bias, const void *y, const float *mean,
                    const float *rstd, int B, int H, int T, int N, lla_dtype dt)
{
    const size_t rows = (size_t)B * H * T, bx = rows * N * elt(dt), bw = (size_t)H * N * 4;
    return apart({{y, bx}, {mean, rows * 4}, {rstd, rows * 4}}, {{weight, bw}, {bias, bw}}) &&
           apart({{mean, rows * 4}, {rstd, rows * 4}}, {{x, bx}}) && same_or_apart({y, bx}, {x, bx});
}

// the outputs of lla_linattn_bwd
bool bwd_apart(const void *q, const void *k, const void *v, const float *state_in, const void *dout,
               const float *dstate_out, const void *dq, const void *dk, const void *dv, const float *dstate_in, int B,
               int H, int T, int dk_dim, int dv_dim, lla_dtype dt)
{
    const size_t rows = (size_t)B * H * T, bk = rows * dk_dim * elt(dt), bv = rows * dv_dim * elt(dt);
    const size_t bs = (size_t)B * H * dk_dim * dv_dim * 4;
    return apart({{dq, bk}, {dk, bk}, {dv, bv}, {dstate_in, bs}},
                 {{q, bk}, {k, bk}, {v, bv}, {dout, bv}, {state_in, bs}, {dstate_out, bs}});
}

lla_status lin_shape_status(int B, int H, int T, int dk, int dv, lla_dtype dt)
{
    if (B < 0 || H < 0 || T < 0 || !is_dtype(dt)) return LLA_ERR_INVALID_ARGUMENT;
    if (!is_dim(dk) || !is_dim(dv) || T > (1 << 24)) return LLA_ERR_UNSUPPORTED_SHAPE;
    if ((long long)B * H > 65535) return LLA_ERR_UNSUPPORTED_SHAPE;
    return LLA_OK;
}

lla_status workspace_status(const void *ws, size_t have, size_t need)
{
    if (have < need) return LLA_ERR_WORKSPACE_TOO_SMALL;
    if (need > 0 && (ws == nullptr || ((uintptr_t)ws & 255u) != 0)) return LLA_ERR_INVALID_ARGUMENT;
    return LLA_OK;
}

lla_status norm_shape_status(int B, int H, int T, int N, lla_dtype dt)
{
    if (B < 0 || H < 0 || T < 0 || !is_dtype(dt)) return LLA_ERR_INVALID_ARGUMENT;
    if (N < 1 || N > kNormMaxN || (long long)B * H > 65535) return LLA_ERR_UNSUPPORTED_SHAPE;
    return LLA_OK;
}

lla_status done(cudaError_t e) { return e == cudaSuccess ? LLA_OK : LLA_ERR_CUDA; }

// an output of a padded batch: rows of `row` bytes, or one block of them a head (a state)
struct Cleared {
    void *base;
    size_t row;
    bool rows;
};

// The padding of a call's outputs (those that are there), for clear_padding.
lla_status clear(const int32_t *lens, int B, int H, int T, void *stream, std::initializer_list<Cleared> outputs)
{
    ZeroPaddingArgs A{};
    for (const Cleared &c : outputs) {
        if (c.base == nullptr || (c.rows && T == 0)) continue;
        A.rows[A.n] = c.base;
        A.row_bytes[A.n] = (int32_t)c.row;
        A.tokens[A.n++] = c.rows ? T : 0;
    }
    A.lens = lens; A.B = B; A.H = H; A.T = T; A.stream = stream;
    return A.n > 0 ? done(zero_padding(A)) : LLA_OK;
}

}  // namespace

extern "C" {

size_t lla_linattn_fwd_workspace_bytes(int B, int H, int T, int dk, int dv, lla_dtype dt)
{
    if (lin_shape_status(B, H, T, dk, dv, dt) != LLA_OK || (long long)B * H * T == 0) return 0;
    return linattn_fwd_workspace_bytes(B, H, T, dk, dv, dt);
}

lla_status lla_linattn_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                           const int32_t *lens, const float *state_in, void *out, float *state_out,
                           int B, int H, int T, int dk, int dv, lla_dtype dt, int clear_padding, void *workspace,
                           size_t workspace_bytes, int32_t *device_error, void *stream)
{
    lla_status st = lin_shape_status(B, H, T, dk, dv, dt);
    if (st != LLA_OK) return st;
    if ((long long)B * H == 0) return LLA_OK;
    if (!log_decay || !aligned(state_in, state_out)) return LLA_ERR_INVALID_ARGUMENT;
    if (T > 0 && !good(q, k, v, (const void *)out)) return LLA_ERR_INVALID_ARGUMENT;
    st = workspace_status(workspace, workspace_bytes, lla_linattn_fwd_workspace_bytes(B, H, T, dk, dv, dt));
    if (st != LLA_OK) return st;
    if (!fwd_apart(q, k, v, state_in, out, state_out, B, H, T, dk, dv, dt)) return LLA_ERR_INVALID_ARGUMENT;
    clear_padding = clear_padding && lens != nullptr;
    if (clear_padding) {
        st = clear(lens, B, H, T, stream, {{out, dv * elt(dt), true}, {state_out, (size_t)dk * dv * 4, false}});
        if (st != LLA_OK) return st;
    }
    LinFwdArgs A;
    A.after_padding = clear_padding != 0;
    A.q = q; A.k = k; A.v = v; A.log_decay = log_decay; A.lens = lens; A.state_in = state_in; A.out = out;
    A.state_out = state_out; A.B = B; A.H = H; A.T = T; A.dk = dk; A.dv = dv; A.dt = dt; A.workspace = workspace;
    A.device_error = device_error; A.stream = stream;
    return done(linattn_fwd(A));
}

size_t lla_linattn_bwd_workspace_bytes(int B, int H, int T, int dk, int dv, lla_dtype dt)
{
    if (lin_shape_status(B, H, T, dk, dv, dt) != LLA_OK || (long long)B * H * T == 0) return 0;
    return linattn_bwd_workspace_bytes(B, H, T, dk, dv, dt);
}

lla_status lla_linattn_bwd(const void *q, const void *k, const void *v, const float *log_decay,
                           const int32_t *lens, const float *state_in, const void *dout,
                           const float *dstate_out, void *dq, void *dk, void *dv, float *dstate_in, int B,
                           int H, int T, int dk_dim, int dv_dim, lla_dtype dt, int clear_padding,
                           void *workspace, size_t workspace_bytes, int32_t *device_error, void *stream)
{
    lla_status st = lin_shape_status(B, H, T, dk_dim, dv_dim, dt);
    if (st != LLA_OK) return st;
    if ((long long)B * H == 0) return LLA_OK;
    if (!log_decay || !aligned(state_in, dstate_out, dstate_in)) return LLA_ERR_INVALID_ARGUMENT;
    if (T > 0 && !good(q, k, v, dout, (const void *)dq, (const void *)dk, (const void *)dv))
        return LLA_ERR_INVALID_ARGUMENT;
    st = workspace_status(workspace, workspace_bytes,
                          lla_linattn_bwd_workspace_bytes(B, H, T, dk_dim, dv_dim, dt));
    if (st != LLA_OK) return st;
    // dk is formed from dstate_out, dq from state_in, while dstate_in is written
    if (!bwd_apart(q, k, v, state_in, dout, dstate_out, dq, dk, dv, dstate_in, B, H, T, dk_dim, dv_dim, dt))
        return LLA_ERR_INVALID_ARGUMENT;
    clear_padding = clear_padding && lens != nullptr;
    if (clear_padding) {
        const size_t rk = dk_dim * elt(dt), rv = dv_dim * elt(dt);
        st = clear(lens, B, H, T, stream,
                   {{dq, rk, true}, {dk, rk, true}, {dv, rv, true}, {dstate_in, (size_t)dk_dim * dv_dim * 4, false}});
        if (st != LLA_OK) return st;
    }
    LinBwdArgs A;
    A.after_padding = clear_padding != 0;
    A.q = q; A.k = k; A.v = v; A.dout = dout; A.log_decay = log_decay; A.lens = lens; A.state_in = state_in;
    A.dstate_out = dstate_out; A.dq = dq; A.dkey = dk; A.dval = dv; A.dstate_in = dstate_in; A.B = B; A.H = H;
    A.T = T; A.dk = dk_dim; A.dv = dv_dim; A.dt = dt; A.workspace = workspace; A.device_error = device_error;
    A.stream = stream;
    return done(linattn_bwd(A));
}

lla_status lla_linattn_decode_step(float *state, const void *q, const void *k, const void *v,
                                   const float *log_decay, const int32_t *slots, float *out, int pool, int B,
                                   int H, int dk, int dv, lla_dtype dt, int clear_skipped,
                                   int32_t *device_error, void *stream)
{
    if (pool < 0 || B < 0 || H < 0 || !is_dtype(dt)) return LLA_ERR_INVALID_ARGUMENT;
    if (!is_dim(dk) || !is_dim(dv) || B > 65535 || H > (1 << 24)) return LLA_ERR_UNSUPPORTED_SHAPE;
    if ((long long)B * H == 0) return LLA_OK;
    if (slots == nullptr && pool < B) return LLA_ERR_INVALID_ARGUMENT;
    // an empty pool has no address; its slots are all padding or out of range
    if (!log_decay || (pool > 0 && !good((const void *)state)) || !good(q, k, v, (const void *)out))
        return LLA_ERR_INVALID_ARGUMENT;
    const size_t heads = (size_t)B * H;
    if (!apart({{state, (size_t)pool * H * dk * dv * 4}, {out, heads * dv * 4}},
               {{q, heads * dk * elt(dt)}, {k, heads * dk * elt(dt)}, {v, heads * dv * elt(dt)}}))
        return LLA_ERR_INVALID_ARGUMENT;
    LinDecodeArgs A;
    A.state = state; A.q = q; A.k = k; A.v = v; A.log_decay = log_decay; A.slots = slots; A.out = out;
    A.pool = pool; A.B = B; A.H = H; A.dk = dk; A.dv = dv; A.dt = dt; A.clear_skipped = clear_skipped;
    A.device_error = device_error; A.stream = stream;
    return done(linattn_decode(A));
}

lla_status lla_zero_padding(void *const *rows, const int32_t *row_bytes, const int32_t *has_rows, int n,
                            const int32_t *lens, int B, int H, int T, void *stream)
{
    if (n < 0 || B < 0 || H < 0 || T < 0) return LLA_ERR_INVALID_ARGUMENT;
    if (n > kPaddingMax || (long long)B * H > 65535) return LLA_ERR_UNSUPPORTED_SHAPE;
    if ((long long)B * H * n == 0) return LLA_OK;
    if (!rows || !row_bytes || !has_rows || !lens) return LLA_ERR_INVALID_ARGUMENT;
    ZeroPaddingArgs A{};
    for (int i = 0; i < n; i++) {
        if (row_bytes[i] < 0) return LLA_ERR_INVALID_ARGUMENT;
        if (row_bytes[i] == 0 || (has_rows[i] && T == 0)) continue;  // nothing in it
        if (rows[i] == nullptr) return LLA_ERR_INVALID_ARGUMENT;
        A.rows[A.n] = rows[i];
        A.row_bytes[A.n] = row_bytes[i];
        A.tokens[A.n] = has_rows[i] ? T : 0;
        A.n++;
    }
    if (A.n == 0) return LLA_OK;
    A.lens = lens; A.B = B; A.H = H; A.T = T; A.stream = stream;
    return done(zero_padding(A));
}

lla_status lla_layer_norm_fwd(const void *x, const float *weight, const float *bias, const int32_t *lens,
                              void *y, float *mean, float *rstd, int B, int H, int T, int N, float eps,
                              lla_dtype dt, int clear_padding, int32_t *device_error, void *stream)
{
    lla_status st = norm_shape_status(B, H, T, N, dt);
    if (st != LLA_OK) return st;
    if (!(eps >= 0.f) || isinf(eps)) return LLA_ERR_INVALID_ARGUMENT;
    if ((long long)B * H * T == 0) return LLA_OK;
    if (!good(x, (const void *)y) || !aligned(weight, bias)) return LLA_ERR_INVALID_ARGUMENT;
    if (!norm_fwd_apart(x, weight, bias, y, mean, rstd, B, H, T, N, dt)) return LLA_ERR_INVALID_ARGUMENT;
    if (clear_padding && lens != nullptr) {
        st = clear(lens, B, H, T, stream, {{y, N * elt(dt), true}, {mean, 4, true}, {rstd, 4, true}});
        if (st != LLA_OK) return st;
    }
    LayerNormArgs A{};
    A.x = x; A.weight = weight; A.bias = bias; A.lens = lens; A.y = y; A.mean = mean; A.rstd = rstd;
    A.B = B; A.H = H; A.T = T; A.N = N; A.eps = eps; A.dt = dt; A.device_error = device_error;
    A.stream = stream;
    return done(layer_norm_fwd(A));
}

size_t lla_layer_norm_bwd_workspace_bytes(int B, int H, int T, int N, lla_dtype dt)
{
    if (norm_shape_status(B, H, T, N, dt) != LLA_OK || (long long)B * H * T == 0) return 0;
    return layer_norm_bwd_workspace_bytes(B, H, T, N, dt);
}

lla_status lla_layer_norm_bwd(const void *x, const float *weight, const float *mean, const float *rstd,
                              const int32_t *lens, const void *dy, void *dx, float *dweight, float *dbias,
                              int B, int H, int T, int N, lla_dtype dt, int clear_padding, void *workspace,
                              size_t workspace_bytes, int32_t *device_error, void *stream)
{
    lla_status st = norm_shape_status(B, H, T, N, dt);
    if (st != LLA_OK) return st;
    if ((long long)B * H * T == 0) {  // sums over no rows
        for (float *p : {dweight, dbias})
            if (p != nullptr && H > 0 &&
                cudaMemsetAsync(p, 0, (size_t)H * N * sizeof(float), (cudaStream_t)stream) != cudaSuccess)
                return LLA_ERR_CUDA;
        return LLA_OK;
    }
    if (!good(x, dy, (const void *)dx) || !mean || !rstd || !aligned(weight)) return LLA_ERR_INVALID_ARGUMENT;
    if (dweight != nullptr || dbias != nullptr) {
        st = workspace_status(workspace, workspace_bytes, layer_norm_bwd_workspace_bytes(B, H, T, N, dt));
        if (st != LLA_OK) return st;
    }
    const size_t rows = (size_t)B * H * T, bx = rows * N * elt(dt), bw = (size_t)H * N * 4;
    if (!apart({{dx, bx}, {dweight, bw}, {dbias, bw}}, {{weight, bw}, {mean, rows * 4}, {rstd, rows * 4}}) ||
        !apart({{dweight, bw}, {dbias, bw}}, {{x, bx}, {dy, bx}}) || !same_or_apart({dx, bx}, {dy, bx}) ||
        !same_or_apart({dx, bx}, {x, bx}))
        return LLA_ERR_INVALID_ARGUMENT;
    if (clear_padding && lens != nullptr) {
        st = clear(lens, B, H, T, stream, {{dx, N * elt(dt), true}});
        if (st != LLA_OK) return st;
    }
    LayerNormArgs A{};
    A.x = x; A.weight = weight; A.mean = const_cast<float *>(mean); A.rstd = const_cast<float *>(rstd);
    A.lens = lens; A.dy = dy; A.y = dx; A.dweight = dweight; A.dbias = dbias; A.B = B; A.H = H; A.T = T;
    A.N = N; A.dt = dt; A.workspace = workspace; A.device_error = device_error; A.stream = stream;
    return done(layer_norm_bwd(A));
}

lla_status lla_linattn_norm_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                                const int32_t *lens, const float *state_in, const float *weight,
                                const float *bias, float eps, void *o, void *y, float *mean, float *rstd,
                                float *state_out, int B, int H, int T, int dk, int dv, lla_dtype dt,
                                int clear_padding, void *workspace, size_t workspace_bytes,
                                int32_t *device_error, void *stream)
{
    // the norm's own checks first: nothing is enqueued on an error
    lla_status st = lin_shape_status(B, H, T, dk, dv, dt);
    if (st != LLA_OK) return st;
    if (!(eps >= 0.f) || isinf(eps)) return LLA_ERR_INVALID_ARGUMENT;
    if ((long long)B * H * T > 0 && (!good((const void *)o, (const void *)y) || !aligned(weight, bias)))
        return LLA_ERR_INVALID_ARGUMENT;
    const size_t rows = (size_t)B * H * T, bs = (size_t)B * H * dk * dv * 4;
    if (!norm_fwd_apart(o, weight, bias, y, mean, rstd, B, H, T, dv, dt) ||
        !apart({{state_out, bs}}, {{y, rows * dv * elt(dt)}, {mean, rows * 4}, {rstd, rows * 4}}))
        return LLA_ERR_INVALID_ARGUMENT;
    st = lla_linattn_fwd(q, k, v, log_decay, lens, state_in, o, state_out, B, H, T, dk, dv, dt, clear_padding,
                         workspace, workspace_bytes, device_error, stream);
    if (st != LLA_OK) return st;
    return lla_layer_norm_fwd(o, weight, bias, lens, y, mean, rstd, B, H, T, dv, eps, dt, clear_padding,
                              device_error, stream);
}

// [dout | the attention's and the norm's scratch, one after the other in time]
size_t lla_linattn_norm_bwd_workspace_bytes(int B, int H, int T, int dk, int dv, lla_dtype dt)
{
    if (lin_shape_status(B, H, T, dk, dv, dt) != LLA_OK || (long long)B * H * T == 0) return 0;
    const size_t a = linattn_bwd_workspace_bytes(B, H, T, dk, dv, dt);
    const size_t n = layer_norm_bwd_workspace_bytes(B, H, T, dv, dt);
    return align_up((size_t)B * H * T * dv * elt(dt), 256) + (a > n ? a : n);
}

lla_status lla_linattn_norm_bwd(const void *q, const void *k, const void *v, const float *log_decay,
                                const int32_t *lens, const float *state_in, const void *o,
                                const float *weight, const float *mean, const float *rstd, const void *dy,
                                const float *dstate_out, void *dq, void *dk, void *dv, float *dweight,
                                float *dbias, float *dstate_in, int B, int H, int T, int dk_dim, int dv_dim,
                                lla_dtype dt, int clear_padding, void *workspace, size_t workspace_bytes,
                                int32_t *device_error, void *stream)
{
    lla_status st = lin_shape_status(B, H, T, dk_dim, dv_dim, dt);
    if (st != LLA_OK) return st;
    // every check of both calls before the first is enqueued
    if ((long long)B * H > 0) {
        if (!log_decay || !aligned(state_in, dstate_out, dstate_in)) return LLA_ERR_INVALID_ARGUMENT;
    }
    if ((long long)B * H * T > 0) {
        if (!good(q, k, v, o, dy, (const void *)dq, (const void *)dk, (const void *)dv) || !mean || !rstd ||
            !aligned(weight))
            return LLA_ERR_INVALID_ARGUMENT;
        st = workspace_status(workspace, workspace_bytes,
                              lla_linattn_norm_bwd_workspace_bytes(B, H, T, dk_dim, dv_dim, dt));
        if (st != LLA_OK) return st;
    }
    const size_t rows = (size_t)B * H * T, bk = rows * dk_dim * elt(dt), bv = rows * dv_dim * elt(dt);
    const size_t bw = (size_t)H * dv_dim * 4, bs = (size_t)B * H * dk_dim * dv_dim * 4;
    if (!bwd_apart(q, k, v, state_in, workspace, dstate_out, dq, dk, dv, dstate_in, B, H, T, dk_dim, dv_dim, dt) ||
        !apart({{dweight, bw}, {dbias, bw}}, {{q, bk}, {k, bk}, {v, bv}, {dq, bk}, {dk, bk}, {dv, bv}, {dstate_in, bs},
                                              {state_in, bs}, {dstate_out, bs}}))
        return LLA_ERR_INVALID_ARGUMENT;
    const size_t off = (long long)B * H * T > 0 ? align_up((size_t)B * H * T * dv_dim * elt(dt), 256) : 0;
    char *rest = (char *)workspace + off;
    const size_t rest_bytes = off > 0 ? workspace_bytes - off : workspace_bytes;
    st = lla_layer_norm_bwd(o, weight, mean, rstd, lens, dy, workspace, dweight, dbias, B, H, T, dv_dim, dt, 0, rest,
                            rest_bytes, device_error, stream);
    if (st != LLA_OK) return st;
    return lla_linattn_bwd(q, k, v, log_decay, lens, state_in, workspace, dstate_out, dq, dk, dv, dstate_in, B, H,
                           T, dk_dim, dv_dim, dt, clear_padding, rest, rest_bytes, device_error, stream);
}

}  // extern "C"
