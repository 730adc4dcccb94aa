// mrn_train_api.cpp -- the C entry points of the training operations declared
// in include/mrn.h: LayerNorm, the residual add with dropout (alone and before
// a LayerNorm), and the gradients of LayerNorm and RMSNorm.  This layer holds
// no arithmetic of the method: it checks arguments and hands the call to the
// launcher of the operation.
#include "mrn.h"

#include <cmath>
#include <cstdint>

#include "mrn_checks.h"
#include "mrn_train.h"

namespace {

using namespace mrn;

// Whether a row's f32 statistic for every row fits 64 bits of bytes (rows * n * size may, at bf16
// and n = 1, where this does not).
bool statistics_fit(int64_t rows) { return rows <= INT64_MAX / 4; }

// The dropout's threshold on the grid of 2^-16, and its scale.
mrn_status drop_args(double p, const uint64_t *rng, uint64_t site, DropArgs *d) {
    if (!(p >= 0.0 && p <= 1.0)) return MRN_ERR_INVALID_EPS;
    d->threshold = static_cast<uint32_t>(p * 65536.0 + 0.5);
    d->scale = d->threshold < 65536u ? 65536.0f / static_cast<float>(65536u - d->threshold) : 0.0f;
    d->rng = rng;
    d->site = site;
    return MRN_OK;
}

// Workspace of a backward pass: two sets of partial rows.
mrn_status workspace_bytes_needed(int64_t rows, int64_t n, int64_t *bytes) {
    if (n < 1 || rows < 0 || n > INT64_MAX / 16) return MRN_ERR_INVALID_SIZE;
    const int64_t parts = backward_parts(rows, n, sm_count_of_current_device());
    const int64_t stride = part_stride_of(n);
    if (parts > 0 && stride > INT64_MAX / 16 / parts) return MRN_ERR_INVALID_SIZE;
    *bytes = 2 * parts * stride * static_cast<int64_t>(sizeof(float));
    return MRN_OK;
}

struct BackwardCall {
    BackwardArgs a;
    const void *workspace;
    int64_t workspace_bytes;
    bool dropout;   // a.dres is required
    mrn_dtype dtype;
};

mrn_status backward(BackwardCall &c, cudaStream_t stream) {
    BackwardArgs &a = c.a;
    int64_t needed = 0;
    mrn_status st = check_common(a.rows, a.n, c.dtype, a.eps, a.eps);
    if (st == MRN_OK && !statistics_fit(a.rows)) st = MRN_ERR_INVALID_SIZE;
    if (st == MRN_OK) st = workspace_bytes_needed(a.rows, a.n, &needed);
    if (st != MRN_OK) return st;
    Buffers b;
    const int64_t e = elem_bytes(c.dtype);
    const int64_t row_bytes = a.rows * a.n * e;
    if (a.rows > 0) {
        b.add(kRowIn, a.dy, row_bytes, e);
        b.add(kRowIn, a.x, row_bytes, e);
        b.add(kRowIn, a.dstream, row_bytes, e, true);
        b.add(kIn, a.gamma, a.n * e, e);
        if (!a.rms) {
            b.add(kIn, a.mean, a.rows * 4, 4);
            b.add(kIn, a.rstd, a.rows * 4, 4);
        }
        if (c.dropout) {
            b.add(kRowOut, a.dres, row_bytes, e);
            b.add(kIn, a.drop.rng, 16, 8, a.drop.threshold == 0);
        }
        b.add(kRowOut, a.dx, row_bytes, e);
        b.add(kOut, c.workspace, needed, 16);
    }
    b.add(kOut, a.dgamma, a.n * 4, 4);
    b.add(kOut, a.dbeta, a.n * 4, 4, true);
    st = b.check();
    if (st != MRN_OK) return st;
    if (c.workspace_bytes < needed) return MRN_ERR_INVALID_SIZE;
    a.stall = launch_stall_bytes();
    a.workspace = static_cast<float *>(const_cast<void *>(c.workspace));
    uint64_t launched = 0;
    const cudaError_t err = launch_norm_backward(c.dtype == MRN_BF16, a, sm_count_of_current_device(),
                                                 launch_pdl(), stream, &launched);
    return launch_result(err, launched);
}

mrn_status layernorm(LayernormArgs &a, bool add, mrn_dtype dtype, cudaStream_t stream) {
    mrn_status st = check_common(a.rows, a.n, dtype, a.eps, a.eps);
    if (st != MRN_OK || a.rows == 0) return st;
    if (!statistics_fit(a.rows)) return MRN_ERR_INVALID_SIZE;
    Buffers b;
    const int64_t e = elem_bytes(dtype);
    const int64_t row_bytes = a.rows * a.n * e;
    b.add(kRowIn, a.x, row_bytes, e);
    if (add) {
        b.add(kRowIn, a.res, row_bytes, e);
        b.add(kRowOut, a.stream_out, row_bytes, e);
        b.add(kIn, a.drop.rng, 16, 8, a.drop.threshold == 0);
    }
    b.add(kIn, a.gamma, a.n * e, e);
    b.add(kIn, a.beta, a.n * e, e, true);
    b.add(kRowOut, a.y, row_bytes, e);
    b.add(kOut, a.mean, a.rows * 4, 4, a.rstd == nullptr);   // both or neither
    b.add(kOut, a.rstd, a.rows * 4, 4, a.mean == nullptr);
    st = b.check();
    if (st != MRN_OK) return st;
    a.stall = launch_stall_bytes();
    uint64_t launched = 0;
    const cudaError_t err = launch_layernorm(dtype == MRN_BF16, a, sm_count_of_current_device(),
                                             launch_pdl(), stream, &launched);
    return launch_result(err, launched);
}

}  // namespace

extern "C" {

mrn_status mrn_layernorm(const void *x, const void *gamma, const void *beta, void *y, float *mean,
                         float *rstd, int64_t rows, int64_t n, float eps, mrn_dtype dtype,
                         cudaStream_t stream) {
    LayernormArgs a = {};
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.drop.scale = 1.0f;
    a.rows = rows;
    a.n = n;
    a.eps = eps;
    return layernorm(a, false, dtype, stream);
}

mrn_status mrn_dropout_add_layernorm(const void *x, const void *residual, const void *gamma,
                                     const void *beta, void *out_stream, void *normed, float *mean,
                                     float *rstd, const uint64_t *rng, uint64_t site, double p,
                                     int64_t rows, int64_t n, float eps, mrn_dtype dtype,
                                     cudaStream_t stream) {
    LayernormArgs a = {};
    const mrn_status st = drop_args(p, rng, site, &a.drop);
    if (st != MRN_OK) return st;
    a.x = x;
    a.res = residual;
    a.gamma = gamma;
    a.beta = beta;
    a.stream_out = out_stream;
    a.y = normed;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.n = n;
    a.eps = eps;
    return layernorm(a, true, dtype, stream);
}

mrn_status mrn_layernorm_backward(const void *dy, const void *x, const void *gamma,
                                  const float *mean, const float *rstd, const void *dstream,
                                  void *dx, float *dgamma, float *dbeta, void *workspace,
                                  int64_t workspace_bytes, int64_t rows, int64_t n,
                                  mrn_dtype dtype, cudaStream_t stream) {
    BackwardCall c = {};
    c.a.dy = dy;
    c.a.x = x;
    c.a.gamma = gamma;
    c.a.mean = mean;
    c.a.rstd = rstd;
    c.a.dstream = dstream;
    c.a.dx = dx;
    c.a.dgamma = dgamma;
    c.a.dbeta = dbeta;
    c.a.rows = rows;
    c.a.n = n;
    c.a.eps = 1.0f;   // (not used: rstd is given)
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    c.dtype = dtype;
    return backward(c, stream);
}

mrn_status mrn_dropout_add_layernorm_backward(
    const void *dnormed, const void *out_stream, const void *gamma, const float *mean,
    const float *rstd, const void *dstream, void *dx, void *dresidual, float *dgamma, float *dbeta,
    const uint64_t *rng, uint64_t site, double p, void *workspace, int64_t workspace_bytes,
    int64_t rows, int64_t n, mrn_dtype dtype, cudaStream_t stream) {
    BackwardCall c = {};
    const mrn_status st = drop_args(p, rng, site, &c.a.drop);
    if (st != MRN_OK) return st;
    c.a.dy = dnormed;
    c.a.x = out_stream;
    c.a.gamma = gamma;
    c.a.mean = mean;
    c.a.rstd = rstd;
    c.a.dstream = dstream;
    c.a.dx = dx;
    c.a.dres = dresidual;
    c.a.dgamma = dgamma;
    c.a.dbeta = dbeta;
    c.a.rows = rows;
    c.a.n = n;
    c.a.eps = 1.0f;
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    c.dropout = true;
    c.dtype = dtype;
    return backward(c, stream);
}

mrn_status mrn_rmsnorm_backward(const void *dy, const void *x, const void *gamma,
                                const void *dstream, void *dx, float *dgamma, void *workspace,
                                int64_t workspace_bytes, int64_t rows, int64_t n, float eps,
                                mrn_dtype dtype, cudaStream_t stream) {
    BackwardCall c = {};
    c.a.dy = dy;
    c.a.x = x;
    c.a.gamma = gamma;
    c.a.dstream = dstream;
    c.a.dx = dx;
    c.a.dgamma = dgamma;
    c.a.rows = rows;
    c.a.n = n;
    c.a.eps = eps;
    c.a.rms = true;
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    c.dtype = dtype;
    return backward(c, stream);
}

mrn_status mrn_dropout_add(const void *x, const void *residual, void *out, const uint64_t *rng,
                           uint64_t site, double p, int64_t rows, int64_t n, mrn_dtype dtype,
                           cudaStream_t stream) {
    DropoutArgs a = {};
    mrn_status st = drop_args(p, rng, site, &a.drop);
    if (st == MRN_OK) st = check_common(rows, n, dtype, 1.0f, 1.0f);
    if (st != MRN_OK || rows == 0) return st;
    Buffers b;
    const int64_t e = elem_bytes(dtype);
    const int64_t row_bytes = rows * n * e;
    b.add(kRowIn, x, row_bytes, e);
    b.add(kRowIn, residual, row_bytes, e, true);
    b.add(kRowOut, out, row_bytes, e);
    b.add(kIn, rng, 16, 8, a.drop.threshold == 0);
    st = b.check();
    if (st != MRN_OK) return st;
    a.x = x;
    a.res = residual;
    a.y = out;
    a.total = rows * n;
    uint64_t launched = 0;
    const cudaError_t err = launch_dropout(dtype == MRN_BF16, a, launch_pdl(), stream, &launched);
    return launch_result(err, launched);
}

mrn_status mrn_norm_backward_workspace(int64_t rows, int64_t n, int64_t *bytes) {
    if (!bytes) return MRN_ERR_NULL_POINTER;
    return workspace_bytes_needed(rows, n, bytes);
}

}  // extern "C"
