// mrn_gate_api.cpp -- the C entry points of the gated sandwich tail, its
// gradient, and the global gradient norm with clipping, declared in
// include/mrn.h.  This layer holds no arithmetic of the method: it checks
// arguments and hands the call to the launcher of the operation.
#include "mrn.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "mrn_checks.h"
#include "mrn_gate.h"
#include "mrn_train.h"

namespace {

using namespace mrn;

bool known(mrn_factor kind, bool rows_too) {
    return kind == MRN_FACTOR_NONE || kind == MRN_FACTOR_SCALAR || kind == MRN_FACTOR_CHANNEL ||
           (rows_too && kind == MRN_FACTOR_ROW);
}

int64_t values_of(mrn_factor kind, int64_t rows, int64_t n) {
    return kind == MRN_FACTOR_SCALAR ? 1 : (kind == MRN_FACTOR_CHANNEL ? n : (kind == MRN_FACTOR_ROW ? rows : 0));
}

Factor factor_of(const void *p, mrn_factor kind) {
    return Factor{kind == MRN_FACTOR_NONE ? nullptr : p, kind};
}

// Workspace of the gated tail's gradient (see mrn_gate.h).
mrn_status gate_workspace_bytes(int64_t rows, int64_t n, int64_t *bytes) {
    if (n < 1 || rows < 0 || n > INT64_MAX / 16) return MRN_ERR_INVALID_SIZE;
    const int64_t parts = gate_parts(rows, n, sm_count_of_current_device());
    const int64_t stride = part_stride_of(n);
    if (parts > 0 && stride > INT64_MAX / 32 / parts) return MRN_ERR_INVALID_SIZE;
    *bytes = kGateColumnSets * parts * stride * static_cast<int64_t>(sizeof(float)) +
             2 * kGateScalars * parts * static_cast<int64_t>(sizeof(double));
    return MRN_OK;
}

// The tensors of one call, checked; NULL out: the norm alone.
mrn_status check_list(const TensorList &l, const float *norm, const void *workspace,
                      int64_t workspace_bytes, int64_t needed) {
    if (!norm || !workspace) return MRN_ERR_NULL_POINTER;
    if (!aligned_to(norm, 4) || !aligned_to(workspace, 8)) return MRN_ERR_MISALIGNED;
    const Span ns = span_of(norm, 4), ws = span_of(workspace, needed);
    if (overlaps(ns, ws)) return MRN_ERR_ALIASING;
    if (l.tensors > 0 && (!l.in || !l.counts || !l.dtypes)) return MRN_ERR_NULL_POINTER;
    int64_t total = 0;
    for (int64_t i = 0; i < l.tensors; ++i) {
        if (l.dtypes[i] != MRN_F32 && l.dtypes[i] != MRN_BF16) return MRN_ERR_UNSUPPORTED_DTYPE;
        const int64_t count = l.counts[i];
        if (count < 0 || count > INT64_MAX / 16 - total) return MRN_ERR_INVALID_SIZE;
        total += count;
    }
    if (workspace_bytes < needed) return MRN_ERR_INVALID_SIZE;
    std::vector<Span> outs;
    if (l.out) outs.reserve(static_cast<size_t>(l.tensors));
    for (int64_t i = 0; i < l.tensors; ++i) {
        if (l.counts[i] == 0) continue;
        const int64_t e = elem_bytes(l.dtypes[i]);
        if (!l.in[i] || (l.out && !l.out[i])) return MRN_ERR_NULL_POINTER;
        if (!aligned_to(l.in[i], e) || (l.out && !aligned_to(l.out[i], e))) return MRN_ERR_MISALIGNED;
        const Span in = span_of(l.in[i], l.counts[i] * e);
        if (overlaps(in, ns) || overlaps(in, ws)) return MRN_ERR_ALIASING;
        if (!l.out) continue;
        const Span out = span_of(l.out[i], l.counts[i] * e);
        if (overlaps(out, ns) || overlaps(out, ws) || !output_vs_row_input_ok(out, in)) return MRN_ERR_ALIASING;
        outs.push_back(out);
    }
    if (!l.out) return MRN_OK;
    // no output meets another, nor another tensor's input
    std::sort(outs.begin(), outs.end(), [](Span a, Span b) { return a.lo < b.lo; });
    for (size_t i = 1; i < outs.size(); ++i)
        if (overlaps(outs[i - 1], outs[i])) return MRN_ERR_ALIASING;
    for (int64_t i = 0; i < l.tensors; ++i) {
        if (l.counts[i] == 0) continue;
        const Span in = span_of(l.in[i], l.counts[i] * elem_bytes(l.dtypes[i]));
        // the first output that ends behind the input's start; its own is checked above
        auto o = std::upper_bound(outs.begin(), outs.end(), in.lo, [](uintptr_t at, Span s) { return at < s.hi; });
        for (; o != outs.end() && o->lo < in.hi; ++o)
            if (o->lo != reinterpret_cast<uintptr_t>(l.out[i])) return MRN_ERR_ALIASING;
    }
    return MRN_OK;
}

mrn_status run_list(const TensorList &l, double max_norm, float *norm, void *workspace,
                    int64_t workspace_bytes, cudaStream_t stream) {
    if (l.tensors < 0) return MRN_ERR_INVALID_SIZE;
    if (!(max_norm >= 0.0)) return MRN_ERR_INVALID_EPS;
    int64_t needed = 0;
    mrn_status st = mrn_grad_norm_workspace(l.tensors, &needed);
    if (st != MRN_OK) return st;
    try {
        st = check_list(l, norm, workspace, workspace_bytes, needed);
    } catch (const std::bad_alloc &) {
        return MRN_ERR_INVALID_SIZE;
    }
    if (st != MRN_OK) return st;
    uint64_t launched = 0;
    const cudaError_t err = launch_grad_norm(l, max_norm, norm, static_cast<double *>(workspace),
                                             sm_count_of_current_device(), launch_pdl(), stream, &launched);
    return launch_result(err, launched);
}

}  // namespace

extern "C" {

mrn_status mrn_norm_gate_residual_norm(const void *block_out, const void *residual,
                                       const void *gamma_post, const void *gamma_pre,
                                       const void *gate, mrn_factor gate_kind,
                                       const void *res_scale, mrn_factor res_scale_kind,
                                       void *out_stream, void *normed, int64_t rows, int64_t n,
                                       float eps_post, float eps_pre, mrn_dtype dtype,
                                       cudaStream_t stream) {
    mrn_status st = check_common(rows, n, dtype, eps_post, eps_pre);
    if (st == MRN_OK && (!known(gate_kind, true) || !known(res_scale_kind, false))) st = MRN_ERR_INVALID_SIZE;
    if (st != MRN_OK || rows == 0) return st;
    GateArgs a = {};
    a.b = block_out;
    a.res = residual;
    a.g1 = gamma_post;
    a.g2 = gamma_pre;
    a.gate = factor_of(gate, gate_kind);
    a.scale = factor_of(res_scale, res_scale_kind);
    a.stream_out = out_stream;
    a.y = normed;
    a.rows = rows;
    a.n = n;
    a.eps1 = eps_post;
    a.eps2 = eps_pre;
    Buffers b;
    const int64_t e = elem_bytes(dtype);
    const int64_t row_bytes = rows * n * e;
    b.add(kRowIn, block_out, row_bytes, e);
    b.add(kRowIn, residual, row_bytes, e);
    b.add(kIn, gamma_post, n * e, e);
    b.add(kIn, gamma_pre, n * e, e);
    b.add(kIn, a.gate.p, values_of(gate_kind, rows, n) * e, e, gate_kind == MRN_FACTOR_NONE);
    b.add(kIn, a.scale.p, values_of(res_scale_kind, rows, n) * e, e, res_scale_kind == MRN_FACTOR_NONE);
    b.add(kRowOut, out_stream, row_bytes, e);
    b.add(kRowOut, normed, row_bytes, e);
    st = b.check();
    if (st != MRN_OK) return st;
    a.stall = launch_stall_bytes();
    uint64_t launched = 0;
    const cudaError_t err = launch_gate(dtype == MRN_BF16, a, sm_count_of_current_device(), launch_pdl(),
                                        stream, &launched);
    return launch_result(err, launched);
}

mrn_status mrn_norm_gate_backward_workspace(int64_t rows, int64_t n, int64_t *bytes) {
    if (!bytes) return MRN_ERR_NULL_POINTER;
    return gate_workspace_bytes(rows, n, bytes);
}

mrn_status mrn_norm_gate_residual_norm_backward(
    const void *dnormed, const void *dstream, const void *block_out, const void *out_stream,
    const void *residual, const void *gamma_post, const void *gamma_pre, const void *gate,
    mrn_factor gate_kind, const void *res_scale, mrn_factor res_scale_kind, void *dblock,
    void *dresidual, float *dgamma_post, float *dgamma_pre, float *dgate, float *dres_scale,
    void *workspace, int64_t workspace_bytes, int64_t rows, int64_t n, float eps_post,
    float eps_pre, mrn_dtype dtype, cudaStream_t stream) {
    int64_t needed = 0;
    mrn_status st = check_common(rows, n, dtype, eps_post, eps_pre);
    if (st == MRN_OK && (!known(gate_kind, true) || !known(res_scale_kind, false))) st = MRN_ERR_INVALID_SIZE;
    if (st == MRN_OK && rows > INT64_MAX / 4) st = MRN_ERR_INVALID_SIZE;      // (a gradient per row)
    if (st == MRN_OK) st = gate_workspace_bytes(rows, n, &needed);
    if (st != MRN_OK) return st;
    if ((dgate && gate_kind == MRN_FACTOR_NONE) || (dres_scale && res_scale_kind == MRN_FACTOR_NONE))
        return MRN_ERR_NULL_POINTER;
    GateBackwardArgs a = {};
    a.dn = dnormed;
    a.dstream = dstream;
    a.b = block_out;
    a.s = out_stream;
    a.res = dres_scale ? residual : nullptr;
    a.g1 = gamma_post;
    a.g2 = gamma_pre;
    a.gate = factor_of(gate, gate_kind);
    a.scale = factor_of(res_scale, res_scale_kind);
    a.db = dblock;
    a.dres = dresidual;
    a.dg1 = dgamma_post;
    a.dg2 = dgamma_pre;
    a.dgate = dgate;
    a.dscale = dres_scale;
    a.workspace = static_cast<float *>(workspace);
    a.rows = rows;
    a.n = n;
    a.eps1 = eps_post;
    a.eps2 = eps_pre;
    Buffers b;
    const int64_t e = elem_bytes(dtype);
    const int64_t row_bytes = rows * n * e;
    if (rows > 0) {
        b.add(kRowIn, dnormed, row_bytes, e);
        b.add(kRowIn, dstream, row_bytes, e, true);
        b.add(kRowIn, block_out, row_bytes, e);
        b.add(kRowIn, out_stream, row_bytes, e);
        b.add(kRowIn, a.res, row_bytes, e, dres_scale == nullptr);
        b.add(kIn, gamma_post, n * e, e);
        b.add(kIn, gamma_pre, n * e, e);
        b.add(kIn, a.gate.p, values_of(gate_kind, rows, n) * e, e, gate_kind == MRN_FACTOR_NONE);
        b.add(kIn, a.scale.p, values_of(res_scale_kind, rows, n) * e, e, res_scale_kind == MRN_FACTOR_NONE);
        b.add(kRowOut, dblock, row_bytes, e);
        b.add(kRowOut, dresidual, row_bytes, e);
        b.add(kOut, workspace, needed, 16);
    }
    b.add(kOut, dgamma_post, n * 4, 4);
    b.add(kOut, dgamma_pre, n * 4, 4);
    if (values_of(gate_kind, rows, n) > 0) b.add(kOut, dgate, values_of(gate_kind, rows, n) * 4, 4, true);
    b.add(kOut, dres_scale, values_of(res_scale_kind, rows, n) * 4, 4, true);
    st = b.check();
    if (st != MRN_OK) return st;
    if (workspace_bytes < needed) return MRN_ERR_INVALID_SIZE;
    a.stall = launch_stall_bytes();
    uint64_t launched = 0;
    const auto launch = dtype == MRN_BF16 ? launch_gate_backward_bf16 : launch_gate_backward_f32;
    const cudaError_t err = launch(a, sm_count_of_current_device(), launch_pdl(), stream, &launched);
    return launch_result(err, launched);
}

mrn_status mrn_grad_norm_workspace(int64_t tensors, int64_t *bytes) {
    if (!bytes) return MRN_ERR_NULL_POINTER;
    if (tensors < 0 || tensors > INT64_MAX / 4096) return MRN_ERR_INVALID_SIZE;
    *bytes = grad_norm_partials(tensors, sm_count_of_current_device()) * static_cast<int64_t>(sizeof(double));
    return MRN_OK;
}

mrn_status mrn_grad_norm(const void *const *grads, const int64_t *counts, const mrn_dtype *dtypes,
                         int64_t tensors, float *norm, void *workspace, int64_t workspace_bytes,
                         cudaStream_t stream) {
    return run_list(TensorList{grads, nullptr, counts, dtypes, tensors}, INFINITY, norm, workspace,
                    workspace_bytes, stream);
}

mrn_status mrn_clip_grad_norm(const void *const *grads, void *const *out, const int64_t *counts,
                              const mrn_dtype *dtypes, int64_t tensors, double max_norm,
                              float *norm, void *workspace, int64_t workspace_bytes,
                              cudaStream_t stream) {
    if (tensors > 0 && !out) return MRN_ERR_NULL_POINTER;
    return run_list(TensorList{grads, out, counts, dtypes, tensors}, max_norm, norm, workspace,
                    workspace_bytes, stream);
}

}  // extern "C"
