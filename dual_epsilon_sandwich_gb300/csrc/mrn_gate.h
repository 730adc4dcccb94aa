// mrn_gate.h -- host-side interface between the C entry points of the gated
// sandwich tail and of the operations over many tensors (mrn_gate_api.cpp) and
// their kernels (mrn_gate_forward.cu, mrn_gate_backward.cuh, mrn_grad_norm.cu).
// Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime_api.h>

#include "mrn.h"

namespace mrn {

// A factor of the tail (the block's gate, the stream's residual scale): device
// memory of the operands' type, read as its kind says.
struct Factor {
    const void *p;          // NULL with MRN_FACTOR_NONE
    mrn_factor kind;
};

struct GateArgs {
    const void *b;          // block_out
    const void *res;
    const void *g1, *g2;    // gamma_post, gamma_pre
    Factor gate, scale;
    void *stream_out, *y;
    int64_t rows, n;
    float eps1, eps2;       // eps_post, eps_pre
    uint32_t stall;         // bytes that a cluster's first wait expects in vain (test hook)
};

struct GateBackwardArgs {
    const void *dn;         // dnormed
    const void *b, *s;      // block_out, out_stream
    const void *dstream;    // NULL: none
    const void *res;        // read for dscale only
    const void *g1, *g2;
    Factor gate, scale;
    void *db, *dres;
    float *dg1, *dg2;
    float *dgate, *dscale;  // NULL: not due
    float *workspace;       // see kGateColumnSets
    int64_t rows, n;
    float eps1, eps2;
    uint32_t stall;
};

cudaError_t launch_gate(bool bf16, const GateArgs &a, int sms, bool pdl, cudaStream_t stream,
                        uint64_t *launches);
cudaError_t launch_gate_backward_f32(const GateBackwardArgs &a, int sms, bool pdl, cudaStream_t stream,
                                     uint64_t *launches);
cudaError_t launch_gate_backward_bf16(const GateBackwardArgs &a, int sms, bool pdl, cudaStream_t stream,
                                      uint64_t *launches);

// Bounded waits of these kernels' clusters that ran out since the last call.
enum { kOpGateTimeouts = 102, kOpGateBackwardF32Timeouts = 103, kOpGateBackwardBF16Timeouts = 104 };
int take_wait_timeouts_gate();
int take_wait_timeouts_gate_backward_f32();
int take_wait_timeouts_gate_backward_bf16();

// Workspace of the tail's gradient: three sets of partial rows (as of the norms' gradients),
// and behind them, for either scalar factor, one f64 partial sum per CTA, of which a partial row
// has kGateScalars at most (a cluster's).
// Partial rows at most: as many as CTAs run at once, twice as many where rows are narrow.
constexpr int gate_parts_per_sm(int64_t n) { return n <= 2048 ? 8 : 4; }
inline int64_t gate_parts(int64_t rows, int64_t n, int sms) {
    int64_t parts = static_cast<int64_t>(sms) * gate_parts_per_sm(n);
    const int64_t by_size = (int64_t(1) << 27) / n;
    if (parts > by_size) parts = by_size;
    if (parts > rows) parts = rows;
    return parts < 1 ? (rows > 0 ? 1 : 0) : parts;
}
constexpr int64_t kGateColumnSets = 3;
constexpr int64_t kGateScalars = 16;

// ---------------------------------------------------------------------------
// Many tensors
// ---------------------------------------------------------------------------
struct TensorList {
    const void *const *in;
    void *const *out;       // NULL: the norm alone
    const int64_t *counts;
    const mrn_dtype *dtypes;
    int64_t tensors;
};

// Doubles of workspace for lists of this many tensors.
int64_t grad_norm_partials(int64_t tensors, int sms);
cudaError_t launch_grad_norm(const TensorList &l, double max_norm, float *norm, double *workspace,
                             int sms, bool pdl, cudaStream_t stream, uint64_t *launches);

}  // namespace mrn
