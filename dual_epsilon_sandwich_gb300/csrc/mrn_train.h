// mrn_train.h -- host-side interface between the C entry points of the
// training operations (mrn_train_api.cpp) and their kernels
// (mrn_layernorm.cu, mrn_norm_backward.cu, mrn_dropout.cu).  Not part of the
// public ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime_api.h>

namespace mrn {

// The dropout of one call: element e of the flattened [rows x n] matrix is
// kept when its 16 random bits are >= threshold (see drop_groups and DropGroup in
// mrn_train_kernels.cuh), and kept values are multiplied by scale.
struct DropArgs {
    const uint64_t *rng;    // device: {seed, offset}; not read when threshold == 0
    uint64_t site;          // added to the offset
    uint32_t threshold;     // round(p * 2^16), 0 (no dropout) .. 65536
    float scale;            // 65536 / (65536 - threshold); 0 when nothing is kept
};

// LayerNorm, alone (res and stream NULL: normalises x) or after
// stream = res + dropout(x).
struct LayernormArgs {
    const void *x;
    const void *res;
    const void *gamma;
    const void *beta;       // NULL: none
    void *stream_out;
    void *y;
    float *mean, *rstd;     // NULL: not kept
    DropArgs drop;
    int64_t rows, n;
    float eps;
    uint32_t stall;             // bytes that a cluster's first wait expects in vain (test hook)
};

// The gradient of LayerNorm (rms false) or RMSNorm (rms true) at x.
struct BackwardArgs {
    const void *dy;
    const void *x;
    const void *gamma;
    const float *mean, *rstd;   // LayerNorm: the forward's; RMSNorm: NULL
    const void *dstream;        // NULL: none
    void *dx;                   // with dres: dropout(ds); else ds
    void *dres;                 // NULL: no dropout follows
    float *dgamma, *dbeta;      // dbeta NULL: none
    float *workspace;           // [parts x part_stride_of(n)] partial sums of dgamma, then of dbeta
    DropArgs drop;
    int64_t rows, n;
    float eps;                  // RMSNorm
    uint32_t stall;             // as above
    bool rms;
};

struct DropoutArgs {
    const void *x;
    const void *res;        // NULL: dropout alone
    void *y;
    DropArgs drop;
    int64_t total;          // rows * n
};

cudaError_t launch_layernorm(bool bf16, const LayernormArgs &a, int sms, bool pdl,
                             cudaStream_t stream, uint64_t *launches);
cudaError_t launch_norm_backward(bool bf16, const BackwardArgs &a, int sms, bool pdl,
                                 cudaStream_t stream, uint64_t *launches);
cudaError_t launch_dropout(bool bf16, const DropoutArgs &a, bool pdl, cudaStream_t stream,
                           uint64_t *launches);

// Bounded waits of these kernels' clusters that ran out since the last call; the tags keep the
// counters of the two apart from each other's and the operations'.
enum { kOpLayernormTimeouts = 100, kOpBackwardTimeouts = 101 };
int take_wait_timeouts_layernorm();
int take_wait_timeouts_norm_backward();

// Partial sums of dgamma (and of dbeta) that a backward pass keeps at most: the
// rows of [parts x part_stride_of(n)] floats in its workspace, for each of the two.
int64_t backward_parts(int64_t rows, int64_t n, int sms);
// Floats from one partial row to the next: whole slots of eight, and up to seven elements
// before them.
constexpr int64_t part_stride_of(int64_t n) { return (n + 15) / 8 * 8; }

}  // namespace mrn
