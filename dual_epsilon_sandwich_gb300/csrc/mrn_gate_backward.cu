// mrn_gate_backward.cu -- the gradient of the gated sandwich tail.  Per row, with
// i1 = inv(b; eps1), i2 = inv(s; eps2), w = dn * g2, c = g1 (times the gate, when that is one
// value per channel), g the gate otherwise, xh = b * i1:
//   ds = i2 * (w - s * i2^2 * mean(w s)) + dstream
//   db = i1 * (g ds c - xh * mean(g ds c xh)),   dres = scale * ds
// and over rows
//   P_j = sum_r dn s i2 = dg2_j,   A_j = sum_r g ds xh,   R_j = sum_r ds res
// which give dg1 = gate A and dgate = g1 A for a gate per channel, dg1 = A otherwise; with
// q_r = sum_j ds c xh, dgate = q_r per row, sum_r q_r for a scalar.
//   Both means are known after one reduction of a row: with
//   S1 = sum s^2, S2 = sum w s, S3 = sum b^2, S4 = sum w c b, S5 = sum s c b, S6 = sum dstream c b
// q = i1 * (i2 * (S4 - (i2 S2 / n) * (i2 S5)) + S6): the sum of ds c xh term by term, so that what
// cancels in it is what cancels in ds itself.
//   The column sums are taken on the same pass: every CTA adds up the rows it handles (fixed
// rows, in order) and leaves a row of partial sums per set in the workspace, which a second
// launch adds in order.  No atomics: the result does not depend on which CTA ran when.
#include "mrn_gate_kernels.cuh"

namespace mrn {

constexpr int kLoopedThreads = 512;

// What a row's six sums give.
struct RowScalars {
    float i1, i2;     // inv of the block's row, of the stream's
    float m;          // -i2 * mean(w s) * i2, the factor of xh_s = s i2 in ds
    float q;          // sum_j ds c xh
};
template <class InvSqrt>
__device__ __forceinline__ RowScalars row_scalars(const float (&s)[6], float inv_n, float eps1, float eps2,
                                                  InvSqrt inv_sqrt_of) {
    RowScalars r;
    r.i1 = inv_sqrt_of(fmaf(s[2], inv_n, eps1));
    r.i2 = inv_sqrt_of(fmaf(s[0], inv_n, eps2));
    const float mean = r.i2 * (s[1] * inv_n);
    r.m = -mean * r.i2;
    r.q = r.i1 * fmaf(r.i2, s[3], fmaf(r.m, r.i2 * s[4], s[5]));
    return r;
}

// Where a call's partial sums stand.
struct GateParts {
    float *pre, *post, *res;   // [parts x stride] each; res NULL: not due
    float *gate, *scale;       // partial sums of the scalar factors, one per entry; NULL: not due
    int64_t stride;
};

// Any width and any alignment: one row per CTA at a time, two passes over it (the second out of
// L2), element by element; the partial sums live in the workspace, each element of them read
// and written by one thread only.
template <class T>
__global__ void __launch_bounds__(kLoopedThreads)
mrn_gate_backward_looped_kernel(const GateBackwardArgs a, const GateParts parts) {
    __shared__ CtaSumSix slots;
    __shared__ CtaSum last;
    cta_sum_setup(slots);
    cta_sum_setup(last);
    pdl_enter();
    int turn = 0;
    const float inv_n = 1.0f / static_cast<float>(a.n);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * parts.stride;
    const bool channel = a.gate.kind == MRN_FACTOR_CHANNEL;
    float gates = 0.0f, scales = 0.0f;
    bool fresh = true;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t e0 = r * a.n;
        float s[6] = {};
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const float v = ld_elem<T>(a.s, e0 + j), b = ld_elem<T>(a.b, e0 + j);
            const float w = ld_elem<T>(a.dn, e0 + j) * ld_elem<T>(a.g2, j);
            const float cb = b * (channel ? ld_elem<T>(a.g1, j) * factor_at<T>(a.gate, r, j) : ld_elem<T>(a.g1, j));
            s[0] = fmaf(v, v, s[0]);
            s[1] = fmaf(w, v, s[1]);
            s[2] = fmaf(b, b, s[2]);
            s[3] = fmaf(w, cb, s[3]);
            s[4] = fmaf(v, cb, s[4]);
            if (a.dstream) s[5] = fmaf(ld_elem<T>(a.dstream, e0 + j), cb, s[5]);
        }
        cta_sum(s, slots, turn);
        const RowScalars k = row_scalars(s, inv_n, a.eps1, a.eps2, [](float v) { return 1.0f / sqrtf(v); });
        const float g = channel ? 1.0f : factor_at<T>(a.gate, r, 0);
        const float c2 = -k.i1 * (g * (k.q * inv_n));
        float scaled = 0.0f;
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const int64_t e = e0 + j;
            const float dn = ld_elem<T>(a.dn, e);
            const float vh = ld_elem<T>(a.s, e) * k.i2;
            const float xh = ld_elem<T>(a.b, e) * k.i1;
            float ds = fmaf(vh, k.m, dn * ld_elem<T>(a.g2, j) * k.i2);
            if (a.dstream) ds += ld_elem<T>(a.dstream, e);
            const float dsg = ds * g;
            const float c = channel ? ld_elem<T>(a.g1, j) * factor_at<T>(a.gate, r, j) : ld_elem<T>(a.g1, j);
            const float res = parts.res || parts.scale ? ld_elem<T>(a.res, e) : 0.0f;
            st_elem<T>(a.db, e, fmaf(xh, c2, dsg * c * k.i1));
            st_elem<T>(a.dres, e, factor_at<T>(a.scale, r, j) * ds);
            float *p = parts.pre + at + j;
            *p = fmaf(dn, vh, fresh ? 0.0f : *p);
            p = parts.post + at + j;
            *p = fmaf(dsg, xh, fresh ? 0.0f : *p);
            if (parts.res) {
                p = parts.res + at + j;
                *p = fmaf(ds, res, fresh ? 0.0f : *p);
            }
            scaled = fmaf(ds, res, scaled);
        }
        scales += scaled;
        gates += k.q;
        if (a.dgate && a.gate.kind == MRN_FACTOR_ROW && threadIdx.x == 0) a.dgate[r] = k.q;
        fresh = false;
    }
    if (parts.gate && threadIdx.x == 0) parts.gate[blockIdx.x] = gates;
    if (parts.scale) {
        float v[1] = {scales};
        cta_sum(v, last, turn);
        if (threadIdx.x == 0) parts.scale[blockIdx.x] = v[0];
    }
}

// The sums of the partial rows, one column per thread, and of the scalar factors' partial sums.
//   blockIdx.y  0: P -> dg2    1: A -> dg1, and dgate of a gate per channel    2: R -> dscale
//   behind the column blocks (blockIdx.x == columns): the scalars, y 0 the gate, 1 the scale
struct GateJoinArgs {
    GateParts from;
    float *dg1, *dg2, *dgate, *dscale;   // dgate, dscale: per channel or scalar; NULL: not due
    const void *g1;
    Factor gate;
    int64_t n, parts, scalars;
    int columns;
};

constexpr int kGateJoinThreads = 256;

template <class T>
__global__ void __launch_bounds__(kGateJoinThreads) mrn_gate_join_kernel(const GateJoinArgs a) {
    __shared__ CtaSum slots;
    cta_sum_setup(slots);
    pdl_enter();
    if (static_cast<int>(blockIdx.x) == a.columns) {
        const float *from = blockIdx.y == 0 ? a.from.gate : (blockIdx.y == 1 ? a.from.scale : nullptr);
        if (!from) return;
        float v[1] = {0.0f};
        for (int64_t i = threadIdx.x; i < a.scalars; i += kGateJoinThreads) v[0] += from[i];
        int turn = 0;
        cta_sum(v, slots, turn);
        if (threadIdx.x == 0) *(blockIdx.y == 0 ? a.dgate : a.dscale) = v[0];
        return;
    }
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kGateJoinThreads + threadIdx.x;
    const float *from = blockIdx.y == 0 ? a.from.pre : (blockIdx.y == 1 ? a.from.post : a.from.res);
    if (j >= a.n || (a.parts > 0 && !from)) return;
    float v = 0.0f;
    for (int64_t p = 0; p < a.parts; ++p) v += from[p * a.from.stride + j];
    if (blockIdx.y == 0) {
        a.dg2[j] = v;
    } else if (blockIdx.y == 1) {
        const bool any = a.parts > 0;      // (without rows the weights are not read)
        const float g = any && (a.gate.kind == MRN_FACTOR_CHANNEL) ? factor_at<T>(a.gate, 0, j) : 1.0f;
        a.dg1[j] = v * g;
        if (a.dgate && a.gate.kind == MRN_FACTOR_CHANNEL) a.dgate[j] = any ? v * ld_elem<T>(a.g1, j) : 0.0f;
    } else {
        a.dscale[j] = v;
    }
}

template <class T>
cudaError_t launch_gate_backward_typed(const GateBackwardArgs &a, int sms, bool pdl, cudaStream_t stream,
                                       uint64_t *launches) {
    const int64_t most = backward_parts(a.rows, a.n, sms);
    const bool scalar_gate = a.dgate && a.gate.kind == MRN_FACTOR_SCALAR;
    const bool scalar_scale = a.dscale && a.scale.kind == MRN_FACTOR_SCALAR;
    const bool column_scale = a.dscale && !scalar_scale;
    GateParts p = {};
    p.stride = part_stride_of(a.n);
    const int64_t set = most * p.stride;
    p.pre = a.workspace;
    p.post = a.workspace + set;
    p.res = column_scale ? a.workspace + 2 * set : nullptr;
    float *const scalars = a.workspace + kGateColumnSets * set;
    p.gate = scalar_gate ? scalars : nullptr;
    p.scale = scalar_scale ? scalars + 16 * most : nullptr;
    GateJoinArgs join = {};
    if (most > 0) {
        const cudaError_t err = launch_plain(mrn_gate_backward_looped_kernel<T>, most, kLoopedThreads, 0, pdl,
                                             stream, launches, a, p);
        if (err != cudaSuccess) return err;
    } else {
        // no rows: the sums are zero, their places only say which are due
        p.gate = scalar_gate ? a.dgate : nullptr;
        p.scale = scalar_scale ? a.dscale : nullptr;
    }
    join.from = p;
    join.dg1 = a.dg1;
    join.dg2 = a.dg2;
    join.dgate = a.dgate;
    join.dscale = a.dscale;
    join.g1 = a.g1;
    join.gate = a.gate;
    join.n = a.n;
    join.parts = join.scalars = most;
    const int64_t columns = (a.n + kGateJoinThreads - 1) / kGateJoinThreads;
    if (columns >= 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    join.columns = static_cast<int>(columns);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(columns + (scalar_gate || scalar_scale)), column_scale ? 3 : 2, 1);
    cfg.blockDim = dim3(kGateJoinThreads, 1, 1);
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, mrn_gate_join_kernel<T>, join);
    if (err == cudaSuccess) ++*launches;
    return err;
}

cudaError_t launch_gate_backward(bool bf16, const GateBackwardArgs &a, int sms, bool pdl,
                                 cudaStream_t stream, uint64_t *launches) {
    return bf16 ? launch_gate_backward_typed<BF16>(a, sms, pdl, stream, launches)
                : launch_gate_backward_typed<F32>(a, sms, pdl, stream, launches);
}

}  // namespace mrn
