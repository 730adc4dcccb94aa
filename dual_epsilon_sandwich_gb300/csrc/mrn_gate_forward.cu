// mrn_gate_forward.cu -- the dual-epsilon sandwich tail with a gate on the
// block and a scale on the residual:
//   stream = scale * res + gate * g1 * b * inv(b; eps1), rounded once and stored
//   y = stream * inv(stream; eps2) * g2
// with inv(v; eps) = 1 / sqrt(sum_j v_j^2 / n + eps).
#include "mrn_gate_kernels.cuh"

namespace mrn {

constexpr int kLoopedThreads = 512;

// Any width and any alignment: one row per CTA at a time, three passes over it (the second and
// third out of L2), element by element.
template <class T>
__global__ void __launch_bounds__(kLoopedThreads) mrn_gate_looped_kernel(const GateArgs a) {
    __shared__ CtaSum slots;
    cta_sum_setup(slots);
    pdl_enter();
    int turn = 0;
    const float count = static_cast<float>(a.n);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t e0 = r * a.n;
        float sum[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const float v = ld_elem<T>(a.b, e0 + j);
            sum[0] = fmaf(v, v, sum[0]);
        }
        cta_sum(sum, slots, turn);
        float k = 1.0f / sqrtf(sum[0] / count + a.eps1);
        if (a.gate.kind != MRN_FACTOR_CHANNEL) k *= factor_at<T>(a.gate, r, 0);
        sum[0] = 0.0f;
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            float c = ld_elem<T>(a.g1, j);
            if (a.gate.kind == MRN_FACTOR_CHANNEL) c *= factor_at<T>(a.gate, r, j);
            const float t = factor_at<T>(a.scale, r, j) * ld_elem<T>(a.res, e0 + j);
            const float v = st_elem<T>(a.stream_out, e0 + j, fmaf(ld_elem<T>(a.b, e0 + j) * k, c, t));
            sum[0] = fmaf(v, v, sum[0]);
        }
        cta_sum(sum, slots, turn);
        const float inv = 1.0f / sqrtf(sum[0] / count + a.eps2);
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x)
            st_elem<T>(a.y, e0 + j, ld_elem<T>(a.stream_out, e0 + j) * inv * ld_elem<T>(a.g2, j));
    }
}

cudaError_t launch_gate(bool bf16, const GateArgs &a, int sms, bool pdl, cudaStream_t stream,
                        uint64_t *launches) {
    const int64_t ctas = a.rows < 4LL * sms ? a.rows : 4LL * sms;
    return launch_plain(bf16 ? mrn_gate_looped_kernel<BF16> : mrn_gate_looped_kernel<F32>, ctas,
                        kLoopedThreads, 0, pdl, stream, launches, a);
}

}  // namespace mrn
