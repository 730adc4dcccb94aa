// mrn_layernorm.cu -- LayerNorm of every row, alone or after the residual add
// with dropout:
//   stream = res + dropout(x), rounded once to the row type and stored
//   mean = sum_j s_j / n,  rstd = 1 / sqrt(sum_j (s_j - mean)^2 / n + eps)
//   y = (s - mean) * rstd * gamma + beta      (s the stored stream, or x)
// The variance is summed from the deviations, not from the squares: a row
// whose mean is far from zero loses no digits.
#include "mrn_train_kernels.cuh"

namespace mrn {

constexpr int kLoopedThreads = 512;

// Any width: one row per CTA at a time, three passes over it (the second and
// third out of L2), element by element.
template <class T>
__global__ void __launch_bounds__(kLoopedThreads) mrn_layernorm_looped_kernel(const LayernormArgs a) {
    __shared__ CtaSumSlots<1> slots;
    pdl_enter();
    int turn = 0;
    const DropKey key = drop_key(a.drop);
    const bool add = a.res != nullptr;
    const void *s = add ? a.stream_out : a.x;
    const float count = static_cast<float>(a.n);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t e0 = r * a.n;
        float sum[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const int64_t e = e0 + j;
            float v = ld_elem<T>(a.x, e);
            if (add) {
                const bool keep = drop_keeps_element(key, e, a.drop.threshold);
                v = st_elem<T>(a.stream_out, e, drop_add(v, ld_elem<T>(a.res, e), keep, a.drop.scale));
            }
            sum[0] += v;
        }
        cta_sum(sum, slots, turn);
        const float mean = sum[0] / count;
        float dev[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const float d = ld_elem<T>(s, e0 + j) - mean;
            dev[0] = fmaf(d, d, dev[0]);
        }
        cta_sum(dev, slots, turn);
        const float rstd = 1.0f / sqrtf(dev[0] / count + a.eps);
        if (threadIdx.x == 0 && a.mean) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const float h = (ld_elem<T>(s, e0 + j) - mean) * rstd;
            const float b = a.beta ? ld_elem<T>(a.beta, j) : 0.0f;
            st_elem<T>(a.y, e0 + j, fmaf(h, ld_elem<T>(a.gamma, j), b));
        }
    }
}

template <class T>
cudaError_t launch_layernorm_typed(const LayernormArgs &a, int sms, bool pdl, cudaStream_t stream,
                                   uint64_t *launches) {
    const int64_t ctas = a.rows < 4LL * sms ? a.rows : 4LL * sms;
    return launch_plain(mrn_layernorm_looped_kernel<T>, ctas, kLoopedThreads, 0, pdl, stream,
                        launches, a);
}

cudaError_t launch_layernorm(bool bf16, const LayernormArgs &a, int sms, bool pdl,
                             cudaStream_t stream, uint64_t *launches) {
    return bf16 ? launch_layernorm_typed<BF16>(a, sms, pdl, stream, launches)
                : launch_layernorm_typed<F32>(a, sms, pdl, stream, launches);
}

}  // namespace mrn
