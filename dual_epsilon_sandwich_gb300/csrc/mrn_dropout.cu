// mrn_dropout.cu -- y = res + dropout(x) over rows * n elements; without res
// it is the dropout alone, which is also its own gradient (the same counters
// give the same mask).
#include "mrn_train_kernels.cuh"

namespace mrn {

constexpr int kDropoutThreads = 256;

// Any alignment: element by element.
template <class T>
__global__ void __launch_bounds__(kDropoutThreads) mrn_dropout_kernel(const DropoutArgs a) {
    pdl_enter();
    const DropKey key = drop_key(a.drop);
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < a.total;
         e += step) {
        const bool keep = drop_keeps_element(key, e, a.drop.threshold);
        const float v = ld_elem<T>(a.x, e);
        st_elem<T>(a.y, e, a.res ? drop_add(v, ld_elem<T>(a.res, e), keep, a.drop.scale)
                                 : drop_scale(v, keep, a.drop.scale));
    }
}

cudaError_t launch_dropout(bool bf16, const DropoutArgs &a, int sms, bool pdl,
                           cudaStream_t stream, uint64_t *launches) {
    const int64_t most = 8LL * sms;
    const int64_t ctas = (a.total + kDropoutThreads - 1) / kDropoutThreads;
    return launch_plain(bf16 ? mrn_dropout_kernel<BF16> : mrn_dropout_kernel<F32>,
                        ctas < most ? ctas : most, kDropoutThreads, 0, pdl, stream, launches, a);
}

}  // namespace mrn
