// mrn_grad_norm.cu -- the norm of all elements of a list of tensors, and the
// tensors scaled to a largest norm:
//   norm = sqrt(sum g^2),   out = g * (norm > max_norm ? max_norm / norm : 1)
// The list travels in the kernels' parameters, so that a call copies nothing and a captured
// graph holds its entries.
#include "mrn_gate_kernels.cuh"

namespace mrn {

constexpr int kListThreads = 256;
constexpr int kListCtasPerSm = 4;
constexpr int kListTensors = 1024;      // per launch: what 32,764 bytes of parameters hold
constexpr int kListFew = 96;            // ... and a form of less than 4096 bytes

template <int N> struct ListArgs {
    const void *in[N];
    void *out[N];
    int64_t first[N + 1];      // elements before tensor t
    uint8_t bf16[N];
    int tensors;
};

template <int N> __device__ __forceinline__ int tensor_of(const ListArgs<N> &l, int64_t e) {
    int lo = 0, hi = l.tensors;        // first[lo] <= e < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (l.first[mid] <= e) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The sum of a value over the CTA, in a fixed order; valid in thread 0.
__device__ __forceinline__ double cta_sum_f64(double v) {
    __shared__ double s[kListThreads];
    s[threadIdx.x] = v;
    for (int o = kListThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (threadIdx.x < o) s[threadIdx.x] += s[threadIdx.x + o];
    }
    return s[0];
}

template <int N>
__global__ void __launch_bounds__(kListThreads)
mrn_grad_squares_kernel(const __grid_constant__ ListArgs<N> l, double *parts) {
    pdl_enter();
    double sum = 0.0;
    const int64_t total = l.first[l.tensors];
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kListThreads + threadIdx.x; e < total;
         e += static_cast<int64_t>(gridDim.x) * kListThreads) {
        const int t = tensor_of(l, e);
        const float g = l.bf16[t] ? ld_elem<BF16>(l.in[t], e - l.first[t]) : ld_elem<F32>(l.in[t], e - l.first[t]);
        sum += static_cast<double>(g) * g;
    }
    sum = cta_sum_f64(sum);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

__device__ __forceinline__ double norm_of(const double *parts, int64_t count) {
    __shared__ double norm;
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kListThreads) sum += parts[i];
    sum = cta_sum_f64(sum);
    if (threadIdx.x == 0) norm = sqrt(sum);
    __syncthreads();
    return norm;
}

__global__ void __launch_bounds__(kListThreads)
mrn_grad_norm_kernel(const double *parts, int64_t count, float *norm) {
    pdl_enter();
    const double v = norm_of(parts, count);
    if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

template <int N>
__global__ void __launch_bounds__(kListThreads)
mrn_grad_scale_kernel(const __grid_constant__ ListArgs<N> l, const double *parts, int64_t count, double max_norm) {
    pdl_enter();
    const double norm = norm_of(parts, count);
    const bool clip = norm > max_norm && isfinite(static_cast<float>(norm));
    const float k = clip ? static_cast<float>(max_norm / norm) : 1.0f;
    const int64_t total = l.first[l.tensors];
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kListThreads + threadIdx.x; e < total;
         e += static_cast<int64_t>(gridDim.x) * kListThreads) {
        const int t = tensor_of(l, e);
        const int64_t i = e - l.first[t];
        if (!clip && l.in[t] == l.out[t]) continue;
        // (unscaled values are copied as bits: a product with one would change a NaN's)
        if (l.bf16[t]) {
            if (clip) st_elem<BF16>(l.out[t], i, ld_elem<BF16>(l.in[t], i) * k);
            else static_cast<uint16_t *>(l.out[t])[i] = static_cast<const uint16_t *>(l.in[t])[i];
        } else {
            if (clip) st_elem<F32>(l.out[t], i, ld_elem<F32>(l.in[t], i) * k);
            else static_cast<uint32_t *>(l.out[t])[i] = static_cast<const uint32_t *>(l.in[t])[i];
        }
    }
}

int64_t grad_norm_partials(int64_t tensors, int sms) {
    const int64_t launches = (tensors + kListTensors - 1) / kListTensors;
    return (launches < 1 ? 1 : launches) * sms * kListCtasPerSm;
}

template <int N, class Launch>
cudaError_t for_list(const TensorList &l, int64_t from, int64_t to, int64_t *at, Launch launch) {
    ListArgs<N> a;
    a.tensors = 0;
    a.first[0] = 0;
    for (; from < to; ++from) {
        if (l.counts[from] == 0) continue;
        a.in[a.tensors] = l.in[from];
        a.out[a.tensors] = l.out ? l.out[from] : nullptr;
        a.bf16[a.tensors] = l.dtypes[from] == MRN_BF16;
        a.first[a.tensors + 1] = a.first[a.tensors] + l.counts[from];
        ++a.tensors;
    }
    if (a.tensors == 0) return cudaSuccess;
    return launch(a, a.first[a.tensors], at);
}

cudaError_t launch_grad_norm(const TensorList &l, double max_norm, float *norm, double *workspace,
                             int sms, bool pdl, cudaStream_t stream, uint64_t *launches) {
    int64_t parts = 0;
    const auto ctas_of = [sms](int64_t total) {
        const int64_t want = (total + kListThreads - 1) / kListThreads, most = int64_t(sms) * kListCtasPerSm;
        return want < most ? want : most;
    };
    const auto squares = [&](const auto &a, int64_t total, int64_t *at) {
        const int64_t ctas = ctas_of(total);
        double *to = workspace + *at;
        *at += ctas;
        return launch_plain(mrn_grad_squares_kernel<sizeof(a.in) / 8>, ctas, kListThreads, 0, pdl, stream,
                            launches, a, to);
    };
    const auto scale = [&](const auto &a, int64_t total, int64_t *) {
        return launch_plain(mrn_grad_scale_kernel<sizeof(a.in) / 8>, ctas_of(total), kListThreads, 0, pdl,
                            stream, launches, a, static_cast<const double *>(workspace), parts, max_norm);
    };
    const auto walk = [&](auto launch) {
        cudaError_t err = cudaSuccess;
        for (int64_t from = 0; from < l.tensors && err == cudaSuccess; from += kListTensors) {
            const int64_t to = from + kListTensors < l.tensors ? from + kListTensors : l.tensors;
            err = to - from <= kListFew ? for_list<kListFew>(l, from, to, &parts, launch)
                                        : for_list<kListTensors>(l, from, to, &parts, launch);
        }
        return err;
    };
    cudaError_t err = walk(squares);
    if (err == cudaSuccess)
        err = launch_plain(mrn_grad_norm_kernel, 1, kListThreads, 0, pdl, stream, launches,
                           static_cast<const double *>(workspace), parts, norm);
    if (err == cudaSuccess && l.out) err = walk(scale);
    return err;
}

}  // namespace mrn
