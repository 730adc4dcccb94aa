// mrn_grad_norm.cu -- the norm of all elements of a list of tensors, and the
// tensors scaled to a largest norm:
//   norm = sqrt(sum g^2),   out = g * (norm > max_norm ? max_norm / norm : 1)
//   The list travels in the kernels' parameters, so that a call copies nothing and a captured
// graph holds its entries.  All tensors together are one sequence of slots of eight elements, cut at
// multiples of eight elements of each tensor's memory, so that all but a tensor's first and last are
// whole and aligned.  Every CTA takes one stretch of the sequence: equal work whatever the tensors'
// sizes, and a fixed order of additions.
#include "mrn_gate_kernels.cuh"

namespace mrn {

constexpr int kListThreads = 256;
constexpr int kListCtasPerSm = 4;
constexpr int kListFlight = 4;          // slots of a thread in flight
constexpr int kListStep = kListThreads * kListFlight;
constexpr int kListTensors = 960;       // per launch: what 32,764 bytes of parameters hold
constexpr int kListFew = 120;           // ... and a form of less than 4096 bytes

struct ListEntry {
    const void *in;
    void *out;                 // NULL: the norm alone
    int64_t first;             // slots before this tensor
    uint64_t count;            // elements; the top bit: bf16
    MRN_HOST_DEVICE bool bf16() const { return count >> 63; }
    MRN_HOST_DEVICE int64_t elements() const { return static_cast<int64_t>(count & ~(uint64_t(1) << 63)); }
};

template <int N> struct ListArgs {
    ListEntry t[N];
    int64_t total;             // slots of all tensors
    int64_t per_cta;           // slots of one CTA, a multiple of kListStep
    int tensors;
};

// Elements from the slot boundary below a tensor to its first.
MRN_HOST_DEVICE inline int list_offset(const void *p, bool bf16) {
    return bf16 ? static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16) / 2
                : static_cast<int>(reinterpret_cast<uintptr_t>(p) % 32) / 4;
}

// The last of tensors lo .. hi whose first slot is at most s.
template <int N> __device__ __forceinline__ int list_find(const ListArgs<N> &l, int64_t s, int lo, int hi) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.t[mid].first <= s) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The sum over the CTA of a value in 64 bits, in a fixed order, for all threads.
__device__ __forceinline__ double list_cta_sum(double v) {
    __shared__ double s[kListThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < kListThreads / 32; ++w) v += s[w];
    return v;
}

// The squares of a thread's slots, in f32: two chains of at most 16 additions.
template <class T> __device__ __forceinline__ float slot_squares(const Slot<T> (&s)[kListFlight]) {
    uint64_t acc = 0;
#pragma unroll
    for (int u = 0; u < kListFlight; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = f2_fma(s[u].pair(i), s[u].pair(i), acc);
    return f2_sum(acc);
}
// The same where f32 has lost squares, in 64 bits.  Below 2^-100 those under f32's normal range may
// have been a share of the sum; at the other end it is infinite.  (Zeros are left out: gradients
// hold whole blocks of them, and 64-bit arithmetic is slow.)
template <class T> __device__ __noinline__ double slot_squares_f64(const Slot<T> (&s)[kListFlight]) {
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < kListFlight; ++u)
#pragma unroll
        for (int w = 0; w < Slot<T>::kWords; ++w) any |= s[u].w[w] << (T::kBytes == 4 ? 1 : 0);
    double sum = 0.0;
    if (T::kBytes == 2) any &= 0x7FFF7FFFu;
    if (any == 0) return sum;
#pragma unroll
    for (int u = 0; u < kListFlight; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += static_cast<double>(s[u].get(i)) * s[u].get(i);
    return sum;
}
template <class T> __device__ __forceinline__ double squares_of(const Slot<T> (&s)[kListFlight]) {
    const float q = slot_squares(s);
    return q >= 0x1p-100f && q < INFINITY ? static_cast<double>(q) : slot_squares_f64(s);
}

// A slot that is not whole: its elements one by one, zeros outside the tensor.
template <class T> __device__ __forceinline__ void list_load(Slot<T> &s, const ListEntry &e, int64_t slot, int offset) {
    const int64_t j0 = slot * 8 - offset, count = e.elements();
    if (j0 >= 0 && j0 + 8 <= count) {
        ld_slot(s, elem_ptr<T>(e.in, j0));
        return;
    }
    s.zero();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (j0 + i < 0 || j0 + i >= count) continue;
        Frag<T, 1> f;
        ld_plain(f, elem_ptr<T>(e.in, j0 + i));
        if constexpr (T::kBytes == 4) s.w[i] = f.w;
        else s.w[i >> 1] |= static_cast<uint32_t>(f.h) << ((i & 1) * 16);
    }
}

template <class T> __device__ __forceinline__ double list_squares_whole(const void *in, int64_t at) {
    Slot<T> s[kListFlight];
#pragma unroll
    for (int u = 0; u < kListFlight; ++u) ld_slot(s[u], elem_ptr<T>(in, at + u * (kListThreads * 8)));
    return squares_of(s);
}

template <int N>
__global__ void __launch_bounds__(kListThreads, kListCtasPerSm)
mrn_grad_squares_kernel(const __grid_constant__ ListArgs<N> l, double *parts) {
    pdl_enter();
    const int64_t lo = blockIdx.x * l.per_cta;
    const int64_t hi = lo + l.per_cta < l.total ? lo + l.per_cta : l.total;
    double sum = 0.0;
    int t = list_find(l, lo, 0, l.tensors - 1);
    for (int64_t base = lo; base < hi; base += kListStep) {
        int last = t;                                   // the tensor of the step's last slot
        const int64_t end = base + kListStep < hi ? base + kListStep : hi;
        if (t + 1 < l.tensors && l.t[t + 1].first < end) last = list_find(l, end - 1, t, l.tensors - 1);
        const ListEntry &e = l.t[t];
        const int offset = list_offset(e.in, e.bf16());
        const int64_t at = (base - e.first) * 8 - offset;
        if (last == t && at >= 0 && at + kListStep * 8 <= e.elements() && base + kListStep <= hi) {
            sum += e.bf16() ? list_squares_whole<BF16>(e.in, at + threadIdx.x * 8)
                            : list_squares_whole<F32>(e.in, at + threadIdx.x * 8);
        } else {
            // the end of a tensor: each slot finds its own
            Slot<BF16> h[kListFlight];
            Slot<F32> f[kListFlight];
#pragma unroll
            for (int u = 0; u < kListFlight; ++u) {
                h[u].zero();
                f[u].zero();
                const int64_t s = base + u * kListThreads + threadIdx.x;
                if (s >= end) continue;
                const ListEntry &own = l.t[list_find(l, s, t, last)];
                if (own.bf16()) list_load(h[u], own, s - own.first, list_offset(own.in, true));
                else list_load(f[u], own, s - own.first, list_offset(own.in, false));
            }
            sum += squares_of(h);
            sum += squares_of(f);
        }
        t = last;
        if (t + 1 < l.tensors && l.t[t + 1].first <= end) ++t;
    }
    sum = list_cta_sum(sum);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

__device__ __forceinline__ double norm_of(const double *parts, int64_t count) {
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kListThreads) sum += parts[i];
    return sqrt(list_cta_sum(sum));
}

__global__ void __launch_bounds__(kListThreads)
mrn_grad_norm_kernel(const double *parts, int64_t count, float *norm) {
    pdl_enter();
    const double v = norm_of(parts, count);
    if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

// Whole slots times k; as they are when k is one (a product would change a NaN's bits).
template <class T> __device__ __forceinline__ void slot_scale(Slot<T> &s, uint64_t k, bool clip) {
    if (!clip) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.put_pair(i, f2_mul(s.pair(i), k));
}
template <class T>
__device__ __forceinline__ void list_scale_whole(const void *in, void *out, int64_t at, uint64_t k, bool clip) {
    Slot<T> s[kListFlight];
#pragma unroll
    for (int u = 0; u < kListFlight; ++u) ld_slot(s[u], elem_ptr<T>(in, at + u * (kListThreads * 8)));
#pragma unroll
    for (int u = 0; u < kListFlight; ++u) {
        slot_scale(s[u], k, clip);
        st_slot(elem_ptr<T>(out, at + u * (kListThreads * 8)), s[u]);
    }
}
template <class T>
__device__ __forceinline__ void list_scale_slot(const ListEntry &e, int64_t slot, uint64_t k, bool clip) {
    const int offset = list_offset(e.in, T::kBytes == 2);
    Slot<T> s;
    list_load(s, e, slot, offset);
    slot_scale(s, k, clip);
    const int64_t j0 = slot * 8 - offset, count = e.elements();
    if (j0 >= 0 && j0 + 8 <= count && list_offset(e.out, T::kBytes == 2) == offset) {
        st_slot(elem_ptr<T>(e.out, j0), s);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (j0 + i < 0 || j0 + i >= count) continue;
        Frag<T, 1> f;
        if constexpr (T::kBytes == 4) f.w = s.w[i];
        else f.h = static_cast<unsigned short>(s.w[i >> 1] >> ((i & 1) * 16));
        st_global(elem_ptr<T>(e.out, j0 + i), f);
    }
}

// Every CTA adds up the partial sums itself, in the same order, and walks its stretch from the end:
// what the squares read last is still in L2.
template <int N>
__global__ void __launch_bounds__(kListThreads, kListCtasPerSm)
mrn_grad_scale_kernel(const __grid_constant__ ListArgs<N> l, const double *parts, int64_t count, double max_norm,
                      float *norm_out) {
    pdl_enter();
    const double norm = norm_of(parts, count);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
    const bool clip = norm > max_norm && isfinite(static_cast<float>(norm));
    const float kf = clip ? static_cast<float>(max_norm / norm) : 1.0f;
    const uint64_t k = f2_pack(kf, kf);
    const int64_t lo = blockIdx.x * l.per_cta;
    const int64_t hi = lo + l.per_cta < l.total ? lo + l.per_cta : l.total;
    int last = list_find(l, hi - 1, 0, l.tensors - 1);
    for (int64_t base = lo + (hi - 1 - lo) / kListStep * kListStep; base >= lo; base -= kListStep) {
        const int64_t end = base + kListStep < hi ? base + kListStep : hi;
        const int t = l.t[last].first <= base ? last : list_find(l, base, 0, last);
        const ListEntry &e = l.t[t];
        const int offset = list_offset(e.in, e.bf16());
        const int64_t at = (base - e.first) * 8 - offset;
        if (t == last && !clip && e.in == e.out) {
            // nothing to write
        } else if (t == last && at >= 0 && at + kListStep * 8 <= e.elements() && base + kListStep <= hi &&
                   list_offset(e.out, e.bf16()) == offset) {
            if (e.bf16()) list_scale_whole<BF16>(e.in, e.out, at + threadIdx.x * 8, k, clip);
            else list_scale_whole<F32>(e.in, e.out, at + threadIdx.x * 8, k, clip);
        } else {
#pragma unroll
            for (int u = 0; u < kListFlight; ++u) {
                const int64_t s = base + u * kListThreads + threadIdx.x;
                if (s >= end) continue;
                const ListEntry &own = l.t[list_find(l, s, t, last)];
                if (!clip && own.in == own.out) continue;
                if (own.bf16()) list_scale_slot<BF16>(own, s - own.first, k, clip);
                else list_scale_slot<F32>(own, s - own.first, k, clip);
            }
        }
        last = t;
        if (last > 0 && l.t[last].first >= base) --last;
    }
}

int64_t grad_norm_partials(int64_t tensors, int sms) {
    const int64_t launches = (tensors + kListTensors - 1) / kListTensors;
    return (launches < 1 ? 1 : launches) * sms * kListCtasPerSm;
}

// The entries from .. to as one launch's parameters; false when all of them are empty.
template <int N>
bool fill_list(ListArgs<N> &a, const TensorList &l, int64_t from, int64_t to, int sms, int64_t *ctas) {
    a.tensors = 0;
    a.total = 0;
    for (; from < to; ++from) {
        if (l.counts[from] == 0) continue;
        const bool bf16 = l.dtypes[from] == MRN_BF16;
        a.t[a.tensors++] = ListEntry{l.in[from], l.out ? l.out[from] : nullptr, a.total,
                                     static_cast<uint64_t>(l.counts[from]) | static_cast<uint64_t>(bf16) << 63};
        a.total += (l.counts[from] + list_offset(l.in[from], bf16) + 7) / 8;
    }
    if (a.tensors == 0) return false;
    const int64_t most = int64_t(sms) * kListCtasPerSm;
    a.per_cta = ((a.total + most - 1) / most + kListStep - 1) / kListStep * kListStep;
    *ctas = (a.total + a.per_cta - 1) / a.per_cta;
    return true;
}

cudaError_t launch_grad_norm(const TensorList &l, double max_norm, float *norm, double *workspace,
                             int sms, bool pdl, cudaStream_t stream, uint64_t *launches) {
    int64_t parts = 0;
    bool pending = true;       // norm is still to be written
    const auto squares = [&](const auto &a, int64_t ctas) {
        double *to = workspace + parts;
        parts += ctas;
        return launch_plain(mrn_grad_squares_kernel<sizeof(a.t) / sizeof(ListEntry)>, ctas, kListThreads, 0, pdl,
                            stream, launches, a, to);
    };
    const auto scale = [&](const auto &a, int64_t ctas) {
        float *to = pending ? norm : nullptr;
        pending = false;
        return launch_plain(mrn_grad_scale_kernel<sizeof(a.t) / sizeof(ListEntry)>, ctas, kListThreads, 0, pdl,
                            stream, launches, a, static_cast<const double *>(workspace), parts, max_norm, to);
    };
    const auto walk = [&](auto launch) {
        cudaError_t err = cudaSuccess;
        for (int64_t from = 0; from < l.tensors && err == cudaSuccess; from += kListTensors) {
            const int64_t to = from + kListTensors < l.tensors ? from + kListTensors : l.tensors;
            int64_t ctas = 0;
            if (to - from <= kListFew) {
                ListArgs<kListFew> a;
                if (fill_list(a, l, from, to, sms, &ctas)) err = launch(a, ctas);
            } else {
                ListArgs<kListTensors> a;
                if (fill_list(a, l, from, to, sms, &ctas)) err = launch(a, ctas);
            }
        }
        return err;
    };
    cudaError_t err = walk(squares);
    if (err == cudaSuccess && l.out) err = walk(scale);
    if (err == cudaSuccess && pending)
        err = launch_plain(mrn_grad_norm_kernel, 1, kListThreads, 0, pdl, stream, launches,
                           static_cast<const double *>(workspace), parts, norm);
    return err;
}

}  // namespace mrn
