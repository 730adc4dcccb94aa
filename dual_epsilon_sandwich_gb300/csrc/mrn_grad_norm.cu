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
// Slots of a thread in flight, 128 bytes of either type, and slots of one step of a CTA.
template <class T> struct ListFlight { static constexpr int kSlots = 16 / T::kBytes; };
constexpr int kListStepSlots = 8;
constexpr int kListStep = kListThreads * kListStepSlots;
// Slots of a thread at least: with one, lists of some hundred thousand elements take twice as many
// CTAs as need be (104 x 6656 f32: 9.4 us with one, 5.5 with two, 5.7 with four, 7.1 with eight; a
// clip of 3.2 M elements 18.4, 12.7, 12.7, 14.9).
constexpr int kListUnit = 2;
constexpr int kListTensors = 960;       // per launch: what 32,764 bytes of parameters hold
constexpr int kListFew = 86;            // ... and a form of less than 4096 bytes
constexpr int kListCtas = 608;          // four for each of 152 SMs

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
    int64_t per_cta;           // slots of one CTA, a multiple of kListThreads
    int tensors;
    uint16_t start[kListCtas + 1];   // the tensor of a CTA's first slot
};
static_assert(sizeof(ListArgs<kListTensors>) <= 32764 - 64 && sizeof(ListArgs<kListFew>) <= 4096 - 64, "kernel parameters");

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

// The sum over the CTA of a value in 64 bits, in a fixed order; valid in the first warp.  (An SM
// does two 64-bit additions a clock: all warps adding up shuffles took a microsecond per CTA.)
__device__ __forceinline__ double list_cta_sum(double v) {
    __shared__ double s[kListThreads];
    s[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
#pragma unroll
    for (int w = 1; w < kListThreads / 32; ++w) v += s[threadIdx.x + 32 * w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Squares in f32 are kept where none can have been lost: below 2^-100 those under f32's normal
// range may have been a share of the sum; at the other end it is infinite.
__device__ __forceinline__ bool squares_hold(float q) { return q >= 0x1p-100f && q < INFINITY; }

// The words of a slot that are not zero, but for signs.
template <class T> __device__ __forceinline__ uint32_t slot_bits(const Slot<T> &s) {
    uint32_t any = 0;
#pragma unroll
    for (int w = 0; w < Slot<T>::kWords; ++w) any |= s.w[w];
    return any & (T::kBytes == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
}

// The squares of `slots` whole slots, a CTA's width apart, in 64 bits, where f32 has lost some.
// (Zeros beside them are left out: 64-bit arithmetic is slow.)
template <class T> __device__ __forceinline__ double list_squares_f64(const void *in, int64_t at, int slots) {
    double sum = 0.0;
#pragma unroll 1
    for (int u = 0; u < slots; ++u) {
        Slot<T> s;
        ld_slot(s, elem_ptr<T>(in, at + u * (kListThreads * 8)));
        if (slot_bits(s) == 0) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += static_cast<double>(s.get(i)) * s.get(i);
    }
    return sum;
}

// The squares of a thread's share of a step: in f32 two chains of at most 32 additions.  Gradients
// hold whole blocks of zeros, whose squares have lost nothing: they are told while their slots
// are in registers, and take no longer than others (67 M elements, half of them zero: f32 42.3 us, bf16
// 22.9; read again 47.4 and 30.3).
template <class T> __device__ __forceinline__ double list_squares_whole(const void *in, int64_t at) {
    constexpr int F = ListFlight<T>::kSlots;
    double sum = 0.0;
#pragma unroll
    for (int h = 0; h < kListStepSlots; h += F) {
        Slot<T> s[F];
#pragma unroll
        for (int u = 0; u < F; ++u) ld_slot(s[u], elem_ptr<T>(in, at + (h + u) * (kListThreads * 8)));
        uint64_t acc = 0;
#pragma unroll
        for (int u = 0; u < F; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = f2_fma(s[u].pair(i), s[u].pair(i), acc);
        const float q = f2_sum(acc);
        if (squares_hold(q)) {
            sum += static_cast<double>(q);
            continue;
        }
        uint32_t any = 0;
#pragma unroll
        for (int u = 0; u < F; ++u) any |= slot_bits(s[u]);
        if (any != 0) sum += list_squares_f64<T>(in, at + h * (kListThreads * 8), F);
    }
    return sum;
}

// Where one slot of a step stands: of the tensor it belongs to, elements j .. j + 8 (cut to its own).
struct ListPlace {
    const void *in;
    void *out;
    int64_t j, count;
    bool bf16;
    __device__ __forceinline__ bool whole() const { return j >= 0 && j + 8 <= count; }
};
template <int N>
__device__ __forceinline__ ListPlace list_place(const ListArgs<N> &l, int64_t s, int first, int last) {
    const ListEntry &e = l.t[list_find(l, s, first, last)];
    ListPlace p = {e.in, e.out, 0, e.elements(), e.bf16()};
    p.j = (s - e.first) * 8 - list_offset(e.in, p.bf16);
    return p;
}
// A slot as raw words, of either type: bf16 fills the first four.
__device__ __forceinline__ void list_load(Slot<F32> &s, const ListPlace &p) {
    const char *at = static_cast<const char *>(p.in) + p.j * (p.bf16 ? 2 : 4);
    if (p.whole()) {
        if (p.bf16) {
            Slot<BF16> h;
            ld_slot(h, at);
#pragma unroll
            for (int i = 0; i < 4; ++i) s.w[i] = h.w[i];
        } else {
            ld_slot(s, at);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (p.j + i < 0 || p.j + i >= p.count) continue;
        if (p.bf16) {
            s.w[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(at)[i]) << ((i & 1) * 16);
        } else {
            s.w[i] = reinterpret_cast<const uint32_t *>(at)[i];
        }
    }
}
__device__ __forceinline__ Slot<BF16> list_half(const Slot<F32> &s) {
    Slot<BF16> h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h.w[i] = s.w[i];
    return h;
}
template <class T> __device__ __forceinline__ double slot_squares(const Slot<T> &s) {
    uint64_t acc = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = f2_fma(s.pair(i), s.pair(i), acc);
    const float q = f2_sum(acc);
    if (squares_hold(q)) return static_cast<double>(q);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (s.get(i) != 0.0f) sum += static_cast<double>(s.get(i)) * s.get(i);
    return sum;
}

constexpr int kListMixed = 2;      // slots of a thread in flight where a step meets several tensors

// Memory bounds it: 0.58 G bf16 elements 171 to 176 us on the device (6.6 to 6.8 TB/s, 97 to 100 % of the
// copy's rate, whose traffic is half writes), 128 bytes of each of 32 warps' threads in flight; 104 x 6656 f32 5.0 us
// with the norm, two launches.
template <int N>
__global__ void __launch_bounds__(kListThreads, kListCtasPerSm)
mrn_grad_squares_kernel(const __grid_constant__ ListArgs<N> l, double *parts) {
    pdl_enter();
    const int64_t lo = blockIdx.x * l.per_cta;
    const int64_t hi = lo + l.per_cta < l.total ? lo + l.per_cta : l.total;
    double sum = 0.0;
    int t = l.start[blockIdx.x];
    for (int64_t base = lo; base < hi; base += kListStep) {
        int last = t;                                   // the tensor of the step's last slot
        const int64_t end = base + kListStep < hi ? base + kListStep : hi;
        if (t + 1 < l.tensors && l.t[t + 1].first < end) last = list_find(l, end - 1, t, l.tensors - 1);
        const ListEntry &e = l.t[t];
        const int64_t at = (base - e.first) * 8 - list_offset(e.in, e.bf16());
        if (last == t && at >= 0 && at + kListStep * 8 <= e.elements() && base + kListStep <= hi) {
            sum += e.bf16() ? list_squares_whole<BF16>(e.in, at + threadIdx.x * 8)
                            : list_squares_whole<F32>(e.in, at + threadIdx.x * 8);
        } else {
            // a tensor's end, or several tensors: each slot finds its own
#pragma unroll 1
            for (int64_t s0 = base + threadIdx.x; s0 < end; s0 += kListMixed * kListThreads) {
                Slot<F32> s[kListMixed];
                bool bf16[kListMixed];
#pragma unroll
                for (int u = 0; u < kListMixed; ++u) {
                    s[u].zero();
                    bf16[u] = false;
                    if (s0 + u * kListThreads >= end) continue;
                    const ListPlace p = list_place(l, s0 + u * kListThreads, t, last);
                    bf16[u] = p.bf16;
                    list_load(s[u], p);
                }
#pragma unroll
                for (int u = 0; u < kListMixed; ++u) sum += bf16[u] ? slot_squares(list_half(s[u])) : slot_squares(s[u]);
            }
        }
        t = last;
        if (t + 1 < l.tensors && l.t[t + 1].first <= end) ++t;
    }
    sum = list_cta_sum(sum);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

// The root of the sum of the partial sums, and its inverse (0 where the norm is zero or not
// finite); valid in the first warp.  One step of Newton's in 64 bits from rsqrtf of the sum scaled
// to 1 .. 4 leaves 2^-42 (a 64-bit root and a quotient would take four times as long, in every
// CTA).
struct Norm {
    double norm, inv;
};
__device__ __forceinline__ Norm norm_of(const double *parts, int64_t count) {
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kListThreads) sum += parts[i];
    sum = list_cta_sum(sum);
    if (!(sum > 0.0) || !(sum < INFINITY)) return Norm{sum, 0.0};
    const int e = ((__double2hiint(sum) >> 20) - 1023) & ~1;
    const double m = sum * __hiloint2double((1023 - e) << 20, 0);
    double y = static_cast<double>(rsqrtf(static_cast<float>(m)));
    y = fma(0.5 * y, fma(-m * y, y, 1.0), y);
    return Norm{m * y * __hiloint2double((1023 + e / 2) << 20, 0), y * __hiloint2double((1023 - e / 2) << 20, 0)};
}

__global__ void __launch_bounds__(kListThreads)
mrn_grad_norm_kernel(const double *parts, int64_t count, float *norm) {
    pdl_enter();
    const double v = norm_of(parts, count).norm;
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
    constexpr int F = ListFlight<T>::kSlots;
#pragma unroll
    for (int h = 0; h < kListStepSlots; h += F) {
        Slot<T> s[F];
#pragma unroll
        for (int u = 0; u < F; ++u) ld_slot(s[u], elem_ptr<T>(in, at + (h + u) * (kListThreads * 8)));
#pragma unroll
        for (int u = 0; u < F; ++u) {
            slot_scale(s[u], k, clip);
            st_slot(elem_ptr<T>(out, at + (h + u) * (kListThreads * 8)), s[u]);
        }
    }
}
__device__ __forceinline__ void list_store(Slot<F32> &s, const ListPlace &p, uint64_t k, bool clip) {
    Slot<BF16> h = list_half(s);
    if (p.bf16) {
        slot_scale(h, k, clip);
#pragma unroll
        for (int i = 0; i < 4; ++i) s.w[i] = h.w[i];
    } else {
        slot_scale(s, k, clip);
    }
    char *at = static_cast<char *>(p.out) + p.j * (p.bf16 ? 2 : 4);
    if (p.whole() && list_offset(at, p.bf16) == 0) {
        if (p.bf16) st_slot(at, h);
        else st_slot(at, s);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (p.j + i < 0 || p.j + i >= p.count) continue;
        if (p.bf16) reinterpret_cast<uint16_t *>(at)[i] = static_cast<uint16_t>(s.w[i >> 1] >> ((i & 1) * 16));
        else reinterpret_cast<uint32_t *>(at)[i] = s.w[i];
    }
}

// Every CTA adds up the partial sums itself, in the same order, and walks its stretch from the end:
// what the squares read last may still be in L2.
//   Memory bounds it: with the squares 0.58 G bf16 elements 540 to 550 us, 3.48 GB (6.3 TB/s, 94 %); 16.8 M
// f32 elements 35 us, 5.7 TB/s.  Eviction hints (the stretch's end kept, the rest and the
// outputs dropped first) gained 2 % at most and are not used.  In place takes the same where the limit is
// reached, and little more than the norm where it is not (0.13 G bf16 elements 129 and 47 us); outputs at
// other offsets than their inputs go element by element (403 us).
template <int N>
__global__ void __launch_bounds__(kListThreads, kListCtasPerSm)
mrn_grad_scale_kernel(const __grid_constant__ ListArgs<N> l, const double *parts, int64_t count, double max_norm,
                      float *norm_out) {
    pdl_enter();
    __shared__ float factor;
    const Norm n = norm_of(parts, count);
    if (threadIdx.x == 0) {
        const float norm = static_cast<float>(n.norm);
        if (norm_out && blockIdx.x == 0) *norm_out = norm;
        factor = n.norm > max_norm && norm < INFINITY ? static_cast<float>(max_norm * n.inv) : 1.0f;
    }
    __syncthreads();
    const float kf = factor;
    const bool clip = kf != 1.0f;
    const uint64_t k = f2_pack(kf, kf);
    const int64_t lo = blockIdx.x * l.per_cta;
    const int64_t hi = lo + l.per_cta < l.total ? lo + l.per_cta : l.total;
    int last = l.start[blockIdx.x + 1];                     // the tensor of the stretch's last slot
    if (l.t[last].first >= hi) --last;
    for (int64_t base = lo + (hi - 1 - lo) / kListStep * kListStep; base >= lo; base -= kListStep) {
        const int64_t end = base + kListStep < hi ? base + kListStep : hi;
        const int t = l.t[last].first <= base ? last : list_find(l, base, 0, last);
        const ListEntry &e = l.t[t];
        const int64_t at = (base - e.first) * 8 - list_offset(e.in, e.bf16());
        if (t == last && !clip && e.in == e.out) {
            // nothing to write
        } else if (t == last && at >= 0 && at + kListStep * 8 <= e.elements() && base + kListStep <= hi &&
                   list_offset(e.out, e.bf16()) == list_offset(e.in, e.bf16())) {
            if (e.bf16()) list_scale_whole<BF16>(e.in, e.out, at + threadIdx.x * 8, k, clip);
            else list_scale_whole<F32>(e.in, e.out, at + threadIdx.x * 8, k, clip);
        } else {
#pragma unroll 1
            for (int64_t s0 = base + threadIdx.x; s0 < end; s0 += kListMixed * kListThreads) {
                Slot<F32> s[kListMixed];
                ListPlace p[kListMixed];
#pragma unroll
                for (int u = 0; u < kListMixed; ++u) {
                    s[u].zero();
                    p[u].in = p[u].out = nullptr;
                    if (s0 + u * kListThreads >= end) continue;
                    p[u] = list_place(l, s0 + u * kListThreads, t, last);
                    list_load(s[u], p[u]);
                }
#pragma unroll
                for (int u = 0; u < kListMixed; ++u)
                    if (p[u].out && (clip || p[u].in != p[u].out)) list_store(s[u], p[u], k, clip);
            }
        }
        last = t;
        if (last > 0 && l.t[last].first >= base) --last;
    }
}

int64_t list_ctas(int sms) { return sms * kListCtasPerSm < kListCtas ? sms * kListCtasPerSm : kListCtas; }

int64_t grad_norm_partials(int64_t tensors, int sms) {
    const int64_t launches = (tensors + kListTensors - 1) / kListTensors;
    return (launches < 1 ? 1 : launches) * list_ctas(sms);
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
    const int64_t most = list_ctas(sms);
    const int64_t each = (a.total + most - 1) / most, unit = each < kListStep ? kListThreads * kListUnit : kListStep;
    a.per_cta = (each + unit - 1) / unit * unit;
    *ctas = (a.total + a.per_cta - 1) / a.per_cta;
    int t = 0;
    for (int64_t c = 0; c <= *ctas; ++c) {
        while (t + 1 < a.tensors && a.t[t + 1].first <= c * a.per_cta) ++t;
        a.start[c] = static_cast<uint16_t>(t);
    }
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
