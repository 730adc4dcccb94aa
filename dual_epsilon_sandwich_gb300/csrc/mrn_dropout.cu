// mrn_dropout.cu -- y = res + dropout(x) over rows * n elements; without res
// it is the dropout alone, which is also its own gradient (the same counters
// give the same mask).
#include "mrn_train_kernels.cuh"

namespace mrn {

constexpr int kDropoutThreads = 256;

// One thread per generator group of eight elements, kDropoutGroups groups apart by
// a CTA's width, so that a warp's accesses are contiguous and several are in flight
// while the generator runs.  VEC: every operand aligned to a slot (the usual case);
// else the eight elements are moved one by one, through L1, the generator still
// once for the eight.
//   Bound by memory: 65536 x 5120 bf16 293 us, 6.9 TB/s (the copy's rate: 297 us);
// 64 x 2048 bf16 1.4 us, a launch and one round trip.  Not VEC, the accesses bound it:
// 16384 x 4096 bf16, one operand an element off, 167 us against 59.
constexpr int kDropoutGroups = 2;

template <class T, bool VEC, bool ADD>
__global__ void __launch_bounds__(kDropoutThreads) mrn_dropout_kernel(const DropoutArgs a) {
    pdl_enter();
    const DropKey key = drop_key(a.drop);
    const int64_t groups = (a.total + 7) / 8;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kDropoutThreads * kDropoutGroups;
    for (int64_t g0 = static_cast<int64_t>(blockIdx.x) * kDropoutThreads * kDropoutGroups +
                      threadIdx.x;
         g0 < groups; g0 += step) {
        Slot<T> x[kDropoutGroups], r[kDropoutGroups];
#pragma unroll
        for (int k = 0; k < kDropoutGroups; ++k) {
            const int64_t e = (g0 + k * kDropoutThreads) * 8;
            if (VEC && e + 8 <= a.total) {
                ld_slot(x[k], elem_ptr<T>(a.x, e));
                if (ADD) ld_slot(r[k], elem_ptr<T>(a.res, e));
            }
        }
        DropGroup drop[kDropoutGroups];
        uint64_t group[kDropoutGroups];
#pragma unroll
        for (int k = 0; k < kDropoutGroups; ++k) group[k] = static_cast<uint64_t>(g0 + k * kDropoutThreads);
        drop_groups<kDropoutGroups>(drop, key, group, a.drop.threshold);
#pragma unroll
        for (int k = 0; k < kDropoutGroups; ++k) {
            const int64_t e = (g0 + k * kDropoutThreads) * 8;
            if (e >= a.total) continue;
            const DropGroup &d = drop[k];
            if (VEC && e + 8 <= a.total) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool keep = d.keeps(i);
                    o[i] = ADD ? drop_add(x[k].get(i), r[k].get(i), keep, a.drop.scale)
                               : drop_scale(x[k].get(i), keep, a.drop.scale);
                }
                x[k].put(o);
                st_slot(elem_ptr<T>(a.y, e), x[k]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (e + i >= a.total) break;
                    const bool keep = d.keeps(i);
                    const float v = ld_elem<T>(a.x, e + i);
                    st_elem<T>(a.y, e + i,
                               ADD ? drop_add(v, ld_elem<T>(a.res, e + i), keep, a.drop.scale)
                                   : drop_scale(v, keep, a.drop.scale));
                }
            }
        }
    }
}

template <class T, bool VEC>
cudaError_t launch_dropout_typed(const DropoutArgs &a, bool pdl, cudaStream_t stream,
                                 uint64_t *launches) {
    const int64_t per = int64_t(kDropoutThreads) * kDropoutGroups * 8;
    const int64_t most = int64_t(1) << 30;
    const int64_t ctas = a.total / per + (a.total % per != 0);
    return launch_plain(a.res ? mrn_dropout_kernel<T, VEC, true> : mrn_dropout_kernel<T, VEC, false>,
                        ctas < most ? ctas : most, kDropoutThreads, 0, pdl, stream, launches, a);
}

cudaError_t launch_dropout(bool bf16, const DropoutArgs &a, bool pdl, cudaStream_t stream,
                           uint64_t *launches) {
    const uintptr_t size = bf16 ? 16 : 32;
    const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                       reinterpret_cast<uintptr_t>(a.res)) % size) == 0;
    if (bf16)
        return vec ? launch_dropout_typed<BF16, true>(a, pdl, stream, launches)
                   : launch_dropout_typed<BF16, false>(a, pdl, stream, launches);
    return vec ? launch_dropout_typed<F32, true>(a, pdl, stream, launches)
               : launch_dropout_typed<F32, false>(a, pdl, stream, launches);
}

}  // namespace mrn
