// mrn_train_kernels.cuh -- device code shared by the training operations:
// the counter-based generator of the dropout, and sums over a CTA.
#pragma once

#include "mrn_kernels.cuh"
#include "mrn_train.h"

namespace mrn {

// ---------------------------------------------------------------------------
// Dropout's random bits: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011): ten rounds of
//   (c0, c1, c2, c3) <- (hi(M1 c2) ^ c1 ^ k0, lo(M1 c2), hi(M0 c0) ^ c3 ^ k1, lo(M0 c0))
// with the key advanced by the Weyl constants between rounds.  The counter of
// element e is (e / 8, offset + site), 64 bits each, and the key is the seed;
// the 128 bits of the result are eight lanes of 16, so that one evaluation
// serves eight elements: a probability on a grid of 2^-16 costs a quarter of
// what 32 bits per element would.  Nothing is stored: the gradient evaluates
// the same counters again.
// ---------------------------------------------------------------------------
struct DropKey {
    uint32_t k0, k1, c2, c3;
};

__device__ __forceinline__ DropKey drop_key(const DropArgs &d) {
    DropKey k = {0u, 0u, 0u, 0u};
    if (d.threshold != 0u) {
        const uint64_t seed = d.rng[0];
        const uint64_t step = d.rng[1] + d.site;
        k.k0 = static_cast<uint32_t>(seed);
        k.k1 = static_cast<uint32_t>(seed >> 32);
        k.c2 = static_cast<uint32_t>(step);
        k.c3 = static_cast<uint32_t>(step >> 32);
    }
    return k;
}

// The eight 16-bit lanes of group e / 8, two per word, low half first.
__device__ __forceinline__ void philox_lanes(const DropKey &key, uint64_t group, uint32_t (&w)[4]) {
    uint32_t c0 = static_cast<uint32_t>(group), c1 = static_cast<uint32_t>(group >> 32);
    uint32_t c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
}

// Whether lane i (0..7) of a group is kept.
__device__ __forceinline__ bool drop_keeps(const uint32_t (&w)[4], int i, uint32_t threshold) {
    const uint32_t u = (i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu;
    return u >= threshold;
}

// One element on its own.
__device__ __forceinline__ bool drop_keeps_element(const DropKey &key, int64_t e,
                                                   uint32_t threshold) {
    if (threshold == 0u) return true;
    uint32_t w[4];
    philox_lanes(key, static_cast<uint64_t>(e) >> 3, w);
    const int i = static_cast<int>(e & 7);
    const uint32_t word = i < 4 ? (i < 2 ? w[0] : w[1]) : (i < 6 ? w[2] : w[3]);
    return ((i & 1) ? word >> 16 : word & 0xFFFFu) >= threshold;
}

// dropout(v).
__device__ __forceinline__ float drop_scale(float v, bool keep, float scale) {
    return keep ? v * scale : 0.0f;
}
// dropout(v), added to r: one rounding in f32.  A dropped value is not read
// into the sum, whatever it is (infinities and NaN included).
__device__ __forceinline__ float drop_add(float v, float r, bool keep, float scale) {
    return keep ? fmaf(v, scale, r) : r;
}

// ---------------------------------------------------------------------------
// Sums over all threads of a CTA (a multiple of 32), one barrier each: the
// slots alternate between calls, so that a call's writes never meet the reads
// of the call before it.
// ---------------------------------------------------------------------------
template <int N> struct CtaSumSlots {
    float v[2][N][32];
};

template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], CtaSumSlots<N> &s, int &turn) {
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int nwarps = blockDim.x >> 5;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = warp_allsum(v[i]);
        if (lane == 0) s.v[turn][i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_allsum(lane < nwarps ? s.v[turn][i][lane] : 0.0f);
}

// One kernel launch with the library's programmatic dependent launch option.
template <class... Params, class... Args>
cudaError_t launch_plain(void (*fn)(Params...), int64_t ctas, int threads, size_t shared, bool pdl,
                         cudaStream_t stream, uint64_t *launches, Args... args) {
    if (ctas < 1 || ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, fn, args...);
    if (err == cudaSuccess) ++*launches;
    return err;
}

// ---------------------------------------------------------------------------
// Eight consecutive elements of one operand, as raw bits: the share of one
// thread in a row, and the elements of one generator group.  16 bytes of bf16;
// 32 bytes of f32, moved in one 256-bit access.
// ---------------------------------------------------------------------------
template <class T> struct Slot {
    static constexpr int kWords = 2 * T::kBytes;
    uint32_t w[kWords];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (T::kBytes == 4) {
            return __uint_as_float(w[i]);
        } else {
            const uint32_t u = w[i >> 1];
            return __uint_as_float((i & 1) ? (u & 0xFFFF0000u) : (u << 16));
        }
    }
    // rounds to T (to nearest even)
    __device__ __forceinline__ void put(const float (&f)[8]) {
        if constexpr (T::kBytes == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void clear(int i) {
        if constexpr (T::kBytes == 4) {
            w[i] = 0u;
        } else {
            w[i >> 1] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;
        }
    }
    __device__ __forceinline__ void st_one(char *p, int i) const {
        if constexpr (T::kBytes == 4) {
            asm volatile("st.global.u32 [%0], %1;" :: "l"(p), "r"(w[i]) : "memory");
        } else {
            const unsigned short h =
                static_cast<unsigned short>((i & 1) ? (w[i >> 1] >> 16) : (w[i >> 1] & 0xFFFFu));
            asm volatile("st.global.u16 [%0], %1;" :: "l"(p), "h"(h) : "memory");
        }
    }
};

// A whole slot, aligned to its size; read once (past L1).
__device__ __forceinline__ void ld_slot(Slot<BF16> &s, const void *p) {
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]) : "l"(p));
}
__device__ __forceinline__ void ld_slot(Slot<F32> &s, const void *p) {
    asm volatile("ld.global.L1::no_allocate.L2::256B.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]), "=r"(s.w[4]),
                   "=r"(s.w[5]), "=r"(s.w[6]), "=r"(s.w[7]) : "l"(p));
}
__device__ __forceinline__ void st_slot(void *p, const Slot<BF16> &s) {
    asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};"
                 :: "l"(p), "r"(s.w[0]), "r"(s.w[1]), "r"(s.w[2]), "r"(s.w[3]) : "memory");
}
__device__ __forceinline__ void st_slot(void *p, const Slot<F32> &s) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "l"(p), "r"(s.w[0]), "r"(s.w[1]), "r"(s.w[2]), "r"(s.w[3]), "r"(s.w[4]),
                    "r"(s.w[5]), "r"(s.w[6]), "r"(s.w[7]) : "memory");
}

// One element of T at p.
template <class T> __device__ __forceinline__ float ld_elem(const void *base, int64_t e) {
    Frag<T, 1> f;
    ld_plain(f, elem_ptr<T>(base, e));
    return f.get(0);
}
template <class T> __device__ __forceinline__ float st_elem(void *base, int64_t e, float v) {
    Frag<T, 1> f;
    const float o[1] = {v};
    f.put(o);
    st_global(elem_ptr<T>(base, e), f);
    return f.get(0);   // as stored
}

}  // namespace mrn
