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
// serves eight elements: a probability on a grid of 2^-16 costs half of
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

// One group's eight 16-bit lanes (two per word, low half first) and the word threshold they
// are compared with: element i is kept when its lane, moved to the upper half of a word, is
// >= at (the lower half left below an upper lane does not change the comparison).
struct DropGroup {
    uint32_t w[4];
    uint32_t at;
    __device__ __forceinline__ bool keeps(int i) const {
        return ((i & 1) ? w[i >> 1] : w[i >> 1] << 16) >= at;
    }
    // the same for a lane that is not known when compiling
    __device__ __forceinline__ bool keeps_any(int i) const {
        const uint32_t word = i < 4 ? (i < 2 ? w[0] : w[1]) : (i < 6 ? w[2] : w[3]);
        return ((i & 1) ? word : word << 16) >= at;
    }
};

// G groups, round by round: the round keys are advanced once for all of them, and the G
// chains of ten dependent multiplications overlap.  All kept (threshold 0) and all dropped
// (65536) need no generator.
template <int G>
__device__ __forceinline__ void drop_groups(DropGroup (&d)[G], const DropKey &key, const uint64_t (&group)[G],
                                            uint32_t threshold) {
    const bool mixed = threshold != 0u && threshold < 65536u;
    uint32_t c0[G], c1[G], c2[G], c3[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        d[g].at = mixed ? threshold << 16 : (threshold == 0u ? 0u : 1u);
        c0[g] = c1[g] = c2[g] = c3[g] = 0u;
    }
    if (mixed) {
        uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            c0[g] = static_cast<uint32_t>(group[g]);
            c1[g] = static_cast<uint32_t>(group[g] >> 32);
            c2[g] = key.c2;
            c3[g] = key.c3;
        }
#pragma unroll
        for (int r = 0; r < 10; ++r) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint64_t a = static_cast<uint64_t>(c0[g]) * 0xD2511F53u;
                const uint64_t b = static_cast<uint64_t>(c2[g]) * 0xCD9E8D57u;
                c0[g] = static_cast<uint32_t>(b >> 32) ^ c1[g] ^ k0;
                c1[g] = static_cast<uint32_t>(b);
                c2[g] = static_cast<uint32_t>(a >> 32) ^ c3[g] ^ k1;
                c3[g] = static_cast<uint32_t>(a);
            }
            k0 += 0x9E3779B9u;
            k1 += 0xBB67AE85u;
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        d[g].w[0] = c0[g];
        d[g].w[1] = c1[g];
        d[g].w[2] = c2[g];
        d[g].w[3] = c3[g];
    }
}

__device__ __forceinline__ DropGroup drop_group(const DropKey &key, uint64_t group,
                                                uint32_t threshold) {
    DropGroup d[1];
    const uint64_t g[1] = {group};
    drop_groups<1>(d, key, g, threshold);
    return d[0];
}

// One element on its own.
__device__ __forceinline__ bool drop_keeps_element(const DropKey &key, int64_t e,
                                                   uint32_t threshold) {
    return drop_group(key, static_cast<uint64_t>(e) >> 3, threshold).keeps_any(static_cast<int>(e & 7));
}

// 1 / sqrt(v): within 2 units in the last place (rsqrtf), and 0 at infinity.  The IEEE
// square root and division would cost each thread of a row some forty instructions more.
__device__ __forceinline__ float inv_sqrt(float v) { return rsqrtf(v); }

// dropout(v).
__device__ __forceinline__ float drop_scale(float v, bool keep, float scale) {
    return keep ? v * scale : 0.0f;
}
// dropout(v), added to r: one rounding in f32.  A dropped value is not read
// into the sum, whatever it is (infinities and NaN included).
__device__ __forceinline__ float drop_add(float v, float r, bool keep, float scale) {
    return keep ? fmaf(v, scale, r) : r;
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float f2_sum(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return lo + hi;
}

// ---------------------------------------------------------------------------
// Sums over all threads of a CTA (a multiple of 32, at most 512), one barrier each: the
// slots alternate between calls, so that a call's writes never meet the reads
// of the call before it.  What stands behind the barrier is on every row's path: the fewer
// shuffles, the better.  cta_sum_setup, before the first sum, zeroes the slots of warps that
// the CTA does not have.
// ---------------------------------------------------------------------------
constexpr int kCtaWarps = 16;

// One value.
struct CtaSum {
    __align__(16) float v[2][kCtaWarps];
};
__device__ __forceinline__ void cta_sum_setup(CtaSum &s) {
    const int warp = static_cast<int>(blockDim.x >> 5) + static_cast<int>(threadIdx.x);
    if (warp < kCtaWarps) s.v[0][warp] = s.v[1][warp] = 0.0f;
}
__device__ __forceinline__ void cta_sum(float (&v)[1], CtaSum &s, int &turn) {
    const int lane = threadIdx.x & 31;
    const int p = ++turn & 1;
    v[0] = warp_allsum(v[0]);
    if (lane == 0) s.v[p][threadIdx.x >> 5] = v[0];
    __syncthreads();
    float t = s.v[p][lane & 7] + s.v[p][(lane & 7) + 8];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    v[0] = t;
}

// Two values: the first exchange leaves one value with each half of the warp, so that both take
// little more than the shuffles of one.  Joined by shuffles: the fewest registers (f32, RMSNorm).
struct CtaSumHalves {
    float v[2][2][32];
};
__device__ __forceinline__ void cta_sum_setup(CtaSumHalves &) {}
__device__ __forceinline__ void cta_sum(float (&v)[2], CtaSumHalves &s, int &turn) {
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int nwarps = blockDim.x >> 5;
    const int half = lane >> 4;
    const int p = ++turn & 1;
    float t = (half ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, half ? v[0] : v[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    if ((lane & 15) == 0) s.v[p][half][warp] = t;
    __syncthreads();
    t = (lane & 15) < nwarps ? s.v[p][half][lane & 15] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    v[0] = __shfl_sync(0xFFFFFFFFu, t, 0);
    v[1] = __shfl_sync(0xFFFFFFFFu, t, 16);
}

// Two values, a warp's side by side: every thread reads all the pairs, four warps in two loads,
// and adds them in order: one trip to shared memory in place of six shuffles, and more
// registers.  Measured on GB300, us a call, against halves: bf16 LayerNorm gradient 16384 x
// 4095 85.8 (90.5), the tail's 138 (144), the tail 16384 x 4096 88.8 (90.3), but RMSNorm's
// gradient 16384 x 4096, whose rows are read again behind the sums, 78.3 (72.9), and in f32 the
// tail's gradient 4096 x 6656, at the register limit, 100 (95).
struct CtaSumPairs {
    __align__(16) float v[2][kCtaWarps][2];
};
__device__ __forceinline__ void cta_sum_setup(CtaSumPairs &s) {
    const int warp = static_cast<int>(blockDim.x >> 5) + static_cast<int>(threadIdx.x);
    if (warp < kCtaWarps) s.v[0][warp][0] = s.v[0][warp][1] = s.v[1][warp][0] = s.v[1][warp][1] = 0.0f;
}
__device__ __forceinline__ void cta_sum(float (&v)[2], CtaSumPairs &s, int &turn) {
    const int lane = threadIdx.x & 31;
    const int half = lane >> 4;
    const int p = ++turn & 1;
    float t = (half ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, half ? v[0] : v[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    if ((lane & 15) == 0) s.v[p][threadIdx.x >> 5][half] = t;
    __syncthreads();
    const ulonglong2 *w = reinterpret_cast<const ulonglong2 *>(s.v[p]);
    const auto four = [&](int i) {
        const ulonglong2 a = w[i], b = w[i + 1];
        return f2_add(f2_add(a.x, a.y), f2_add(b.x, b.y));
    };
    uint64_t both = f2_add(four(0), four(2));
    if (blockDim.x > 256) both = f2_add(both, f2_add(four(4), four(6)));
    f2_unpack(both, v[0], v[1]);
}

// The form for N values.
template <int N, bool PAIRS> struct CtaSumOf { using Slots = CtaSum; };
template <> struct CtaSumOf<2, true> { using Slots = CtaSumPairs; };
template <> struct CtaSumOf<2, false> { using Slots = CtaSumHalves; };

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
    // elements 2 p and 2 p + 1 as an f32 pair, for the two-lane arithmetic
    __device__ __forceinline__ uint64_t pair(int p) const { return f2_pack(get(2 * p), get(2 * p + 1)); }
    __device__ __forceinline__ void put_pair(int p, uint64_t v) {
        float lo, hi;
        f2_unpack(v, lo, hi);
        if constexpr (T::kBytes == 4) {
            w[2 * p] = __float_as_uint(lo);
            w[2 * p + 1] = __float_as_uint(hi);
        } else {
            w[p] = pack_bf16x2(lo, hi);
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

// The same when `on` (predicated, no branch).
__device__ __forceinline__ void st_slot_if(bool on, void *p, const Slot<BF16> &s) {
    asm volatile("{.reg .pred q; setp.ne.u32 q, %5, 0; @q st.global.v4.b32 [%0], {%1,%2,%3,%4};}"
                 :: "l"(p), "r"(s.w[0]), "r"(s.w[1]), "r"(s.w[2]), "r"(s.w[3]),
                    "r"(static_cast<uint32_t>(on)) : "memory");
}
__device__ __forceinline__ void st_slot_if(bool on, void *p, const Slot<F32> &s) {
    asm volatile("{.reg .pred q; setp.ne.u32 q, %9, 0;"
                 " @q st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};}"
                 :: "l"(p), "r"(s.w[0]), "r"(s.w[1]), "r"(s.w[2]), "r"(s.w[3]), "r"(s.w[4]),
                    "r"(s.w[5]), "r"(s.w[6]), "r"(s.w[7]), "r"(static_cast<uint32_t>(on)) : "memory");
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
