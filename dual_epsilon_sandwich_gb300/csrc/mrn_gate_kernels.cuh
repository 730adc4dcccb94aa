// mrn_gate_kernels.cuh -- device code shared by the gated tail and its
// gradient: the factors, and sums of six values over a CTA.
#pragma once

#include "mrn_gate.h"
#include "mrn_row_tile.cuh"

namespace mrn {

// Element (r, j) of a factor.
template <class T> __device__ __forceinline__ float factor_at(const Factor &f, int64_t r, int64_t j) {
    if (f.kind == MRN_FACTOR_NONE) return 1.0f;
    return ld_elem<T>(f.p, f.kind == MRN_FACTOR_CHANNEL ? j : (f.kind == MRN_FACTOR_ROW ? r : 0));
}

// Sums of six values over a warp, eight shuffles: each exchange halves the values that a lane
// still adds up.  Lane 0 ends with the sum of v[0], 16 with v[1]'s, 8 with v[2]'s, 24 with
// v[3]'s, 4 with v[4]'s, 20 with v[5]'s (and lanes near them with the same).
__device__ __forceinline__ float warp_sum_six(const float (&v)[6], int lane) {
    float a[3];
#pragma unroll
    for (int i = 0; i < 3; ++i)
        a[i] = ((lane & 16) ? v[2 * i + 1] : v[2 * i]) +
               __shfl_xor_sync(0xFFFFFFFFu, (lane & 16) ? v[2 * i] : v[2 * i + 1], 16);
    float b = ((lane & 8) ? a[1] : a[0]) + __shfl_xor_sync(0xFFFFFFFFu, (lane & 8) ? a[0] : a[1], 8);
    const float c = a[2] + __shfl_xor_sync(0xFFFFFFFFu, a[2], 8);
    b = ((lane & 4) ? c : b) + __shfl_xor_sync(0xFFFFFFFFu, (lane & 4) ? b : c, 4);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, 2);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, 1);
    return b;
}
// The value whose sum warp_sum_six leaves with this lane; -1: none (of lanes that are a multiple
// of four, which all have one, 12 and 28 hold what 4 and 20 do).
__device__ __forceinline__ int sum_six_index(int lane) {
    if (lane & 3) return -1;
    if (lane & 4) return (lane & 8) ? -1 : 4 + (lane >> 4);
    return (lane >> 4) + ((lane & 8) ? 2 : 0);
}

// ... and all six for all lanes.
__device__ __forceinline__ void from_lanes(float (&v)[6], float t) {
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, t, i < 4 ? (i & 1) * 16 + (i >> 1) * 8 : (i & 1) * 16 + 4);
}

// Six values over a CTA of at most 16 warps: one barrier; behind it each lane adds four warps' sums
// of one value, two shuffles join them and six hand them to all lanes.
struct CtaSumSix {
    __align__(16) float v[2][6][kCtaWarps];
};
__device__ __forceinline__ void cta_sum_setup(CtaSumSix &s) {
    const int warp = static_cast<int>(blockDim.x >> 5) + static_cast<int>(threadIdx.x);
    if (warp < kCtaWarps) {
#pragma unroll
        for (int i = 0; i < 6; ++i) s.v[0][i][warp] = s.v[1][i][warp] = 0.0f;
    }
}
__device__ __forceinline__ void cta_sum(float (&v)[6], CtaSumSix &s, int &turn) {
    const int lane = threadIdx.x & 31;
    const int p = ++turn & 1;
    const float w = warp_sum_six(v, lane);
    const int mine = sum_six_index(lane);
    if (mine >= 0) s.v[p][mine][threadIdx.x >> 5] = w;
    __syncthreads();
    const int of = lane >> 2 < 6 ? lane >> 2 : 5;
    const float4 q = *reinterpret_cast<const float4 *>(&s.v[p][of][(lane & 3) * 4]);
    float t = (q.x + q.y) + (q.z + q.w);
    t += __shfl_xor_sync(0xFFFFFFFFu, t, 1);
    t += __shfl_xor_sync(0xFFFFFFFFu, t, 2);
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, t, 4 * i);
}

template <> struct CtaSumOf<6, false> { using Slots = CtaSumSix; };

// row_sum of six values, with fewer shuffles behind a cluster's messages.
template <bool WARP>
__device__ __forceinline__ bool row_sum_six(float (&v)[6], RowSumSlots<6, false> &s, int &turn, int width,
                                            unsigned cl, unsigned crank, uint32_t stall) {
    if constexpr (WARP) {
        if (width == 32) {
            const float t = warp_sum_six(v, static_cast<int>(threadIdx.x & 31));
            from_lanes(v, t);
            return true;
        }
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = group_allsum(v[i], width);
    } else {
        cta_sum(v, s.cta, turn);
        if (cl > 1) {
            const int p = turn & 1;
            const unsigned lane = threadIdx.x & 31;
            if (threadIdx.x == 0) mbar_arrive_expect_tx(&s.bar[p], (cl - 1) * 24u + stall);
            if (threadIdx.x < cl && threadIdx.x != crank) {
#pragma unroll
                for (int i = 0; i < 6; ++i) send_f32(&s.box[p][i][crank], &s.bar[p], threadIdx.x, v[i]);
            }
            const bool late = !mbar_wait_bounded_cluster(&s.bar[p], static_cast<uint32_t>((turn - 1) >> 1 & 1));
            float x[6];
#pragma unroll
            for (int i = 0; i < 6; ++i) x[i] = lane >= cl ? 0.0f : (lane == crank ? v[i] : s.box[p][i][lane]);
            const float t = warp_sum_six(x, static_cast<int>(lane));
            from_lanes(v, t);
            if (__syncthreads_or(late)) {
                if (threadIdx.x == 0) atomicAdd(&g_wait_timeouts, 1u);
                return false;
            }
        }
    }
    return true;
}

// A gate of one value per row travels with its row: one word per lanes that copy together (bf16:
// the word that holds the element).  A load of it in the loop would hold up every row.
template <bool EDGE, bool WARP> struct RowGates {
    static constexpr int kTeams = !WARP ? kCtaWarps : (EDGE ? kWarpTileThreads / kEndLanes : kWarpTileThreads);
    uint32_t w[kTileMaxStages][kTeams];
};
template <class T> __device__ __forceinline__ uintptr_t row_gate_at(const Factor &gate, int64_t row) {
    return reinterpret_cast<uintptr_t>(gate.p) + static_cast<uintptr_t>(row * T::kBytes);
}
template <class T> __device__ __forceinline__ void copy_row_gate(uint32_t *to, const Factor &gate, int64_t row) {
    cp_async4(smem_addr(to), reinterpret_cast<const void *>(row_gate_at<T>(gate, row) & ~uintptr_t(3)));
}
template <class T> __device__ __forceinline__ float row_gate(uint32_t w, const Factor &gate, int64_t row) {
    if constexpr (T::kBytes == 4) return __uint_as_float(w);
    return __uint_as_float((row_gate_at<T>(gate, row) & 2) ? w & 0xFFFF0000u : w << 16);
}

// gamma_post of a thread's columns, times the gate of a channel, in f32.
template <class T, int K, class Tile>
__device__ __forceinline__ void block_weights(uint64_t (&c)[K][4], const Tile &tile, const void *g1, const Factor &gate) {
    Slot<T> g[K];
    tile.weights(g, g1);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[k][i] = g[k].pair(i);
    if (gate.kind == MRN_FACTOR_CHANNEL) {
        tile.weights(g, gate.p);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[k][i] = f2_mul(c[k][i], g[k].pair(i));
    }
}
template <class Tile>
__device__ __forceinline__ float end_block_weight(const Tile &tile, const void *g1, const Factor &gate) {
    const float g = tile.end_weight(g1);
    return gate.kind == MRN_FACTOR_CHANNEL ? g * tile.end_weight(gate.p) : g;
}
// A factor that all rows and channels share; one where it is not of that kind.
template <class T> __device__ __forceinline__ float scalar_factor(const Factor &f) {
    return f.kind == MRN_FACTOR_SCALAR ? ld_elem<T>(f.p, 0) : 1.0f;
}

}  // namespace mrn
