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

}  // namespace mrn
