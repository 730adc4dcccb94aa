// mrn_gate_forward.cu -- the dual-epsilon sandwich tail with a gate on the
// block and a scale on the residual:
//   stream = scale * res + gate * g1 * b * inv(b; eps1), rounded once and stored
//   y = stream * inv(stream; eps2) * g2
// with inv(v; eps) = 1 / sqrt(sum_j v_j^2 / n + eps).
#include "mrn_gate_kernels.cuh"

namespace mrn {

constexpr int kLoopedThreads = 512;

// Any width and any alignment: one row per CTA at a time, three passes over it (the second and
// third out of L2), element by element.
template <class T>
__global__ void __launch_bounds__(kLoopedThreads) mrn_gate_looped_kernel(const GateArgs a) {
    __shared__ CtaSum slots;
    cta_sum_setup(slots);
    pdl_enter();
    int turn = 0;
    const float count = static_cast<float>(a.n);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t e0 = r * a.n;
        float sum[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const float v = ld_elem<T>(a.b, e0 + j);
            sum[0] = fmaf(v, v, sum[0]);
        }
        cta_sum(sum, slots, turn);
        float k = 1.0f / sqrtf(sum[0] / count + a.eps1);
        if (a.gate.kind != MRN_FACTOR_CHANNEL) k *= factor_at<T>(a.gate, r, 0);
        sum[0] = 0.0f;
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            float c = ld_elem<T>(a.g1, j);
            if (a.gate.kind == MRN_FACTOR_CHANNEL) c *= factor_at<T>(a.gate, r, j);
            const float t = factor_at<T>(a.scale, r, j) * ld_elem<T>(a.res, e0 + j);
            const float v = st_elem<T>(a.stream_out, e0 + j, fmaf(ld_elem<T>(a.b, e0 + j) * k, c, t));
            sum[0] = fmaf(v, v, sum[0]);
        }
        cta_sum(sum, slots, turn);
        const float inv = 1.0f / sqrtf(sum[0] / count + a.eps2);
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x)
            st_elem<T>(a.y, e0 + j, ld_elem<T>(a.stream_out, e0 + j) * inv * ld_elem<T>(a.g2, j));
    }
}

// Threads that an SM's registers are shared between (the launch bound), from what a thread
// holds: k slots of r rows, of gamma_post with the gate in f32, of gamma_pre and, ACH, of a
// scale per channel.
template <class T> constexpr int gate_resident(int k, int r, bool ach) {
    const int words = k * ((r + 1 + ach) * Slot<T>::kWords + 8);
    return words <= 16 ? 1024 : (words <= 32 ? 768 : (words <= 44 ? 640 : (words <= 72 ? 512 : (words <= 104 ? 384 : 256))));
}
template <class T> constexpr int gate_threads(int k, int r, bool ach) {
    return gate_resident<T>(k, r, ach) < 512 ? gate_resident<T>(k, r, ach) : 512;
}

// Rows held in registers between their copy and their outputs (see mrn_row_tile.cuh): every
// operand is read once, every output written once, and a row has two sums, the second over the
// rounded stream.
template <class T, int K, int R, bool EDGE, bool WARP, bool ACH>
__global__ void __launch_bounds__(gate_resident<T>(K, R, ACH))
mrn_gate_tile_kernel(const GateArgs a, const TileArgs t) {
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    __shared__ RowSumSlots<R, T::kBytes == 2> slots;
    __shared__ EndSlots<2, R, EDGE, WARP> end_w;
    __shared__ RowGates<R, EDGE, WARP> gates;
    RowTile<T, K, R, EDGE, WARP> tile(a.rows, a.n, t);
    const int64_t back = static_cast<int64_t>(t.mis) * T::kBytes;
    const char *const ops[2] = {static_cast<const char *>(a.b) - back, static_cast<const char *>(a.res) - back};
    char *const y = static_cast<char *>(a.y) - back;
    char *const stream_out = static_cast<char *>(a.stream_out) - back;
    RingWalk walk(tile.stage_bytes(2), t.stages);
    const int ahead = t.stages - 1;
    const uint32_t ring = tile.warp_ring(static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes)), t.stages, 2);
    const bool by_row = a.gate.kind == MRN_FACTOR_ROW;
    tile.clear(ring, t.stages, 2);
    row_sum_setup(slots, tile.cl);
    pdl_enter();
    int64_t gate_row = tile.row;
    auto issue = [&](int to) {
        if (by_row && tile.leads) {
#pragma unroll
            for (int rr = 0; rr < R; ++rr)
                if (rr < tile.copy_left)
                    copy_row_gate<T>(&gates.w[to][rr][tile.team], a.gate, gate_row + rr * tile.stride);
        }
        gate_row += R * tile.stride;
        tile.issue(ring + to * walk.bytes, to, ops, 2, end_w);
    };
    for (int s = 0; s < ahead; ++s) issue(s);
    uint64_t c[K][4];
    Slot<T> g2[K], alpha[ACH ? K : 1];
    block_weights<T>(c, tile, a.g1, a.gate);
    tile.weights(g2, a.g2);
    if constexpr (ACH) tile.weights(alpha, a.scale.p);
    const float gate = scalar_factor<T>(a.gate);
    const float scale = ACH ? 1.0f : scalar_factor<T>(a.scale);
    const float end_c = EDGE ? end_block_weight(tile, a.g1, a.gate) : 0.0f;
    const float end_g2 = EDGE ? tile.end_weight(a.g2) : 0.0f;
    const float end_alpha = EDGE && ACH ? tile.end_weight(a.scale.p) : scale;
    row_sum_ready(tile.cl);
    const float inv_n = 1.0f / static_cast<float>(a.n);
    const uint64_t scale2 = f2_pack(scale, scale);
    int turn = 0;
    for (; tile.cta_left > 0; tile.advance(), walk.next()) {
        __syncwarp();
        issue(walk.write);
        cp_async_wait(ahead);
        __syncwarp();
        const uint32_t from = ring + walk.read * walk.bytes;
        Slot<T> v[R][K];
        float sum[R], end[R], row_g[R];
#pragma unroll
        for (int rr = 0; rr < R; ++rr) {
            tile.fetch(v[rr], from, 0, rr, 2);
            uint64_t acc = 0;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc = f2_fma(v[rr][k].pair(i), v[rr][k].pair(i), acc);
            sum[rr] = f2_sum(acc);
            end[rr] = 0.0f;
            if (EDGE && tile.ends) {
                end[rr] = tile.fetch_end(end_w, walk.read, 0, rr);
                sum[rr] = fmaf(end[rr], end[rr], sum[rr]);
            }
            row_g[rr] = by_row && (!WARP || tile.valid(rr))
                            ? row_gate<T>(gates.w[walk.read][rr][tile.team], a.gate, tile.row + rr * tile.stride)
                            : gate;
        }
        if (!row_sum<WARP>(sum, slots, turn, tile.width, tile.cl, tile.crank, turn == 0 ? t.stall : 0u)) break;
#pragma unroll
        for (int rr = 0; rr < R; ++rr) {
            const float m = inv_sqrt(fmaf(sum[rr], inv_n, a.eps1)) * row_g[rr];
            const uint64_t m2 = f2_pack(m, m);
            Slot<T> res[K];
            tile.fetch(res, from, 1, rr, 2);
            uint64_t acc = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t r = f2_mul(res[k].pair(i), ACH ? alpha[ACH ? k : 0].pair(i) : scale2);
                    v[rr][k].put_pair(i, f2_fma(f2_mul(v[rr][k].pair(i), m2), c[k][i], r));
                    acc = f2_fma(v[rr][k].pair(i), v[rr][k].pair(i), acc);
                }
            }
            tile.store(stream_out, rr, tile.valid(rr), v[rr]);
            sum[rr] = f2_sum(acc);
            if (EDGE && tile.ends) {
                const float o = fmaf(end[rr] * m, end_c, end_alpha * tile.fetch_end(end_w, walk.read, 1, rr));
                end[rr] = tile.store_end(stream_out, rr, tile.valid(rr), o);
                if (tile.end_col < 0) end[rr] = 0.0f;
                sum[rr] = fmaf(end[rr], end[rr], sum[rr]);
            }
        }
        if (!row_sum<WARP>(sum, slots, turn, tile.width, tile.cl, tile.crank, 0u)) break;
#pragma unroll
        for (int rr = 0; rr < R; ++rr) {
            const float m = inv_sqrt(fmaf(sum[rr], inv_n, a.eps2));
            const uint64_t m2 = f2_pack(m, m);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[rr][k].put_pair(i, f2_mul(f2_mul(v[rr][k].pair(i), m2), g2[k].pair(i)));
            tile.store(y, rr, tile.valid(rr), v[rr]);
            if (EDGE && tile.ends) tile.store_end(y, rr, tile.valid(rr), end[rr] * m * end_g2);
        }
    }
    cp_async_wait(0);
    row_sum_leave(tile.cl);
}

// Whether the call was launched; false: it takes the looped kernel.
template <class T, int K, int R, bool EDGE, bool WARP, bool ACH>
bool launch_gate_tile(const GateArgs &a, const TileShape &p, int sms, bool pdl, cudaStream_t stream,
                      uint64_t *launches, cudaError_t *err) {
    static TileLaunchCache cache;
    const auto fn = mrn_gate_tile_kernel<T, K, R, EDGE, WARP, ACH>;
    TileGrid g;
    *err = tile_grid(cache, fn, p, a.rows, a.n, R, T::kBytes, 2, 32, sms, &g);
    if (*err != cudaSuccess) return true;
    if (g.stages < 1) return false;
    const TileArgs t = {p.lanes, g.stages, p.mis, a.stall};
    *err = launch_tile(fn, p, g.ctas, g.shared, pdl, stream, launches, a, t);
    return true;
}

template <class T, int K, int R, bool WARP>
bool launch_gate_k(const GateArgs &a, const TileShape &p, int sms, bool pdl, cudaStream_t stream,
                   uint64_t *launches, cudaError_t *err) {
    if (a.scale.kind == MRN_FACTOR_CHANNEL)
        return p.edge ? launch_gate_tile<T, K, R, true, WARP, true>(a, p, sms, pdl, stream, launches, err)
                      : launch_gate_tile<T, K, R, false, WARP, true>(a, p, sms, pdl, stream, launches, err);
    return p.edge ? launch_gate_tile<T, K, R, true, WARP, false>(a, p, sms, pdl, stream, launches, err)
                  : launch_gate_tile<T, K, R, false, WARP, false>(a, p, sms, pdl, stream, launches, err);
}

template <class T>
cudaError_t launch_gate_typed(const GateArgs &a, int sms, bool pdl, cudaStream_t stream, uint64_t *launches) {
    const int mis = common_offset(T::kBytes, a.b, a.res, static_cast<const void *>(a.stream_out),
                                  static_cast<const void *>(a.y));
    if (mis >= 0) {
        const int64_t slots = a.n / 8;
        const bool ach = a.scale.kind == MRN_FACTOR_CHANNEL;
        int k = T::kBytes == 2 ? (slots <= 512 ? 2 : 4) : (slots <= 512 ? 1 : (slots <= 1024 ? 2 : 4));
        int most_threads = gate_threads<T>(k, 1, ach);
        if (T::kBytes == 4 && slots > 1536) k = 2, most_threads = 256;
        if (T::kBytes == 2 && slots > 2048) most_threads = 128;
        while (most_threads < gate_threads<T>(k, 1, ach) && slots > int64_t(kMaxCluster) * k * most_threads) most_threads *= 2;
        if (most_threads > gate_threads<T>(k, 1, ach)) most_threads = gate_threads<T>(k, 1, ach);
        const bool few = tile_few_rows(a.rows, a.n, sms);
        if (few) {
            k = 1;
            most_threads = tile_few_threads(a.rows, a.n, sms);
        }
        const TileShape p = tile_shape(a.n, mis, k, most_threads, few);
        cudaError_t err = cudaSuccess;
        bool done = false;
        if (p.ok && p.warp) {
            done = p.k == 1   ? launch_gate_k<T, 1, 1, true>(a, p, sms, pdl, stream, launches, &err)
                   : p.k == 2 ? launch_gate_k<T, 2, 1, true>(a, p, sms, pdl, stream, launches, &err)
                   : p.k == 3 ? launch_gate_k<T, 3, 1, true>(a, p, sms, pdl, stream, launches, &err)
                              : launch_gate_k<T, 4, 1, true>(a, p, sms, pdl, stream, launches, &err);
        } else if (p.ok) {
            done = k == 1   ? launch_gate_k<T, 1, 1, false>(a, p, sms, pdl, stream, launches, &err)
                   : k == 2 ? launch_gate_k<T, 2, 1, false>(a, p, sms, pdl, stream, launches, &err)
                            : launch_gate_k<T, 4, 1, false>(a, p, sms, pdl, stream, launches, &err);
        }
        if (done) return err;
    }
    const int64_t ctas = a.rows < 4LL * sms ? a.rows : 4LL * sms;
    return launch_plain(mrn_gate_looped_kernel<T>, ctas, kLoopedThreads, 0, pdl, stream, launches, a);
}

cudaError_t launch_gate(bool bf16, const GateArgs &a, int sms, bool pdl, cudaStream_t stream,
                        uint64_t *launches) {
    return bf16 ? launch_gate_typed<BF16>(a, sms, pdl, stream, launches)
                : launch_gate_typed<F32>(a, sms, pdl, stream, launches);
}

int take_wait_timeouts_gate() { return take_wait_timeouts<kOpGateTimeouts>(); }

}  // namespace mrn
