// mrn_gate_forward.cu -- the dual-epsilon sandwich tail with a gate on the
// block and a scale on the residual:
//   stream = scale * res + gate * g1 * b * inv(b; eps1), rounded once and stored
//   y = stream * inv(stream; eps2) * g2
// with inv(v; eps) = 1 / sqrt(sum_j v_j^2 / n + eps).
#include "mrn_gate_kernels.cuh"

namespace mrn {

constexpr int kLoopedThreads = 512;

// Any width and any alignment: one row per CTA at a time, three passes over it (the second and
// third out of L2), element by element.  For operands that do not share an offset and rows wider
// than a cluster holds.  Bound by its accesses of one element: 16384 x 4096 bf16 414 us (the tiles:
// 89).
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
// holds: k slots of the row, of gamma_post with the gate in f32, of gamma_pre and, ACH, of a
// scale per channel, and what rows that share a warp take beside them (distances of their own: without
// it eight bf16 forms spilled, and 65536 x 1023 took 124 us against 100, 65536 x 511 56 against 45; two
// still do, four slots with a scale per channel).
template <class T> constexpr int gate_resident(int k, bool ach, bool warp) {
    const int words = k * ((2 + ach) * Slot<T>::kWords + 8) + (warp ? 20 : 0);
    return words <= 16 ? 1024 : (words <= 32 ? 768 : (words <= 44 ? 640 : (words <= 72 ? 512 : (words <= 104 ? 384 : 256))));
}
template <class T> constexpr int gate_threads(int k, bool ach) {
    return gate_resident<T>(k, ach, false) < 512 ? gate_resident<T>(k, ach, false) : 512;
}

// Stages of the tiles' ring at most: with more copies in flight than two stages of each CTA, reads and
// writes get in each other's way in DRAM (4096 x 6655 f32 78.9 us with four, 76.5 with two; 16384 x
// 4095 bf16 93.1, 89.0; 32768 x 4096 f32 351, 332; but one slot of bf16, 16384 x 4096, 87.6 and 89.0).
constexpr int kGateStages = 2;
// Threads of the row kernel at most (two CTAs of that size share an SM's registers).
constexpr int kGateRowThreads = 32 * kCtaWarps;

__device__ __forceinline__ void ld_weights(Slot<BF16> &s, const void *p) {
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]) : "l"(p));
}
__device__ __forceinline__ void ld_weights(Slot<F32> &s, const void *p) {
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]) : "l"(p));
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4+16];"
                 : "=r"(s.w[4]), "=r"(s.w[5]), "=r"(s.w[6]), "=r"(s.w[7]) : "l"(p));
}

// Rows held in registers between their copy and their outputs (see mrn_row_tile.cuh): every
// operand is read once, every output written once, and a row has two sums, the second over the
// rounded stream.  ACH: the residual has a scale per channel.  Measured on GB300: 16384 x 4096 bf16
// 88 to 90 us (6.0 TB/s, 88 % of the copy's rate), 4096 x 6655 f32 73 to 75 us (5.9 TB/s), 1 x 6656 f32
// 2.7 us, a launch and two sums over a cluster.
//   What bounds it: bf16 the instructions (issued in 68 % of cycles, the conversions most of them),
// f32 at odd pitches 13 warps that wait for shared memory and the barrier, and everywhere what reads
// ahead and writes of a persistent grid cost in DRAM: aligned f32 rows take 10 % less in the kernel
// below, whose CTAs come and go.
template <class T, int K, bool EDGE, bool WARP, bool ACH>
__global__ void __launch_bounds__(gate_resident<T>(K, ACH, WARP))
mrn_gate_tile_kernel(const GateArgs a, const TileArgs t) {
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    __shared__ RowSumSlots<1, T::kBytes == 2> slots;
    __shared__ EndSlots<2, 1, EDGE, WARP> end_w;
    __shared__ RowGates<EDGE, WARP> gates;
    RowTile<T, K, 1, EDGE, WARP> tile(a.rows, a.n, t);
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
        if (by_row && tile.leads && tile.copy_left > 0) copy_row_gate<T>(&gates.w[to][tile.team], a.gate, gate_row);
        gate_row += tile.stride;
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
        const bool ok = !WARP || tile.valid(0);
        Slot<T> v[K];
        tile.fetch(v, from, 0, 0, 2);
        uint64_t acc = 0;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = f2_fma(v[k].pair(i), v[k].pair(i), acc);
        float sum[1] = {f2_sum(acc)};
        float end = 0.0f;
        if (EDGE && tile.ends) {
            end = tile.fetch_end(end_w, walk.read, 0, 0);
            sum[0] = fmaf(end, end, sum[0]);
        }
        const float row_g = by_row && ok ? row_gate<T>(gates.w[walk.read][tile.team], a.gate, tile.row) : gate;
        if (!row_sum<WARP>(sum, slots, turn, tile.width, tile.cl, tile.crank, turn == 0 ? t.stall : 0u)) break;
        float m = inv_sqrt(fmaf(sum[0], inv_n, a.eps1)) * row_g;
        uint64_t m2 = f2_pack(m, m);
        Slot<T> res[K];
        tile.fetch(res, from, 1, 0, 2);
        acc = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t r = f2_mul(res[k].pair(i), ACH ? alpha[ACH ? k : 0].pair(i) : scale2);
                v[k].put_pair(i, f2_fma(f2_mul(v[k].pair(i), m2), c[k][i], r));
                acc = f2_fma(v[k].pair(i), v[k].pair(i), acc);
            }
        }
        tile.store(stream_out, 0, ok, v);
        sum[0] = f2_sum(acc);
        if (EDGE && tile.ends) {
            const float o = fmaf(end * m, end_c, end_alpha * tile.fetch_end(end_w, walk.read, 1, 0));
            end = tile.store_end(stream_out, 0, ok, o);
            if (tile.end_col < 0) end = 0.0f;
            sum[0] = fmaf(end, end, sum[0]);
        }
        if (!row_sum<WARP>(sum, slots, turn, tile.width, tile.cl, tile.crank, 0u)) break;
        m = inv_sqrt(fmaf(sum[0], inv_n, a.eps2));
        m2 = f2_pack(m, m);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k].put_pair(i, f2_mul(f2_mul(v[k].pair(i), m2), g2[k].pair(i)));
        tile.store(y, 0, ok, v);
        if (EDGE && tile.ends) tile.store_end(y, 0, ok, end * m * end_g2);
    }
    cp_async_wait(0);
    row_sum_leave(tile.cl);
}

// Whether the call was launched; false: it takes the looped kernel.
template <class T, int K, bool EDGE, bool WARP, bool ACH>
bool launch_gate_tile(const GateArgs &a, const TileShape &p, int sms, bool pdl, cudaStream_t stream,
                      uint64_t *launches, cudaError_t *err) {
    static TileLaunchCache cache;
    const auto fn = mrn_gate_tile_kernel<T, K, EDGE, WARP, ACH>;
    TileGrid g;
    *err = tile_grid(cache, fn, p, a.rows, a.n, 1, T::kBytes, 2, 32, sms, &g, 0,
                     T::kBytes == 2 && K == 1 && !EDGE && !WARP ? kTileMaxStages : kGateStages);
    if (*err != cudaSuccess) return true;
    if (g.stages < 1) return false;
    const TileArgs t = {p.lanes, g.stages, p.mis, a.stall};
    *err = launch_tile(fn, p, g.ctas, g.shared, pdl, stream, launches, a, t);
    return true;
}

template <class T, int K, bool WARP>
bool launch_gate_k(const GateArgs &a, const TileShape &p, int sms, bool pdl, cudaStream_t stream,
                   uint64_t *launches, cudaError_t *err) {
    if (a.scale.kind == MRN_FACTOR_CHANNEL)
        return p.edge ? launch_gate_tile<T, K, true, WARP, true>(a, p, sms, pdl, stream, launches, err)
                      : launch_gate_tile<T, K, false, WARP, true>(a, p, sms, pdl, stream, launches, err);
    return p.edge ? launch_gate_tile<T, K, true, WARP, false>(a, p, sms, pdl, stream, launches, err)
                  : launch_gate_tile<T, K, false, WARP, false>(a, p, sms, pdl, stream, launches, err);
}

// One row per CTA, K slots of eight elements to a thread, nothing kept from row to row: aligned
// rows only.  The grid holds all rows, and an SM as many of them as its registers do; the weights come
// out of L1 for each row, behind the barriers, where the row's own registers are free for them.
// Measured on GB300: 8192 x 4096 f32 80.8 us (6.65 TB/s, 98 % of the copy's rate), 4096 x 6656 f32 70 to
// 71 (a gate per channel; 66.7 without one, 96 %), 32768 x 2048 bf16 85.6 (6.3 TB/s).
//   What bounds it: memory; at 6656, where two CTAs fill an SM's registers, the waits for the weights
// behind the barriers (long scoreboard 12 cycles per issue).  Rows of fewer bytes than 8 KB would be
// bound by the start of their CTAs, about one a nanosecond: they take the tiles.
template <class T, int K>
__global__ void __launch_bounds__(kGateRowThreads, 2)
mrn_gate_row_kernel(const GateArgs a) {
    __shared__ CtaSum slots;
    cta_sum_setup(slots);
    const int lane = threadIdx.x & 31;
    const int first = (static_cast<int>(threadIdx.x) - lane) * K + lane;     // a warp's slots are consecutive
    const int count = static_cast<int>(a.n / 8);
    const int64_t row = blockIdx.x;
    const int64_t e0 = row * a.n + first * 8;
    pdl_enter();
    Slot<T> b[K], res[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        b[k].zero();
        res[k].zero();
        if (first + 32 * k < count) {
            ld_slot(b[k], elem_ptr<T>(a.b, e0 + 256 * k));
            ld_slot(res[k], elem_ptr<T>(a.res, e0 + 256 * k));
        }
    }
    const bool channel = a.gate.kind == MRN_FACTOR_CHANNEL, scaled = a.scale.kind == MRN_FACTOR_CHANNEL;
    const float gate = channel ? 1.0f : factor_at<T>(a.gate, row, 0);
    const float scale = scaled ? 1.0f : factor_at<T>(a.scale, row, 0);
    const float inv_n = 1.0f / static_cast<float>(a.n);
    uint64_t acc = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = f2_fma(b[k].pair(i), b[k].pair(i), acc);
    float sum[1] = {f2_sum(acc)};
    int turn = 0;
    cta_sum(sum, slots, turn);
    const float m = inv_sqrt(fmaf(sum[0], inv_n, a.eps1)) * gate;
    const uint64_t m2 = f2_pack(m, m), scale2 = f2_pack(scale, scale);
    acc = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (first + 32 * k >= count) continue;
        Slot<T> g, f;
        const int64_t j = (first + 32 * k) * 8;
        ld_weights(g, elem_ptr<T>(a.g1, j));
        uint64_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = g.pair(i);
        if (channel) {
            ld_weights(f, elem_ptr<T>(a.gate.p, j));
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = f2_mul(c[i], f.pair(i));
        }
        if (scaled) ld_weights(f, elem_ptr<T>(a.scale.p, j));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t r = f2_mul(res[k].pair(i), scaled ? f.pair(i) : scale2);
            b[k].put_pair(i, f2_fma(f2_mul(b[k].pair(i), m2), c[i], r));
            acc = f2_fma(b[k].pair(i), b[k].pair(i), acc);
        }
        st_slot(elem_ptr<T>(a.stream_out, e0 + 256 * k), b[k]);
    }
    sum[0] = f2_sum(acc);
    cta_sum(sum, slots, turn);
    const float v = inv_sqrt(fmaf(sum[0], inv_n, a.eps2));
    const uint64_t v2 = f2_pack(v, v);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (first + 32 * k >= count) continue;
        Slot<T> g;
        ld_weights(g, elem_ptr<T>(a.g2, (first + 32 * k) * 8));
#pragma unroll
        for (int i = 0; i < 4; ++i) b[k].put_pair(i, f2_mul(f2_mul(b[k].pair(i), v2), g.pair(i)));
        st_slot(elem_ptr<T>(a.y, e0 + 256 * k), b[k]);
    }
}

// Slots per thread of the row kernel; 0: the call takes the tiles.  It needs rows and weights on
// 16-byte boundaries (32 of f32 rows).  Measured on GB300 beside the tiles (us, gate per channel):
//   up to two rows per SM, one slot: f32 1 x 768 1.7 (2.0), 1 x 4096 2.5 (2.7), 64 x 4096 2.6 (3.3), 300
//     x 4096 5.7 (6.5);  bf16 64 x 768 1.9 (2.2), 300 x 4096 3.0 (3.6), but 1000 x 4096 11.8 (8.6)
//   f32 batches: n = 384 69.3 (67.7), 512 78.7 (89.0), 768 78.6 (90.3), 1024 one slot 78.7, two 79.9
//     (90.3), 1032 89.0, 81.4 (95.8), 1536 80.1 (89.7), 4096 80.8 (88.2), 6656 70.8 (71.3), 8192
//     84.9 (90.2);  without a gate 6656 66.7 (71.8)
//   bf16 batches, two slots: n = 768 72.8 (68.8), 1024 84.9 (100.5), 1280 116 (112), 1536 87.2 (92.0),
//     1792 90.2 (90.3), 2048 85.6 (90.7), 2304 92.9 (91.0), 4096 89.7 (89.0): only where whole warps are
//     filled; below, the CTAs of a row each come at most one a nanosecond
template <class T> int gate_row_slots(const GateArgs &a, int mis, int sms) {
    const auto off = [](const Factor &f) {
        return f.kind == MRN_FACTOR_CHANNEL ? reinterpret_cast<uintptr_t>(f.p) : uintptr_t(0);
    };
    const uintptr_t weights = reinterpret_cast<uintptr_t>(a.g1) | reinterpret_cast<uintptr_t>(a.g2) | off(a.gate) | off(a.scale);
    if (mis != 0 || a.n % 8 != 0 || weights % 16 != 0 || a.rows > 0x7FFFFFFF) return 0;
    const int64_t slots = a.n / 8;
    if (a.rows <= 2LL * sms && slots > 16 && slots <= kGateRowThreads) return 1;
    if (a.rows <= sms) return 0;
    if (T::kBytes == 2) return slots >= 128 && slots <= 256 && slots % 64 == 0 ? 2 : 0;
    return slots < 64 || slots > 2 * kGateRowThreads ? 0 : (slots <= 128 ? 1 : 2);
}

template <class T, int K>
cudaError_t launch_gate_row(const GateArgs &a, bool pdl, cudaStream_t stream, uint64_t *launches) {
    const int threads = static_cast<int>((a.n / 8 + 32 * K - 1) / (32 * K)) * 32;
    return launch_plain(mrn_gate_row_kernel<T, K>, a.rows, threads, 0, pdl, stream, launches, a);
}

// Slots per thread (k) for rows of a CTA, and threads of one at most.  Measured on GB300 (us, k 1, 2,
// 4; 537 MB a call, 436 at 6655):
//   bf16  n = 2560 93.0, 92.9, 91.9;  4095 108, 90.3, 90.3;  4096 87.6, 92.1, 90.3;  5120 113, 93.7,
//         91.0;  6656 116, 95.8, 92.4;  8192 125, 87.5, 91.7;  4096 with a scale per channel 103, 93.1, 92.0
//   f32   n = 1032 99.2, 99.2, 96.1;  4095 89.6, 97.0, 97.8;  6655 113, 76.5, 76.4;  12288 122, 97.2, 92.4
template <class T> void gate_tile(int64_t slots, bool edge, bool ach, int *k, int *threads) {
    if (T::kBytes == 2) {
        *k = slots > 448 && slots <= 512 && !edge && !ach ? 1 : (slots >= 960 && slots <= 1024 ? 2 : 4);
        *threads = slots > 2048 ? 128 : 512;
    } else {
        *k = slots <= 512 ? 1 : (slots <= 1024 || slots > 1536 ? 2 : 4);
        *threads = slots > 1536 ? 256 : 512;
    }
    const int most = gate_threads<T>(*k, ach);
    while (*threads < most && slots > int64_t(kMaxCluster) * *k * *threads) *threads *= 2;
    if (*threads > most) *threads = most;
}

template <class T>
cudaError_t launch_gate_typed(const GateArgs &a, int sms, bool pdl, cudaStream_t stream, uint64_t *launches) {
    const int mis = common_offset(T::kBytes, a.b, a.res, static_cast<const void *>(a.stream_out),
                                  static_cast<const void *>(a.y));
    if (gate_row_slots<T>(a, mis, sms) == 1) return launch_gate_row<T, 1>(a, pdl, stream, launches);
    if (gate_row_slots<T>(a, mis, sms) == 2) return launch_gate_row<T, 2>(a, pdl, stream, launches);
    if (mis >= 0) {
        const bool ach = a.scale.kind == MRN_FACTOR_CHANNEL;
        const bool few = tile_few_rows(a.rows, a.n, sms);
        int k = 1, most_threads = tile_few_threads(a.rows, a.n, sms);
        if (!few) gate_tile<T>(a.n / 8, mis != 0 || a.n % 8 != 0, ach, &k, &most_threads);
        const TileShape p = tile_shape(a.n, mis, k, most_threads, few);
        cudaError_t err = cudaSuccess;
        bool done = false;
        if (p.ok && p.warp) {
            done = p.k == 1   ? launch_gate_k<T, 1, true>(a, p, sms, pdl, stream, launches, &err)
                   : p.k == 2 ? launch_gate_k<T, 2, true>(a, p, sms, pdl, stream, launches, &err)
                   : p.k == 3 ? launch_gate_k<T, 3, true>(a, p, sms, pdl, stream, launches, &err)
                              : launch_gate_k<T, 4, true>(a, p, sms, pdl, stream, launches, &err);
        } else if (p.ok) {
            done = k == 1   ? launch_gate_k<T, 1, false>(a, p, sms, pdl, stream, launches, &err)
                   : k == 2 ? launch_gate_k<T, 2, false>(a, p, sms, pdl, stream, launches, &err)
                            : launch_gate_k<T, 4, false>(a, p, sms, pdl, stream, launches, &err);
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
