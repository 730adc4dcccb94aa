// mrn_layernorm.cu -- LayerNorm of every row, alone or after the residual add
// with dropout:
//   stream = res + dropout(x), rounded once to the row type and stored
//   mean = sum_j s_j / n,  rstd = 1 / sqrt(sum_j (s_j - mean)^2 / n + eps)
//   y = (s - mean) * rstd * gamma + beta      (s the stored stream, or x)
// The variance is summed from the deviations, not from the squares: what a row whose mean
// is far from zero loses is the roundings of its f32 mean alone.  Those are the sum's: the
// quotient by n is rounded once (mean_of below).
#include "mrn_row_tile.cuh"

namespace mrn {

constexpr int kLoopedThreads = 512;
// Threads that an SM's registers are shared between (the launch bound), from what a thread
// holds: k slots of r rows and of two weights.
// It does not count what rows that share a warp take beside them (distances of their own, with
// ends one more generator group): ten of those bf16 forms spill, 4 to 96 bytes.
template <class T> constexpr int forward_resident(int k, int r) {
    const int words = k * (r + 2) * Slot<T>::kWords;
    return words <= 12 ? 1024 : (words <= 28 ? 768 : (words <= 36 ? 640 : (words <= 68 ? 512 : (words <= 100 ? 384 : 256))));
}
// Threads of a CTA at most.
template <class T> constexpr int forward_threads(int k, int r) {
    return forward_resident<T>(k, r) < 512 ? forward_resident<T>(k, r) : 512;
}

// sum / n, rounded to nearest, from the reciprocal inv = 1 / n that is itself rounded to
// nearest: Markstein's step ("Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  q is within one and a half units of the quotient; what the fma leaves of
// sum is a whole multiple of q's unit, of at most 1.5 n units, and exact; times inv it takes q to
// within 2^-23 units of the quotient.  A quotient by n < 2^19 (the row tiles hold up to 2^18
// elements and the ends) lies 2^-20 units at least from the border between two f32 numbers, so
// that the last addition rounds as the quotient itself would be rounded.
//   The product alone missed it by up to a unit: a constant row of 1000.0, n = 6656, whose sum is
// exact, came out 0.02 off beta at eps 1e-5 and 0.5 off at 1e-8.  Every row waits for this; measured
// on GB300, us with the product, so, and with a division: f32 8192 x 4096 45.8, 46.6, 47.5, bf16
// 16384 x 4096 after the add 89.6, 90.3, 92.1, f32 64 x 1024 1.83, 1.89, 1.89.
__device__ __forceinline__ float mean_of(float sum, float n, float inv) {
    const float q = sum * inv;
    const float left = fmaf(-q, n, sum);
    return left == left ? fmaf(left, inv, q) : q;     // (an infinite sum leaves NaN)
}

// Any width: one row per CTA at a time, three passes over it (the second and
// third out of L2), element by element.  For operands that do not share an offset and rows
// wider than a cluster holds.  Bound by its accesses of one element: 16384 x 4096 bf16, x an
// element off the others, 312 us alone and 539 after the add (the tile kernel: 45 and 89).
template <class T>
__global__ void __launch_bounds__(kLoopedThreads) mrn_layernorm_looped_kernel(const LayernormArgs a) {
    __shared__ CtaSum slots;
    cta_sum_setup(slots);
    pdl_enter();
    int turn = 0;
    const DropKey key = drop_key(a.drop);
    const bool add = a.res != nullptr;
    const void *s = add ? a.stream_out : a.x;
    const float count = static_cast<float>(a.n);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t e0 = r * a.n;
        float sum[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const int64_t e = e0 + j;
            float v = ld_elem<T>(a.x, e);
            if (add) {
                const bool keep = drop_keeps_element(key, e, a.drop.threshold);
                v = st_elem<T>(a.stream_out, e, drop_add(v, ld_elem<T>(a.res, e), keep, a.drop.scale));
            }
            sum[0] += v;
        }
        cta_sum(sum, slots, turn);
        const float mean = sum[0] / count;
        float dev[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const float d = ld_elem<T>(s, e0 + j) - mean;
            dev[0] = fmaf(d, d, dev[0]);
        }
        cta_sum(dev, slots, turn);
        const float rstd = 1.0f / sqrtf(dev[0] / count + a.eps);
        if (threadIdx.x == 0 && a.mean) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const float h = (ld_elem<T>(s, e0 + j) - mean) * rstd;
            const float b = a.beta ? ld_elem<T>(a.beta, j) : 0.0f;
            st_elem<T>(a.y, e0 + j, fmaf(h, ld_elem<T>(a.gamma, j), b));
        }
    }
}

// Rows held in registers between their copy and their outputs (see mrn_row_tile.cuh): the
// deviations are taken from the values themselves, so that every operand is read once and every
// output written once.  Measured on GB300: 16384 x 4096 bf16 45.7 us alone (5.9 TB/s, 87 % of
// the copy's rate) and 90.1 after the add (6.0 TB/s); 4096 x 6655 f32 after the add 77.7 us
// (5.6 TB/s); 4 x 6656 f32 2.6 us, a launch and two sums over a cluster.
//   What bounds it: not memory alone (dram 69 % busy under ncu) but the instructions of 16 warps
// on an SM, issued in 55 % of cycles, with the generator's and the conversions' the most of
// them; a row's two sums, each a barrier of its CTA, are covered by the copies in flight and
// by the other CTA of the SM.  More warps would need fewer registers than a row's slots take.
template <class T, int K, int R, bool EDGE, bool WARP, bool ADD>
__global__ void __launch_bounds__(forward_resident<T>(K, R))
mrn_layernorm_tile_kernel(const LayernormArgs a, const TileArgs t) {
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    __shared__ RowSumSlots<R, T::kBytes == 2> slots;
    constexpr int kOps = ADD ? 2 : 1;
    __shared__ EndSlots<kOps, R, EDGE, WARP> end_w;
    RowTile<T, K, R, EDGE, WARP> tile(a.rows, a.n, t);
    const int64_t back = static_cast<int64_t>(t.mis) * T::kBytes;
    const char *ops[kOps];
    ops[0] = static_cast<const char *>(a.x) - back;
    if constexpr (ADD) ops[1] = static_cast<const char *>(a.res) - back;
    char *const y = static_cast<char *>(a.y) - back;
    char *const stream_out = ADD ? static_cast<char *>(a.stream_out) - back : nullptr;
    RingWalk walk(tile.stage_bytes(kOps), t.stages);
    const int ahead = t.stages - 1;
    const uint32_t ring = tile.warp_ring(static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes)), t.stages, kOps);
    tile.clear(ring, t.stages, kOps);
    row_sum_setup(slots, tile.cl);
    pdl_enter();
    for (int s = 0; s < ahead; ++s) tile.issue(ring + s * walk.bytes, s, ops, kOps, end_w);
    const DropKey key = ADD ? drop_key(a.drop) : DropKey{};
    Slot<T> gamma[K], beta[K];
    tile.weights(gamma, a.gamma);
    if (a.beta) {
        tile.weights(beta, a.beta);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) beta[k].zero();
    }
    const float end_gamma = EDGE ? tile.end_weight(a.gamma) : 0.0f;
    const float end_beta = EDGE && a.beta ? tile.end_weight(a.beta) : 0.0f;
    row_sum_ready(tile.cl);
    const float count = static_cast<float>(a.n), inv_n = 1.0f / count;
    int turn = 0;
    for (; tile.cta_left > 0; tile.advance(), walk.next()) {
        __syncwarp();
        tile.issue(ring + walk.write * walk.bytes, walk.write, ops, kOps, end_w);
        cp_async_wait(ahead);
        __syncwarp();
        const uint32_t from = ring + walk.read * walk.bytes;
        Slot<T> v[R][K];
        float sum[R], end[R];
        bool end_keep[R];
#pragma unroll
        for (int rr = 0; rr < R; ++rr) {
            tile.fetch(v[rr], from, 0, rr, kOps);
            if constexpr (ADD) {
                Slot<T> res[K];
                DropGroup d[K];
                end_keep[rr] = tile.masks(d, key, rr, a.drop.threshold);
                tile.fetch(res, from, 1, rr, kOps);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o[i] = drop_add(v[rr][k].get(i), res[k].get(i), d[k].keeps(i), a.drop.scale);
                    v[rr][k].put(o);
                }
                tile.store(stream_out, rr, tile.valid(rr), v[rr]);
            }
            uint64_t acc = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc = f2_add(acc, v[rr][k].pair(i));
            }
            sum[rr] = f2_sum(acc);
            end[rr] = 0.0f;
            if (EDGE && tile.ends) {
                end[rr] = tile.fetch_end(end_w, walk.read, 0, rr);
                if constexpr (ADD) {
                    end[rr] = tile.store_end(stream_out, rr, tile.valid(rr),
                                             drop_add(end[rr], tile.fetch_end(end_w, walk.read, 1, rr),
                                                      end_keep[rr], a.drop.scale));
                    if (tile.end_col < 0) end[rr] = 0.0f;
                }
                sum[rr] += end[rr];
            }
        }
        if (!row_sum<WARP>(sum, slots, turn, tile.width, tile.cl, tile.crank, turn == 0 ? t.stall : 0u)) break;
        float dev[R];
#pragma unroll
        for (int rr = 0; rr < R; ++rr) {
            sum[rr] = mean_of(sum[rr], count, inv_n);
            const uint64_t minus = f2_pack(-sum[rr], -sum[rr]);
            uint64_t acc = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                uint64_t part = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t d = f2_add(v[rr][k].pair(i), minus);
                    part = f2_fma(d, d, part);
                }
                acc = f2_add(acc, tile.holds(k) ? part : 0);
            }
            dev[rr] = f2_sum(acc);
            if (EDGE && tile.end_col >= 0) dev[rr] = fmaf(end[rr] - sum[rr], end[rr] - sum[rr], dev[rr]);
        }
        if (!row_sum<WARP>(dev, slots, turn, tile.width, tile.cl, tile.crank, 0u)) break;
        uint64_t minus[R], scale[R];
#pragma unroll
        for (int rr = 0; rr < R; ++rr) {
            const float rstd = inv_sqrt(fmaf(dev[rr], inv_n, a.eps));
            if (a.mean && tile.first == 0 && tile.valid(rr)) {
                a.mean[tile.row + rr * tile.stride] = sum[rr];
                a.rstd[tile.row + rr * tile.stride] = rstd;
            }
            minus[rr] = f2_pack(-sum[rr], -sum[rr]);
            scale[rr] = f2_pack(rstd, rstd);
            if (EDGE && tile.ends)
                tile.store_end(y, rr, tile.valid(rr), fmaf((end[rr] - sum[rr]) * rstd, end_gamma, end_beta));
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t g = gamma[k].pair(i), b = beta[k].pair(i);
#pragma unroll
                for (int rr = 0; rr < R; ++rr)
                    v[rr][k].put_pair(i, f2_fma(f2_mul(f2_add(v[rr][k].pair(i), minus[rr]), scale[rr]), g, b));
            }
        }
#pragma unroll
        for (int rr = 0; rr < R; ++rr) tile.store(y, rr, tile.valid(rr), v[rr]);
    }
    cp_async_wait(0);
    row_sum_leave(tile.cl);
}

// Whether the call was launched; false: it takes the looped kernel.
template <class T, int K, int R, bool EDGE, bool WARP, bool ADD>
bool launch_layernorm_tile(const LayernormArgs &a, const TileShape &p, int sms, bool pdl,
                           cudaStream_t stream, uint64_t *launches, cudaError_t *err) {
    static TileLaunchCache cache;
    const auto fn = mrn_layernorm_tile_kernel<T, K, R, EDGE, WARP, ADD>;
    constexpr int kOps = ADD ? 2 : 1;
    TileGrid g;
    *err = tile_grid(cache, fn, p, a.rows, a.n, R, T::kBytes, kOps, 32, sms, &g);
    if (*err != cudaSuccess) return true;
    if (g.stages < 1) return false;
    const TileArgs t = {p.lanes, g.stages, p.mis, a.stall};
    *err = launch_tile(fn, p, g.ctas, g.shared, pdl, stream, launches, a, t);
    return true;
}

template <class T, int K, int R, bool WARP>
bool launch_layernorm_k(const LayernormArgs &a, const TileShape &p, int sms, bool pdl,
                        cudaStream_t stream, uint64_t *launches, cudaError_t *err) {
    if (a.res)
        return p.edge ? launch_layernorm_tile<T, K, R, true, WARP, true>(a, p, sms, pdl, stream, launches, err)
                      : launch_layernorm_tile<T, K, R, false, WARP, true>(a, p, sms, pdl, stream, launches, err);
    return p.edge ? launch_layernorm_tile<T, K, R, true, WARP, false>(a, p, sms, pdl, stream, launches, err)
                  : launch_layernorm_tile<T, K, R, false, WARP, false>(a, p, sms, pdl, stream, launches, err);
}

// Slots per thread (k) and rows at a time (r) for rows of a CTA.  Measured on GB300, a call of
// 269 MB (alone) or 537 MB (after the add), k x r (us):
//   bf16 alone      n = 1280 2 x 2 49.0, 4 x 1 54.2;  1408 49.7, 51.3;  1536 50.0, 49.2;  2048 49.6,
//                   47.4;  4096 46.9, 45.9;  4095 59.0, 51.3;  8192 55.5, 46.2
//   bf16 after add  n = 1280 2 x 2 96.7, 4 x 1 108.1;  1536 97.1, 92.5;  2048 95.6, 94.5;  2568
//                   102.7, 94.5;  3584 94.8, 91.0;  3712 94.8, 92.2;  3840 92.8, 93.3;  3968 92.2,
//                   93.8;  4096 90.2, 94.3;  4104 110.9, 105.3;  4608 98.6, 94.5;  5120 96.1,
//                   91.4;  8192 102.2, 89.9;  odd: 4095 115.2, 90.2
//   f32 alone       n = 2048 1 x 1 49.1, 2 x 1 47.2;  4096 1 x 1 46.9, 2 x 1 46.8, 4 x 1 47.1;
//                   4104 2 x 2 54.4, 2 x 1 48.9;  6656 2 x 2 47.5, 2 x 1 46.3, 4 x 1 52.4;  6655
//                   52.4, 61.6, 56.6;  8192 47.6, 48.2, 49.3;  8200 72.8, 62.2, 54.4;  12288 58.5,
//                   61.0, 48.2
//   f32 after add   n = 2048 1 x 1 92.2, 2 x 1 91.2;  4096 92.2, 92.5;  4104 2 x 1 96.6, 4 x 1 100.9;
//                   5120 92.5, 92.8;  6655 92.6, 100.8;  6656 94.5, 88.4;  7168 93.7, 87.2;  7176
//                   100.7, 94.3;  8191 98.4, 93.5;  8192 93.8, 92.2
// Where a border serves aligned and odd widths, the odd ones, which lose more, set it (f32 6655 beside
// 6656).
// Rows in clusters, and their CTAs' threads (us): f32 alone 4096 x 16384 2 x 2 of 128 98.8, 2 x 1
// of 512 104.7, 4 x 1 of 384 132, but 2048 x 16384 59.6, 59.0, 65.7 and 2 x 1 of 256 51.8; 1024 x
// 32768 2 x 1 of 256 54.7, of 512 62.4, 2 x 2 of 256 62.4; 512 x 65536 2 x 1 of 256 71.1, of 512
// 72.7, 2 x 2 of 256 67.5, 4 x 1 of 384 67.7.  f32 after add 2048 x 16384 2 x 1 of 256 91.7, of 128
// 88.4, of 512 94.3, 4 x 1 of 256 98.4; 512 x 65536 2 x 1 of 256 115.8, of 512 118.9.  bf16 4 x 1
// alone 3276 x 20480 of 128 64.3, of 256 74.6; 2048 x 32768 of 128 72.6, of 256 66.5, of 512 68.7;
// 1024 x 65536 90.9, 80.0, 73.8; after add the last two 101.2, 114.3, 113.2 and 115.2, 119.1, 122.7.
template <class T> void forward_tile(int64_t slots, bool add, bool edge, int *k, int *r, int *threads) {
    if (T::kBytes == 4 && slots > 1536) {
        *k = 2;
        *r = !add && slots <= 2048 ? 2 : 1;
        *threads = *r == 2 ? 128 : 256;
    } else if (T::kBytes == 2) {
        const bool two = slots < 192 || (add && !edge && slots > 464 && slots <= 512);
        *k = two ? 2 : 4;
        *r = two ? 2 : 1;
    } else if (add) {
        *k = slots <= 512 ? 1 : (slots <= 896 ? 2 : 4);
        *r = 1;
    } else {
        *k = slots <= 512 ? 1 : (slots <= 1024 ? 2 : 4);
        *r = *k == 2 ? 2 : 1;
    }
    if (T::kBytes == 2 && slots > 2048) *threads = 128;
    while (*threads > 0 && *threads < forward_threads<T>(*k, *r) && slots > int64_t(kMaxCluster) * *k * *threads) *threads *= 2;
}

template <class T>
cudaError_t launch_layernorm_typed(const LayernormArgs &a, int sms, bool pdl, cudaStream_t stream,
                                   uint64_t *launches) {
    const int mis = common_offset(T::kBytes, a.x, a.y, a.res, static_cast<const void *>(a.stream_out));
    // (a generator group is a slot only when the operands start on a slot boundary)
    if (mis == 0 || (mis > 0 && a.drop.threshold == 0)) {
        int k = 4, r = 1, most_threads = 0;
        forward_tile<T>(a.n / 8, a.res != nullptr, mis != 0 || a.n % 8 != 0, &k, &r, &most_threads);
        if (most_threads == 0 || most_threads > forward_threads<T>(k, r)) most_threads = forward_threads<T>(k, r);
        const bool few = tile_few_rows(a.rows, a.n, sms);
        if (few) {
            k = r = 1;
            most_threads = tile_few_threads(a.rows, a.n, sms);
        }
        const TileShape p = tile_shape(a.n, mis, k, most_threads, few);
        cudaError_t err = cudaSuccess;
        bool done = false;
        if (p.ok && p.warp) {
            done = p.k == 1   ? launch_layernorm_k<T, 1, 1, true>(a, p, sms, pdl, stream, launches, &err)
                   : p.k == 2 ? launch_layernorm_k<T, 2, 1, true>(a, p, sms, pdl, stream, launches, &err)
                   : p.k == 3 ? launch_layernorm_k<T, 3, 1, true>(a, p, sms, pdl, stream, launches, &err)
                              : launch_layernorm_k<T, 4, 1, true>(a, p, sms, pdl, stream, launches, &err);
        } else if (p.ok) {
            if (k == 1) {
                done = launch_layernorm_k<T, 1, 1, false>(a, p, sms, pdl, stream, launches, &err);
            } else if (k == 4) {
                done = launch_layernorm_k<T, 4, 1, false>(a, p, sms, pdl, stream, launches, &err);
            } else if constexpr (T::kBytes == 2) {
                done = launch_layernorm_k<T, 2, 2, false>(a, p, sms, pdl, stream, launches, &err);
            } else if (r == 1) {
                done = launch_layernorm_k<T, 2, 1, false>(a, p, sms, pdl, stream, launches, &err);
            } else {      // (two rows at a time: without an add)
                done = p.edge ? launch_layernorm_tile<T, 2, 2, true, false, false>(a, p, sms, pdl, stream, launches, &err)
                              : launch_layernorm_tile<T, 2, 2, false, false, false>(a, p, sms, pdl, stream, launches, &err);
            }
        }
        if (done) return err;
    }
    const int64_t ctas = a.rows < 4LL * sms ? a.rows : 4LL * sms;
    return launch_plain(mrn_layernorm_looped_kernel<T>, ctas, kLoopedThreads, 0, pdl, stream,
                        launches, a);
}

cudaError_t launch_layernorm(bool bf16, const LayernormArgs &a, int sms, bool pdl,
                             cudaStream_t stream, uint64_t *launches) {
    return bf16 ? launch_layernorm_typed<BF16>(a, sms, pdl, stream, launches)
                : launch_layernorm_typed<F32>(a, sms, pdl, stream, launches);
}

int take_wait_timeouts_layernorm() { return take_wait_timeouts<kOpLayernormTimeouts>(); }

}  // namespace mrn
