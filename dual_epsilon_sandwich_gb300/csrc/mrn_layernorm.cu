// mrn_layernorm.cu -- LayerNorm of every row, alone or after the residual add
// with dropout:
//   stream = res + dropout(x), rounded once to the row type and stored
//   mean = sum_j s_j / n,  rstd = 1 / sqrt(sum_j (s_j - mean)^2 / n + eps)
//   y = (s - mean) * rstd * gamma + beta      (s the stored stream, or x)
// The variance is summed from the deviations, not from the squares: a row
// whose mean is far from zero loses no digits.
#include "mrn_row_tile.cuh"

namespace mrn {

constexpr int kLoopedThreads = 512;

// Any width: one row per CTA at a time, three passes over it (the second and
// third out of L2), element by element.
template <class T>
__global__ void __launch_bounds__(kLoopedThreads) mrn_layernorm_looped_kernel(const LayernormArgs a) {
    __shared__ CtaSumSlots<1> slots;
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

// The row held in registers between its copy and its outputs (see mrn_row_tile.cuh).
template <class T, int K, bool EDGE, bool WARP, bool ADD>
__global__ void __launch_bounds__(WARP ? 128 : tile_max_threads(K))
mrn_layernorm_tile_kernel(const LayernormArgs a, const TileArgs t) {
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    __shared__ RowSumSlots<1> slots;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes));
    RowTile<T, K, EDGE, WARP> tile(a.rows, a.n, t);
    constexpr int kOps = ADD ? 2 : 1;
    const int64_t back = static_cast<int64_t>(t.mis) * T::kBytes;
    const char *const ops[kTileMaxOperands] = {static_cast<const char *>(a.x) - back,
                                               ADD ? static_cast<const char *>(a.res) - back : nullptr,
                                               nullptr};
    char *const y = static_cast<char *>(a.y) - back;
    char *const stream_out = ADD ? static_cast<char *>(a.stream_out) - back : nullptr;
    RingWalk walk(kOps * K * tile.region, t.stages);
    const int ahead = t.stages - 1;
    tile.clear(ring, t.stages, kOps);
    if (tile.cl > 1) cluster_arrive_relaxed();   // (peers' shared memory is written later)
    pdl_enter();
    for (int s = 0; s < ahead; ++s) tile.issue(ring + s * walk.bytes, s, ops, kOps);
    const DropKey key = ADD ? drop_key(a.drop) : DropKey{};
    Slot<T> gamma[K], beta[K];
    tile.weights(gamma, a.gamma);
    if (a.beta) {
        tile.weights(beta, a.beta);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) beta[k].zero();
    }
    if (tile.cl > 1) cluster_wait_acquire();
    const float inv_n = 1.0f / static_cast<float>(a.n);
    int turn = 0;
    for (; tile.cta_row() < a.rows; tile.advance(), walk.next()) {
        __syncwarp();
        tile.issue(ring + walk.write * walk.bytes, ahead, ops, kOps);
        cp_async_wait(ahead);
        __syncwarp();
        const uint32_t from = ring + walk.read * walk.bytes;
        Slot<T> v[K];
        tile.fetch(v, from, 0);
        if constexpr (ADD) {
            Slot<T> res[K];
            tile.fetch(res, from, 1);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (tile.in[k] == 0u) continue;
                const DropGroup d = drop_group(key, tile.group(k), a.drop.threshold);
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = drop_add(v[k].get(i), res[k].get(i), d.keeps(i), a.drop.scale);
                v[k].put(o);
                if (!WARP || tile.row < a.rows) tile.store(stream_out, k, v[k]);
            }
        }
        uint64_t acc = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = f2_add(acc, v[k].pair(i));
        }
        float sum[1] = {f2_sum(acc)};
        row_sum<1, WARP>(sum, slots, turn, tile.width, tile.cl, tile.crank);
        const float mean = sum[0] * inv_n;
        const uint64_t minus = f2_pack(-mean, -mean);
        acc = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (tile.in[k] == 0u) continue;
            if (!EDGE || tile.in[k] == 0xFFu) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t d = f2_add(v[k].pair(i), minus);
                    acc = f2_fma(d, d, acc);
                }
            } else {
                float part = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = ((tile.in[k] >> i) & 1u) ? v[k].get(i) - mean : 0.0f;
                    part = fmaf(d, d, part);
                }
                acc = f2_add(acc, f2_pack(part, 0.0f));
            }
        }
        float dev[1] = {f2_sum(acc)};
        row_sum<1, WARP>(dev, slots, turn, tile.width, tile.cl, tile.crank);
        const float rstd = inv_sqrt(fmaf(dev[0], inv_n, a.eps));
        if (!WARP || tile.row < a.rows) {
            if (a.mean && tile.first == 0) {
                a.mean[tile.row] = mean;
                a.rstd[tile.row] = rstd;
            }
            const uint64_t scale = f2_pack(rstd, rstd);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                Slot<T> out;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    out.put_pair(i, f2_fma(f2_mul(f2_add(v[k].pair(i), minus), scale),
                                           gamma[k].pair(i), beta[k].pair(i)));
                tile.store(y, k, out);
            }
        }
    }
    cp_async_wait(0);
}

template <class T, int K, bool EDGE, bool WARP, bool ADD>
cudaError_t launch_layernorm_tile(const LayernormArgs &a, const TilePlan &p, bool pdl,
                                  cudaStream_t stream, uint64_t *launches) {
    static TileLaunchCache cache;
    const TileArgs t = {p.lanes, p.stages, p.mis};
    const int64_t shared = tile_ring_bytes(T::kBytes, K, p.threads, p.stages, ADD ? 2 : 1);
    return launch_tile(cache, mrn_layernorm_tile_kernel<T, K, EDGE, WARP, ADD>, p, shared, pdl,
                       stream, launches, a, t);
}

template <class T, int K, bool WARP>
cudaError_t launch_layernorm_k(const LayernormArgs &a, const TilePlan &p, bool pdl,
                               cudaStream_t stream, uint64_t *launches) {
    if (a.res)
        return p.edge ? launch_layernorm_tile<T, K, true, WARP, true>(a, p, pdl, stream, launches)
                      : launch_layernorm_tile<T, K, false, WARP, true>(a, p, pdl, stream, launches);
    return p.edge ? launch_layernorm_tile<T, K, true, WARP, false>(a, p, pdl, stream, launches)
                  : launch_layernorm_tile<T, K, false, WARP, false>(a, p, pdl, stream, launches);
}

template <class T>
cudaError_t launch_layernorm_typed(const LayernormArgs &a, int sms, bool pdl, cudaStream_t stream,
                                   uint64_t *launches) {
    const int mis = common_offset(T::kBytes, a.x, a.y, a.res, static_cast<const void *>(a.stream_out));
    // (a generator group is a slot only when the operands start on a slot boundary)
    if (mis == 0 || (mis > 0 && a.drop.threshold == 0)) {
        const TileWish wish = {a.res ? 2 : 1, 2, 1024, 8};
        const TilePlan p = plan_tiles(a.rows, a.n, T::kBytes, mis, wish, sms);
        if (p.ok && p.warp) {
            if (p.k == 1) return launch_layernorm_k<T, 1, true>(a, p, pdl, stream, launches);
            if (p.k == 2) return launch_layernorm_k<T, 2, true>(a, p, pdl, stream, launches);
            return launch_layernorm_k<T, 4, true>(a, p, pdl, stream, launches);
        }
        if (p.ok) {
            if (p.k == 1) return launch_layernorm_k<T, 1, false>(a, p, pdl, stream, launches);
            if (p.k == 2) return launch_layernorm_k<T, 2, false>(a, p, pdl, stream, launches);
            if (p.k == 3) return launch_layernorm_k<T, 3, false>(a, p, pdl, stream, launches);
            return launch_layernorm_k<T, 4, false>(a, p, pdl, stream, launches);
        }
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

}  // namespace mrn
