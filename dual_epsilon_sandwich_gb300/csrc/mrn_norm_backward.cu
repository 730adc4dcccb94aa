// mrn_norm_backward.cu -- the gradients of LayerNorm and RMSNorm.  With
// w = dy * gamma and, per row,
//   LayerNorm  xh = (x - mean) * rstd        ds = rstd * (w - mean(w) - xh * mean(w xh))
//   RMSNorm    xh = x * rstd, rstd = 1 / sqrt(mean(x^2) + eps)
//                                            ds = rstd * (w - xh * mean(w xh))
// ds gets the stream's own gradient added (dstream) and is written to dx, or
// to dresidual with dropout(ds) written to dx;
//   dgamma_j = sum_r dy xh,  dbeta_j = sum_r dy.
// The two column sums are taken on the same pass: every CTA adds up the rows
// it handles (fixed rows, in order) and leaves one row of partial sums in the
// workspace, which a second launch adds in order.  No atomics: the result does
// not depend on which CTA ran when.
#include "mrn_row_tile.cuh"

namespace mrn {

constexpr int kLoopedThreads = 512;

// A backward pass leaves at most this many partial rows, and for very wide rows
// no more than fill 2^27 floats.
constexpr int kPartsPerSm = 4;
constexpr int64_t kPartsFloats = int64_t(1) << 27;

int64_t backward_parts(int64_t rows, int64_t n, int sms) {
    int64_t parts = static_cast<int64_t>(sms) * kPartsPerSm;
    const int64_t by_size = kPartsFloats / n;
    if (parts > by_size) parts = by_size;
    if (parts > rows) parts = rows;
    return parts < 1 ? (rows > 0 ? 1 : 0) : parts;
}

// Any width: one row per CTA at a time, two passes over it (the second out of
// L2), element by element; the partial sums live in the workspace, each
// element of them read and written by one thread only.
template <class T, bool RMS>
__global__ void __launch_bounds__(kLoopedThreads)
mrn_norm_backward_looped_kernel(const BackwardArgs a, float *part_gamma, float *part_beta) {
    __shared__ CtaSumSlots<2> slots;
    pdl_enter();
    int turn = 0;
    const DropKey key = drop_key(a.drop);
    const float count = static_cast<float>(a.n);
    float *pg = part_gamma + static_cast<int64_t>(blockIdx.x) * a.n;
    float *pb = part_beta ? part_beta + static_cast<int64_t>(blockIdx.x) * a.n : nullptr;
    bool fresh = true;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t e0 = r * a.n;
        const float mean = RMS ? 0.0f : a.mean[r];
        float rstd = RMS ? 0.0f : a.rstd[r];
        // LayerNorm: sums of w and w xh; RMSNorm: of x^2 and w x
        float s[2] = {0.0f, 0.0f};
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const float x = ld_elem<T>(a.x, e0 + j);
            const float w = ld_elem<T>(a.dy, e0 + j) * ld_elem<T>(a.gamma, j);
            if (RMS) {
                s[0] = fmaf(x, x, s[0]);
                s[1] = fmaf(w, x, s[1]);
            } else {
                s[0] += w;
                s[1] = fmaf(w, (x - mean) * rstd, s[1]);
            }
        }
        cta_sum(s, slots, turn);
        float c1 = 0.0f, c2;
        if (RMS) {
            rstd = 1.0f / sqrtf(s[0] / count + a.eps);
            c2 = s[1] / count * rstd;
        } else {
            c1 = s[0] / count;
            c2 = s[1] / count;
        }
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const int64_t e = e0 + j;
            const float dy = ld_elem<T>(a.dy, e);
            const float xh = (ld_elem<T>(a.x, e) - mean) * rstd;
            float ds = (fmaf(dy, ld_elem<T>(a.gamma, j), -c1) - xh * c2) * rstd;
            if (a.dstream) ds += ld_elem<T>(a.dstream, e);
            if (a.dres) {
                const bool keep = drop_keeps_element(key, e, a.drop.threshold);
                st_elem<T>(a.dx, e, drop_scale(ds, keep, a.drop.scale));
                st_elem<T>(a.dres, e, ds);
            } else {
                st_elem<T>(a.dx, e, ds);
            }
            pg[j] = fmaf(dy, xh, fresh ? 0.0f : pg[j]);
            if (pb) pb[j] = dy + (fresh ? 0.0f : pb[j]);
        }
        fresh = false;
    }
}

// The row held in registers between its copy and its outputs, the column sums in
// registers over all rows of the CTA (see mrn_row_tile.cuh).
template <class T, int K, bool EDGE, bool WARP, bool RMS>
__global__ void __launch_bounds__(WARP ? 128 : tile_max_threads(K))
mrn_norm_backward_tile_kernel(const BackwardArgs a, const TileArgs t, float *part_gamma,
                              float *part_beta) {
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    __shared__ RowSumSlots<2> slots;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes));
    const RowTile<T, K, EDGE, WARP> tile(a.rows, a.n, t);
    const int ops_count = a.dstream ? 3 : 2;
    const int64_t back = static_cast<int64_t>(t.mis) * T::kBytes;
    const char *const ops[kTileMaxOperands] = {
        static_cast<const char *>(a.dy) - back, static_cast<const char *>(a.x) - back,
        a.dstream ? static_cast<const char *>(a.dstream) - back : nullptr};
    char *const dx = static_cast<char *>(a.dx) - back;
    char *const dres = a.dres ? static_cast<char *>(a.dres) - back : nullptr;
    uint32_t in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) in[k] = tile.inside(k);
    if (tile.cl > 1) cluster_arrive_relaxed();   // (peers' shared memory is written later)
    pdl_enter();
    const int ahead = t.stages - 1;
    for (int s = 0; s < ahead; ++s) {
        const int64_t r = tile.row + s * tile.stride;
        tile.issue(ring, s, r, r < a.rows, ops, ops_count);
        cp_async_commit();
    }
    const DropKey key = drop_key(a.drop);
    Slot<T> gamma[K];
    tile.weights(gamma, in, a.gamma);
    float sum_g[K][8], sum_b[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum_g[k][i] = sum_b[k][i] = 0.0f;
    if (tile.cl > 1) cluster_wait_acquire();
    const float inv_n = 1.0f / static_cast<float>(a.n);
    int turn = 0, stage = 0, fill = ahead;
    float mean = 0.0f, rstd = 0.0f;
    if (!RMS && tile.row < a.rows) {
        mean = a.mean[tile.row];
        rstd = a.rstd[tile.row];
    }
    for (int64_t it = 0; tile.cta_row(it) < a.rows; ++it) {
        const int64_t r = tile.row + it * tile.stride;
        const bool ok = r < a.rows;
        __syncwarp();
        const int64_t next = r + ahead * tile.stride;
        tile.issue(ring, fill, next, next < a.rows, ops, ops_count);
        cp_async_commit();
        fill = fill + 1 == t.stages ? 0 : fill + 1;
        float next_mean = 0.0f, next_rstd = 0.0f;
        if (!RMS && r + tile.stride < a.rows) {
            next_mean = a.mean[r + tile.stride];
            next_rstd = a.rstd[r + tile.stride];
        }
        cp_async_wait(ahead);
        __syncwarp();
        Slot<T> dy[K], x[K];
        tile.fetch(dy, ring, stage, 0, ops_count);
        tile.mask(dy, in);
        tile.fetch(x, ring, stage, 1, ops_count);
        tile.mask(x, in);
        // LayerNorm: sums of w and w xh; RMSNorm: of x^2 and w x
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = dy[k].get(i);
                const float w = d * gamma[k].get(i);
                if (RMS) {
                    s[0] = fmaf(x[k].get(i), x[k].get(i), s[0]);
                    s[1] = fmaf(w, x[k].get(i), s[1]);
                } else {
                    const float xh = (x[k].get(i) - mean) * rstd;
                    s[0] += w;
                    s[1] = fmaf(w, xh, s[1]);
                    sum_g[k][i] = fmaf(d, xh, sum_g[k][i]);
                    sum_b[k][i] += d;
                }
            }
        }
        row_sum<2, WARP>(s, slots, turn, tile.width, tile.cl, tile.crank);
        float c1 = 0.0f, c2;
        if (RMS) {
            rstd = 1.0f / sqrtf(s[0] * inv_n + a.eps);
            c2 = s[1] * inv_n * rstd;
        } else {
            c1 = s[0] * inv_n;
            c2 = s[1] * inv_n;
        }
        Slot<T> ds[K];
        if (a.dstream) tile.fetch(ds, ring, stage, 2, ops_count);
        stage = stage + 1 == t.stages ? 0 : stage + 1;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = dy[k].get(i);
                const float xh = RMS ? x[k].get(i) * rstd : (x[k].get(i) - mean) * rstd;
                o[i] = fmaf(-xh, c2, fmaf(d, gamma[k].get(i), -c1)) * rstd;
                if (RMS && ok) sum_g[k][i] = fmaf(d, xh, sum_g[k][i]);
            }
            if (a.dstream) {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += ds[k].get(i);
            }
            if (!ok) continue;
            Slot<T> out;
            out.put(o);
            if (a.dres) {
                tile.store(dres, r, k, in[k], out);
                if (in[k] != 0u) {
                    uint32_t w[4] = {0u, 0u, 0u, 0u};
                    if (a.drop.threshold != 0u)
                        philox_lanes(key, static_cast<uint64_t>((tile.slot0(r) >> 3) + tile.first +
                                                                k * tile.width), w);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o[i] = drop_scale(o[i], drop_keeps(w, i, a.drop.threshold), a.drop.scale);
                    out.put(o);
                }
            }
            tile.store(dx, r, k, in[k], out);
        }
        mean = next_mean;
        rstd = next_rstd;
    }
    cp_async_wait(0);
    __syncthreads();   // the ring is free: the CTA's column sums go through it
    float *const buf = reinterpret_cast<float *>(ring_bytes);
    const int64_t part = (WARP ? blockIdx.x : blockIdx.x / tile.cl) * a.n;
    const int lo = WARP ? 0 : static_cast<int>(tile.crank) * K * static_cast<int>(blockDim.x) * 8 - tile.off;
    const int span = K * tile.width * 8;      // columns lo .. lo + span of this CTA
    const int turns = WARP ? static_cast<int>(blockDim.x) / tile.width : 1;
    const int mine = WARP ? static_cast<int>(threadIdx.x) / tile.width : 0;
    for (int which = 0; which < (!RMS && part_beta ? 2 : 1); ++which) {
        float *const out = which == 0 ? part_gamma : part_beta;
        for (int g = 0; g < turns; ++g) {
            if (g == mine) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    // (WARP: rows of one CTA may start at different offsets, so columns
                    // are counted from the row's first)
                    const int at = tile.column(k) - lo;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (!((in[k] >> i) & 1u)) continue;
                        const float v = which == 0 ? sum_g[k][i] : sum_b[k][i];
                        buf[at + i] = g == 0 ? v : buf[at + i] + v;
                    }
                }
            }
            __syncthreads();
        }
        for (int j = threadIdx.x; j < span; j += blockDim.x) {
            const int64_t col = static_cast<int64_t>(lo) + j;
            if (col >= 0 && col < a.n) out[part + col] = buf[j];
        }
        __syncthreads();
    }
}

template <class T, int K, bool EDGE, bool WARP, bool RMS>
cudaError_t launch_backward_tile(const BackwardArgs &a, const TilePlan &p, float *pg, float *pb,
                                 bool pdl, cudaStream_t stream, uint64_t *launches) {
    static TileLaunchCache cache;
    const TileArgs t = {p.lanes, p.stages, p.mis};
    const int64_t shared = tile_ring_bytes(T::kBytes, K, p.threads, p.stages, a.dstream ? 3 : 2);
    return launch_tile(cache, mrn_norm_backward_tile_kernel<T, K, EDGE, WARP, RMS>, p, shared, pdl,
                       stream, launches, a, t, pg, pb);
}

template <class T, int K, bool WARP>
cudaError_t launch_backward_k(const BackwardArgs &a, const TilePlan &p, float *pg, float *pb,
                              bool pdl, cudaStream_t stream, uint64_t *launches) {
    if (a.rms)
        return p.edge ? launch_backward_tile<T, K, true, WARP, true>(a, p, pg, pb, pdl, stream, launches)
                      : launch_backward_tile<T, K, false, WARP, true>(a, p, pg, pb, pdl, stream, launches);
    return p.edge ? launch_backward_tile<T, K, true, WARP, false>(a, p, pg, pb, pdl, stream, launches)
                  : launch_backward_tile<T, K, false, WARP, false>(a, p, pg, pb, pdl, stream, launches);
}

// dgamma (blockIdx.y == 0) and dbeta (1): the sum of `parts` partial rows.  A
// CTA owns 32 columns; its 32 warps take every 32nd partial row each and are
// joined in shared memory, in order.
constexpr int kJoinColumns = 32;
constexpr int kJoinThreads = 1024;

__global__ void __launch_bounds__(kJoinThreads)
mrn_norm_backward_join_kernel(const float *part_gamma, const float *part_beta, float *dgamma,
                              float *dbeta, int64_t parts, int64_t n) {
    __shared__ float sums[32][kJoinColumns + 1];
    pdl_enter();
    const float *part = blockIdx.y == 0 ? part_gamma : part_beta;
    float *out = blockIdx.y == 0 ? dgamma : dbeta;
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kJoinColumns + lane;
    float s = 0.0f;
    if (j < n) {
        for (int64_t p = warp; p < parts; p += 32) s += part[p * n + j];
    }
    sums[warp][lane] = s;
    __syncthreads();
    // warp c adds up column c: lane w holds warp w's sum
    const float t = warp_allsum(sums[lane][warp]);
    const int64_t jc = static_cast<int64_t>(blockIdx.x) * kJoinColumns + warp;
    if (lane == 0 && jc < n) out[jc] = t;
}

cudaError_t launch_join(const float *pg, const float *pb, float *dgamma, float *dbeta,
                        int64_t parts, int64_t n, bool pdl, cudaStream_t stream,
                        uint64_t *launches) {
    const int64_t ctas = (n + kJoinColumns - 1) / kJoinColumns;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), dbeta ? 2 : 1, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, mrn_norm_backward_join_kernel, pg, pb, dgamma,
                                               dbeta, parts, n);
    if (err == cudaSuccess) ++*launches;
    return err;
}

template <class T>
cudaError_t launch_backward_typed(const BackwardArgs &a, int sms, bool pdl, cudaStream_t stream,
                                  uint64_t *launches) {
    const int64_t most = backward_parts(a.rows, a.n, sms);
    if (most == 0) return launch_join(nullptr, nullptr, a.dgamma, a.dbeta, 0, a.n, pdl, stream, launches);
    const int mis = common_offset(T::kBytes, a.dy, a.x, a.dstream, static_cast<const void *>(a.dx),
                                  static_cast<const void *>(a.dres));
    TilePlan p = {};
    // (a generator group is a slot only when the operands start on a slot boundary)
    if (mis == 0 || (mis > 0 && a.drop.threshold == 0)) {
        const TileWish wish = {a.dstream ? 3 : 2, 512, kPartsPerSm};
        p = plan_tiles(a.rows, a.n, T::kBytes, mis, wish, sms);
    }
    const int64_t parts = p.ok ? p.ctas / p.cluster : most;
    if (parts > most) return cudaErrorInvalidConfiguration;   // (the workspace holds `most`)
    float *pg = a.workspace;
    float *pb = a.dbeta ? a.workspace + parts * a.n : nullptr;
    cudaError_t err;
    if (p.ok && p.warp) {
        err = p.k == 1   ? launch_backward_k<T, 1, true>(a, p, pg, pb, pdl, stream, launches)
              : p.k == 2 ? launch_backward_k<T, 2, true>(a, p, pg, pb, pdl, stream, launches)
                         : launch_backward_k<T, 4, true>(a, p, pg, pb, pdl, stream, launches);
    } else if (p.ok) {
        err = p.k == 1 ? launch_backward_k<T, 1, false>(a, p, pg, pb, pdl, stream, launches)
                       : launch_backward_k<T, 2, false>(a, p, pg, pb, pdl, stream, launches);
    } else {
        const auto fn = a.rms ? mrn_norm_backward_looped_kernel<T, true>
                              : mrn_norm_backward_looped_kernel<T, false>;
        err = launch_plain(fn, parts, kLoopedThreads, 0, pdl, stream, launches, a, pg, pb);
    }
    if (err != cudaSuccess) return err;
    return launch_join(pg, pb, a.dgamma, a.dbeta, parts, a.n, pdl, stream, launches);
}

cudaError_t launch_norm_backward(bool bf16, const BackwardArgs &a, int sms, bool pdl,
                                 cudaStream_t stream, uint64_t *launches) {
    return bf16 ? launch_backward_typed<BF16>(a, sms, pdl, stream, launches)
                : launch_backward_typed<F32>(a, sms, pdl, stream, launches);
}

}  // namespace mrn
