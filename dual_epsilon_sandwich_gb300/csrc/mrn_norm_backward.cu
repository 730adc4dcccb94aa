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
mrn_norm_backward_looped_kernel(const BackwardArgs a, float *part_gamma, float *part_beta,
                                const int64_t part_stride) {
    __shared__ CtaSumSlots<2> slots;
    pdl_enter();
    int turn = 0;
    const DropKey key = drop_key(a.drop);
    const float count = static_cast<float>(a.n);
    float *pg = part_gamma + static_cast<int64_t>(blockIdx.x) * part_stride;
    float *pb = part_beta ? part_beta + static_cast<int64_t>(blockIdx.x) * part_stride : nullptr;
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
                              float *part_beta, const int64_t part_stride) {
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    __shared__ RowSumSlots<2> slots;
    __shared__ float stats[kTileMaxStages][2][128];   // mean and rstd of the ring's rows, per team
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes));
    RowTile<T, K, EDGE, WARP> tile(a.rows, a.n, t);
    const int ops_count = a.dstream ? 3 : 2;
    const int64_t back = static_cast<int64_t>(t.mis) * T::kBytes;
    const char *const ops[kTileMaxOperands] = {
        static_cast<const char *>(a.dy) - back, static_cast<const char *>(a.x) - back,
        a.dstream ? static_cast<const char *>(a.dstream) - back : nullptr};
    char *const dx = static_cast<char *>(a.dx) - back;
    char *const dres = a.dres ? static_cast<char *>(a.dres) - back : nullptr;
    RingWalk walk(ops_count * K * tile.region, t.stages);
    const int ahead = t.stages - 1;
    tile.clear(ring, t.stages, ops_count);
    if (tile.cl > 1) cluster_arrive_relaxed();   // (peers' shared memory is written later)
    pdl_enter();
    // mean and rstd travel with their row, so that no load of them is waited for
    auto issue = [&](int to, int rows_ahead) {
        const int64_t r = tile.row + rows_ahead * tile.stride;
        if (!RMS && tile.leads && r < a.rows) {
            cp_async4(static_cast<uint32_t>(__cvta_generic_to_shared(&stats[to][0][tile.team])), a.mean + r);
            cp_async4(static_cast<uint32_t>(__cvta_generic_to_shared(&stats[to][1][tile.team])), a.rstd + r);
        }
        tile.issue(ring + to * walk.bytes, rows_ahead, ops, ops_count);
    };
    for (int s = 0; s < ahead; ++s) issue(s, s);
    const DropKey key = drop_key(a.drop);
    Slot<T> gamma[K];
    tile.weights(gamma, a.gamma);
    uint64_t sum_g[K][4], sum_b[K][4];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum_g[k][i] = sum_b[k][i] = 0;
    const float inv_n = 1.0f / static_cast<float>(a.n);
    int turn = 0;
    if (tile.cl > 1) cluster_wait_acquire();
    for (; tile.cta_row() < a.rows; tile.advance(), walk.next()) {
        __syncwarp();
        issue(walk.write, ahead);
        cp_async_wait(ahead);
        __syncwarp();
        const uint32_t from = ring + walk.read * walk.bytes;
        Slot<T> dy[K], x[K];
        tile.fetch(dy, from, 0);
        tile.fetch(x, from, 1);
        const bool ok = !WARP || tile.row < a.rows;
        const float mean = RMS || !ok ? 0.0f : stats[walk.read][0][tile.team];
        float rstd = RMS || !ok ? 0.0f : stats[walk.read][1][tile.team];
        // w = dy gamma and xh (RMSNorm: x) stay until the outputs.
        // LayerNorm: sums of w and w xh; RMSNorm: of x^2 and w x
        uint64_t w[K][4], xh[K][4];
        uint64_t s0 = 0, s1 = 0;
        const uint64_t minus = f2_pack(-mean, -mean);
        uint64_t scale = f2_pack(rstd, rstd);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t d = dy[k].pair(i);
                w[k][i] = f2_mul(d, gamma[k].pair(i));
                if (RMS) {
                    xh[k][i] = x[k].pair(i);
                    s0 = f2_fma(xh[k][i], xh[k][i], s0);
                } else {
                    xh[k][i] = f2_mul(f2_add(x[k].pair(i), minus), scale);
                    s0 = f2_add(s0, w[k][i]);
                    sum_g[k][i] = f2_fma(d, xh[k][i], sum_g[k][i]);
                    sum_b[k][i] = f2_add(sum_b[k][i], d);
                }
                s1 = f2_fma(w[k][i], xh[k][i], s1);
            }
        }
        float s[2] = {f2_sum(s0), f2_sum(s1)};
        row_sum<2, WARP>(s, slots, turn, tile.width, tile.cl, tile.crank);
        // ds = rstd w - rstd c1 - xh rstd c2
        float c1 = 0.0f, c2;
        if (RMS) {
            rstd = inv_sqrt(fmaf(s[0], inv_n, a.eps));
            scale = f2_pack(rstd, rstd);
            c2 = -(s[1] * inv_n * rstd) * rstd * rstd;
        } else {
            c1 = -(s[0] * inv_n) * rstd;
            c2 = -(s[1] * inv_n) * rstd;
        }
        const uint64_t c1p = f2_pack(c1, c1), c2p = f2_pack(c2, c2);
        if (a.dstream) tile.fetch(x, from, 2);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint64_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[i] = f2_fma(xh[k][i], c2p, RMS ? f2_mul(w[k][i], scale)
                                                 : f2_fma(w[k][i], scale, c1p));
                if (RMS) sum_g[k][i] = f2_fma(dy[k].pair(i), f2_mul(xh[k][i], scale), sum_g[k][i]);
            }
            if (a.dstream) {
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = f2_add(o[i], x[k].pair(i));
            }
            if (!ok) continue;
            Slot<T> out;
#pragma unroll
            for (int i = 0; i < 4; ++i) out.put_pair(i, o[i]);
            if (a.dres) {
                tile.store(dres, k, out);
                if (tile.in[k] != 0u) {
                    const DropGroup g = drop_group(key, tile.group(k), a.drop.threshold);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float lo, hi;
                        f2_unpack(o[i], lo, hi);
                        out.put_pair(i, f2_pack(drop_scale(lo, g.keeps(2 * i), a.drop.scale),
                                                drop_scale(hi, g.keeps(2 * i + 1), a.drop.scale)));
                    }
                }
            }
            tile.store(dx, k, out);
        }
    }
    cp_async_wait(0);
    if constexpr (!WARP) {
        // one partial row per CTA (or cluster), in slots: the join knows the row's offset
        const int64_t part = blockIdx.x / tile.cl;
#pragma unroll
        for (int which = 0; which < (RMS ? 1 : 2); ++which) {
            if (which == 1 && !part_beta) break;
            float *const out = (which == 0 ? part_gamma : part_beta) + part * part_stride;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (tile.in[k] == 0u) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    Frag<F32, 4> v;
                    float f[4];
                    f2_unpack(which == 0 ? sum_g[k][2 * i] : sum_b[k][2 * i], f[0], f[1]);
                    f2_unpack(which == 0 ? sum_g[k][2 * i + 1] : sum_b[k][2 * i + 1], f[2], f[3]);
                    v.put(f);
                    st_global(out + (tile.first + k * tile.width) * 8 + 4 * i, v);
                }
            }
        }
    } else {
        // the rows' sums of this CTA through the ring, in slots; then one column per thread,
        // over the rows in order
        const int span = K * tile.width * 8;
        const int teams = static_cast<int>(blockDim.x) / tile.width;
        const int64_t row0 = static_cast<int64_t>(blockIdx.x) * teams;
        float *const buf = reinterpret_cast<float *>(ring_bytes);
#pragma unroll
        for (int which = 0; which < (RMS ? 1 : 2); ++which) {
            if (which == 1 && !part_beta) break;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                uint64_t *to = reinterpret_cast<uint64_t *>(buf + tile.team * span +
                                                            (tile.first + k * tile.width) * 8);
#pragma unroll
                for (int i = 0; i < 4; ++i) to[i] = which == 0 ? sum_g[k][i] : sum_b[k][i];
            }
            __syncthreads();
            float *const out = (which == 0 ? part_gamma : part_beta) +
                               static_cast<int64_t>(blockIdx.x) * part_stride;
            for (int j = threadIdx.x; j < static_cast<int>(a.n); j += blockDim.x) {
                float v = 0.0f;
                for (int g = 0; g < teams; ++g) {
                    const int off = EDGE ? static_cast<int>((t.mis + (row0 + g) * a.n) & 7) : 0;
                    v += buf[g * span + j + off];
                }
                out[j] = v;
            }
        }
    }
}

template <class T, int K, bool EDGE, bool WARP, bool RMS>
cudaError_t launch_backward_tile(const BackwardArgs &a, const TilePlan &p, float *pg, float *pb,
                                 bool pdl, cudaStream_t stream, uint64_t *launches) {
    static TileLaunchCache cache;
    const TileArgs t = {p.lanes, p.stages, p.mis};
    const int64_t shared = tile_ring_bytes(T::kBytes, K, p.threads, p.stages, a.dstream ? 3 : 2);
    return launch_tile(cache, mrn_norm_backward_tile_kernel<T, K, EDGE, WARP, RMS>, p, shared, pdl,
                       stream, launches, a, t, pg, pb, part_stride_of(a.n));
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

// dgamma (blockIdx.y == 0) and dbeta (1): the sum of `parts` partial rows.  A CTA owns 32
// columns; its 32 warps take every 32nd partial row each, eight loads in flight, and are
// joined in shared memory, in order.  shifted: partial row p starts as row p of the matrix
// does, (mis + p n) mod 8 elements into its first slot.
constexpr int kJoinColumns = 32;
constexpr int kJoinThreads = 1024;
constexpr int kJoinFlight = 8;

struct JoinArgs {
    const float *part_gamma, *part_beta;
    float *dgamma, *dbeta;
    int64_t parts, n, stride;
    int mis;
    bool shifted;
};

__global__ void __launch_bounds__(kJoinThreads) mrn_norm_backward_join_kernel(const JoinArgs a) {
    __shared__ float sums[32][kJoinColumns + 1];
    pdl_enter();
    const float *part = blockIdx.y == 0 ? a.part_gamma : a.part_beta;
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kJoinColumns + lane;
    float s = 0.0f;
    for (int64_t p0 = warp; p0 < a.parts; p0 += 32 * kJoinFlight) {
        float v[kJoinFlight];
#pragma unroll
        for (int i = 0; i < kJoinFlight; ++i) {
            const int64_t p = p0 + 32 * i;
            const int64_t off = a.shifted ? (a.mis + p * a.n) & 7 : 0;
            v[i] = p < a.parts && j < a.n ? part[p * a.stride + off + j] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kJoinFlight; ++i) s += v[i];
    }
    sums[warp][lane] = s;
    __syncthreads();
    // warp c adds up column c: lane w holds warp w's sum
    const float t = warp_allsum(sums[lane][warp]);
    const int64_t jc = static_cast<int64_t>(blockIdx.x) * kJoinColumns + warp;
    if (lane == 0 && jc < a.n) (blockIdx.y == 0 ? a.dgamma : a.dbeta)[jc] = t;
}

cudaError_t launch_join(const JoinArgs &a, bool pdl, cudaStream_t stream, uint64_t *launches) {
    const int64_t ctas = (a.n + kJoinColumns - 1) / kJoinColumns;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), a.dbeta ? 2 : 1, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, mrn_norm_backward_join_kernel, a);
    if (err == cudaSuccess) ++*launches;
    return err;
}

template <class T>
cudaError_t launch_backward_typed(const BackwardArgs &a, int sms, bool pdl, cudaStream_t stream,
                                  uint64_t *launches) {
    const int64_t most = backward_parts(a.rows, a.n, sms);
    JoinArgs join = {};
    join.dgamma = a.dgamma;
    join.dbeta = a.dbeta;
    join.n = a.n;
    join.stride = part_stride_of(a.n);
    if (most == 0) return launch_join(join, pdl, stream, launches);
    const int mis = common_offset(T::kBytes, a.dy, a.x, a.dstream, static_cast<const void *>(a.dx),
                                  static_cast<const void *>(a.dres));
    TilePlan p = {};
    // (a generator group is a slot only when the operands start on a slot boundary)
    if (mis == 0 || (mis > 0 && a.drop.threshold == 0)) {
        const TileWish wish = {a.dstream ? 3 : 2, 2, 512, kPartsPerSm};
        p = plan_tiles(a.rows, a.n, T::kBytes, mis, wish, sms);
    }
    const int64_t parts = p.ok ? p.ctas / p.cluster : most;
    if (parts > most) return cudaErrorInvalidConfiguration;   // (the workspace holds `most`)
    float *pg = a.workspace;
    float *pb = a.dbeta ? a.workspace + parts * join.stride : nullptr;
    cudaError_t err;
    if (p.ok && p.warp) {
        err = p.k == 1   ? launch_backward_k<T, 1, true>(a, p, pg, pb, pdl, stream, launches)
              : p.k == 2 ? launch_backward_k<T, 2, true>(a, p, pg, pb, pdl, stream, launches)
                         : launch_backward_k<T, 4, true>(a, p, pg, pb, pdl, stream, launches);
    } else if (p.ok) {
        err = p.k == 1   ? launch_backward_k<T, 1, false>(a, p, pg, pb, pdl, stream, launches)
              : p.k == 2 ? launch_backward_k<T, 2, false>(a, p, pg, pb, pdl, stream, launches)
              : p.k == 3 ? launch_backward_k<T, 3, false>(a, p, pg, pb, pdl, stream, launches)
                         : launch_backward_k<T, 4, false>(a, p, pg, pb, pdl, stream, launches);
    } else {
        const auto fn = a.rms ? mrn_norm_backward_looped_kernel<T, true>
                              : mrn_norm_backward_looped_kernel<T, false>;
        err = launch_plain(fn, parts, kLoopedThreads, 0, pdl, stream, launches, a, pg, pb, join.stride);
    }
    if (err != cudaSuccess) return err;
    join.part_gamma = pg;
    join.part_beta = pb;
    join.parts = parts;
    join.mis = p.mis;
    join.shifted = p.ok && p.edge && !p.warp;
    return launch_join(join, pdl, stream, launches);
}

cudaError_t launch_norm_backward(bool bf16, const BackwardArgs &a, int sms, bool pdl,
                                 cudaStream_t stream, uint64_t *launches) {
    return bf16 ? launch_backward_typed<BF16>(a, sms, pdl, stream, launches)
                : launch_backward_typed<F32>(a, sms, pdl, stream, launches);
}

}  // namespace mrn
