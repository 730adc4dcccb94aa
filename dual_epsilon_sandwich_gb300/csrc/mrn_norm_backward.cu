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

// Threads that an SM's registers are shared between (the launch bound): what a thread with k
// slots needs.
constexpr int backward_resident(int k) { return k <= 1 ? 768 : (k <= 2 ? 512 : (k <= 3 ? 384 : 256)); }

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
// element of them read and written by one thread only.  For the calls that the tile kernel
// does not take, as in the forward; 16384 x 4096 bf16, x an element off the others, 296 us
// (the tile kernel: 76).
template <class T, bool RMS>
__global__ void __launch_bounds__(kLoopedThreads)
mrn_norm_backward_looped_kernel(const BackwardArgs a, float *part_gamma, float *part_beta,
                                const int64_t part_stride) {
    __shared__ CtaSumHalves slots;
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

// Rows held in registers between their copy and their outputs, the column sums in
// registers over all rows of the CTA (see mrn_row_tile.cuh).  Each operand is read once, and
// both sums of a row are taken together, so a row costs one barrier.  Measured on GB300, with
// the join: 16384 x 4096 bf16 76 us (5.3 TB/s, 78 % of the copy's rate), with dropout and a
// stream's gradient 121 us (5.5 TB/s); 16384 x 4095 bf16 with both 139 us (4.8 TB/s); 4096 x
// 6656 f32 with both 95 us (5.7 TB/s); RMSNorm 163840 x 128 bf16 24 us (5.2 TB/s), 4096 x 16384
// f32 in clusters 178 to 188 us on several GPUs (5.7 to 6.0 TB/s).
//   What bounds it: the instructions of the 16 warps that the registers of the column sums leave
// room for (issued in 54 % of cycles under ncu, dram 60 to 65 % busy; waits for shared memory
// and for results of arithmetic come first), then the join with its launch, 4 to 6 us.  Where
// rows start off a slot boundary, the warp that holds their ends lets the others wait (barriers
// are then the first stall) and half of the rows' sectors are written in two parts.
template <class T, int K, bool EDGE, bool WARP, bool RMS>
__global__ void __launch_bounds__(backward_resident(K))
mrn_norm_backward_tile_kernel(const BackwardArgs a, const TileArgs t, float *part_gamma,
                              float *part_beta, const int64_t part_stride) {
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    __shared__ RowSumSlots<2, T::kBytes == 2 && !RMS> slots;
    __shared__ float stats[kTileMaxStages][2][kWarpTileThreads];   // mean and rstd, per team
    __shared__ EndSlots<3, 1, EDGE, WARP> end_w;
    RowTile<T, K, 1, EDGE, WARP> tile(a.rows, a.n, t);
    const int ops_count = a.dstream ? 3 : 2;
    const int64_t back = static_cast<int64_t>(t.mis) * T::kBytes;
    const char *const ops[3] = {
        static_cast<const char *>(a.dy) - back, static_cast<const char *>(a.x) - back,
        a.dstream ? static_cast<const char *>(a.dstream) - back : nullptr};
    char *const dx = static_cast<char *>(a.dx) - back;
    char *const dres = a.dres ? static_cast<char *>(a.dres) - back : nullptr;
    RingWalk walk(tile.stage_bytes(ops_count), t.stages);
    const int ahead = t.stages - 1;
    const uint32_t ring = tile.warp_ring(static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes)), t.stages, ops_count);
    tile.clear(ring, t.stages, ops_count);
    row_sum_setup(slots, tile.cl);
    pdl_enter();
    // mean and rstd travel with their row: a load of them in the loop held up every row
    // (16384 x 4096 bf16: 116 us against 80)
    const float *mean_of = RMS ? nullptr : a.mean + tile.row, *rstd_of = RMS ? nullptr : a.rstd + tile.row;
    auto issue = [&](int to) {
        if (!RMS && tile.leads) {
            if (tile.copy_left > 0) {
                cp_async4(static_cast<uint32_t>(__cvta_generic_to_shared(&stats[to][0][tile.team])), mean_of);
                cp_async4(static_cast<uint32_t>(__cvta_generic_to_shared(&stats[to][1][tile.team])), rstd_of);
            }
            mean_of += tile.stride;
            rstd_of += tile.stride;
        }
        tile.issue(ring + to * walk.bytes, to, ops, ops_count, end_w);
    };
    for (int s = 0; s < ahead; ++s) issue(s);
    const DropKey key = drop_key(a.drop);
    Slot<T> gamma[K];
    tile.weights(gamma, a.gamma);
    uint64_t sum_g[K][4], sum_b[K][4];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum_g[k][i] = sum_b[k][i] = 0;
    const float end_gamma = EDGE ? tile.end_weight(a.gamma) : 0.0f;
    float end_sum_g = 0.0f, end_sum_b = 0.0f;
    const float inv_n = 1.0f / static_cast<float>(a.n);
    int turn = 0;
    row_sum_ready(tile.cl);
    for (; tile.cta_left > 0; tile.advance(), walk.next()) {
        __syncwarp();
        issue(walk.write);
        cp_async_wait(ahead);
        __syncwarp();
        const uint32_t from = ring + walk.read * walk.bytes;
        const bool ok = !WARP || tile.valid(0);
        // w = dy gamma and xh (RMSNorm: x) stay until the outputs.
        // LayerNorm: sums of w and w xh; RMSNorm: of x^2 and w x
        uint64_t w[K][4], xh[K][4];
        Slot<T> dy[K], x[K];
        tile.fetch(dy, from, 0, 0, ops_count);
        tile.fetch(x, from, 1, 0, ops_count);
        const float mean = RMS || !ok ? 0.0f : stats[walk.read][0][tile.team];
        float rstd = RMS || !ok ? 0.0f : stats[walk.read][1][tile.team];
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
        float end_d = 0.0f, end_xh = 0.0f, end_o = 0.0f;
        if (EDGE && tile.ends) {
            end_d = tile.fetch_end(end_w, walk.read, 0, 0);
            end_xh = tile.fetch_end(end_w, walk.read, 1, 0);
            const float ew = end_d * end_gamma;
            if (RMS) {
                s[0] = fmaf(end_xh, end_xh, s[0]);
            } else {
                // (lanes without an element have d = 0, and xh is then of no effect)
                end_xh = (end_xh - mean) * rstd;
                s[0] += ew;
                end_sum_g = fmaf(end_d, end_xh, end_sum_g);
                end_sum_b += end_d;
            }
            s[1] = fmaf(ew, end_xh, s[1]);
        }
        if (!row_sum<WARP>(s, slots, turn, tile.width, tile.cl, tile.crank, turn == 0 ? t.stall : 0u)) break;
        // ds = rstd w - rstd c1 - xh rstd c2
        float c1 = 0.0f, c2;
        if (RMS) {
            rstd = inv_sqrt(fmaf(s[0], inv_n, a.eps));
            scale = f2_pack(rstd, rstd);
            s[1] *= rstd;
            // xh itself, and dy once more for dgamma
            tile.fetch(dy, from, 0, 0, ops_count);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    xh[k][i] = f2_mul(xh[k][i], scale);
                    sum_g[k][i] = f2_fma(dy[k].pair(i), xh[k][i], sum_g[k][i]);
                }
            end_xh *= rstd;
        } else {
            c1 = -(s[0] * inv_n) * rstd;
        }
        c2 = -(s[1] * inv_n) * rstd;
        const uint64_t c1p = f2_pack(c1, c1), c2p = f2_pack(c2, c2);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[k][i] = f2_fma(xh[k][i], c2p, RMS ? f2_mul(w[k][i], scale) : f2_fma(w[k][i], scale, c1p));
        }
        if (a.dstream) {
            tile.fetch(x, from, 2, 0, ops_count);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) w[k][i] = f2_add(w[k][i], x[k].pair(i));
        }
        Slot<T> out[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[k].put_pair(i, w[k][i]);
        if (EDGE && tile.ends) {
            const float ew = end_d * end_gamma;
            float o = fmaf(end_xh, c2, RMS ? ew * rstd : fmaf(ew, rstd, c1));
            if (RMS) end_sum_g = fmaf(end_d, end_xh, end_sum_g);
            if (a.dstream) o += tile.fetch_end(end_w, walk.read, 2, 0);
            end_o = o;
            tile.store_end(a.dres ? dres : dx, 0, ok, o);
        }
        if (a.dres) {
            DropGroup g[K];
            const bool end_keep = tile.masks(g, key, 0, a.drop.threshold);
            tile.store(dres, 0, ok, out);
            if (EDGE && tile.ends) tile.store_end(dx, 0, ok, drop_scale(end_o, end_keep, a.drop.scale));
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    f2_unpack(w[k][i], lo, hi);
                    out[k].put_pair(i, f2_pack(drop_scale(lo, g[k].keeps(2 * i), a.drop.scale),
                                               drop_scale(hi, g[k].keeps(2 * i + 1), a.drop.scale)));
                }
            }
        }
        tile.store(dx, 0, ok, out);
    }
    cp_async_wait(0);
    row_sum_leave(tile.cl);
    // Column j of a partial row stands at j + 8 - before, so that slots are aligned; the join
    // knows `before` from the row's number.
    if constexpr (!WARP) {
        const int64_t part = blockIdx.x / tile.cl;
#pragma unroll
        for (int which = 0; which < (RMS ? 1 : 2); ++which) {
            if (which == 1 && !part_beta) break;
            float *const out = (which == 0 ? part_gamma : part_beta) + part * part_stride + (EDGE ? 8 : 0);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!tile.holds(k)) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    Frag<F32, 4> v;
                    float f[4];
                    f2_unpack(which == 0 ? sum_g[k][2 * i] : sum_b[k][2 * i], f[0], f[1]);
                    f2_unpack(which == 0 ? sum_g[k][2 * i + 1] : sum_b[k][2 * i + 1], f[2], f[3]);
                    v.put(f);
                    st_global(out + (tile.first + k * tile.slot_step()) * 8 + 4 * i, v);
                }
            }
            if (EDGE && tile.end_col >= 0)
                out[tile.end_col - tile.before] = which == 0 ? end_sum_g : end_sum_b;
        }
    } else {
        // the rows' sums of this CTA through the ring, laid out the same; then one column per
        // thread, over the rows in order
        const int span = K * tile.width * 8 + (EDGE ? 16 : 0);
        const int teams = static_cast<int>(blockDim.x) / tile.width;
        const int64_t row0 = static_cast<int64_t>(blockIdx.x) * teams;
        float *const buf = reinterpret_cast<float *>(ring_bytes);
#pragma unroll
        for (int which = 0; which < (RMS ? 1 : 2); ++which) {
            if (which == 1 && !part_beta) break;
            __syncthreads();
            float *const mine = buf + tile.team * span + (EDGE ? 8 : 0);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!tile.holds(k)) continue;
                uint64_t *to = reinterpret_cast<uint64_t *>(mine + (tile.first + k * tile.slot_step()) * 8);
#pragma unroll
                for (int i = 0; i < 4; ++i) to[i] = which == 0 ? sum_g[k][i] : sum_b[k][i];
            }
            if (EDGE && tile.end_col >= 0)
                mine[tile.end_col - tile.before] = which == 0 ? end_sum_g : end_sum_b;
            __syncthreads();
            float *const out = (which == 0 ? part_gamma : part_beta) +
                               static_cast<int64_t>(blockIdx.x) * part_stride;
            for (int j = threadIdx.x; j < static_cast<int>(a.n); j += blockDim.x) {
                float v = 0.0f;
                for (int g = 0; g < teams; ++g) {
                    const int off = EDGE ? 8 - static_cast<int>(-(t.mis + (row0 + g) * a.n) & 7) : 0;
                    v += buf[g * span + j + off];
                }
                out[j] = v;
            }
        }
    }
}

struct BackwardLaunch {
    int sms;
    bool pdl;
    cudaStream_t stream;
    uint64_t *launches;
    int64_t most_parts;
    int64_t parts;      // out: partial rows written
    cudaError_t err;    // out
};

// Whether the call was launched; false: it takes the looped kernel.
template <class T, int K, bool EDGE, bool WARP, bool RMS>
bool launch_backward_tile(const BackwardArgs &a, const TileShape &p, BackwardLaunch &l) {
    static TileLaunchCache cache;
    const auto fn = mrn_norm_backward_tile_kernel<T, K, EDGE, WARP, RMS>;
    const int operands = a.dstream ? 3 : 2;
    TileGrid g;
    l.err = tile_grid(cache, fn, p, a.rows, a.n, 1, T::kBytes, operands, kPartsPerSm, l.sms, &g);
    if (l.err != cudaSuccess) return true;
    l.parts = g.ctas / p.cluster;
    if (g.stages < 1 || l.parts > l.most_parts) return false;   // (the workspace holds no more)
    const TileArgs t = {p.lanes, g.stages, p.mis, a.stall};
    const int64_t stride = part_stride_of(a.n);
    // (WARP: the epilogue's rows have room for the ends)
    l.err = launch_tile(fn, p, g.ctas, g.shared + (WARP ? 1024 : 0),
                        l.pdl, l.stream, l.launches, a, t, a.workspace,
                        a.dbeta ? a.workspace + l.parts * stride : nullptr, stride);
    return true;
}

template <class T, int K, bool WARP>
bool launch_backward_k(const BackwardArgs &a, const TileShape &p, BackwardLaunch &l) {
    if (a.rms)
        return p.edge ? launch_backward_tile<T, K, true, WARP, true>(a, p, l)
                      : launch_backward_tile<T, K, false, WARP, true>(a, p, l);
    return p.edge ? launch_backward_tile<T, K, true, WARP, false>(a, p, l)
                  : launch_backward_tile<T, K, false, WARP, false>(a, p, l);
}

// dgamma (blockIdx.y == 0) and dbeta (1): the sum of `parts` partial rows.  A CTA owns
// 32 * C columns; its warps take every nth partial row each, all their loads in flight at
// once where there are few enough, and are joined in shared memory, in order: one trip to L2,
// which bounds it.  304 rows of 4096 columns, two sums (10 MB): 6.7 us alone out of DRAM under
// ncu, about 4 behind its backward, whose last rows are still in L2.  shifted: column
// j of partial row p stands where the tile kernel left it, at j + 8 - (the elements from row
// p's start to the next slot boundary).
struct JoinArgs {
    const float *part_gamma, *part_beta;
    float *dgamma, *dbeta;
    int64_t parts, n, stride;
    int mis;
    bool shifted;
};

template <int WARPS, int C, int kJoinFlight>
__global__ void __launch_bounds__(WARPS * 32) mrn_norm_backward_join_kernel(const JoinArgs a) {
    __shared__ float sums[WARPS][C * 32];
    pdl_enter();
    const float *part = blockIdx.y == 0 ? a.part_gamma : a.part_beta;
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * (32 * C) + lane;
    float s[C];
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = 0.0f;
    for (int64_t p0 = warp; p0 < a.parts; p0 += WARPS * kJoinFlight) {
        float v[kJoinFlight][C];
#pragma unroll
        for (int i = 0; i < kJoinFlight; ++i) {
            const int64_t p = p0 + WARPS * i;
            const int64_t off = a.shifted ? 8 - (-(a.mis + p * a.n) & 7) : 0;
            const float *from = part + p * a.stride + off + j0;
#pragma unroll
            for (int c = 0; c < C; ++c)
                v[i][c] = p < a.parts && j0 + 32 * c < a.n ? from[32 * c] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kJoinFlight; ++i)
#pragma unroll
            for (int c = 0; c < C; ++c) s[c] += v[i][c];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) sums[warp][32 * c + lane] = s[c];
    __syncthreads();
    for (int c = threadIdx.x; c < 32 * C; c += WARPS * 32) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) t += sums[w][c];
        const int64_t j = static_cast<int64_t>(blockIdx.x) * (32 * C) + c;
        if (j < a.n) (blockIdx.y == 0 ? a.dgamma : a.dbeta)[j] = t;
    }
}

template <int WARPS, int C, int FLIGHT>
cudaError_t launch_join_typed(const JoinArgs &a, bool pdl, cudaStream_t stream, uint64_t *launches) {
    const int64_t ctas = (a.n + 32 * C - 1) / (32 * C);
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), a.dbeta ? 2 : 1, 1);
    cfg.blockDim = dim3(WARPS * 32, 1, 1);
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, mrn_norm_backward_join_kernel<WARPS, C, FLIGHT>, a);
    if (err == cudaSuccess) ++*launches;
    return err;
}

cudaError_t launch_join(const JoinArgs &a, bool pdl, cudaStream_t stream, uint64_t *launches) {
    // (measured on GB300, us a call with 608 partial rows, 32 warps of 32 columns against 16 of 64:
    // 163840 x 128 bf16 24.2, 26.0;  65536 x 1024 bf16 71.0, 71.7;  32768 x 2048 80.0, 81.5;  16384 x
    // 4096 76.3, 75.8;  4096 x 6656 f32 61.9, 59.1)
    return a.n <= 1024 ? launch_join_typed<32, 1, 20>(a, pdl, stream, launches)
                       : launch_join_typed<16, 2, 10>(a, pdl, stream, launches);
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
    BackwardLaunch l = {sms, pdl, stream, launches, most, most, cudaSuccess};
    bool done = false;
    // (a generator group is a slot only when the operands start on a slot boundary)
    if (mis == 0 || (mis > 0 && a.drop.threshold == 0)) {
        // Slots per thread (k) for rows of a CTA, and threads of one at most.  Measured on GB300 (us),
        // with dropout and a stream's gradient 671 MB a call, LayerNorm's alone ("ln") 403 MB:
        //   bf16  n = 1536 2 119.1, 4 125.2;  2048 126.5, 117.6;  2560 126.3, 137.7;  4095 139.1,
        //         141.1;  4096 121.2, 117.0;  5120 141.6, 145.5;  5632 136.5, 140.1;  6656 139.6,
        //         135.2;  6655 161.0, 149.6;  8192 130.9, 129.1;  ln: 2559 83.0, 104.5;  4096 76.6,
        //         80.2;  4095 86.1, 84.6;  5120 91.9, 90.4;  6656 88.1, 84.3;  8191 94.0, 88.4;
        //         rmsnorm with a stream's gradient 5120 102.5, 110.9;  8192 94.3, 98.4;  rows of
        //         16384 in clusters of CTAs of 64 threads 4 129.3, of 128 135.5, of 256 145.5
        //   f32   n = 1152 3 122.4, 4 133.7;  1280 126.0, 123.7;  1536 125.8, 118.9;  1792 121.9,
        //         124.0;  2048 122.4, 125.8;  2304 123.0, 113.0;  2560 121.0, 113.2;  2816 121.6,
        //         120.4;  3328 122.2, 123.9;  4096 110.9, 125.4;  4104 122.4, 133.3;  4480 115.5,
        //         116.6;  4608 119.6, 114.8;  5120 121.2, 113.7;  6656 123.3, 116.2;  ln: 1408 83.0,
        //         74.0;  1544 81.5, 82.0;  2560 79.3, 73.6;  4352 77.9, 82.3;  odd widths 2047 2
        //         128.9, 4 132.4;  2559 131.1, 125.3;  4095 2 131.2, 3 152.4, 4 125.8;  5119 2
        //         119.1, 4 127.3;  6655 2 119.6, 3 133.2, 4 119.1;  8191 3 145.7, 4 121.4
        //         16384 in clusters of CTAs of 256 threads 4 117.8, 2 120.4, of 64 4 118.3;  16383
        //         of 64 123.0, of 256 135.8;  rmsnorm with a stream's gradient (537 MB) 12288 4 93.0,
        //         2 of 512 96.1;  16384 99.4, 94.9;  24576 of 128 94.8, 2 of 512 102.7;  32768 of 128
        //         96.3, of 256 98.4;  65536 of 128 117.6, of 256 114.0, 2 of 512 117.3
        // bf16: two slots also where four win at aligned widths only (2048, 4096): beside them, and at
        // odd widths, four lose more.
        const int64_t slots = a.n / 8;
        const bool edge = mis != 0 || a.n % 8 != 0;
        int k;
        if (T::kBytes == 2) {
            k = slots > 1024 || (a.dres && slots > 640) ? 4 : 2;
        } else {
            const bool four = edge || slots > 560 || (slots >= 160 && slots <= 192) ||
                              (slots > 256 && slots <= 352);
            k = four ? 4 : 3;
        }
        int most_threads = backward_resident(k);
        if (slots > 1024 && (T::kBytes == 2 || edge || slots > 2048))
            most_threads = slots <= 2048 ? 64 : (slots <= (T::kBytes == 2 ? 4096 : 8192) ? 128 : 256);
        const bool few = tile_few_rows(a.rows, a.n, sms);
        if (few) {
            k = 1;
            most_threads = tile_few_threads(a.rows, a.n, sms);
        }
        const TileShape p = tile_shape(a.n, mis, k, most_threads, few);
        if (p.ok && p.warp) {
            done = p.k == 1   ? launch_backward_k<T, 1, true>(a, p, l)
                   : p.k == 2 ? launch_backward_k<T, 2, true>(a, p, l)
                   : p.k == 3 ? launch_backward_k<T, 3, true>(a, p, l)
                              : launch_backward_k<T, 4, true>(a, p, l);
        } else if (p.ok) {
            if (k == 1) {
                done = launch_backward_k<T, 1, false>(a, p, l);
            } else if (k == 4) {
                done = launch_backward_k<T, 4, false>(a, p, l);
            } else if constexpr (T::kBytes == 2) {
                done = launch_backward_k<T, 2, false>(a, p, l);
            } else {             // (three: aligned rows)
                done = a.rms ? launch_backward_tile<T, 3, false, false, true>(a, p, l)
                             : launch_backward_tile<T, 3, false, false, false>(a, p, l);
            }
        }
        join.mis = mis;
        join.shifted = done && p.edge && !p.warp;
    }
    if (!done) {
        const auto fn = a.rms ? mrn_norm_backward_looped_kernel<T, true>
                              : mrn_norm_backward_looped_kernel<T, false>;
        l.parts = most;
        l.err = launch_plain(fn, most, kLoopedThreads, 0, pdl, stream, launches, a, a.workspace,
                             a.dbeta ? a.workspace + most * join.stride : nullptr, join.stride);
    }
    if (l.err != cudaSuccess) return l.err;
    join.part_gamma = a.workspace;
    join.part_beta = a.dbeta ? a.workspace + l.parts * join.stride : nullptr;
    join.parts = l.parts;
    return launch_join(join, pdl, stream, launches);
}

cudaError_t launch_norm_backward(bool bf16, const BackwardArgs &a, int sms, bool pdl,
                                 cudaStream_t stream, uint64_t *launches) {
    return bf16 ? launch_backward_typed<BF16>(a, sms, pdl, stream, launches)
                : launch_backward_typed<F32>(a, sms, pdl, stream, launches);
}

int take_wait_timeouts_norm_backward() { return take_wait_timeouts<kOpBackwardTimeouts>(); }

}  // namespace mrn
