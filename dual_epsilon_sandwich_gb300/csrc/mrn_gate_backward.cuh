// mrn_gate_backward.cuh -- the gradient of the gated sandwich tail (one translation unit per type).  Per row, with
// i1 = inv(b; eps1), i2 = inv(s; eps2), w = dn * g2, c = g1 (times the gate, when that is one
// value per channel), g the gate otherwise, xh = b * i1:
//   ds = i2 * (w - s * i2^2 * mean(w s)) + dstream
//   db = i1 * (g ds c - xh * mean(g ds c xh)),   dres = scale * ds
// and over rows
//   P_j = sum_r dn s i2 = dg2_j,   A_j = sum_r g ds xh,   R_j = sum_r ds res
// which give dg1 = gate A and dgate = g1 A for a gate per channel, dg1 = A otherwise; with
// q_r = sum_j ds c xh, dgate = q_r per row, sum_r q_r for a scalar.
//   Both means are known after one reduction of a row: with
//   S1 = sum s^2, S2 = sum w s, S3 = sum b^2, S4 = sum w c b, S5 = sum s c b, S6 = sum dstream c b
// q = i1 * (i2 * (S4 - (i2 S2 / n) * (i2 S5)) + S6): the sum of ds c xh term by term, so that what
// cancels in it is what cancels in ds itself.
// The products are of the operands as they are, since i1 and i2 are not known yet: rows whose
// |dn| |b| add up past f32's largest number are outside of the operation's range, as the public
// header says.  (Products of xh would take a second reduction.)
//   The column sums are taken on the same pass: every CTA adds up the rows it handles (fixed
// rows, in order) and leaves a row of partial sums per set in the workspace, which a second
// launch adds in order.  No atomics: the result does not depend on which CTA ran when.
#pragma once

#include "mrn_gate_kernels.cuh"

namespace mrn {

constexpr int kLoopedThreads = 512;

// 1 / sqrt(v) within one unit: rsqrtf and a step of Newton's (0 at infinity, as rsqrtf).  Its error is
// the whole row's, and does not average out in the sums over rows that scalar factors take.
__device__ __forceinline__ float inv_sqrt_refined(float v) {
    const float y = rsqrtf(v);
    return v < INFINITY ? fmaf(0.5f * y, fmaf(-v * y, y, 1.0f), y) : y;
}

// What a row's six sums give.
struct RowScalars {
    float i1, i2;     // inv of the block's row, of the stream's
    float m;          // -i2 * mean(w s) * i2, the factor of xh_s = s i2 in ds
    float q;          // sum_j ds c xh
};
__device__ __forceinline__ RowScalars row_scalars(const float (&s)[6], float inv_n, float eps1, float eps2) {
    RowScalars r;
    r.i1 = inv_sqrt_refined(fmaf(s[2], inv_n, eps1));
    r.i2 = inv_sqrt_refined(fmaf(s[0], inv_n, eps2));
    const float mean = r.i2 * (s[1] * inv_n);
    r.m = -mean * r.i2;
    r.q = r.i1 * fmaf(r.i2, s[3], fmaf(r.m, r.i2 * s[4], s[5]));
    return r;
}

// Where a call's partial sums stand.
struct GateParts {
    float *pre, *post, *res;   // [parts x stride] each; res NULL: not due
    double *gate, *scale;      // partial sums of the scalar factors, one per CTA; NULL: not due
    int64_t stride;
};

// a += v with the rounding's loss kept in b (Knuth's two-sum, "The Art of Computer Programming",
// volume 2, 4.2.2).
__device__ __forceinline__ void add_kept(float &a, float &b, float v) {
    const float s = a + v;
    const float w = s - a;
    b += (a - (s - w)) + (v - w);
    a = s;
}

// The sum over a warp of values kept that way.
__device__ __forceinline__ double warp_sum_kept(float a, float b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float c = __shfl_xor_sync(0xFFFFFFFFu, a, o), d = __shfl_xor_sync(0xFFFFFFFFu, b, o);
        add_kept(a, b, c);
        b += d;
    }
    // (an infinite sum has lost NaN)
    return fabsf(a) < INFINITY ? static_cast<double>(a) + static_cast<double>(b) : static_cast<double>(a);
}

// A CTA's share of the scalar factors' gradients, each a sum and what its roundings lost: they are
// sums over all elements, and what these leave behind cancelling is small.  (In f32 pairs: an SM does
// two 64-bit additions a clock.)
__device__ __forceinline__ void leave_scalars(float gate, float gate_lost, float scale, float scale_lost,
                                              const GateParts &parts, double (&s)[2][kCtaWarps]) {
    if (!parts.gate && !parts.scale) return;
    const double g = warp_sum_kept(gate, gate_lost), c = warp_sum_kept(scale, scale_lost);
    if ((threadIdx.x & 31) == 0) {
        s[0][threadIdx.x >> 5] = g;
        s[1][threadIdx.x >> 5] = c;
    }
    __syncthreads();
    if (threadIdx.x >= 2) return;
    double sum = 0.0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) sum += s[threadIdx.x][w];
    double *const to = threadIdx.x == 0 ? parts.gate : parts.scale;
    if (to) to[blockIdx.x] = sum;
}

// Any width and any alignment: one row per CTA at a time, two passes over it (the second out of
// L2), element by element; the partial sums live in the workspace, each element of them read
// and written by one thread only.  For the calls that the tiles do not take; 16384 x 4096 bf16 with all
// gradients 1115 us (the tiles: 169).
template <class T>
__global__ void __launch_bounds__(kLoopedThreads)
mrn_gate_backward_looped_kernel(const GateBackwardArgs a, const GateParts parts) {
    __shared__ CtaSumSix slots;
    __shared__ double last[2][kCtaWarps];
    cta_sum_setup(slots);
    pdl_enter();
    int turn = 0;
    const float inv_n = 1.0f / static_cast<float>(a.n);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * parts.stride;
    const bool channel = a.gate.kind == MRN_FACTOR_CHANNEL;
    float gates = 0.0f, gates_lost = 0.0f, scales = 0.0f, scales_lost = 0.0f;
    bool fresh = true;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t e0 = r * a.n;
        float s[6] = {};
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const float v = ld_elem<T>(a.s, e0 + j), b = ld_elem<T>(a.b, e0 + j);
            const float w = ld_elem<T>(a.dn, e0 + j) * ld_elem<T>(a.g2, j);
            const float cb = b * (channel ? ld_elem<T>(a.g1, j) * factor_at<T>(a.gate, r, j) : ld_elem<T>(a.g1, j));
            s[0] = fmaf(v, v, s[0]);
            s[1] = fmaf(w, v, s[1]);
            s[2] = fmaf(b, b, s[2]);
            s[3] = fmaf(w, cb, s[3]);
            s[4] = fmaf(v, cb, s[4]);
            if (a.dstream) s[5] = fmaf(ld_elem<T>(a.dstream, e0 + j), cb, s[5]);
        }
        cta_sum(s, slots, turn);
        const RowScalars k = row_scalars(s, inv_n, a.eps1, a.eps2);
        const float g = channel ? 1.0f : factor_at<T>(a.gate, r, 0);
        const float c2 = -k.i1 * (g * (k.q * inv_n));
        float gated = 0.0f, scaled = 0.0f;
        for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
            const int64_t e = e0 + j;
            const float dn = ld_elem<T>(a.dn, e);
            const float vh = ld_elem<T>(a.s, e) * k.i2;
            const float xh = ld_elem<T>(a.b, e) * k.i1;
            float ds = fmaf(vh, k.m, dn * ld_elem<T>(a.g2, j) * k.i2);
            if (a.dstream) ds += ld_elem<T>(a.dstream, e);
            const float dsg = ds * g;
            const float c = channel ? ld_elem<T>(a.g1, j) * factor_at<T>(a.gate, r, j) : ld_elem<T>(a.g1, j);
            const float res = parts.res || parts.scale ? ld_elem<T>(a.res, e) : 0.0f;
            st_elem<T>(a.db, e, fmaf(xh, c2, dsg * c * k.i1));
            st_elem<T>(a.dres, e, factor_at<T>(a.scale, r, j) * ds);
            float *p = parts.pre + at + j;
            *p = fmaf(dn, vh, fresh ? 0.0f : *p);
            p = parts.post + at + j;
            *p = fmaf(dsg, xh, fresh ? 0.0f : *p);
            if (parts.res) {
                p = parts.res + at + j;
                *p = fmaf(ds, res, fresh ? 0.0f : *p);
            }
            gated = fmaf(ds * c, xh, gated);
            scaled = fmaf(ds, res, scaled);
        }
        add_kept(gates, gates_lost, gated);
        add_kept(scales, scales_lost, scaled);
        if (a.dgate && a.gate.kind == MRN_FACTOR_ROW && threadIdx.x == 0) a.dgate[r] = k.q;
        fresh = false;
    }
    leave_scalars(gates, gates_lost, scales, scales_lost, parts, last);
}

// Threads that an SM's registers are shared between (the launch bound): what a thread with k
// slots needs.
template <class T> constexpr int gate_backward_resident(int k, int res, bool warp) {
    const int words = k * (8 * (res == 2 ? 4 : 3) + Slot<T>::kWords) + (warp ? 24 : 0);
    return words <= 56 ? 512 : (words <= 64 ? 448 : (words <= 108 ? 384 : 256));
}

// Rows behind a ring of copies, the column sums in registers over all rows of the CTA (see
// mrn_row_tile.cuh); one reduction to a row, behind which the operands are read from the ring
// once more.  RES: whether the residual is read for the gradient of its scale: 0 no, 1 a scalar,
// 2 one value per channel, whose column sums are kept too.
//   Measured on GB300, with the join: 16384 x 4096 bf16 with gate and scale learned per channel 170 to 173
// us (5.5 TB/s, 80 to 81 % of the copy's rate), without the scale 139 (5.8 TB/s); 16384 x 4095 bf16, a gate per row,
// 148 (5.4 TB/s); 4096 x 6656 f32 without factors 110 to 114 (5.7 to 6.0 TB/s, where rmsnorm_backward twice
// moves 8 matrices to its 6); 65536 x 768 bf16 103 (5.9 TB/s); 64 x 768 f32 5.0 us, two launches.
//   What bounds it: warps.  The column sums and weights leave 8 to 16 of them on an SM, issuing in 26 to 57
// % of cycles between waits for shared memory, arithmetic and (f32, whose rows fill the ring with two
// stages) their copies; dram is 68 to 72 % busy under ncu.  Operands held in registers over the
// barrier instead of a second read of the ring would cost warps again.
//   A scale per channel stands in shared memory behind the ring, each thread's columns where it
// alone reads them: registers are what bounds the number of warps.
template <class T, int K, bool EDGE, bool WARP, int RES>
__global__ void __launch_bounds__(gate_backward_resident<T>(K, RES, WARP))
mrn_gate_backward_tile_kernel(const GateBackwardArgs a, const TileArgs t, const GateParts parts,
                              const uint32_t ring_total) {
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    constexpr int kOps = RES ? 5 : 4;
    __shared__ RowSumSlots<6, false> slots;
    __shared__ EndSlots<kOps, 1, EDGE, WARP> end_w;
    __shared__ RowGates<EDGE, WARP> gates;
    __shared__ double last[2][kCtaWarps];
    RowTile<T, K, 1, EDGE, WARP> tile(a.rows, a.n, t);
    const int64_t back = static_cast<int64_t>(t.mis) * T::kBytes;
    const bool has_d = a.dstream != nullptr;
    const int res_op = has_d ? 4 : 3;
    const int ops_count = 3 + has_d + (RES ? 1 : 0);
    const char *ops[kOps];
    ops[0] = static_cast<const char *>(a.dn) - back;
    ops[1] = static_cast<const char *>(a.s) - back;
    ops[2] = static_cast<const char *>(a.b) - back;
    ops[3] = (has_d || !RES ? static_cast<const char *>(a.dstream) : static_cast<const char *>(a.res)) - back;
    if constexpr (RES) ops[4] = static_cast<const char *>(a.res) - back;
    char *const db = static_cast<char *>(a.db) - back;
    char *const dres = static_cast<char *>(a.dres) - back;
    RingWalk walk(tile.stage_bytes(ops_count), t.stages);
    const int ahead = t.stages - 1;
    const uint32_t ring0 = static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes));
    const uint32_t ring = tile.warp_ring(ring0, t.stages, ops_count);
    const bool by_row = a.gate.kind == MRN_FACTOR_ROW;
    const bool by_channel = RES == 2 || (RES == 0 && a.scale.kind == MRN_FACTOR_CHANNEL);
    tile.clear(ring, t.stages, ops_count);
    row_sum_setup(slots, tile.cl);
    pdl_enter();
    int64_t gate_row = tile.row;
    auto issue = [&](int to) {
        if (by_row && tile.leads && tile.copy_left > 0) copy_row_gate<T>(&gates.w[to][tile.team], a.gate, gate_row);
        gate_row += tile.stride;
        tile.issue(ring + to * walk.bytes, to, ops, ops_count, end_w);
    };
    for (int s = 0; s < ahead; ++s) issue(s);
    uint64_t c[K][4];
    Slot<T> g2[K];
    const uint32_t alpha_at = ring0 + ring_total + threadIdx.x * (8 * T::kBytes);
    const uint32_t alpha_step = blockDim.x * (8 * T::kBytes);
    if (by_channel) {
        tile.weights(g2, a.scale.p);
#pragma unroll
        for (int k = 0; k < K; ++k) st_shared_slot(alpha_at + k * alpha_step, g2[k]);
    }
    block_weights<T>(c, tile, a.g1, a.gate);
    tile.weights(g2, a.g2);
    const float gate = scalar_factor<T>(a.gate);
    const float scale = scalar_factor<T>(a.scale);
    const uint64_t scale2 = f2_pack(scale, scale);
    const float end_c = EDGE ? end_block_weight(tile, a.g1, a.gate) : 0.0f;
    const float end_g2 = EDGE ? tile.end_weight(a.g2) : 0.0f;
    const float end_alpha = EDGE && by_channel ? tile.end_weight(a.scale.p) : scale;
    uint64_t sum_p[K][4], sum_a[K][4], sum_r[RES == 2 ? K : 1][4];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sum_p[k][i] = sum_a[k][i] = 0;
            if (RES == 2) sum_r[RES == 2 ? k : 0][i] = 0;
        }
    float end_p = 0.0f, end_a = 0.0f, end_r = 0.0f;
    float gate_hi = 0.0f, gate_lo = 0.0f, scale_hi = 0.0f, scale_lo = 0.0f;
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
        float s[6];
        {
            uint64_t acc[6] = {0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < K; ++k) {
                Slot<T> dn, sv, b, d;
                tile.fetch_slot(dn, from, 0, k);
                tile.fetch_slot(sv, from, 1, k);
                tile.fetch_slot(b, from, 2, k);
                if (has_d) tile.fetch_slot(d, from, 3, k);
                else d.zero();
                if (WARP && !ok) {
                    dn.zero();
                    sv.zero();
                    b.zero();
                    d.zero();
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t v = sv.pair(i), bp = b.pair(i);
                    const uint64_t w = f2_mul(dn.pair(i), g2[k].pair(i)), cb = f2_mul(bp, c[k][i]);
                    acc[0] = f2_fma(v, v, acc[0]);
                    acc[1] = f2_fma(w, v, acc[1]);
                    acc[2] = f2_fma(bp, bp, acc[2]);
                    acc[3] = f2_fma(w, cb, acc[3]);
                    acc[4] = f2_fma(v, cb, acc[4]);
                    acc[5] = f2_fma(d.pair(i), cb, acc[5]);
                }
            }
#pragma unroll
            for (int i = 0; i < 6; ++i) s[i] = f2_sum(acc[i]);
        }
        float e_dn = 0.0f, e_s = 0.0f, e_b = 0.0f, e_d = 0.0f;
        if (EDGE && tile.ends) {
            e_dn = tile.fetch_end(end_w, walk.read, 0, 0);
            e_s = tile.fetch_end(end_w, walk.read, 1, 0);
            e_b = tile.fetch_end(end_w, walk.read, 2, 0);
            if (has_d) e_d = tile.fetch_end(end_w, walk.read, 3, 0);
            const float w = e_dn * end_g2, cb = e_b * end_c;
            s[0] = fmaf(e_s, e_s, s[0]);
            s[1] = fmaf(w, e_s, s[1]);
            s[2] = fmaf(e_b, e_b, s[2]);
            s[3] = fmaf(w, cb, s[3]);
            s[4] = fmaf(e_s, cb, s[4]);
            s[5] = fmaf(e_d, cb, s[5]);
        }
        const float g = by_row && ok ? row_gate<T>(gates.w[walk.read][tile.team], a.gate, tile.row) : gate;
        if (!row_sum_six<WARP>(s, slots, turn, tile.width, tile.cl, tile.crank, turn == 0 ? t.stall : 0u)) break;
        const RowScalars q = row_scalars(s, inv_n, a.eps1, a.eps2);
        if (a.dgate && by_row && tile.first == 0 && ok) a.dgate[tile.row] = q.q;
        const float c2 = -q.i1 * (g * (q.q * inv_n)), ig = q.i1 * g;
        const uint64_t i1 = f2_pack(q.i1, q.i1), i2 = f2_pack(q.i2, q.i2), m = f2_pack(q.m, q.m);
        const uint64_t g_p = f2_pack(g, g), c2_p = f2_pack(c2, c2), ig_p = f2_pack(ig, ig);
        uint64_t gated = 0, scaled = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            Slot<T> dn, sv, b, d, r, al, out;
            tile.fetch_slot(dn, from, 0, k);
            tile.fetch_slot(sv, from, 1, k);
            tile.fetch_slot(b, from, 2, k);
            if (has_d) tile.fetch_slot(d, from, 3, k);
            else d.zero();
            if (RES) tile.fetch_slot(r, from, res_op, k);
            if (by_channel) ld_shared_slot(al, alpha_at + k * alpha_step);
            if (WARP && !ok) {
                dn.zero();
                sv.zero();
                b.zero();
                d.zero();
                if (RES) r.zero();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t dnp = dn.pair(i);
                const uint64_t vh = f2_mul(sv.pair(i), i2), xh = f2_mul(b.pair(i), i1);
                const uint64_t ds = f2_add(f2_fma(vh, m, f2_mul(f2_mul(dnp, g2[k].pair(i)), i2)), d.pair(i));
                sum_p[k][i] = f2_fma(dnp, vh, sum_p[k][i]);
                sum_a[k][i] = f2_fma(ds, f2_mul(xh, g_p), sum_a[k][i]);
                const uint64_t v = f2_mul(ds, c[k][i]);
                gated = f2_fma(v, xh, gated);
                if (RES == 1) scaled = f2_fma(ds, r.pair(i), scaled);
                if (RES == 2) sum_r[RES == 2 ? k : 0][i] = f2_fma(ds, r.pair(i), sum_r[RES == 2 ? k : 0][i]);
                out.put_pair(i, f2_fma(xh, c2_p, f2_mul(v, ig_p)));
                d.put_pair(i, f2_mul(ds, by_channel ? al.pair(i) : scale2));
            }
            tile.store_slot(db, ok, out, k);
            tile.store_slot(dres, ok, d, k);
        }
        float row_gated = f2_sum(gated), row_scaled = f2_sum(scaled);
        if (EDGE && tile.ends) {
            const float vh = e_s * q.i2, xh = e_b * q.i1;
            const float ds = fmaf(vh, q.m, e_dn * end_g2 * q.i2) + e_d;
            end_p = fmaf(e_dn, vh, end_p);
            end_a = fmaf(ds, xh * g, end_a);
            const float v = ds * end_c;
            row_gated = fmaf(v, xh, row_gated);
            if (RES) {
                const float r = tile.fetch_end(end_w, walk.read, res_op, 0);
                if (RES == 1) row_scaled = fmaf(ds, r, row_scaled);
                else end_r = fmaf(ds, r, end_r);
            }
            tile.store_end(db, 0, ok, fmaf(xh, c2, v * ig));
            tile.store_end(dres, 0, ok, ds * end_alpha);
        }
        add_kept(gate_hi, gate_lo, row_gated);
        if (RES == 1) add_kept(scale_hi, scale_lo, row_scaled);
    }
    cp_async_wait(0);
    row_sum_leave(tile.cl);
    leave_scalars(gate_hi, gate_lo, scale_hi, scale_lo, parts, last);
    // Column j of a partial row stands at j + 8 - before, so that slots are aligned; the join
    // knows `before` from the row's number.
    constexpr int kSets = RES == 2 ? 3 : 2;
    if constexpr (!WARP) {
        const int64_t part = blockIdx.x / tile.cl;
#pragma unroll
        for (int which = 0; which < kSets; ++which) {
            float *const out = (which == 0 ? parts.pre : (which == 1 ? parts.post : parts.res)) + part * parts.stride + (EDGE ? 8 : 0);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!tile.holds(k)) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    Frag<F32, 4> v;
                    float f[4];
                    const auto &sum = which == 0 ? sum_p[k] : (which == 1 ? sum_a[k] : sum_r[RES == 2 ? k : 0]);
                    f2_unpack(sum[2 * i], f[0], f[1]);
                    f2_unpack(sum[2 * i + 1], f[2], f[3]);
                    v.put(f);
                    st_global(out + (tile.first + k * tile.slot_step()) * 8 + 4 * i, v);
                }
            }
            if (EDGE && tile.end_col >= 0) out[tile.end_col - tile.before] = which == 0 ? end_p : (which == 1 ? end_a : end_r);
        }
    } else {
        // the rows' sums of this CTA through the ring, laid out the same; then one column per
        // thread, over the rows in order
        const int span = K * tile.width * 8 + (EDGE ? 16 : 0);
        const int teams = static_cast<int>(blockDim.x) / tile.width;
        const int64_t row0 = static_cast<int64_t>(blockIdx.x) * teams;
        float *const buf = reinterpret_cast<float *>(ring_bytes);
#pragma unroll
        for (int which = 0; which < kSets; ++which) {
            __syncthreads();
            float *const mine = buf + tile.team * span + (EDGE ? 8 : 0);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!tile.holds(k)) continue;
                uint64_t *to = reinterpret_cast<uint64_t *>(mine + (tile.first + k * tile.slot_step()) * 8);
#pragma unroll
                for (int i = 0; i < 4; ++i) to[i] = which == 0 ? sum_p[k][i] : (which == 1 ? sum_a[k][i] : sum_r[RES == 2 ? k : 0][i]);
            }
            if (EDGE && tile.end_col >= 0) mine[tile.end_col - tile.before] = which == 0 ? end_p : (which == 1 ? end_a : end_r);
            __syncthreads();
            float *const out = (which == 0 ? parts.pre : (which == 1 ? parts.post : parts.res)) +
                               static_cast<int64_t>(blockIdx.x) * parts.stride;
            for (int j = threadIdx.x; j < static_cast<int>(a.n); j += blockDim.x) {
                float v = 0.0f;
                for (int r = 0; r < teams; ++r) {
                    const int off = EDGE ? 8 - static_cast<int>(-(t.mis + (row0 + r) * a.n) & 7) : 0;
                    v += buf[r * span + j + off];
                }
                out[j] = v;
            }
        }
    }
}

// The sums of the partial rows and of the scalar factors' partial sums.  A CTA owns 32 * C columns;
// its warps take every nth partial row each, all their loads in flight at once where there are few
// enough, and are joined in shared memory, in order: one trip to L2 bounds it, 4 to 5 us behind a
// backward of 304 partial rows.
//   blockIdx.y  0: P -> dg2    1: A -> dg1, and dgate of a gate per channel    2: R -> dscale
//   behind the column blocks (blockIdx.x == columns): the scalars, y 0 the gate, 1 the scale
// shifted: column j of partial row p stands where the tile kernel left it, at j + 8 - (the
// elements from row p's start to the next slot boundary).
struct GateJoinArgs {
    GateParts from;
    float *dg1, *dg2, *dgate, *dscale;   // dgate, dscale: per channel or scalar; NULL: not due
    const void *g1;
    Factor gate;
    int64_t n, parts, scalars;
    int columns, mis;
    bool shifted;
};

template <class T, int WARPS, int C, int kJoinFlight>
__global__ void __launch_bounds__(WARPS * 32) mrn_gate_join_kernel(const GateJoinArgs a) {
    __shared__ float sums[WARPS][C * 32];
    __shared__ double scalar[4];
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    if (static_cast<int>(blockIdx.x) == a.columns) {
        const double *from = blockIdx.y == 0 ? a.from.gate : (blockIdx.y == 1 ? a.from.scale : nullptr);
        if (!from) return;
        // (four warps: see leave_scalars on 64-bit additions)
        if (warp < 4) {
            double v = 0.0;
            for (int64_t i = threadIdx.x; i < a.scalars; i += 128) v += from[i];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (lane == 0) scalar[warp] = v;
        }
        __syncthreads();
        if (threadIdx.x == 0)
            *(blockIdx.y == 0 ? a.dgate : a.dscale) =
                static_cast<float>((scalar[0] + scalar[1]) + (scalar[2] + scalar[3]));
        return;
    }
    const float *part = blockIdx.y == 0 ? a.from.pre : (blockIdx.y == 1 ? a.from.post : a.from.res);
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
            const float *from = part + p * a.from.stride + off + j0;
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
        if (j >= a.n) continue;
        if (blockIdx.y == 0) {
            a.dg2[j] = t;
        } else if (blockIdx.y == 2) {
            a.dscale[j] = t;
        } else if (a.gate.kind == MRN_FACTOR_CHANNEL && a.parts > 0) {   // (no rows: nothing is read)
            a.dg1[j] = t * factor_at<T>(a.gate, 0, j);
            if (a.dgate) a.dgate[j] = t * ld_elem<T>(a.g1, j);
        } else {
            a.dg1[j] = t;
            if (a.dgate && a.gate.kind == MRN_FACTOR_CHANNEL) a.dgate[j] = t;
        }
    }
}

template <class T, int WARPS, int C, int FLIGHT>
cudaError_t launch_gate_join_typed(GateJoinArgs &a, bool pdl, cudaStream_t stream, uint64_t *launches) {
    const int64_t columns = (a.n + 32 * C - 1) / (32 * C);
    if (columns >= 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    a.columns = static_cast<int>(columns);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const bool scalars = a.from.gate || a.from.scale;
    cfg.gridDim = dim3(static_cast<unsigned>(columns + scalars), a.from.res ? 3 : 2, 1);
    cfg.blockDim = dim3(WARPS * 32, 1, 1);
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, mrn_gate_join_kernel<T, WARPS, C, FLIGHT>, a);
    if (err == cudaSuccess) ++*launches;
    return err;
}

struct GateBackwardLaunch {
    int sms;
    bool pdl;
    cudaStream_t stream;
    uint64_t *launches;
    int64_t most_parts;
    int64_t parts;      // out: partial rows written
    int64_t ctas;       // out: CTAs that left scalars
    cudaError_t err;    // out
};

// Slots per thread (k) for rows of a CTA.  Measured on GB300 (us), a stream's
// gradient with it, 805 MB a call (654 at 6656 and 6655; 940 and 763 with the residual's scale):
//   bf16  k 1, 2, 3, 4:  n = 1032 202, 187, 165, 209;  1280 (1 GB) 208, 189, 179, 211;  2048 168, 146, 143,
//         143;  2560 198, 147, 141, 174;  4096 178, 139, 142, 144;  4095 198, 151, 145, 148;  5120 261,
//         164, 165, 173;  6656 246, 163, 160, 155;  8192 222, 152, 149, 142
//         a scale per channel: 2048 175, 164, 195, 174;  4096 191, 177, 188, 169;  4095 206, 195, 232,
//         172;  8192 244, 219, 191, 159;  a scalar one: 4096 193, 170, 166, 169
//   f32   n = 1032 146, 179, 166, 225;  1280 (1 GB) 187, 172, 169, 220;  2048 140, 147, 135, 135;  4096 142,
//         134, 130, 139;  4095 162, 194, 148, 156;  5120 147, 144, 139, 134;  6656 143, 117, 139, 141;  6655
//         165, 154, 155, 156;  8192 166, 168, 162, 159;  12288 183, 152, 156, 140;  16384 175, 170, 188, 174
//         a scale per channel: 2048 167, 168, 195, 163;  4096 160, 157, 160, 165;  6656, two CTAs a row,
//         151 with one slot, 157, 163, 167
//   Around the band of two slots, f32, 4096 rows, with dstream, and without it:
//         5600 121, 96, 94, 93;  6400 140, 107, 139, 140;  6655 162, 156, 155, 156;  6656 142, 114, 141, 141;
//         6912 141, 149, 145, 144;  7168 143, 153, 152, 148;  7176 160, 182, 162, 164
//         5600 108, 81, 78, 78;  6400 126, 91, 89, 89;  6655 145, 114, 99, 101;  6656 127, 94, 94, 93;
//         6912 127, 99, 99, 99;  6911 148, 123, 101, 103;  7168 129, 105, 104, 103;  7176 141, 126, 112, 111
// Up to 6656 f32 a row's four operands take 106 KB at most: two stages fit, and with two slots 13 warps
// (with three, whose CTAs hold a multiple of 96 slots, the second stage misses by 1 KB).  Above, a CTA has
// room for one, and up to 7168 all forms are within 8 %.  The rule does not look at dstream: without
// it three slots would take 13 to 18 % less for rows with ends.
template <class T> constexpr int gate_backward_slots(int64_t slots, bool edge, bool residual, bool columns) {
    if (T::kBytes == 2) {
        if (columns) return slots <= 384 ? 2 : 4;
        return slots > 640 ? 4 : (slots <= 400 || edge ? 3 : 2);
    }
    if (residual) return slots <= 160 || slots > 560 ? (slots <= 4096 ? 1 : 4) : 2;
    if (slots <= 144) return 1;
    if (slots <= 192) return 3;
    return slots <= 560 && slots > 384 ? 3 : (slots > 700 && slots <= 896 ? 2 : 4);
}

// Threads of a CTA at most, for that many slots per thread.
template <class T> int gate_backward_threads(int64_t slots, int k, bool residual, bool columns) {
    const int most = gate_backward_resident<T>(k, columns ? 2 : 0, false);
    int threads = most;
    if (T::kBytes == 4 && residual && slots > 560) threads = 256;
    if (T::kBytes == 2 && slots > 1024) threads = slots <= 2048 ? 64 : (slots <= 4096 ? 128 : 256);
    while (threads < most && slots > int64_t(kMaxCluster) * k * threads) threads *= 2;
    return threads > most ? most : threads;
}

// Whether rows of so few slots that they could share warps have CTAs of their own: f32 rows of more
// slots than three for each lane of a warp, where four spill (32768 x 1024 167 us in warps, 142 in
// CTAs of 128 threads; with ends 131 in warps).
template <class T> constexpr bool gate_backward_apart(int64_t slots, bool edge) {
    return T::kBytes == 4 && slots > 96 && !edge;
}

// Whether any call takes this form: the forms that are compiled.  Few rows take one slot, and rows
// that share a warp and other rows of a CTA what the rules above give for some width.
template <class T> constexpr bool gate_backward_chosen(int k, bool edge, bool warp, int res) {
    if (k == 1) return true;
    if (warp) {
        for (int slots = 1; slots <= kWarpTileSlots; ++slots)
            if (warp_tile_slots(slots) == k && !gate_backward_apart<T>(slots, edge)) return true;
        return false;
    }
    for (int slots = 1; slots <= kMaxCluster * kTileMaxThreads * 4; ++slots)
        if (gate_backward_slots<T>(slots, edge, res != 0, res == 2) == k) return true;
    return false;
}

// Whether the call was launched; false: it takes the looped kernel.
template <class T, int K, bool EDGE, bool WARP, int RES>
bool launch_gate_backward_tile(const GateBackwardArgs &a, const GateParts &parts, const TileShape &p,
                               GateBackwardLaunch &l) {
    if constexpr (!gate_backward_chosen<T>(K, EDGE, WARP, RES)) {
        l.err = cudaErrorInvalidDeviceFunction;     // (no call comes here)
        return true;
    } else {
        static TileLaunchCache cache;
        const auto fn = mrn_gate_backward_tile_kernel<T, K, EDGE, WARP, RES>;
        const int operands = 3 + (a.dstream ? 1 : 0) + (RES ? 1 : 0);
        const int64_t alpha = a.scale.kind == MRN_FACTOR_CHANNEL ? int64_t(K) * p.threads * 8 * T::kBytes : 0;
        TileGrid g;
        // (WARP: the epilogue's rows have room for the ends)
        l.err = tile_grid(cache, fn, p, a.rows, a.n, 1, T::kBytes, operands, gate_parts_per_sm(a.n), l.sms, &g,
                          alpha + (WARP ? 1024 : 0));
        if (l.err != cudaSuccess) return true;
        l.parts = g.ctas / p.cluster;
        l.ctas = g.ctas;
        if (g.stages < 1 || l.parts > l.most_parts) return false;   // (the workspace holds no more)
        const TileArgs t = {p.lanes, g.stages, p.mis, a.stall};
        l.err = launch_tile(fn, p, g.ctas, g.shared, l.pdl, l.stream, l.launches, a, t, parts,
                            static_cast<uint32_t>(g.shared - alpha));
        return true;
    }
}

template <class T, int K, bool EDGE, bool WARP>
bool launch_gate_backward_res(const GateBackwardArgs &a, const GateParts &parts, const TileShape &p,
                              GateBackwardLaunch &l) {
    if (!a.dscale) return launch_gate_backward_tile<T, K, EDGE, WARP, 0>(a, parts, p, l);
    return parts.res ? launch_gate_backward_tile<T, K, EDGE, WARP, 2>(a, parts, p, l)
                     : launch_gate_backward_tile<T, K, EDGE, WARP, 1>(a, parts, p, l);
}

template <class T, int K, bool WARP>
bool launch_gate_backward_k(const GateBackwardArgs &a, const GateParts &parts, const TileShape &p,
                            GateBackwardLaunch &l) {
    return p.edge ? launch_gate_backward_res<T, K, true, WARP>(a, parts, p, l)
                  : launch_gate_backward_res<T, K, false, WARP>(a, parts, p, l);
}

template <class T>
cudaError_t launch_gate_backward_typed(const GateBackwardArgs &a, int sms, bool pdl, cudaStream_t stream,
                                       uint64_t *launches) {
    const int64_t most = gate_parts(a.rows, a.n, sms);
    const bool scalar_gate = a.dgate && a.gate.kind == MRN_FACTOR_SCALAR;
    const bool scalar_scale = a.dscale && a.scale.kind == MRN_FACTOR_SCALAR;
    GateParts parts = {};
    parts.stride = part_stride_of(a.n);
    const int64_t set = most * parts.stride;
    double *const scalars = reinterpret_cast<double *>(a.workspace + kGateColumnSets * set);
    parts.pre = a.workspace;
    parts.post = a.workspace + set;
    parts.res = a.dscale && !scalar_scale ? a.workspace + 2 * set : nullptr;
    parts.gate = scalar_gate ? scalars : nullptr;
    parts.scale = scalar_scale ? scalars + kGateScalars * most : nullptr;
    GateJoinArgs join = {};
    GateBackwardLaunch l = {sms, pdl, stream, launches, most, most, most, cudaSuccess};
    if (most > 0) {
        const int mis = common_offset(T::kBytes, a.dn, a.s, a.b, a.dstream, a.res, static_cast<const void *>(a.db),
                                      static_cast<const void *>(a.dres));
        bool done = false;
        if (mis >= 0) {
            const int64_t slots = a.n / 8;
            const bool edge = mis != 0 || a.n % 8 != 0;
            const bool residual = a.dscale != nullptr, columns = parts.res != nullptr;
            const bool few = tile_few_rows(a.rows, a.n, sms);
            const int k = few ? 1 : gate_backward_slots<T>(slots, edge, residual, columns);
            const int most_threads = few ? tile_few_threads(a.rows, a.n, sms)
                                         : gate_backward_threads<T>(slots, k, residual, columns);
            const TileShape p = tile_shape(a.n, mis, k, most_threads, few || gate_backward_apart<T>(slots, edge));
            if (p.ok && p.warp) {
                done = p.k == 1   ? launch_gate_backward_k<T, 1, true>(a, parts, p, l)
                       : p.k == 2 ? launch_gate_backward_k<T, 2, true>(a, parts, p, l)
                       : p.k == 3 ? launch_gate_backward_k<T, 3, true>(a, parts, p, l)
                                  : launch_gate_backward_k<T, 4, true>(a, parts, p, l);
            } else if (p.ok) {
                done = k == 1   ? launch_gate_backward_k<T, 1, false>(a, parts, p, l)
                       : k == 2 ? launch_gate_backward_k<T, 2, false>(a, parts, p, l)
                       : k == 3 ? launch_gate_backward_k<T, 3, false>(a, parts, p, l)
                                : launch_gate_backward_k<T, 4, false>(a, parts, p, l);
            }
            join.mis = mis;
            join.shifted = done && p.edge && !p.warp;
        }
        if (!done) {
            l.parts = l.ctas = most;
            l.err = launch_plain(mrn_gate_backward_looped_kernel<T>, most, kLoopedThreads, 0, pdl, stream, launches, a,
                                 parts);
        }
        if (l.err != cudaSuccess) return l.err;
    } else {
        // no rows, and perhaps no workspace: the sums are zero, their places only say which are due
        parts.res = a.dscale && !scalar_scale ? a.dscale : nullptr;
        parts.gate = scalar_gate ? reinterpret_cast<double *>(a.dgate) : nullptr;
        parts.scale = scalar_scale ? reinterpret_cast<double *>(a.dscale) : nullptr;
    }
    join.from = parts;
    join.dg1 = a.dg1;
    join.dg2 = a.dg2;
    join.dgate = a.dgate;
    join.dscale = a.dscale;
    join.g1 = a.g1;
    join.gate = a.gate;
    join.n = a.n;
    join.parts = l.parts;
    join.scalars = l.ctas;
    return a.n <= 1024 ? launch_gate_join_typed<T, 32, 1, 20>(join, pdl, stream, launches)
                       : launch_gate_join_typed<T, 16, 2, 10>(join, pdl, stream, launches);
}

}  // namespace mrn
