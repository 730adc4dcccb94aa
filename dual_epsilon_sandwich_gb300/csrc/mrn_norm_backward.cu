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
#include "mrn_train_kernels.cuh"

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
    const int64_t parts = backward_parts(a.rows, a.n, sms);
    float *pg = a.workspace;
    float *pb = a.dbeta ? a.workspace + parts * a.n : nullptr;
    if (parts > 0) {
        const auto fn = a.rms ? mrn_norm_backward_looped_kernel<T, true>
                              : mrn_norm_backward_looped_kernel<T, false>;
        const cudaError_t err = launch_plain(fn, parts, kLoopedThreads, 0, pdl, stream, launches, a,
                                             pg, pb);
        if (err != cudaSuccess) return err;
    }
    return launch_join(pg, pb, a.dgamma, a.dbeta, parts, a.n, pdl, stream, launches);
}

cudaError_t launch_norm_backward(bool bf16, const BackwardArgs &a, int sms, bool pdl,
                                 cudaStream_t stream, uint64_t *launches) {
    return bf16 ? launch_backward_typed<BF16>(a, sms, pdl, stream, launches)
                : launch_backward_typed<F32>(a, sms, pdl, stream, launches);
}

}  // namespace mrn
