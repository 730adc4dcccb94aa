// mrn_row_tile.cuh -- how the training operations' kernels hold rows: a persistent
// CTA (or cluster of CTAs, or part of a warp) walks over rows that are a fixed
// number apart, each thread owning the same columns of all of them.
//
//  * A thread owns K slots of eight consecutive elements, a row's width in threads
//    apart.  Slots are cut at multiples of eight elements of the flattened matrix, so
//    that they are aligned in memory and are the dropout's generator groups; when
//    the row pitch is not a multiple of eight (EDGE), a row starts `off` elements into
//    its first slot.  The rows of one CTA are a multiple of eight apart, so `off`
//    and with it every thread's columns are the same for all of them: weights are
//    loaded once, and column sums stay in registers over all rows.
//  * Row operands are copied ahead by cp.async into a ring of `stages` rows in shared
//    memory, each warp its own columns, so that a stage is handed over by the warp's
//    own wait and needs no barrier.  The copies in flight cover the latency of the
//    row sums, whose barriers would otherwise leave the memory idle.
//  * f32 slots are 32 bytes: a warp copies 16-byte chunks with consecutive lanes on
//    consecutive chunks, so that each access covers whole sectors.
#pragma once

#include "mrn_train_kernels.cuh"

namespace mrn {

struct TileArgs {
    int lanes;      // threads per row when several rows share a warp (WARP); else unused
    int stages;     // ring depth
    int mis;        // elements from the slot boundary below the operands' base to the base
};

constexpr int kTileMaxThreads = 512;
constexpr int tile_max_threads(int k) { return k >= 3 ? 256 : kTileMaxThreads; }
constexpr int kTileMaxStages = 4;
constexpr int kTileMaxOperands = 3;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;"
                 :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the `pending` youngest groups of this thread have landed.
__device__ __forceinline__ void cp_async_wait(int pending) {
    switch (pending) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}
__device__ __forceinline__ void ld_shared_slot(Slot<BF16> &s, uint32_t p) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]) : "r"(p));
}
__device__ __forceinline__ void ld_shared_slot(Slot<F32> &s, uint32_t p) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]) : "r"(p));
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4+16];"
                 : "=r"(s.w[4]), "=r"(s.w[5]), "=r"(s.w[6]), "=r"(s.w[7]) : "r"(p));
}

// Sums of N values over the threads of a row.  WARP: over `width` lanes; else over
// the CTA and, for rows split over a cluster, over its CTAs.
template <int N> struct RowSumSlots {
    CtaSumSlots<N> cta;
    float peer[2][N][kMaxCluster];
};

template <int N, bool WARP>
__device__ __forceinline__ void row_sum(float (&v)[N], RowSumSlots<N> &s, int &turn, int width,
                                        unsigned cl, unsigned crank) {
    if constexpr (WARP) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = group_allsum(v[i], width);
    } else {
        cta_sum(v, s.cta, turn);
        if (cl > 1) {
            // (two turns: a peer writes turn t + 2 after the barrier of t + 1, which this
            // CTA enters after its reads of t)
            const unsigned lane = threadIdx.x & 31;
            if (threadIdx.x < cl) {
#pragma unroll
                for (int i = 0; i < N; ++i) st_cluster_f32(&s.peer[turn][i][crank], threadIdx.x, v[i]);
            }
            cluster_arrive_release();
            cluster_wait_acquire();
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = warp_allsum(lane < cl ? s.peer[turn][i][lane] : 0.0f);
        }
    }
}

template <class T, int K, bool EDGE, bool WARP> struct RowTile {
    static constexpr int kChunks = T::kBytes / 2;          // 16-byte chunks per slot
    static constexpr int kChunkElems = 8 / kChunks;

    int width;            // threads per row (in this CTA)
    int first;            // this thread's first slot; slot k is first + k * width
    int off;              // elements of the row's first slot that precede the row
    unsigned cl, crank;
    int64_t n, rows;
    int64_t row;          // this thread's row; the next is row + stride
    int64_t stride;
    int64_t at;           // byte offset of the row's slot 0 from the slot boundary below its operand
    int64_t step;         // bytes to the next row's
    int team;             // index in the CTA of the lanes that copy together
    bool leads;           // the first of them
    uint32_t in[K];       // elements of slot k inside the row: bit i for element i
    uint32_t copies;      // chunks this thread copies: bit k * kChunks + c
    uint32_t region;      // bytes of one slot index k of all threads in the ring
    uint32_t copy_base;   // this thread's place in a region: as copier,
    uint32_t slot_base;   // ... and as owner
    int copy_off;         // byte offset in the row of the first chunk this thread copies
    int copy_step;        // ... and from chunk to chunk of a slot

    __device__ __forceinline__ RowTile(int64_t rows_, int64_t n_, const TileArgs &t)
        : n(n_), rows(rows_) {
        const int tid = threadIdx.x, lane = tid & 31;
        int lanes = 32, li = lane;      // lanes that copy together, and this one's index
        team = tid >> 5;
        if constexpr (WARP) {
            cl = 1;
            crank = 0;
            width = t.lanes;
            first = tid & (t.lanes - 1);
            const int rows_per_cta = blockDim.x / t.lanes;
            row = static_cast<int64_t>(blockIdx.x) * rows_per_cta + tid / t.lanes;
            stride = static_cast<int64_t>(gridDim.x) * rows_per_cta;
            lanes = t.lanes;
            li = first;
            team = tid / t.lanes;
        } else {
            cl = cluster_nctarank();
            crank = cluster_ctarank();
            width = blockDim.x;
            first = tid + static_cast<int>(crank) * K * static_cast<int>(blockDim.x);
            row = blockIdx.x / cl;
            stride = gridDim.x / cl;
        }
        leads = li == 0;
        const int64_t e0 = t.mis + row * n;
        off = EDGE ? static_cast<int>(e0 & 7) : 0;
        at = (e0 - off) * T::kBytes;
        step = stride * n * T::kBytes;
        region = blockDim.x * kChunks * 16;
        const int chunk0 = (first - li) * 8 + li * kChunkElems;     // element in the slot row
        copy_off = chunk0 * T::kBytes;
        copy_step = lanes * 16;
        copy_base = static_cast<uint32_t>(((tid - li) * kChunks + li) * 16);
        slot_base = static_cast<uint32_t>(tid * kChunks * 16);
        copies = 0u;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t j = column(k);
            uint32_t m = 0xFFu;
            if (j < 0) m &= 0xFFu << static_cast<int>(-j);
            if (j + 8 > n) m = j < n ? m & (0xFFu >> static_cast<int>(j + 8 - n)) : 0u;
            in[k] = m;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int64_t jc = chunk0 + k * width * 8 + c * lanes * kChunkElems - off;
                if (jc < n && jc + kChunkElems > 0) copies |= 1u << (k * kChunks + c);
            }
        }
    }

    // First row of this CTA's iteration: uniform over the CTA, so that all its threads
    // make the same number of iterations.
    __device__ __forceinline__ int64_t cta_row() const {
        if constexpr (WARP) {
            return row - team;
        } else {
            return row;
        }
    }
    __device__ __forceinline__ int column(int k) const { return (first + k * width) * 8 - off; }

    // Zeroes a ring of `stages` stages of `count` operands: the chunks outside the row are
    // never copied, and read as zeros ever after.
    __device__ __forceinline__ void clear(uint32_t ring, int stages, int count) const {
        for (int i = 0; i < stages * count * K; ++i) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};"
                             :: "r"(ring + i * region + copy_base + c * copy_step), "r"(0u) : "memory");
        }
        __syncwarp();
    }
    // Copies the row `ahead` rows from this one into the ring's stage at `to` (one group of
    // asynchronous copies with what was issued since the last).
    __device__ __forceinline__ void issue(uint32_t to, int ahead, const char *const (&ops)[kTileMaxOperands],
                                          int count) const {
        if (row + ahead * stride < rows) {
            const int64_t from = at + ahead * step + copy_off;
#pragma unroll
            for (int o = 0; o < kTileMaxOperands; ++o) {
                if (o >= count) break;
                const char *src = ops[o] + from;
                const uint32_t dst = to + o * K * region + copy_base;
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        if ((copies >> (k * kChunks + c)) & 1u)
                            cp_async16(dst + k * region + c * copy_step,
                                       src + k * (width * 8 * T::kBytes) + c * copy_step);
                    }
                }
            }
        }
        cp_async_commit();
    }
    // This thread's slots of operand o in the stage at `from`, zero outside the row.
    __device__ __forceinline__ void fetch(Slot<T> (&s)[K], uint32_t from, int o) const {
        const uint32_t src = from + o * K * region + slot_base;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            ld_shared_slot(s[k], src + k * region);
            if constexpr (EDGE) {
                if (in[k] != 0xFFu && in[k] != 0u) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (!((in[k] >> i) & 1u)) s[k].clear(i);
                }
            }
        }
        if constexpr (WARP) {
            if (row >= rows) {      // (past the last row: the stage holds an earlier one)
#pragma unroll
                for (int k = 0; k < K; ++k) s[k].zero();
            }
        }
    }
    // Stores slot k of this row (the elements inside it) at `base`, the slot boundary below
    // the operand's first element.
    __device__ __forceinline__ void store(char *base, int k, const Slot<T> &s) const {
        char *p = base + at + (first + k * width) * (8 * T::kBytes);
        if (!EDGE || in[k] == 0xFFu) {
            if (in[k] != 0u) st_slot(p, s);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((in[k] >> i) & 1u) s.st_one(p + i * T::kBytes, i);
        }
    }
    // Generator group of slot k (the operands start on a slot boundary).
    __device__ __forceinline__ uint64_t group(int k) const {
        return static_cast<uint64_t>(at) / (8 * T::kBytes) + static_cast<uint64_t>(first + k * width);
    }
    // The thread's columns of a weight vector, zeros outside the row; once per CTA.  All
    // loads are independent of each other.
    __device__ __forceinline__ void weights(Slot<T> (&s)[K], const void *w) const {
        const bool whole = !EDGE && reinterpret_cast<uintptr_t>(w) % 16 == 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t j = column(k);
            if (whole) {
                const int64_t jj = in[k] ? j : 0;
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(s[k].w[4 * c]), "=r"(s[k].w[4 * c + 1]),
                                   "=r"(s[k].w[4 * c + 2]), "=r"(s[k].w[4 * c + 3])
                                 : "l"(elem_ptr<T>(w, jj) + c * 16));
                if (!in[k]) s[k].zero();
            } else {
                Frag<T, 1> f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) ld_ro(f[i], elem_ptr<T>(w, ((in[k] >> i) & 1u) ? j + i : 0));
                s[k].zero();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (T::kBytes == 4) {
                        s[k].w[i] = ((in[k] >> i) & 1u) ? f[i].w : 0u;
                    } else {
                        if ((in[k] >> i) & 1u)
                            s[k].w[i >> 1] |= static_cast<uint32_t>(f[i].h) << ((i & 1) * 16);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void advance() {
        row += stride;
        at += step;
    }
};

// The ring's stages: the one the current row is read from and the one that the row `stages - 1`
// rows on is copied to.
struct RingWalk {
    uint32_t bytes;
    int stages, read, write;
    __device__ __forceinline__ RingWalk(uint32_t stage_bytes, int stages_)
        : bytes(stage_bytes), stages(stages_), read(0), write(stages_ - 1) {}
    __device__ __forceinline__ void next() {
        read = read + 1 == stages ? 0 : read + 1;
        write = write + 1 == stages ? 0 : write + 1;
    }
};

// Dynamic shared memory that a ring may use: the rest is the static row-sum slots.
constexpr int64_t kTileSharedBudget = kSharedBytesPerCta - 8192;

// Dynamic shared memory of a ring.
inline int64_t tile_ring_bytes(int elem_bytes, int k, int threads, int stages, int operands) {
    return int64_t(stages) * operands * k * threads * (elem_bytes / 2) * 16;
}

// How a call's rows are laid over threads.
struct TilePlan {
    bool ok;          // false: the looped kernel
    bool warp;        // several rows per warp
    bool edge;
    int k, threads, lanes, cluster, stages;
    int64_t ctas;
    int mis;
};

struct TileWish {
    int operands;          // row operands copied ahead
    int slots_per_thread;  // for rows of a CTA
    int threads_per_sm;    // resident threads to aim for
    int most_ctas_per_sm;
};

inline TilePlan plan_tiles(int64_t rows, int64_t n, int elem_bytes, int mis, const TileWish &wish,
                           int sms) {
    TilePlan p = {};
    p.mis = mis;
    p.edge = mis != 0 || n % 8 != 0;
    p.cluster = 1;
    const int64_t slots = p.edge ? (n + 14) / 8 : n / 8;
    if (slots <= 128) {
        p.warp = true;
        p.k = slots <= 8 ? 1 : (slots <= 64 ? 2 : 4);
        p.lanes = 1;
        while (p.lanes * p.k < slots) p.lanes *= 2;
        p.threads = 128;
    } else {
        p.k = wish.slots_per_thread;
        const int64_t most = int64_t(p.k) * tile_max_threads(p.k);
        p.cluster = static_cast<int>((slots + most - 1) / most);
        if (p.cluster > kMaxCluster) return p;
        const int64_t per = (slots + p.cluster - 1) / p.cluster;
        p.threads = static_cast<int>((per + 32 * p.k - 1) / (32 * p.k)) * 32;
    }
    const int64_t stage = tile_ring_bytes(elem_bytes, p.k, p.threads, 1, wish.operands);
    int64_t per_sm = wish.threads_per_sm / p.threads;
    if (per_sm > wish.most_ctas_per_sm) per_sm = wish.most_ctas_per_sm;
    if (per_sm < 1) per_sm = 1;
    const int64_t budget = (kTileSharedBudget - (per_sm - 1) * 8192) / per_sm;
    p.stages = static_cast<int>(budget / stage);
    if (p.stages > kTileMaxStages) p.stages = kTileMaxStages;
    if (p.stages < 1) return p;
    //TUNE
    const int64_t rows_per_cta = p.warp ? p.threads / p.lanes : 1;
    int64_t groups = sms * per_sm / p.cluster;      // CTAs or clusters
    if (groups * rows_per_cta % 8 != 0 && groups > 8) groups -= groups % 8;
    if (groups < 8) groups = 8;
    const int64_t need = (rows + rows_per_cta - 1) / rows_per_cta;
    if (groups > need) groups = need;
    p.ctas = groups * p.cluster;
    p.ok = true;
    return p;
}

// Elements from the slot boundary below a row operand to its base; -1 when the
// operands (NULL: none) do not share it.
template <class... P> inline int common_offset(int elem_bytes, const void *first, P... rest) {
    const uintptr_t slot = 8 * static_cast<uintptr_t>(elem_bytes);
    const uintptr_t at = reinterpret_cast<uintptr_t>(first) % slot;
    for (const void *q : {static_cast<const void *>(rest)...})
        if (q && reinterpret_cast<uintptr_t>(q) % slot != at) return -1;
    return static_cast<int>(at) / elem_bytes;
}

// Which kernels have been opened to the shared memory and cluster sizes below, per
// device.  Every thread sets the same values, so that calls that race only repeat them.
struct TileLaunchCache {
    std::atomic<bool> opened[kMaxCachedDevices];
};

template <class... Params, class... Args>
cudaError_t launch_tile(TileLaunchCache &cache, void (*fn)(Params...), const TilePlan &p, int64_t shared,
                        bool pdl, cudaStream_t stream, uint64_t *launches, Args... args) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool cached = dev >= 0 && dev < kMaxCachedDevices;
    if (!cached || !cache.opened[dev].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(kTileSharedBudget));
        if (err != cudaSuccess) return err;
        err = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (err != cudaSuccess) return err;
        if (cached) cache.opened[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(p.threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(shared);
    cfg.stream = stream;
    cfg.attrs = attr;
    if (p.cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(p.cluster);
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    err = cudaLaunchKernelEx(&cfg, fn, args...);
    if (err == cudaSuccess) ++*launches;
    return err;
}

}  // namespace mrn
