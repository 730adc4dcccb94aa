// mrn_row_tile.cuh -- how the training operations' kernels hold rows: a persistent
// CTA (or cluster of CTAs, or part of a warp) walks over rows that are a fixed
// number apart, each thread owning the same columns of all of them.
//
//  * A thread owns K slots of eight consecutive elements: a warp owns 32 K consecutive
//    ones, a lane every 32nd of them, so that the distances between a thread's slots, in
//    memory and in the ring, are constants of the code.  Slots are cut at multiples of
//    eight elements of the flattened matrix: they are aligned in memory and are the
//    dropout's generator groups.  When the row pitch is not a multiple of eight (EDGE),
//    up to seven elements before the row's first whole slot and seven behind its last are
//    taken one by one, each by a lane of its own: every slot is whole, and only the warp
//    that holds the ends does more (16384 x 4095 bf16, the gradient: 86 us, where 4096 takes 76;
//    when it was chosen 91, 79 without that work, 118 with masked slots instead).
//    The rows of one CTA are a multiple of eight apart, so that they all start alike and
//    a thread's columns stay the same: weights are loaded once, and column sums stay in
//    registers over all rows.
//  * R rows at a time: their loads, sums and barriers overlap, and the column sums and
//    weights are held once for all of them.
//  * Row operands are copied ahead by cp.async into a ring of `stages` turns in shared
//    memory, each warp its own columns, so that a stage is handed over by the warp's
//    own wait and needs no barrier.  The copies in flight cover the latency of the
//    row sums, whose barriers would otherwise leave the memory idle.
//  * f32 slots are 32 bytes: a warp copies 16-byte chunks with consecutive lanes on
//    consecutive chunks, so that each access covers whole sectors.
#pragma once

#include "mrn_train_kernels.cuh"

namespace mrn {

struct TileArgs {
    int lanes;      // threads per row when rows share a warp (WARP); else unused
    int stages;     // ring depth
    int mis;        // elements from the slot boundary below the operands' base to the base
    uint32_t stall; // see row_sum
};

constexpr int kTileMaxThreads = 512;
constexpr int kTileMaxStages = 4;

// 16 bytes to shared memory when `on` is not 0 (predicated, no branch).
__device__ __forceinline__ void cp_async16_if(uint32_t on, uint32_t dst, const void *src) {
    asm volatile("{.reg .pred q; setp.ne.u32 q, %2, 0;"
                 " @q cp.async.cg.shared.global.L2::256B [%0], [%1], 16;}"
                 :: "r"(dst), "l"(src), "r"(on) : "memory");
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

__device__ __forceinline__ void st_shared_slot(uint32_t p, const Slot<BF16> &s) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                 :: "r"(p), "r"(s.w[0]), "r"(s.w[1]), "r"(s.w[2]), "r"(s.w[3]) : "memory");
}
__device__ __forceinline__ void st_shared_slot(uint32_t p, const Slot<F32> &s) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                 :: "r"(p), "r"(s.w[0]), "r"(s.w[1]), "r"(s.w[2]), "r"(s.w[3]) : "memory");
    asm volatile("st.shared.v4.b32 [%0+16], {%1,%2,%3,%4};"
                 :: "r"(p), "r"(s.w[4]), "r"(s.w[5]), "r"(s.w[6]), "r"(s.w[7]) : "memory");
}

// Sums of N values over the threads of a row.  WARP: over `width` lanes; else over
// the CTA and, for rows split over a cluster, over its CTAs: every CTA sends its sums to
// every peer as st.async messages, which land in the peer's box for this turn and complete
// the peer's mbarrier for it; a CTA waits for its own and adds the sums in rank order (all
// CTAs get the same bits).  A cluster barrier instead would make each row wait for the
// stores of the row before it (16384 f32: 193 us against 178 for the gradient of
// 4096 rows).  Boxes and mbarriers alternate: a CTA sends turn t + 2 only after it has every
// peer's t + 1, which a peer sends only after all its threads have read t.
template <int N, bool PAIRS> struct RowSumSlots {
    typename CtaSumOf<N, PAIRS>::Slots cta;
    float box[2][N][kMaxCluster];   // [turn parity][value][sender rank]
    __align__(8) uint64_t bar[2];
};

// Before the first row_sum, by every thread: the slots and every peer's mbarriers are set up.
template <int N, bool PAIRS> __device__ __forceinline__ void row_sum_setup(RowSumSlots<N, PAIRS> &s, unsigned cl) {
    cta_sum_setup(s.cta);
    if (cl > 1) {
        if (threadIdx.x == 0) {
            mbar_init(&s.bar[0], 1);
            mbar_init(&s.bar[1], 1);
            fence_mbar_init();
        }
        __syncthreads();
        cluster_arrive_release();
    }
}
__device__ __forceinline__ void row_sum_ready(unsigned cl) {
    if (cl > 1) cluster_wait_acquire();
}
// After the last: no CTA leaves while a peer may still send to it.
__device__ __forceinline__ void row_sum_leave(unsigned cl) {
    if (cl > 1) {
        cluster_arrive_release();
        cluster_wait_acquire();
    }
}

// False (in the whole CTA) when a peer's message did not arrive in time (about a second): the
// CTA then stops, and its peers after it.  `stall`: bytes more than ever arrive that a wait
// expects (a test hook, 0 in use).
template <bool WARP, int N, bool PAIRS>
__device__ __forceinline__ bool row_sum(float (&v)[N], RowSumSlots<N, PAIRS> &s, int &turn, int width,
                                        unsigned cl, unsigned crank, uint32_t stall) {
    if constexpr (WARP) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = group_allsum(v[i], width);
    } else {
        cta_sum(v, s.cta, turn);
        if (cl > 1) {
            const int p = turn & 1;
            const unsigned lane = threadIdx.x & 31;
            if (threadIdx.x == 0) mbar_arrive_expect_tx(&s.bar[p], (cl - 1) * 4u * N + stall);
            if (threadIdx.x < cl && threadIdx.x != crank) {
#pragma unroll
                for (int i = 0; i < N; ++i) send_f32(&s.box[p][i][crank], &s.bar[p], threadIdx.x, v[i]);
            }
            const bool late = !mbar_wait_bounded_cluster(&s.bar[p], static_cast<uint32_t>((turn - 1) >> 1 & 1));
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = warp_allsum(lane >= cl ? 0.0f : (lane == crank ? v[i] : s.box[p][i][lane]));
            if (__syncthreads_or(late)) {
                if (threadIdx.x == 0) atomicAdd(&g_wait_timeouts, 1u);
                return false;
            }
        }
    }
    return true;
}

// The single elements at a row's ends in the ring: one word per lane that holds one (bf16: the
// word that holds the element).
constexpr int kEndLanes = 16;    // lanes 0..6 the ones before the slots, 8..14 the ones behind
template <int OPS, int R, bool EDGE, bool WARP> struct EndSlots {
    static constexpr int kThreads = !EDGE ? 1 : (WARP ? 128 : kEndLanes);
    uint32_t w[kTileMaxStages][R][OPS][kThreads];
};

template <class T, int K, int R, bool EDGE, bool WARP> struct RowTile {
    static constexpr int kChunks = T::kBytes / 2;          // 16-byte chunks per slot
    static constexpr int kBlock = 512 * kChunks;           // a warp's slots k of one operand, in bytes

    int width;            // threads per row (in this CTA)
    int lanes;            // lanes that copy together: the distance of a thread's slots
    int first;            // this thread's first slot; slot k is first + k * lanes
    int before;           // EDGE: elements from the row's start to the next slot boundary
    unsigned cl, crank;
    int64_t row;          // this thread's first row; the R rows are `stride` apart
    int64_t stride;
    int left;             // rows from this one on that exist
    int cta_left;         // ... of the CTA's first row: uniform, so that all threads of a CTA
                          // make the same number of turns
    int64_t at;           // byte offset of the row's slot 0 from the slot boundary below its operand
    int64_t step;         // bytes to the next row's
    int team;             // index in the CTA of the lanes that copy together
    bool leads;           // the first of them
    bool ends;            // EDGE: this warp holds single elements (uniform over the warp)
    int end_col;          // column of this thread's single element; -1: none
    uint32_t full;        // slots of this thread inside the row: bit k
    uint32_t copies;      // chunks this thread copies: bit k * kChunks + c
    uint32_t copy_to;     // this thread's place in its warp's ring: as copier,
    uint32_t slot_from;   // ... and as owner
    int64_t copy_at;      // the next row to copy: byte offset of this thread's first chunk
    int copy_left;        // ... and the rows from it on

    __device__ __forceinline__ RowTile(int64_t rows, int64_t n, const TileArgs &t) {
        const int tid = threadIdx.x, lane = tid & 31;
        int li = lane;                  // index among the lanes that copy together
        lanes = 32;
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
            first = (static_cast<int>(crank * blockDim.x) + (tid - lane)) * K + lane;
            row = blockIdx.x / cl;
            stride = gridDim.x / cl;
        }
        leads = li == 0;
        const int64_t cta_row = WARP ? row - team : row;
        left = row < rows ? static_cast<int>((rows - 1 - row) / stride) + 1 : 0;
        cta_left = cta_row < rows ? static_cast<int>((rows - 1 - cta_row) / stride) + 1 : 0;
        const int64_t e0 = t.mis + row * n;
        before = EDGE ? static_cast<int>(-e0 & 7) : 0;
        at = (e0 + before) * T::kBytes;
        step = stride * n * T::kBytes;
        const int head = before < n ? before : static_cast<int>(n);
        const int slots = static_cast<int>((n - head) / 8);
        ends = EDGE && (WARP || (tid < 32 && crank == 0));
        end_col = -1;
        if (ends) {
            const int j = WARP ? first : tid;
            if (j < 8) {
                if (j < head) end_col = j;
            } else if (j < kEndLanes) {
                const int64_t c = head + slots * int64_t(8) + (j - 8);
                if (c < n) end_col = static_cast<int>(c);
            }
        }
        const int chunk0 = (first - li) * kChunks + li;             // chunk in the slot row
        copy_at = at + chunk0 * 16;
        copy_left = left;
        copy_to = static_cast<uint32_t>(((lane - li) * kChunks + li) * 16);
        slot_from = static_cast<uint32_t>(lane * kChunks * 16);
        full = copies = 0u;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (first + k * lanes < slots) full |= 1u << k;
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                if (chunk0 + (k * kChunks + c) * lanes < slots * kChunks)
                    copies |= 1u << (k * kChunks + c);
        }
    }
    __device__ __forceinline__ bool valid(int rr) const { return rr < left; }
    __device__ __forceinline__ bool holds(int k) const { return (full >> k) & 1u; }
    // First column of slot k.
    __device__ __forceinline__ int slot_step() const { return WARP ? lanes : 32; }
    __device__ __forceinline__ int column(int k) const { return (first + k * slot_step()) * 8 + before; }
    // A warp's ring of `stages` stages of R rows of `count` operands.
    static __device__ __forceinline__ uint32_t stage_bytes(int count) { return R * count * K * kBlock; }
    __device__ __forceinline__ uint32_t warp_ring(uint32_t ring, int stages, int count) const {
        return ring + (threadIdx.x >> 5) * (stages * stage_bytes(count));
    }

    // Zeroes this warp's ring where some of its chunks lie outside the row: they are never
    // copied, and read as zeros ever after.
    __device__ __forceinline__ void clear(uint32_t ring, int stages, int count) const {
        if (__all_sync(0xFFFFFFFFu, copies == (1u << (K * kChunks)) - 1u)) return;
        for (int i = 0; i < stages * R * count * K; ++i) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};"
                             :: "r"(ring + i * kBlock + (threadIdx.x & 31) * 16 + c * 512), "r"(0u) : "memory");
        }
        __syncwarp();
    }
    // Copies the next R rows into the stage at `to` of this warp's ring (and the single elements
    // to end_w[stage]), as one group of asynchronous copies with what was issued since the last.
    template <int OPS, class Ends>
    __device__ __forceinline__ void issue(uint32_t to, int stage, const char *const (&ops)[OPS], int count,
                                          Ends &end_w) {
#pragma unroll
        for (int rr = 0; rr < R; ++rr) {
            if (rr < copy_left) {
                const int64_t row_at = copy_at + rr * step;
#pragma unroll
                for (int o = 0; o < OPS; ++o) {
                    if (o >= count) break;
                    const char *src = ops[o] + row_at;
                    const uint32_t dst = to + (rr * count + o) * K * kBlock + copy_to;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            const int i = k * kChunks + c;
                            cp_async16_if(copies & (1u << i),
                                          dst + k * kBlock + (WARP ? c * lanes * 16 : c * 512),
                                          src + (WARP ? i * lanes * 16 : i * 512));
                        }
                    }
                }
                if (EDGE && ends) {
                    if (end_col >= 0) {
                        // (the row's slot 0, from this thread's first chunk)
                        const int li = WARP ? first : static_cast<int>(threadIdx.x & 31);
                        const int64_t e = row_at - ((first - li) * kChunks + li) * 16 + (end_col - before) * T::kBytes;
#pragma unroll
                        for (int o = 0; o < OPS; ++o) {
                            if (o >= count) break;
                            cp_async4(static_cast<uint32_t>(__cvta_generic_to_shared(
                                          &end_w.w[stage][rr][o][threadIdx.x])),
                                      ops[o] + (e & ~int64_t(3)));
                        }
                    }
                }
            }
        }
        copy_at += R * step;
        copy_left -= R;
        cp_async_commit();
    }
    // This thread's slots of operand o of row rr in the stage at `from`, zero outside the row.
    __device__ __forceinline__ void fetch(Slot<T> (&s)[K], uint32_t from, int o, int rr, int count) const {
        const uint32_t src = from + (rr * count + o) * K * kBlock + slot_from;
#pragma unroll
        for (int k = 0; k < K; ++k) ld_shared_slot(s[k], src + k * kBlock);
        if constexpr (WARP || R > 1) {
            if (!valid(rr)) {      // (past the last row: the stage holds an earlier one)
#pragma unroll
                for (int k = 0; k < K; ++k) s[k].zero();
            }
        }
    }
    // The same of one slot, not zeroed past the last row.
    __device__ __forceinline__ void fetch_slot(Slot<T> &s, uint32_t from, int o, int k) const {
        ld_shared_slot(s, from + o * K * kBlock + slot_from + k * kBlock);
    }
    // This thread's single element of operand o; 0 when it has none.
    template <class Ends>
    __device__ __forceinline__ float fetch_end(const Ends &end_w, int stage, int o, int rr) const {
        if (end_col < 0 || !valid(rr)) return 0.0f;
        const uint32_t w = end_w.w[stage][rr][o][threadIdx.x];
        if constexpr (T::kBytes == 4) return __uint_as_float(w);
        const bool high = ((at >> 1) + end_col - before) & 1;
        return __uint_as_float(high ? w & 0xFFFF0000u : w << 16);
    }
    // Stores the slots of row rr (if `on`) at `base`, the slot boundary below the operand's
    // first element.
    __device__ __forceinline__ void store(char *base, int rr, bool on, const Slot<T> (&s)[K]) const {
        char *p = base + at + rr * step + first * (8 * T::kBytes);
#pragma unroll
        for (int k = 0; k < K; ++k)
            st_slot_if(on && holds(k), p + k * slot_step() * (8 * T::kBytes), s[k]);
    }
    __device__ __forceinline__ void store_slot(char *base, bool on, const Slot<T> &s, int k) const {
        st_slot_if(on && holds(k), base + at + (first + k * slot_step()) * (8 * T::kBytes), s);
    }
    // Stores this thread's single element; returns it as stored.
    __device__ __forceinline__ float store_end(char *base, int rr, bool on, float v) const {
        Frag<T, 1> f;
        const float o[1] = {v};
        f.put(o);
        if (on && end_col >= 0) st_global(base + at + rr * step + (end_col - before) * T::kBytes, f);
        return f.get(0);
    }
    // Generator group of slot k (the operands start on a slot boundary), and the element number
    // of the single element.
    __device__ __forceinline__ uint64_t group(int rr, int k) const {
        return static_cast<uint64_t>(at + rr * step) / (8 * T::kBytes) + static_cast<uint64_t>(first + k * slot_step());
    }
    __device__ __forceinline__ int64_t end_element(int rr) const {
        return (at + rr * step) / T::kBytes + end_col - before;
    }
    // The masks of row rr's slots, and whether the single element is kept: its group is
    // evaluated beside theirs in the one warp that needs it.
    __device__ __forceinline__ bool masks(DropGroup (&d)[K], const DropKey &key, int rr, uint32_t threshold) const {
        if (EDGE && ends) {
            DropGroup e[K + 1];
            uint64_t g[K + 1];
#pragma unroll
            for (int k = 0; k < K; ++k) g[k] = group(rr, k);
            const int64_t element = end_element(rr);
            g[K] = static_cast<uint64_t>(element) >> 3;
            drop_groups<K + 1>(e, key, g, threshold);
#pragma unroll
            for (int k = 0; k < K; ++k) d[k] = e[k];
            return e[K].keeps_any(static_cast<int>(element & 7));
        }
        uint64_t g[K];
#pragma unroll
        for (int k = 0; k < K; ++k) g[k] = group(rr, k);
        drop_groups<K>(d, key, g, threshold);
        return false;
    }
    // The thread's columns of a weight vector, zeros outside the row; once per CTA.  All
    // loads are independent of each other.
    __device__ __forceinline__ void weights(Slot<T> (&s)[K], const void *w) const {
        const bool whole = !EDGE && reinterpret_cast<uintptr_t>(w) % 16 == 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t j = holds(k) ? column(k) : 0;
            s[k].zero();
            if (whole) {
                if (holds(k)) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(s[k].w[4 * c]), "=r"(s[k].w[4 * c + 1]),
                                       "=r"(s[k].w[4 * c + 2]), "=r"(s[k].w[4 * c + 3])
                                     : "l"(elem_ptr<T>(w, j) + c * 16));
                }
            } else if (holds(k)) {
                Frag<T, 1> f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) ld_ro(f[i], elem_ptr<T>(w, j + i));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (T::kBytes == 4) {
                        s[k].w[i] = f[i].w;
                    } else {
                        s[k].w[i >> 1] |= static_cast<uint32_t>(f[i].h) << ((i & 1) * 16);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ float end_weight(const void *w) const {
        if (end_col < 0) return 0.0f;
        Frag<T, 1> f;
        ld_ro(f, elem_ptr<T>(w, end_col));
        return f.get(0);
    }
    __device__ __forceinline__ void advance() {
        row += R * stride;
        at += R * step;
        left -= R;
        cta_left -= R;
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

// Static shared memory of a tile kernel at most.
constexpr int64_t kTileStaticShared = 12288;
// Dynamic shared memory that a ring may use: the rest is the static row-sum slots.
constexpr int64_t kTileSharedBudget = kSharedBytesPerCta - kTileStaticShared;

// Dynamic shared memory of a ring.
inline int64_t tile_ring_bytes(int elem_bytes, int k, int threads, int stages, int operands) {
    return int64_t(stages) * operands * k * threads * (elem_bytes / 2) * 16;
}

// How a call's rows are laid over threads.
struct TileShape {
    bool ok;          // false: the looped kernel
    bool warp;        // several rows per warp
    bool edge;
    int k, threads, lanes, cluster;
    int mis;
};

constexpr int kWarpTileThreads = 128;
constexpr int kWarpTileSlots = 128;    // rows of at most this many slots share warps
// ... with so many slots per thread.
constexpr int warp_tile_slots(int64_t slots) {
    return slots <= 8 ? 1 : (slots <= 64 ? 2 : (slots <= 96 ? 3 : 4));
}

// Few rows, at most one per SM, of more slots than a warp's: what counts is how soon one row is
// done.  One slot per thread, and a row of 512 slots or more over as many CTAs of 64
// threads or more as there are SMs for it (measured on GB300, us a call: layernorm 1 x 6656
// f32 2.7 against 3.2 in one CTA of 416 threads, its gradient 4.0 against 6.0; the gradient of
// 64 x 768 f32 4.2 against 5.1 in warps).
inline bool tile_few_rows(int64_t rows, int64_t n, int sms) {
    return rows <= sms && n / 8 > 32 && n / 8 <= int64_t(kMaxCluster) * 512;
}
inline int tile_few_threads(int64_t rows, int64_t n, int sms) {
    const int64_t slots = n / 8;
    int threads = 64;
    while (threads < 512 && (slots < 512 || rows * ((slots + threads - 1) / threads) > sms ||
                             (slots + threads - 1) / threads > kMaxCluster))
        threads *= 2;
    return threads;
}

// Shape of rows of n elements whose operands lie `mis` elements past a slot boundary:
// `k` slots per thread for rows of a CTA, CTAs of at most `most_threads`.
inline TileShape tile_shape(int64_t n, int mis, int k, int most_threads, bool few) {
    TileShape s = {};
    s.mis = mis;
    s.edge = mis != 0 || n % 8 != 0;
    s.cluster = 1;
    s.lanes = 32;
    const int64_t slots = n < 8 ? 1 : n / 8;
    if (slots <= kWarpTileSlots && !few) {
        s.warp = true;
        s.k = warp_tile_slots(slots);
        s.lanes = s.edge ? kEndLanes : 1;      // (a lane for each element at the ends)
        while (s.lanes * s.k < slots) s.lanes *= 2;
        s.threads = kWarpTileThreads;
    } else {
        s.k = k;
        const int64_t most = int64_t(k) * most_threads;
        if (slots > most * kMaxCluster) return s;
        s.cluster = static_cast<int>((slots + most - 1) / most);
        const int64_t per = (slots + s.cluster - 1) / s.cluster;
        s.threads = static_cast<int>((per + 32 * k - 1) / (32 * k)) * 32;
    }
    s.ok = true;
    return s;
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

// What is known of a kernel on each device: the CTAs that an SM's registers hold, by the warps
// of a CTA (0: not asked yet, and entry 0 whether the kernel has been opened to the shared
// memory and the cluster sizes below), and the clusters that the device holds, in a few
// entries of (threads, cluster, shared memory).  Every thread finds the same values, so that
// calls that race only repeat them.
constexpr int kClusterEntries = 8;
struct TileLaunchCache {
    std::atomic<int> resident[kMaxCachedDevices][kTileMaxThreads / 32 + 1];
    std::atomic<uint64_t> clusters[kMaxCachedDevices][kClusterEntries];
};

template <class... Params>
cudaError_t open_tile(TileLaunchCache &cache, void (*fn)(Params...), int threads, int *resident) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool cached = dev >= 0 && dev < kMaxCachedDevices;
    *resident = cached ? cache.resident[dev][threads / 32].load(std::memory_order_acquire) : 0;
    if (*resident > 0) return cudaSuccess;
    if (!cached || cache.resident[dev][0].load(std::memory_order_acquire) == 0) {
        err = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(kTileSharedBudget));
        if (err != cudaSuccess) return err;
        err = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (err != cudaSuccess) return err;
        if (cached) cache.resident[dev][0].store(1, std::memory_order_release);
    }
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(resident, fn, threads, 0);
    if (err != cudaSuccess) return err;
    if (*resident < 1) return cudaErrorInvalidConfiguration;
    if (cached) cache.resident[dev][threads / 32].store(*resident, std::memory_order_release);
    return cudaSuccess;
}

// Clusters of p.cluster CTAs that the device holds at once: fewer than its SMs divided by their
// number, since a cluster does not leave its group of SMs; a grid of more would end in a second
// wave (4096 x 16384 f32, the gradient of RMSNorm: 256 us against 180).
template <class... Params>
cudaError_t resident_clusters(TileLaunchCache &cache, void (*fn)(Params...), const TileShape &p, int64_t shared,
                              int *count) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool cached = dev >= 0 && dev < kMaxCachedDevices;
    const uint64_t key = (static_cast<uint64_t>(shared) * 2048 + p.threads) * 32 + p.cluster;
    std::atomic<uint64_t> &entry = cache.clusters[cached ? dev : 0][key * 0x9E3779B97F4A7C15u >> 61];
    static_assert(kClusterEntries == 8, "three bits of the hash");
    const uint64_t known = cached ? entry.load(std::memory_order_relaxed) : 0;
    if (known / 4096 == key) {
        *count = static_cast<int>(known % 4096);
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(p.cluster), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(p.threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(shared);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaOccupancyMaxActiveClusters(count, fn, &cfg);
    if (err != cudaSuccess) return err;
    if (*count < 1) return cudaErrorInvalidConfiguration;
    if (*count > 4095) *count = 4095;
    if (cached) entry.store(key * 4096 + *count, std::memory_order_relaxed);
    return cudaSuccess;
}

// The rest of a launch: as many CTAs as the registers let an SM hold (at most most_per_sm), a
// ring as deep as shared memory then allows (two stages at least where it can be), and a
// persistent grid.
struct TileGrid {
    int stages;       // 0: the ring does not fit
    int64_t ctas;
    int64_t shared;   // bytes of the ring, and of what the kernel keeps beside it
};

template <class... Params>
cudaError_t tile_grid(TileLaunchCache &cache, void (*fn)(Params...), const TileShape &s, int64_t rows, int64_t n,
                      int rows_at_a_time, int elem_bytes, int operands, int most_per_sm, int sms, TileGrid *g,
                      int64_t beside = 0, int most_stages = kTileMaxStages) {
    *g = TileGrid{};
    int per_sm = 0;
    cudaError_t err = open_tile(cache, fn, s.threads, &per_sm);
    if (err != cudaSuccess) return err;
    if (per_sm > most_per_sm) per_sm = most_per_sm;
    const int64_t stage = tile_ring_bytes(elem_bytes, s.k, s.threads, 1, operands * rows_at_a_time);
    for (;; --per_sm) {
        const int64_t budget = (kTileSharedBudget - (per_sm - 1) * kTileStaticShared) / per_sm - beside;
        g->stages = budget < 0 ? 0 : static_cast<int>(budget / stage);
        if (g->stages >= 2 || per_sm == 1) break;
    }
    if (g->stages > most_stages) g->stages = most_stages;
    if (g->stages < 1) return cudaSuccess;
    g->shared = stage * g->stages + beside;
    int64_t groups = static_cast<int64_t>(sms) * per_sm;      // CTAs or clusters
    if (s.cluster > 1) {
        int clusters = 0;
        err = resident_clusters(cache, fn, s, g->shared, &clusters);
        if (err != cudaSuccess) return err;
        const int64_t most = static_cast<int64_t>(sms) * most_per_sm / s.cluster;
        groups = clusters < most ? clusters : most;
    }
    const int64_t rows_per_cta = s.warp ? s.threads / s.lanes : 1;
    // rows of one CTA start alike only when they are a multiple of eight elements apart
    int64_t alike = 1;
    while (alike * rows_per_cta % 8 * (n % 8) % 8 != 0) alike *= 2;
    groups = groups < alike ? alike : groups - groups % alike;
    const int64_t need = (rows + rows_per_cta - 1) / rows_per_cta;
    if (groups > need) groups = need;
    g->ctas = groups * s.cluster;
    return cudaSuccess;
}

template <class... Params, class... Args>
cudaError_t launch_tile(void (*fn)(Params...), const TileShape &p, int64_t ctas, int64_t shared, bool pdl,
                        cudaStream_t stream, uint64_t *launches, Args... args) {
    if (ctas < 1 || ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
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
    const cudaError_t err = cudaLaunchKernelEx(&cfg, fn, args...);
    if (err == cudaSuccess) ++*launches;
    return err;
}

}  // namespace mrn
