// Tokens sorted by expert and back: the stable counting sort of a router's
// choices (dopt_route_sort), the copy of each token's row to its experts'
// places (dopt_route_dispatch), the weighted sum of the experts' rows
// (dopt_route_combine) and its gradients (dopt_route_combine_grad).  dopt.h
// states their contracts.
#include <mutex>

#include "op_common.cuh"

namespace {

// ---------------------------------------------------------------------------
// Sort.  Slots in order; bin e < E is expert e, bin E the dropped slots.  A
// slot's row is the number of slots in lower bins plus the number of earlier
// slots of its own bin, so the order inside a bin is the slots' order (stable,
// the same at every call).  Every prefix is a sum of integers.
//
// Up to 2^15 slots: one launch of one cluster of 8 blocks (one block up to
// 4096 slots).  Blocks, and warps in a block, take consecutive stretches; a
// warp counts its slots by bin, 32 at a time, the counts become first rows by
// a scan over the warps, over the blocks (through the cluster's shared
// memory) and over the bins, and the warp goes through its slots again.
// More slots: a launch that counts stretches of 2048 slots (of more above
// 304 * 2048, so that there are at most 304 of them) and one that places
// them, each block adding up the stretches before it.  Sorting 2^18 slots of
// 64 experts and copying their 512 bf16 columns takes 86 us with the cluster
// (41 us for the sort: its 8 SMs store to a sector a slot) and 56 us with the
// two launches (58 and 63 us with stretches of 4096 and 1024); 2^15 slots and
// 2048 columns 40.4 us with the cluster and 42.5 us with the two.  (Putting a
// stretch's rows in order before they are stored changed nothing.)
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 4;  // slots a thread takes at a time, in the cluster
constexpr int kTileRounds = 2;  // in the two launches
constexpr int64_t kSortTile = int64_t(kSortThreads) * kTileRounds;
constexpr int kSortCluster = 8;
constexpr int64_t kClusterSlots = int64_t(1) << 15;
constexpr int64_t kSortMaxTiles = 304;

struct SortArgs {
    const void *ids;
    int32_t *slot_row, *row_token, *offsets;
    int32_t *counts;  // [tiles][bins]
    int32_t slots, k, experts, tiles;
    int32_t rounds;  // of 2048 slots, a tile
    int32_t wide;    // 64-bit ids
};

__device__ __forceinline__ int bin_of(const SortArgs &a, int64_t slot) {
    const int64_t id = a.wide ? static_cast<const int64_t *>(a.ids)[slot]
                              : int64_t(static_cast<const int32_t *>(a.ids)[slot]);
    return id >= 0 && id < a.experts ? int(id) : a.experts;
}

// This lane's slot among its warp's 32: how many slots of its bin came before
// it; count[] moves on.  The lanes of a bin are those that agree in every one
// of its `bits` bits, a ballot each (a match instruction costs an SM some 60
// cycles a warp: with it a cluster sorted 262144 slots in 62 us).
__device__ __forceinline__ int rank_in_warp(int bin, int bits, int lane, int32_t *count) {
    unsigned peers = __ballot_sync(kFull, bin >= 0);
    for (int b = 0; b < bits; ++b) {
        const bool set = bin >> b & 1;
        const unsigned with = __ballot_sync(kFull, set);
        peers &= set ? with : ~with;
    }
    const int before = __popc(peers & ((1u << lane) - 1u));
    const int at = bin >= 0 ? count[bin] + before : 0;
    __syncwarp();
    if (bin >= 0 && before == 0) count[bin] = at + __popc(peers);
    __syncwarp();
    return at;
}

__device__ __forceinline__ int inclusive_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFull, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// base[b] += the sum of total[0..b); written to `offsets` too unless NULL.
// By all threads of the block.
__device__ __forceinline__ void scan_bins(const int32_t *total, int32_t *base, int bins, int32_t *offsets,
                                          int32_t (&warp_sum)[kSortWarps]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int carry = 0;
    for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
        const int b = b0 + int(threadIdx.x);
        const int v = b < bins ? total[b] : 0;
        const int incl = inclusive_scan(v, lane);
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        if (warp == 0) warp_sum[lane] = inclusive_scan(warp_sum[lane], lane);
        __syncthreads();
        const int excl = carry + incl - v + (warp ? warp_sum[warp - 1] : 0);
        if (b < bins) {
            base[b] += excl;
            if (offsets) offsets[b] = excl;
        }
        carry += warp_sum[kSortWarps - 1];
        __syncthreads();
    }
}

// Shared memory: total[bins], base[bins], then counts [32 warps][bins].
__global__ void __launch_bounds__(kSortThreads) dopt_route_sort_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ int32_t smem[];
    __shared__ int32_t warp_sum[kSortWarps];
    const int bins = a.experts + 1;
    int32_t *total = smem, *base = smem + bins, *count = smem + 2 * bins;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bits = 32 - __clz(a.experts);
    const int blocks = int(gridDim.x), block = int(blockIdx.x);  // the grid is the cluster
    let_dependents_start();
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) count[i] = 0;
    wait_for_grids_before();
    __syncthreads();

    // this warp's slots: whole rounds of 32 * kSortRounds
    constexpr int kRound = 32 * kSortRounds;
    const int64_t rounds = (a.slots + int64_t(kRound) * kSortWarps * blocks - 1) / (int64_t(kRound) * kSortWarps * blocks);
    const int64_t first = (int64_t(block) * kSortWarps + warp) * rounds * kRound;
    int32_t *mine = count + warp * bins;
    auto load = [&](int64_t round, int (&bin)[kSortRounds]) {
#pragma unroll
        for (int q = 0; q < kSortRounds; ++q) {
            const int64_t s = first + round * kRound + q * 32 + lane;
            bin[q] = round < rounds && s < a.slots ? bin_of(a, s) : -1;
        }
    };
    int bin[kSortRounds], next[kSortRounds];
    load(0, next);
    for (int64_t r = 0; r < rounds; ++r) {
#pragma unroll
        for (int q = 0; q < kSortRounds; ++q) bin[q] = next[q];
        load(r + 1, next);
#pragma unroll
        for (int q = 0; q < kSortRounds; ++q)
            if (bin[q] >= 0) atomicAdd(&mine[bin[q]], 1);
    }
    load(0, next);  // for the second time through, under the scans
    __syncthreads();
    for (int b = warp; b < bins; b += kSortWarps) {  // lane l: warp l's count
        const int c = count[lane * bins + b], incl = inclusive_scan(c, lane);
        count[lane * bins + b] = incl - c;
        if (lane == 31) total[b] = incl;
    }
    __syncthreads();
    if (blocks > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        for (int b = threadIdx.x; b < bins; b += kSortThreads) {
            const uint32_t own = static_cast<uint32_t>(__cvta_generic_to_shared(&total[b]));
            int before = 0, all = 0;
            for (int o = 0; o < blocks; ++o) {
                uint32_t at;
                int32_t v;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(own), "r"(o));
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
                if (o < block) before += v;
                all += v;
            }
            base[b] = before;
            smem[(2 + kSortWarps) * bins + b] = all;
        }
        // the others' totals have been read before any of them goes
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        total = smem + (2 + kSortWarps) * bins;
    } else {
        for (int b = threadIdx.x; b < bins; b += kSortThreads) base[b] = 0;
    }
    __syncthreads();
    scan_bins(total, base, bins, block == 0 ? a.offsets : nullptr, warp_sum);
    for (int64_t r = 0; r < rounds; ++r) {
#pragma unroll
        for (int q = 0; q < kSortRounds; ++q) bin[q] = next[q];
        load(r + 1, next);
#pragma unroll
        for (int q = 0; q < kSortRounds; ++q) {
            const int row = rank_in_warp(bin[q], bits, lane, mine);
            if (bin[q] < 0) continue;
            const int64_t s = first + r * kRound + q * 32 + lane;
            const bool kept = bin[q] < a.experts;
            a.slot_row[s] = kept ? base[bin[q]] + row : -1;
            a.row_token[base[bin[q]] + row] = kept ? int32_t(s / a.k) : -1;
        }
    }
}

__global__ void __launch_bounds__(kSortThreads) dopt_route_count_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ int32_t hist[];
    const int bins = a.experts + 1;
    let_dependents_start();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) hist[b] = 0;
    wait_for_grids_before();
    __syncthreads();
    for (int round = 0; round < a.rounds; ++round) {
        const int64_t s0 = (int64_t(blockIdx.x) * a.rounds + round) * kSortTile + threadIdx.x;
#pragma unroll
        for (int r = 0; r < kTileRounds; ++r)
            if (s0 + r * kSortThreads < a.slots) atomicAdd(&hist[bin_of(a, s0 + r * kSortThreads)], 1);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads)
        a.counts[int64_t(blockIdx.x) * bins + b] = hist[b];
}

// Shared memory as above.
__global__ void __launch_bounds__(kSortThreads) dopt_route_place_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ int32_t smem[];
    __shared__ int32_t warp_sum[kSortWarps];
    const int bins = a.experts + 1;
    int32_t *total = smem, *base = smem + bins, *count = smem + 2 * bins;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bits = 32 - __clz(a.experts);
    let_dependents_start();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) total[b] = base[b] = 0;
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) count[i] = 0;
    wait_for_grids_before();
    __syncthreads();
    int bin[kTileRounds], rank[kTileRounds];
    auto take = [&](int64_t s0) {
#pragma unroll
        for (int r = 0; r < kTileRounds; ++r) bin[r] = s0 + 32 * r < a.slots ? bin_of(a, s0 + 32 * r) : -1;
#pragma unroll
        for (int r = 0; r < kTileRounds; ++r) rank[r] = rank_in_warp(bin[r], bits, lane, count + warp * bins);
    };
    int64_t s0 = int64_t(blockIdx.x) * a.rounds * kSortTile + int64_t(warp) * 32 * kTileRounds + lane;
    take(s0);
    // slots of each bin in all tiles, and in the tiles before this one
    const int n = a.tiles * bins, mine = int(blockIdx.x) * bins;
    for (int i0 = threadIdx.x; i0 < n; i0 += 4 * kSortThreads) {
        int32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = i0 + j * kSortThreads < n ? a.counts[i0 + j * kSortThreads] : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * kSortThreads;
            if (c[j]) {
                atomicAdd(&total[i % bins], c[j]);
                if (i < mine) atomicAdd(&base[i % bins], c[j]);
            }
        }
    }
    __syncthreads();
    scan_bins(total, base, bins, blockIdx.x == 0 ? a.offsets : nullptr, warp_sum);
    for (int round = 0;; ++round) {
        for (int b = warp; b < bins; b += kSortWarps) {  // lane l: warp l's count
            const int c = count[lane * bins + b], incl = inclusive_scan(c, lane);
            count[lane * bins + b] = incl - c;
            if (lane == 31) total[b] = incl;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kTileRounds; ++r) {
            if (bin[r] < 0) continue;
            const int64_t s = s0 + 32 * r;
            const int row = base[bin[r]] + count[warp * bins + bin[r]] + rank[r];
            const bool kept = bin[r] < a.experts;
            a.slot_row[s] = kept ? row : -1;
            a.row_token[row] = kept ? int32_t(s / a.k) : -1;
        }
        if (round + 1 == a.rounds) return;
        __syncthreads();
        for (int b = threadIdx.x; b < bins; b += kSortThreads) base[b] += total[b];
        for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) count[i] = 0;
        __syncthreads();
        s0 += kSortTile;
        take(s0);
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Rows.  Every kernel moves rows in accesses of VB bytes, the widest (16, 8,
// 4 or 2) that the pointers, the row strides and the row length allow.
// ---------------------------------------------------------------------------

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

struct RowArgs {
    const void *x;           // dispatch: tokens; combine: sorted rows; gradient: d_out
    const void *rows;        // gradient: sorted rows
    void *out;               // dispatch: sorted rows; combine: tokens; gradient: d_rows
    const int32_t *slot_row;
    const float *weights;
    float *d_weights;
    int64_t tokens, n_rows;
    int64_t ld;              // row stride of the token-ordered array, in accesses
    int32_t vecs;            // accesses a row
    int32_t k;
};

// A warp takes 32 * U accesses of one token's row: read once, written to the
// row of each of the token's k slots.  Bound by memory, mostly writing: 32768
// tokens x 512 bf16 to 8 slots take 45 us (6.7 TB/s).  With the sort 56 us; 60
// us for 510 columns (4-byte accesses), 101 us for 511 (2-byte ones).
template <int VB, int U>
__global__ void __launch_bounds__(kRowThreads) dopt_route_dispatch_kernel(const RowArgs a) {
    using V = typename Raw<VB>::type;
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    let_dependents_start();
    wait_for_grids_before();
    if (t >= a.tokens) return;
    const int c0 = int(blockIdx.y) * 32 * U + lane;
    const V *src = static_cast<const V *>(a.x) + t * a.ld;
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (c0 + 32 * u < a.vecs) v[u] = src[c0 + 32 * u];
    for (int j0 = 0; j0 < a.k; j0 += 32) {
        const int mine = j0 + lane < a.k ? a.slot_row[t * a.k + j0 + lane] : -1;
        const int n = min(32, a.k - j0);
        for (int j = 0; j < n; ++j) {
            const int r = __shfl_sync(kFull, mine, j);
            if (r < 0 || r >= a.n_rows) continue;
            V *dst = static_cast<V *>(a.out) + int64_t(r) * a.vecs;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * u < a.vecs) dst[c0 + 32 * u] = v[u];
        }
    }
}

// A warp takes 32 * U accesses of a token's row, of one token after another:
// the sum over the token's slots, in order, of weight * row, in fp32, rounded
// once.  Dropped slots are left out (a weight of NaN there does not matter).
// The rows of A slots are in flight at once, and the next token's slots and
// weights are loaded under them.  Bound by memory: 32768 tokens x 512 bf16
// from 8 slots take 47 us (6.4 TB/s; 61 us with the rows kept in L1, though
// none is read twice); 59 us for 510 columns, 82 us for 511.
template <typename T, int VB, int U, int A>
__global__ void __launch_bounds__(kRowThreads) dopt_route_combine_kernel(const __grid_constant__ RowArgs a) {
    using V = typename Raw<VB>::type;
    constexpr int N = VB / int(sizeof(T));
    const int lane = threadIdx.x & 31;
    const int64_t stride = int64_t(gridDim.x) * kRowWarps;
    int64_t t = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    let_dependents_start();
    wait_for_grids_before();
    const int c0 = int(blockIdx.y) * 32 * U + lane;
    const V *rows = static_cast<const V *>(a.x);
    int next_row = -1;
    float next_weight = 1.0f;
    auto slots_of = [&](int64_t token, int j0) {
        next_row = -1;
        if (token < a.tokens && j0 + lane < a.k) {
            next_row = a.slot_row[token * a.k + j0 + lane];
            if (a.weights) next_weight = a.weights[token * a.k + j0 + lane];
        }
    };
    slots_of(t, 0);
    for (; t < a.tokens; t += stride) {
        float acc[U][N] = {};
        for (int j0 = 0; j0 < a.k; j0 += 32) {
            int row = next_row;
            const float weight = next_weight;
            if (row >= a.n_rows) row = -1;
            if (j0 + 32 < a.k) slots_of(t, j0 + 32);
            else slots_of(t + stride, 0);
            const int n = min(32, a.k - j0);
            for (int j = 0; j < n; j += A) {
                V v[A][U];
                int r[A];
#pragma unroll
                for (int q = 0; q < A; ++q) {
                    r[q] = j + q < n ? __shfl_sync(kFull, row, j + q) : -1;
                    if (r[q] < 0) continue;
                    const V *p = rows + int64_t(r[q]) * a.vecs + c0;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (c0 + 32 * u < a.vecs) v[q][u] = __ldcs(p + 32 * u);
                }
#pragma unroll
                for (int q = 0; q < A; ++q) {
                    if (r[q] < 0) continue;
                    const float w = __shfl_sync(kFull, weight, j + q);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float f[N];
                        unpack<T, VB>(v[q][u], f);
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[u][i] = fmaf(w, f[i], acc[u][i]);
                    }
                }
            }
        }
        V *dst = static_cast<V *>(a.out) + t * a.ld + c0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * u < a.vecs) __stcs(dst + 32 * u, pack<T, VB>(acc[u]));
    }
}

// A warp takes G neighbouring slots, and G others after them: d_row =
// weight * d_out in one pass that also sums <d_out, row>.  The G slots' loads
// are in flight at once, and the next ones' rows and weights are looked up
// under them; d_out, read by all of a token's slots, mostly hits in L1.  Bound
// by memory, half of it writing: 95 us (6.0 TB/s) for 32768 tokens x 512 bf16
// and 8 slots; 115 us for 510 columns, 149 us for 511.
template <typename T, int VB, int U, int G>
__global__ void __launch_bounds__(kRowThreads) dopt_route_combine_grad_kernel(const __grid_constant__ RowArgs a) {
    using V = typename Raw<VB>::type;
    constexpr int N = VB / int(sizeof(T));
    const int lane = threadIdx.x & 31;
    const int64_t slots = a.tokens * a.k, stride = int64_t(gridDim.x) * kRowWarps * G;
    int64_t s = (int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5)) * G;
    let_dependents_start();
    wait_for_grids_before();
    int next_row[G];
    float next_weight[G];
    auto look_up = [&](int64_t first) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            next_row[g] = first + g < slots ? a.slot_row[first + g] : -1;
            next_weight[g] = first + g < slots ? a.weights[first + g] : 0.0f;
        }
    };
    look_up(s);
    for (; s < slots; s += stride) {
        int row[G];
        float w[G], dot[G] = {};
        const V *d[G], *y[G];
        V *out[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            row[g] = next_row[g] < a.n_rows ? next_row[g] : -1;
            w[g] = next_weight[g];
            // (slots are below 2^31)
            d[g] = static_cast<const V *>(a.x) + int64_t(uint32_t(s + g) / uint32_t(a.k)) * a.ld;
            y[g] = static_cast<const V *>(a.rows) + int64_t(max(row[g], 0)) * a.vecs;
            out[g] = static_cast<V *>(a.out) + int64_t(max(row[g], 0)) * a.vecs;
        }
        look_up(s + stride);
        for (int c0 = lane; c0 < a.vecs; c0 += 32 * U) {
            V dv[G][U], yv[G][U];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (row[g] < 0) continue;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + 32 * u < a.vecs) {
                        yv[g][u] = __ldcs(y[g] + c0 + 32 * u);
                        dv[g][u] = d[g][c0 + 32 * u];
                    }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (row[g] < 0) continue;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c0 + 32 * u >= a.vecs) continue;
                    float df[N], yf[N];
                    unpack<T, VB>(dv[g][u], df);
                    unpack<T, VB>(yv[g][u], yf);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        dot[g] = fmaf(df[i], yf[i], dot[g]);
                        df[i] = w[g] * df[i];
                    }
                    __stcs(out[g] + c0 + 32 * u, pack<T, VB>(df));
                }
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) dot[g] += __shfl_xor_sync(kFull, dot[g], m);
            if (lane == 0 && s + g < slots) a.d_weights[s + g] = dot[g];  // 0 for a dropped slot
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Rounds of 2048 slots a stretch.
int64_t sort_rounds(int64_t slots) { return (slots + kSortTile * kSortMaxTiles - 1) / (kSortTile * kSortMaxTiles); }

int64_t sort_tiles(int64_t slots) {
    const int64_t tile = kSortTile * sort_rounds(slots);
    return (slots + tile - 1) / tile;
}

// What a call uses.
int64_t sort_workspace(int64_t slots, int32_t experts) {
    return slots > kClusterSlots ? sort_tiles(slots) * (experts + 1) * int64_t(sizeof(int32_t)) : 0;
}

// What any call of up to so many slots uses: with more than 304 stretches'
// slots they get longer and, at first, fewer.
int64_t sort_workspace_up_to(int64_t slots, int32_t experts) {
    if (slots <= kClusterSlots) return 0;
    const int64_t tiles = std::min<int64_t>(kSortMaxTiles, (slots + kSortTile - 1) / kSortTile);
    return tiles * (experts + 1) * int64_t(sizeof(int32_t));
}

// Bytes of the sorting kernels' shared memory.
constexpr size_t sort_smem(size_t bins) { return (3 + kSortWarps) * bins * sizeof(int32_t); }

std::mutex g_sort_mutex;
bool g_sort_ready[64] = {};  // devices whose kernels are set up

// Raises the sorting kernels' shared-memory limit, once a device and to what
// the most experts need: the limit is the kernel's, for all threads and calls.
int set_up_sort(const char *who) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess && (device < 0 || device >= 64)) return dopt::fail(DOPT_E_ARG, "%s: device %d", who, device);
    std::lock_guard<std::mutex> lock(g_sort_mutex);
    if (e == cudaSuccess && !g_sort_ready[device]) {
        constexpr int kMost = int(sort_smem(DOPT_MAX_EXPERTS + 1));
        e = cudaFuncSetAttribute(dopt_route_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(dopt_route_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        g_sort_ready[device] = e == cudaSuccess;
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return dopt::fail(DOPT_E_CUDA, "%s: shared-memory limit: %s", who, cudaGetErrorString(e));
    }
    return DOPT_OK;
}

int check_slots(const char *who, int64_t tokens, int32_t k) {
    if (tokens < 0 || k < 1 || k > DOPT_MAX_TOPK || tokens > INT32_MAX / k)
        return dopt::fail(DOPT_E_ARG, "%s: tokens %lld, k %d (k in 1..%d, tokens * k below 2^31)",
                          who, static_cast<long long>(tokens), k, DOPT_MAX_TOPK);
    return DOPT_OK;
}

int check_rows(const char *who, dopt_dtype dtype, int64_t n_rows, int64_t cols, int64_t ld) {
    if (!valid_dtype(dtype)) return dopt::fail(DOPT_E_ARG, "%s: unknown dtype %d", who, int(dtype));
    if (n_rows < 0 || n_rows > INT32_MAX)
        return dopt::fail(DOPT_E_ARG, "%s: n_rows out of range", who);
    if (cols < 1 || cols > DOPT_MAX_COLS || ld < cols)
        return dopt::fail(DOPT_E_ARG, "%s: cols %lld, row stride %lld (cols in 1..%d, stride >= cols)",
                          who, static_cast<long long>(cols), static_cast<long long>(ld), DOPT_MAX_COLS);
    return DOPT_OK;
}

int check_pointer(const char *who, const char *name, const void *p, size_t align) {
    if (!p) return dopt::fail(DOPT_E_ARG, "%s: %s is NULL", who, name);
    if (!aligned_to(p, align))
        return dopt::fail(DOPT_E_ALIGN, "%s: %s is not aligned to its elements", who, name);
    return DOPT_OK;
}

template <int VB, int U>
int launch_dispatch(const char *who, const RowArgs &a, cudaStream_t stream) {
    const dim3 grid(unsigned((a.tokens + kRowWarps - 1) / kRowWarps),
                    unsigned((a.vecs + 32 * U - 1) / (32 * U)));
    return launch_op(who, dopt_route_dispatch_kernel<VB, U>, grid, dim3(kRowThreads), 0, stream, a);
}

// Blocks for `blocks` blocks' work: at most 6 an SM's worth, each taking
// several tokens in turn (32768 tokens x 512 bf16, 8 slots, combine and its
// gradient: 47 and 95 us; 4 an SM 55 and 119, 12 an SM 48 and 96).
unsigned row_blocks(int64_t blocks) { return unsigned(std::min<int64_t>(blocks, 152 * 6)); }

template <typename T, int VB, int U, int A>
int launch_combine(const char *who, const RowArgs &a, cudaStream_t stream) {
    const dim3 grid(row_blocks((a.tokens + kRowWarps - 1) / kRowWarps), unsigned((a.vecs + 32 * U - 1) / (32 * U)));
    return launch_op(who, dopt_route_combine_kernel<T, VB, U, A>, grid, dim3(kRowThreads), 0, stream, a);
}

// Slots in flight: 2 for up to 2 a token, 4 otherwise (47 us for 8 a token; 8
// in flight 48.5).
template <typename T, int VB, int U>
int pick_ahead(const char *who, const RowArgs &a, cudaStream_t stream) {
    return a.k <= 2 ? launch_combine<T, VB, U, 2>(who, a, stream) : launch_combine<T, VB, U, 4>(who, a, stream);
}

template <typename T>
int pick_combine(const char *who, const RowArgs &a, int vb, cudaStream_t stream) {
    if (vb == 16) return pick_ahead<T, 16, 2>(who, a, stream);
    if (vb == 8) return pick_ahead<T, 8, 4>(who, a, stream);
    if (vb == 4) return pick_ahead<T, 4, 4>(who, a, stream);
    if constexpr (sizeof(T) == 2) return pick_ahead<T, 2, 4>(who, a, stream);
    return DOPT_E_ALIGN;  // not reached: fp32 rows are 4-byte aligned
}

template <typename T, int VB, int U, int G>
int launch_combine_grad(const char *who, const RowArgs &a, cudaStream_t stream) {
    const dim3 grid(row_blocks((a.tokens * a.k + G * kRowWarps - 1) / (G * kRowWarps)));
    return launch_op(who, dopt_route_combine_grad_kernel<T, VB, U, G>, grid, dim3(kRowThreads), 0, stream, a);
}

// G = 2 slots a warp with 16-byte accesses, two of each row at a time: 95 us
// where one slot takes 128 and four, one access each, 108.
template <typename T>
int pick_combine_grad(const char *who, const RowArgs &a, int vb, cudaStream_t stream) {
    if (vb == 16) return launch_combine_grad<T, 16, 2, 2>(who, a, stream);
    if (vb == 8) return launch_combine_grad<T, 8, 4, 1>(who, a, stream);
    if (vb == 4) return launch_combine_grad<T, 4, 8, 1>(who, a, stream);
    if constexpr (sizeof(T) == 2) return launch_combine_grad<T, 2, 8, 1>(who, a, stream);
    return DOPT_E_ALIGN;  // not reached: fp32 rows are 4-byte aligned
}

}  // namespace

extern "C" int dopt_route_workspace(int64_t tokens, int32_t k, int32_t n_experts, int64_t *bytes) {
    dopt::clear_error();
    const char *who = "dopt_route_workspace";
    if (!bytes) return dopt::fail(DOPT_E_ARG, "%s: bytes is NULL", who);
    int rc = check_slots(who, tokens, k);
    if (rc != DOPT_OK) return rc;
    if (n_experts < 1 || n_experts > DOPT_MAX_EXPERTS)
        return dopt::fail(DOPT_E_ARG, "%s: n_experts %d (1..%d)", who, n_experts, DOPT_MAX_EXPERTS);
    *bytes = sort_workspace_up_to(tokens * k, n_experts);
    return DOPT_OK;
}

extern "C" int dopt_route_sort(const void *expert_ids, int32_t id_bytes, int64_t tokens, int32_t k,
                               int32_t n_experts, int32_t *slot_row, int32_t *row_token,
                               int32_t *offsets, void *workspace, int64_t workspace_bytes,
                               cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_route_sort";
    OpRange range(who);
    if (id_bytes != 4 && id_bytes != 8)
        return fail(DOPT_E_ARG, "%s: id_bytes %d is not 4 or 8", who, id_bytes);
    int rc = check_slots(who, tokens, k);
    if (rc != DOPT_OK) return rc;
    if (n_experts < 1 || n_experts > DOPT_MAX_EXPERTS)
        return fail(DOPT_E_ARG, "%s: n_experts %d (1..%d)", who, n_experts, DOPT_MAX_EXPERTS);
    if ((rc = check_pointer(who, "offsets", offsets, 4)) != DOPT_OK) return rc;
    if (tokens > 0) {
        if ((rc = check_pointer(who, "expert_ids", expert_ids, size_t(id_bytes))) != DOPT_OK) return rc;
        if ((rc = check_pointer(who, "slot_row", slot_row, 4)) != DOPT_OK) return rc;
        if ((rc = check_pointer(who, "row_token", row_token, 4)) != DOPT_OK) return rc;
    }
    const int64_t need = sort_workspace(tokens * k, n_experts);
    if (need > 0) {
        if ((rc = check_pointer(who, "workspace", workspace, 4)) != DOPT_OK) return rc;
        if (workspace_bytes < need)
            return fail(DOPT_E_ARG, "%s: workspace of %lld bytes, %lld needed", who,
                        static_cast<long long>(workspace_bytes), static_cast<long long>(need));
    }
    SortArgs a{};
    a.ids = expert_ids;
    a.slot_row = slot_row;
    a.row_token = row_token;
    a.offsets = offsets;
    a.counts = static_cast<int32_t *>(workspace);
    a.slots = int32_t(tokens * k);
    a.k = k;
    a.experts = n_experts;
    a.wide = id_bytes == 8;
    const size_t bins = size_t(n_experts) + 1, smem = sort_smem(bins);
    if ((rc = set_up_sort(who)) != DOPT_OK) return rc;
    if (need == 0) {
        const unsigned blocks = a.slots <= kSortThreads * kSortRounds ? 1 : kSortCluster;
        return launch_cluster(who, dopt_route_sort_kernel, dim3(blocks), blocks, dim3(kSortThreads), smem, stream, a);
    }
    a.rounds = int32_t(sort_rounds(a.slots));
    a.tiles = int32_t(sort_tiles(a.slots));
    rc = launch_op(who, dopt_route_count_kernel, dim3(unsigned(a.tiles)), dim3(kSortThreads), bins * sizeof(int32_t),
                   stream, a);
    if (rc != DOPT_OK) return rc;
    return launch_op(who, dopt_route_place_kernel, dim3(unsigned(a.tiles)), dim3(kSortThreads), smem, stream, a);
}

extern "C" int dopt_route_dispatch(const void *x, dopt_dtype dtype, int64_t tokens, int64_t cols,
                                   int64_t ld, const int32_t *slot_row, int32_t k, void *rows,
                                   int64_t n_rows, cudaStream_t stream) {
    dopt::clear_error();
    const char *who = "dopt_route_dispatch";
    OpRange range(who);
    int rc = check_slots(who, tokens, k);
    if (rc == DOPT_OK) rc = check_rows(who, dtype, n_rows, cols, ld);
    if (rc != DOPT_OK || tokens == 0 || n_rows == 0) return rc;
    const size_t b = elem_bytes(dtype);
    if ((rc = check_pointer(who, "x", x, b)) != DOPT_OK) return rc;
    if ((rc = check_pointer(who, "slot_row", slot_row, 4)) != DOPT_OK) return rc;
    if ((rc = check_pointer(who, "rows", rows, b)) != DOPT_OK) return rc;
    const int vb = access_bytes(address_bits(x) | address_bits(rows) | uint64_t(ld) * b |
                                uint64_t(cols) * b);
    RowArgs a{};
    a.x = x;
    a.out = rows;
    a.slot_row = slot_row;
    a.tokens = tokens;
    a.n_rows = n_rows;
    a.ld = ld * int64_t(b) / vb;
    a.vecs = int32_t(cols * int64_t(b) / vb);
    a.k = k;
    switch (vb) {
        case 16: return launch_dispatch<16, 2>(who, a, stream);
        case 8: return launch_dispatch<8, 4>(who, a, stream);
        case 4: return launch_dispatch<4, 8>(who, a, stream);
        default: return launch_dispatch<2, 8>(who, a, stream);
    }
}

extern "C" int dopt_route_combine(const void *rows, dopt_dtype dtype, int64_t n_rows,
                                  const int32_t *slot_row, const float *weights, int64_t tokens,
                                  int32_t k, int64_t cols, void *out, int64_t ld,
                                  cudaStream_t stream) {
    dopt::clear_error();
    const char *who = "dopt_route_combine";
    OpRange range(who);
    int rc = check_slots(who, tokens, k);
    if (rc == DOPT_OK) rc = check_rows(who, dtype, n_rows, cols, ld);
    if (rc != DOPT_OK || tokens == 0) return rc;
    const size_t b = elem_bytes(dtype);
    if (n_rows > 0 && (rc = check_pointer(who, "rows", rows, b)) != DOPT_OK) return rc;
    if ((rc = check_pointer(who, "slot_row", slot_row, 4)) != DOPT_OK) return rc;
    if (weights && (rc = check_pointer(who, "weights", weights, 4)) != DOPT_OK) return rc;
    if ((rc = check_pointer(who, "out", out, b)) != DOPT_OK) return rc;
    const int vb = access_bytes(address_bits(rows) | address_bits(out) | uint64_t(ld) * b |
                                uint64_t(cols) * b);
    RowArgs a{};
    a.x = rows;
    a.out = out;
    a.slot_row = slot_row;
    a.weights = weights;
    a.tokens = tokens;
    a.n_rows = n_rows;
    a.ld = ld * int64_t(b) / vb;
    a.vecs = int32_t(cols * int64_t(b) / vb);
    a.k = k;
    switch (dtype) {
        case DOPT_BF16: return pick_combine<__nv_bfloat16>(who, a, vb, stream);
        case DOPT_FP16: return pick_combine<__half>(who, a, vb, stream);
        default: return pick_combine<float>(who, a, vb, stream);
    }
}

extern "C" int dopt_route_combine_grad(const void *d_out, int64_t ld, const void *rows,
                                       dopt_dtype dtype, int64_t n_rows, const int32_t *slot_row,
                                       const float *weights, int64_t tokens, int32_t k,
                                       int64_t cols, void *d_rows, float *d_weights,
                                       cudaStream_t stream) {
    dopt::clear_error();
    const char *who = "dopt_route_combine_grad";
    OpRange range(who);
    int rc = check_slots(who, tokens, k);
    if (rc == DOPT_OK) rc = check_rows(who, dtype, n_rows, cols, ld);
    if (rc != DOPT_OK || tokens == 0) return rc;
    const size_t b = elem_bytes(dtype);
    if ((rc = check_pointer(who, "d_out", d_out, b)) != DOPT_OK) return rc;
    if (n_rows > 0) {
        if ((rc = check_pointer(who, "rows", rows, b)) != DOPT_OK) return rc;
        if ((rc = check_pointer(who, "d_rows", d_rows, b)) != DOPT_OK) return rc;
    }
    if ((rc = check_pointer(who, "slot_row", slot_row, 4)) != DOPT_OK) return rc;
    if ((rc = check_pointer(who, "weights", weights, 4)) != DOPT_OK) return rc;
    if ((rc = check_pointer(who, "d_weights", d_weights, 4)) != DOPT_OK) return rc;
    const int vb = access_bytes(address_bits(d_out) | address_bits(rows) | address_bits(d_rows) |
                                uint64_t(ld) * b | uint64_t(cols) * b);
    RowArgs a{};
    a.x = d_out;
    a.rows = rows;
    a.out = d_rows;
    a.slot_row = slot_row;
    a.weights = weights;
    a.d_weights = d_weights;
    a.tokens = tokens;
    a.n_rows = n_rows;
    a.ld = ld * int64_t(b) / vb;
    a.vecs = int32_t(cols * int64_t(b) / vb);
    a.k = k;
    switch (dtype) {
        case DOPT_BF16: return pick_combine_grad<__nv_bfloat16>(who, a, vb, stream);
        case DOPT_FP16: return pick_combine_grad<__half>(who, a, vb, stream);
        default: return pick_combine_grad<float>(who, a, vb, stream);
    }
}
