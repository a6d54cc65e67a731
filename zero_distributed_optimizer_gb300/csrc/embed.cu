// The token embedding (dopt_embed) and its gradient into the flat grad buffer
// (dopt_embed_grad); dopt.h states the contracts.
//
// The embedding is a copy: a warp takes 256 columns of four tokens, so that four
// rows' loads are in flight together.  16384 tokens of 768 bf16 columns whose ids
// name some 6000 rows, as text's do: 6.8 us, where the 34 MB of those rows and the
// output take 5.1 at the copy rate; what is left is the latency of ids and then
// rows, most of which come from L2, and instructions (half of the issue slots).
// Rows that are not 16-byte aligned go in shifted pieces (rows.cuh).
//
// The gradient sorts the tokens by row and sums each row's tokens in that order,
// so that it does not depend on which block runs when, and every row of the
// table is written once (or zeroed and then written).  Two launches: the sort,
// a block a residue class of rows, bound by latencies (8.7 us for 16384 tokens
// of 50257 rows), with zeros written beside it; and the sums, bound by the
// latency of a few dependent loads and, for frequent rows, of joining parts.
// 16384 tokens x 768 columns into 50257 rows, bf16: 27 us, of which the 77 MB of
// grads alone take 10; 1001 tokens x 515 columns into 5003 rows, fp32: 13.5 us.
#include <mutex>

#include "rows.cuh"

namespace {

constexpr int kEmbedThreads = 256;
constexpr int kWarps = kEmbedThreads / 32;
constexpr int kCols = 8;                 // columns a thread
constexpr int kWarpCols = 32 * kCols;    // columns a warp
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMostRange = 1024;         // rows of the table that one sorting block owns
constexpr int kListed = 128;             // of its own tokens that a sorting warp lists in shared memory
constexpr int kLeastShift = 7;           // at least 128 sorting blocks
constexpr int kMostShare = 32;           // sorted tokens that a warp sums
constexpr int kZeroRows = 4;             // rows of the table that a warp looks over for zeros
constexpr int kRingBytes = 4096;         // of a warp's loads ahead

struct EmbedArgs {
    const void *table;
    const void *ids;
    void *out;
    int64_t ld_table, ld_out;
    int64_t tokens, vocab;
    int32_t cols, wide;  // wide: 64-bit ids
    int32_t vec;         // the table's and the output's rows are 16-byte aligned
    int32_t accumulate;
    float scale;
};

template <typename I>
__device__ __forceinline__ int64_t id_at(const void *ids, int64_t t) {
    return int64_t(static_cast<const I *>(ids)[t]);
}

// out[t] = scale * table[id]: a warp takes 256 columns of four tokens, whose
// ids and then rows are loaded together.
template <typename T, typename I>
__global__ void __launch_bounds__(kEmbedThreads) dopt_embed_kernel(const __grid_constant__ EmbedArgs a) {
    let_dependents_start();
    wait_for_grids_before();
    constexpr int kTokens = 4;
    const int lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens;
    const int c0 = int(blockIdx.y) * kWarpCols, c = c0 + lane * kCols;
    int64_t id[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) id[i] = t0 + i < a.tokens ? id_at<I>(a.ids, t0 + i) : -1;
    using V = Values<T, kCols>;
    typename V::Ahead ahead[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const bool there = uint64_t(id[i]) < uint64_t(a.vocab);
        V::fetch(ahead[i], static_cast<const T *>(a.table) + (there ? id[i] * a.ld_table : 0), c, there ? a.cols : 0,
                 a.vec, lane, 32);
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        if (t0 + i >= a.tokens) break;
        const bool there = uint64_t(id[i]) < uint64_t(a.vocab);
        if (a.accumulate && !there) continue;  // nothing is added
        V v;
        v.take(ahead[i], a.vec, lane, 32);
        T *row = static_cast<T *>(a.out) + (t0 + i) * a.ld_out;
        if (there && (a.scale != 1.0f || a.accumulate)) {  // (zeros stay zeros whatever the scale is)
            float f[kCols], old[kCols] = {};
            v.get(f);
            if (a.accumulate) {
                V o;
                o.load(row, c, a.cols, a.vec, lane, 32);
                o.get(old);
            }
#pragma unroll
            for (int q = 0; q < kCols; ++q) f[q] = f[q] * a.scale + old[q];
            v.set(f);
        }
        v.store(row, c, a.cols, a.vec, lane, 32);
    }
}

// The same where rows are 16-byte aligned, of a multiple of 8 columns.
template <typename T, typename I>
__global__ void __launch_bounds__(kEmbedThreads) dopt_embed_whole_kernel(const __grid_constant__ EmbedArgs a) {
    let_dependents_start();
    wait_for_grids_before();
    constexpr int kTokens = 4, kPieces = kCols * int(sizeof(T)) / 16, kPer = 16 / int(sizeof(T));
    const int64_t t0 = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens;
    const int c = int(blockIdx.y) * kWarpCols + int(threadIdx.x & 31) * kCols;
    if (c >= a.cols) return;
    int64_t id[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) id[i] = t0 + i < a.tokens ? id_at<I>(a.ids, t0 + i) : -1;
    uint4 v[kTokens][kPieces];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const bool there = uint64_t(id[i]) < uint64_t(a.vocab);
        const uint4 *row = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.table) + id[i] * a.ld_table + c);
#pragma unroll
        for (int k = 0; k < kPieces; ++k) v[i][k] = there ? __ldg(row + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const bool there = uint64_t(id[i]) < uint64_t(a.vocab);
        if (t0 + i >= a.tokens || (a.accumulate && !there)) continue;
        uint4 *row = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + (t0 + i) * a.ld_out + c);
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            if (there && (a.scale != 1.0f || a.accumulate)) {
                float f[kPer], old[kPer] = {};
                unpack<T, 16>(v[i][k], f);
                if (a.accumulate) unpack<T, 16>(row[k], old);
#pragma unroll
                for (int q = 0; q < kPer; ++q) f[q] = f[q] * a.scale + old[q];
                v[i][k] = pack<T, 16>(f);
            }
            __stcs(row + k, v[i][k]);
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------

struct EmbedGradArgs {
    const void *ids;
    const void *d_out;
    void *grad;             // of the table's first element
    int32_t *first;         // [ranges * range + 1] the first sorted place of each row of the table, by key
    int32_t *token;         // [tokens] the tokens by row, in order within one
    int32_t *row;           // [tokens] their rows
    int2 *list;             // [tokens] (token, row in its range and more), by range
    int32_t *arrived;       // [chunks * pieces] parts of the run that goes on after a chunk
    float *partial;         // [2 * chunks][part_ld] sums of runs that reach over a chunk's ends
    int64_t ld, tokens, vocab, part_ld;
    int32_t cols, pieces;   // pieces: of 256 columns
    int32_t range, ranges, shift;  // ranges = 2^shift
    int64_t zeroed;                // rows that are zeroed beside the sort
    int32_t share, chunks;  // sorted tokens of a summing warp; blocks of 8 of those
    int32_t vec, vec_grad;  // d_out's, the grads' rows are 16-byte aligned
    int32_t accumulate;
    int32_t grad_bytes;     // of an element
    float scale;
};

// A row's place in the order of the sorted tokens: rows go to the sorting
// blocks in turn, so that frequent ids next to each other (a tokenizer's most
// frequent tokens often are) do not meet in one block.
__device__ __forceinline__ int64_t key_of(const EmbedGradArgs &a, int row) {
    return int64_t(row & (a.ranges - 1)) * a.range + (row >> a.shift);
}

// Exclusive sum over a block's warps of one number each; `total` of all.
__device__ __forceinline__ uint32_t over_warps(uint32_t mine, uint32_t *buffer, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) buffer[warp] = mine;
    __syncthreads();
    uint32_t v = buffer[lane], sum = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, sum, d);
        if (lane >= d) sum += u;
    }
    total = __shfl_sync(kFull, sum, 31);
    return __shfl_sync(kFull, sum - v, warp);
}

// Zeros to the bytes from p to `end` (whole elements of 2 bytes), by `threads`
// threads, of which this is number i: 16 bytes a store, the ends 2 at a time.
__device__ __forceinline__ void zero_bytes(char *p, char *end, int64_t i, int64_t threads) {
    char *from = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(p) + 15) & ~uintptr_t(15));
    char *to = reinterpret_cast<char *>(reinterpret_cast<uintptr_t>(end) & ~uintptr_t(15));
    if (from > to) from = to = end;  // (fewer than 16 bytes, between two boundaries)
    const int64_t n = (to - from) / 16;
    for (int64_t k = i; k < n; k += threads) reinterpret_cast<uint4 *>(from)[k] = make_uint4(0, 0, 0, 0);
    for (char *q = p + 2 * i; q < from; q += 2 * threads) *reinterpret_cast<uint16_t *>(q) = 0;
    for (char *q = to + 2 * i; q < end; q += 2 * threads) *reinterpret_cast<uint16_t *>(q) = 0;
}
__device__ __forceinline__ char *grad_row(const EmbedGradArgs &a, int64_t row) {
    return static_cast<char *>(a.grad) + row * a.cols * a.grad_bytes;
}

// The tokens sorted by the key of their row (stable).  A block owns `range`
// rows of the table.  It goes through all ids, so that it knows without any
// other block how many belong to those before it, lists those that are its own
// in order and sorts the list: counts of each (warp, row), their prefixes,
// places.  A lane's rank among its warp's tokens of one row comes from a ballot
// per bit of the row and is kept with the token for the second pass.  The sort is bound by
// latencies, so blocks that write zeros to the first rows of the table run
// beside it.
template <typename I>
__global__ void __launch_bounds__(kSortThreads, 2) dopt_embed_sort_kernel(const __grid_constant__ EmbedGradArgs a) {
    extern __shared__ uint32_t count[];  // [warps][range], then the warps' lists
    __shared__ uint32_t buffer[32];
    __shared__ uint32_t first[kMostRange];  // the rows' first places
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t before = (1u << lane) - 1;
    let_dependents_start();
    wait_for_grids_before();
    if (int(blockIdx.x) >= a.ranges) {
        zero_bytes(grad_row(a, 0), grad_row(a, a.zeroed), int64_t(blockIdx.x - a.ranges) * kSortThreads + threadIdx.x,
                   int64_t(gridDim.x - a.ranges) * kSortThreads);
        return;
    }
    const int block = int(blockIdx.x), mask = a.ranges - 1;
    for (int64_t i = int64_t(blockIdx.x) * kSortThreads + threadIdx.x; i < int64_t(a.chunks) * a.pieces;
         i += int64_t(a.ranges) * kSortThreads)
        a.arrived[i] = 0;
    for (int i = threadIdx.x; i < kSortWarps * a.range; i += kSortThreads) count[i] = 0;

    constexpr int kAhead = 4;
    int2 *const own_list = reinterpret_cast<int2 *>(count + kSortWarps * a.range + (a.range & 1) * kSortWarps) + warp * kListed;
    const int64_t stretch = ((a.tokens + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t from = min(a.tokens, warp * stretch), to = min(a.tokens, from + stretch);
    uint32_t own = 0, below = 0;
    for (int64_t i = from; i < to; i += 32 * kAhead) {
        int64_t id[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) id[j] = i + 32 * j + lane < to ? id_at<I>(a.ids, i + 32 * j + lane) : -1;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int of = uint64_t(id[j]) < uint64_t(a.vocab) ? int(id[j]) & mask : mask + 1;
            below += of < block;
            const uint32_t all = __ballot_sync(kFull, of == block);
            const uint32_t at = own + __popc(all & before);
            if (of == block && at < kListed) own_list[at] = make_int2(int(i + 32 * j + lane), int(id[j]) >> a.shift);
            own += __popc(all);
        }
    }
    below = __reduce_add_sync(kFull, below);
    uint32_t total, base;
    uint32_t place = over_warps(own, buffer, total);
    over_warps(below, buffer, base);
    // The warps' own lists where they hold all; otherwise one list in memory, of
    // which each warp then takes the same share.
    const bool in_memory = __syncthreads_or(own > kListed);
    if (in_memory && own > 0) {
        for (int64_t i = from; i < to; i += 32 * kAhead) {
            int64_t id[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) id[j] = i + 32 * j + lane < to ? id_at<I>(a.ids, i + 32 * j + lane) : -1;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const bool here = uint64_t(id[j]) < uint64_t(a.vocab) && (int(id[j]) & mask) == block;
                const uint32_t all = __ballot_sync(kFull, here);
                if (here)
                    a.list[base + place + __popc(all & before)] = make_int2(int(i + 32 * j + lane), int(id[j]) >> a.shift);
                place += __popc(all);
            }
        }
    }
    __syncthreads();
    uint32_t *mine = count + warp * a.range;
    const uint32_t share = ((total + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const uint32_t begin = in_memory ? min(total, warp * share) : 0, end = in_memory ? min(total, begin + share) : own;
    int2 *const list = in_memory ? a.list + base : own_list;
    const int bits = 32 - __clz(a.range - 1);
    int2 next = begin + lane < end ? list[begin + lane] : make_int2(0, 0);
    for (uint32_t i = begin; i < end; i += 32) {
        const bool there = i + lane < end;
        const int row = next.y;
        if (i + 32 < end) next = i + 32 + lane < end ? list[i + 32 + lane] : make_int2(0, 0);
        uint32_t peers = __ballot_sync(kFull, there);
        for (int k = 0; k < bits; ++k) {
            const uint32_t ones = __ballot_sync(kFull, row >> k & 1);
            peers &= row >> k & 1 ? ones : ~ones;
        }
        if (there) {
            const int rank = __popc(peers & before);
            if (rank == 0) mine[row] += __popc(peers);
            // the row, the rank, and for the first of them how many they are
            list[i + lane].y = row | rank << 16 | (rank == 0 ? __popc(peers) << 21 : 0);
        }
        __syncwarp();
    }
    __syncthreads();
    uint32_t of_row = 0;  // thread r: the tokens of row r
    if (int(threadIdx.x) < a.range && total > 0)
        for (int w = 0; w < kSortWarps; w += 8) {
            uint32_t *p = count + w * a.range + threadIdx.x, n[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) n[k] = p[k * a.range];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                p[k * a.range] = of_row;
                of_row += n[k];
            }
        }
    uint32_t upto = of_row;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, upto, d);
        if (lane >= d) upto += u;
    }
    uint32_t all;
    const uint32_t start = base + over_warps(__shfl_sync(kFull, upto, 31), buffer, all) + upto - of_row;
    if (int(threadIdx.x) < a.range) {
        a.first[int64_t(block) * a.range + threadIdx.x] = int(start);
        first[threadIdx.x] = start;
    }
    if (block == a.ranges - 1 && threadIdx.x == 0) a.first[int64_t(a.ranges) * a.range] = int(base + total);
    __syncthreads();
    next = begin + lane < end ? list[begin + lane] : make_int2(0, 0);
    for (uint32_t i = begin; i < end; i += 32) {
        const bool there = i + lane < end;
        const int2 e = next;
        if (i + 32 < end) next = i + 32 + lane < end ? list[i + 32 + lane] : make_int2(0, 0);
        const int row = e.y & 0xffff;
        const uint32_t at = there ? first[row] + mine[row] + (e.y >> 16 & 31) : 0;
        __syncwarp();
        if (there) {
            a.token[at] = e.x;
            a.row[at] = row << a.shift | block;
            if (const uint32_t of_chunk = uint32_t(e.y) >> 21) mine[row] += of_chunk;  // by the first of a row
        }
        __syncwarp();
    }
}

__device__ __forceinline__ void add_part(float (&f)[kCols], const float4 *part) {
    const float4 u = part[0], v = part[1];
    f[0] += u.x, f[1] += u.y, f[2] += u.z, f[3] += u.w;
    f[4] += v.x, f[5] += v.y, f[6] += v.z, f[7] += v.w;
}

// scale * f to a row of the grads.
template <typename G, bool WHOLE>
__device__ __forceinline__ void put_row(const EmbedGradArgs &a, int64_t row, int c, int lane, float (&f)[kCols]) {
    G *p = static_cast<G *>(a.grad) + row * a.cols;
    if constexpr (WHOLE) {
        constexpr int kPer = 16 / int(sizeof(G));
        if (c < a.cols)
#pragma unroll
            for (int k = 0; k < kCols / kPer; ++k) {
                uint4 *at = reinterpret_cast<uint4 *>(p + c) + k;
                float v[kPer];
#pragma unroll
                for (int q = 0; q < kPer; ++q) v[q] = f[k * kPer + q] * a.scale;
                if (a.accumulate) {
                    float old[kPer];
                    unpack<G, 16>(*at, old);
#pragma unroll
                    for (int q = 0; q < kPer; ++q) v[q] += old[q];
                }
                *at = pack<G, 16>(v);
            }
    } else {
        using V = Values<G, kCols>;
        float old[kCols] = {};
        if (a.accumulate) {
            V o;
            o.load(p, c, a.cols, a.vec_grad, lane, 32);
            o.get(old);
        }
#pragma unroll
        for (int q = 0; q < kCols; ++q) f[q] = f[q] * a.scale + old[q];
        V v;
        v.set(f);
        v.store(p, c, a.cols, a.vec_grad, lane, 32);
    }
}

// A block takes a chunk of sorted tokens and 256 columns, a warp an eighth of
// them, whose rows of d_out are loaded ahead whatever rows of the table they go
// to.  A row of no more tokens than a share is summed and written by the warp in
// whose share it begins, past the share's end too.  Longer ones are summed in parts: those
// of a chunk's warps meet in shared memory and are added in order by the warp in
// which the row begins (or the first); sums of a chunk's part are kept where the
// row reaches over chunks, and the block that brings the last one adds them in
// order.
template <typename T, typename G, bool WHOLE>
__global__ void __launch_bounds__(kEmbedThreads) dopt_embed_grad_kernel(const __grid_constant__ EmbedGradArgs a) {
    let_dependents_start();
    wait_for_grids_before();
    __shared__ float4 parts[kWarps][2][kWarpCols / 4];  // of a warp's first row, if it began before; of its last, if it goes on
    __shared__ __align__(16) unsigned char rings[WHOLE ? kWarps : 1][WHOLE ? kRingBytes : 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= unsigned(a.chunks) * unsigned(a.pieces)) {
        // zeros to the rows without tokens among those that the sort has left
        const int64_t row0 = a.zeroed + (int64_t(blockIdx.x - unsigned(a.chunks) * unsigned(a.pieces)) * kWarps + warp) * kZeroRows;
        bool empty = false;
        if (lane < kZeroRows && row0 + lane < a.vocab) {
            const int64_t key = key_of(a, int(row0 + lane));
            empty = a.first[key] == a.first[key + 1];
        }
        for (uint32_t rest = __ballot_sync(kFull, empty); rest; rest &= rest - 1) {
            const int64_t row = row0 + __ffs(rest) - 1;
            zero_bytes(grad_row(a, row), grad_row(a, row + 1), lane, 32);
        }
        return;
    }
    const int chunk = int(blockIdx.x / a.pieces), piece = int(blockIdx.x % a.pieces);
    const int c = piece * kWarpCols + lane * kCols;
    const int per_chunk = kWarps * a.share;
    const int base = chunk * per_chunk, p0 = base + warp * a.share;
    // lane i: the warp's tokens i and 32 + i, with what may follow its share
    // (loaded before it is known how many there are)
    int token[2], row[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int64_t p = int64_t(p0) + 32 * k + lane;
        token[k] = p < a.tokens ? a.token[p] : 0;
        row[k] = p < a.tokens ? a.row[p] : -1;
    }
    int row_before = p0 > 0 && p0 < a.tokens ? a.row[p0 - 1] : -1;
    const int total = a.first[int64_t(a.ranges) * a.range], n = min(a.share, total - p0);
    if (base >= total) return;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (p0 + 32 * k + lane >= total) token[k] = 0, row[k] = -1;
    if (n <= 0) row_before = -1;
    auto row_at = [&](int i) { return __shfl_sync(kFull, i < 32 ? row[0] : row[1], i & 31); };
    const int head_row = row_at(0), tail_row = row_at(max(n - 1, 0));
    const bool from_before = n > 0 && head_row == row_before, goes_on = n == a.share && row_at(n) == tail_row && tail_row >= 0;
    // the first and last rows' places, where they reach over the share's ends
    int2 head = make_int2(0, 0), tail = make_int2(0, 0);
    if (from_before) head = make_int2(a.first[key_of(a, head_row)], a.first[key_of(a, head_row) + 1]);
    if (goes_on) tail = make_int2(a.first[key_of(a, tail_row)], a.first[key_of(a, tail_row) + 1]);
    const bool head_part = head.y - head.x > a.share, tail_part = tail.y - tail.x > a.share;
    const int from = from_before && !head_part ? min(n, head.y - p0) : 0;          // (an earlier warp's before that)
    const int to = from < n && goes_on && !tail_part ? tail.y - p0 : max(n, 0);  // (less than a share past it)
    // the tokens after which another row begins
    const int after_lo = __shfl_down_sync(kFull, row[0], 1), after_hi = __shfl_down_sync(kFull, row[1], 1);
    const int middle = __shfl_sync(kFull, row[1], 0);
    const uint64_t ends = __ballot_sync(kFull, row[0] != (lane < 31 ? after_lo : middle)) |
                          uint64_t(__ballot_sync(kFull, row[1] != after_hi)) << 32 | (to > 0 ? uint64_t(1) << (to - 1) : 0);
    float f[kCols] = {};
    // token i's values are added; those of a row that ends there go where they belong
    auto add = [&](int i, const float(&g)[kCols]) {
#pragma unroll
        for (int q = 0; q < kCols; ++q) f[q] += g[q];
        if (!(ends >> i & 1)) return;
        const bool of_head = head_part && (ends & ((uint64_t(1) << i) - 1)) == 0, of_tail = tail_part && i == n - 1;
        if (of_head || of_tail) {
            float4 *const part = parts[warp][of_head ? 0 : 1] + lane * 2;
            part[0] = make_float4(f[0], f[1], f[2], f[3]), part[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            put_row<G, WHOLE>(a, row_at(i), c, lane, f);
        }
#pragma unroll
        for (int q = 0; q < kCols; ++q) f[q] = 0.0f;
    };
    if constexpr (WHOLE) {
        // rows of d_out on their way through shared memory, a thread's 8 columns its own
        constexpr int kBytes = kCols * int(sizeof(T)), kAhead = kRingBytes / (32 * kBytes);
        const uint32_t ring = uint32_t(__cvta_generic_to_shared(rings[warp] + lane * 16));
        auto fetch = [&](int i) {
            const int64_t t = __shfl_sync(kFull, i < 32 ? token[0] : token[1], i & 31);
            const char *at = reinterpret_cast<const char *>(static_cast<const T *>(a.d_out) + t * a.ld + c);
            if (i < to && c < a.cols)
#pragma unroll
                for (int k = 0; k < kBytes / 16; ++k)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     ring + uint32_t((i % kAhead) * 32 * kBytes + k * 512)),
                                 "l"(at + 16 * k)
                                 : "memory");
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int i = from; i < from + kAhead; ++i) fetch(i);
        for (int i = from; i < to; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            float g[kCols] = {};
            if (c < a.cols) {
                constexpr int kPer = 16 / int(sizeof(T));
#pragma unroll
                for (int k = 0; k < kBytes / 16; ++k) {
                    float part[kPer];
                    unpack<T, 16>(*reinterpret_cast<const uint4 *>(rings[warp] + lane * 16 + (i % kAhead) * 32 * kBytes + k * 512), part);
#pragma unroll
                    for (int q = 0; q < kPer; ++q) g[k * kPer + q] = part[q];
                }
            }
            add(i, g);
            fetch(i + kAhead);  // into the place that was just read
        }
    } else {
        using V = Values<T, kCols>;
        constexpr int kAhead = 4;
        for (int i = from; i < to; i += kAhead) {
            typename V::Ahead ahead[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int64_t t = __shfl_sync(kFull, i + j < 32 ? token[0] : token[1], (i + j) & 31);
                V::fetch(ahead[j], static_cast<const T *>(a.d_out) + (i + j < to ? t * a.ld : 0), c, i + j < to ? a.cols : 0,
                         a.vec, lane, 32);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (i + j >= to) break;
                V v;
                v.take(ahead[j], a.vec, lane, 32);
                float g[kCols];
                v.get(g);
                add(i + j, g);
            }
        }
    }
    __syncthreads();
    // The rows in parts: each by the warp in which it begins, or by the first warp
    // if that is in an earlier chunk.
    for (int which = 0; which < 2; ++which) {
        const bool through = head_part && head.x == tail.x;  // the share is all of one row, of earlier warps
        if (which == 0 ? !(warp == 0 && head_part) : !(tail_part && !through)) continue;
        const int of = which == 0 ? head_row : tail_row;
        const int lo = which == 0 ? head.x : tail.x, hi = which == 0 ? head.y : tail.y;
        const int last_warp = min(kWarps - 1, (hi - 1 - base) / a.share);
#pragma unroll
        for (int q = 0; q < kCols; ++q) f[q] = 0.0f;
        add_part(f, parts[warp][which] + lane * 2);
        for (int w = warp + 1; w <= last_warp; ++w) add_part(f, parts[w][0] + lane * 2);
        const int first_chunk = lo / per_chunk, last_chunk = (hi - 1) / per_chunk;
        if (first_chunk != last_chunk) {
            // a chunk's slot 0: the row that began before it; slot 1: the one that goes on after it
            auto slot = [&](int at) { return a.partial + (2 * int64_t(at) + (at == first_chunk)) * a.part_ld + c; };
            float4 *own = reinterpret_cast<float4 *>(slot(chunk));
            own[0] = make_float4(f[0], f[1], f[2], f[3]);
            own[1] = make_float4(f[4], f[5], f[6], f[7]);
            __threadfence();
            __syncwarp();
            int before = 0;
            if (lane == 0) before = atomicAdd(a.arrived + int64_t(first_chunk) * a.pieces + piece, 1);
            if (__shfl_sync(kFull, before, 0) != last_chunk - first_chunk) continue;
            __threadfence();
#pragma unroll
            for (int q = 0; q < kCols; ++q) f[q] = 0.0f;
#pragma unroll 4
            for (int at = first_chunk; at <= last_chunk; ++at) {
                const float4 *s = reinterpret_cast<const float4 *>(slot(at));
                const float4 part[2] = {__ldcg(s), __ldcg(s + 1)};
                add_part(f, part);
            }
        }
        put_row<G, WHOLE>(a, of, c, lane, f);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Sorted tokens that a warp sums: 32, and fewer where 48 warps an SM would not
// have so many.
int32_t share_of(int64_t tokens, int64_t pieces) {
    int32_t share = 2;
    while (share < kMostShare && tokens * pieces > int64_t(share) * 152 * 48) share *= 2;
    return share;
}

// Places of the gradient's tables in its workspace, with at most `share`
// sorted tokens a warp.
struct EmbedSpace {
    int64_t first, token, row, list, arrived, partial, bytes, chunks, pieces, part_ld;
    int32_t share, shift, range;
    EmbedSpace(int64_t tokens, int64_t vocab, int64_t cols) {
        pieces = (cols + kWarpCols - 1) / kWarpCols;
        part_ld = pieces * kWarpCols;
        share = share_of(tokens, pieces);
        chunks = (tokens + kWarps * share - 1) / (kWarps * share);
        for (shift = kLeastShift; (vocab + (int64_t(1) << shift) - 1) >> shift > kMostRange;) ++shift;
        range = int32_t((vocab + (int64_t(1) << shift) - 1) >> shift);
        first = 0;
        token = first + round_up(4 * ((int64_t(range) << shift) + 1), 16);
        row = token + round_up(4 * tokens, 16);
        list = row + round_up(4 * tokens, 16);
        arrived = list + round_up(8 * tokens, 16);
        partial = arrived + round_up(4 * chunks * pieces, 16);
        bytes = partial + 8 * chunks * part_ld;
    }
};
// Bytes for so many tokens and for any fewer: there the chunks may be shorter
// and so, up to the number that the shortest come to, more.
int64_t most_space(int64_t tokens, int64_t vocab, int64_t cols) {
    const EmbedSpace s(tokens, vocab, cols);
    const int64_t most = std::max(s.chunks, std::min((tokens + 2 * kWarps - 1) / (2 * kWarps),
                                                     (152 * 48 + s.pieces * kWarps - 1) / (s.pieces * kWarps) + 1));
    return s.arrived + round_up(4 * most * s.pieces, 16) + 8 * most * s.part_ld;
}

// Bytes of the sorting kernels' shared memory: counts, and the warps' lists from
// an 8-byte boundary on.
constexpr size_t sort_smem(int range) {
    return size_t(kSortWarps) * (range + (range & 1)) * sizeof(uint32_t) + size_t(kSortWarps) * kListed * sizeof(int2);
}

std::mutex g_embed_mutex;
bool g_embed_ready[64] = {};  // devices whose sorting kernels are set up

// Raises the sorting kernels' shared-memory limit, once a device.
int set_up_sort(const char *who) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess && (device < 0 || device >= 64)) return dopt::fail(DOPT_E_ARG, "%s: device %d", who, device);
    std::lock_guard<std::mutex> lock(g_embed_mutex);
    if (e == cudaSuccess && !g_embed_ready[device]) {
        constexpr int kMost = int(sort_smem(kMostRange));
        e = cudaFuncSetAttribute(dopt_embed_sort_kernel<int32_t>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(dopt_embed_sort_kernel<int64_t>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        g_embed_ready[device] = e == cudaSuccess;
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return dopt::fail(DOPT_E_CUDA, "%s: shared-memory limit: %s", who, cudaGetErrorString(e));
    }
    return DOPT_OK;
}

int check_ids(const char *who, const void *ids, int32_t id_bytes, int64_t tokens, int64_t vocab, int64_t cols) {
    using dopt::fail;
    if (id_bytes != 4 && id_bytes != 8) return fail(DOPT_E_ARG, "%s: id_bytes %d (4 or 8)", who, id_bytes);
    if (tokens < 0 || tokens > DOPT_EMBED_MAX_TOKENS || vocab < 1 || vocab > INT32_MAX || cols < 1 || cols > DOPT_MAX_COLS)
        return fail(DOPT_E_ARG, "%s: tokens %lld, vocab %lld, cols %lld", who, static_cast<long long>(tokens),
                    static_cast<long long>(vocab), static_cast<long long>(cols));
    if (tokens > 0 && !ids) return fail(DOPT_E_ARG, "%s: ids is NULL", who);
    if (!aligned_to(ids, size_t(id_bytes))) return fail(DOPT_E_ALIGN, "%s: ids is not aligned to its elements", who);
    return DOPT_OK;
}

template <typename T>
int launch_embed(const char *who, const EmbedArgs &a, cudaStream_t stream) {
    const dim3 grid(unsigned((a.tokens + 4 * kWarps - 1) / (4 * kWarps)), unsigned((a.cols + kWarpCols - 1) / kWarpCols));
    if (a.vec && a.cols % kCols == 0)
        return a.wide ? launch_op(who, dopt_embed_whole_kernel<T, int64_t>, grid, dim3(kEmbedThreads), 0, stream, a)
                      : launch_op(who, dopt_embed_whole_kernel<T, int32_t>, grid, dim3(kEmbedThreads), 0, stream, a);
    return a.wide ? launch_op(who, dopt_embed_kernel<T, int64_t>, grid, dim3(kEmbedThreads), 0, stream, a)
                  : launch_op(who, dopt_embed_kernel<T, int32_t>, grid, dim3(kEmbedThreads), 0, stream, a);
}

template <typename T, typename G>
int launch_grad(const char *who, const EmbedGradArgs &a, cudaStream_t stream) {
    const int64_t left = a.accumulate ? 0 : a.vocab - a.zeroed;
    const dim3 grid(unsigned(a.chunks) * unsigned(a.pieces) + unsigned((left + kZeroRows * kWarps - 1) / (kZeroRows * kWarps)));
    return a.vec && a.vec_grad && a.cols % kCols == 0
               ? launch_op(who, dopt_embed_grad_kernel<T, G, true>, grid, dim3(kEmbedThreads), 0, stream, a)
               : launch_op(who, dopt_embed_grad_kernel<T, G, false>, grid, dim3(kEmbedThreads), 0, stream, a);
}
template <typename T>
int launch_grad(const char *who, dopt_dtype grad, const EmbedGradArgs &a, cudaStream_t stream) {
    switch (grad) {
        case DOPT_BF16: return launch_grad<T, __nv_bfloat16>(who, a, stream);
        case DOPT_FP16: return launch_grad<T, __half>(who, a, stream);
        default: return launch_grad<T, float>(who, a, stream);
    }
}

}  // namespace

extern "C" int dopt_embed(const void *table, dopt_dtype dtype, int64_t vocab, int64_t cols, int64_t ld_table,
                          const void *ids, int32_t id_bytes, int64_t tokens, float scale, void *out, int64_t ld_out,
                          uint32_t flags, cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_embed";
    OpRange range(who);
    int rc = check_ids(who, ids, id_bytes, tokens, vocab, cols);
    if (rc != DOPT_OK) return rc;
    if (!valid_dtype(dtype)) return fail(DOPT_E_ARG, "%s: unknown dtype %d", who, int(dtype));
    if (ld_table < cols || ld_out < cols)
        return fail(DOPT_E_ARG, "%s: row strides %lld, %lld for %lld columns", who, static_cast<long long>(ld_table),
                    static_cast<long long>(ld_out), static_cast<long long>(cols));
    if (flags & ~uint32_t(DOPT_EMBED_ACCUMULATE)) return fail(DOPT_E_ARG, "%s: unknown flags 0x%x", who, flags);
    if (tokens > 0 && (!table || !out)) return fail(DOPT_E_ARG, "%s: NULL table or out", who);
    const size_t b = elem_bytes(dtype);
    if (!aligned_to(table, b) || !aligned_to(out, b))
        return fail(DOPT_E_ALIGN, "%s: table or out is not aligned to its elements", who);
    if (tokens == 0) return DOPT_OK;
    EmbedArgs a{};
    a.table = table;
    a.ids = ids;
    a.out = out;
    a.ld_table = ld_table;
    a.ld_out = ld_out;
    a.tokens = tokens;
    a.vocab = vocab;
    a.cols = int32_t(cols);
    a.wide = id_bytes == 8;
    a.vec = (address_bits(table) | address_bits(out) | uint64_t(ld_table) * b | uint64_t(ld_out) * b) % 16 == 0;
    a.accumulate = (flags & DOPT_EMBED_ACCUMULATE) != 0;
    a.scale = scale;
    switch (dtype) {
        case DOPT_BF16: return launch_embed<__nv_bfloat16>(who, a, stream);
        case DOPT_FP16: return launch_embed<__half>(who, a, stream);
        default: return launch_embed<float>(who, a, stream);
    }
}

extern "C" int dopt_embed_workspace(int64_t tokens, int64_t vocab, int64_t cols, int64_t *bytes) {
    dopt::clear_error();
    const char *who = "dopt_embed_workspace";
    if (!bytes) return dopt::fail(DOPT_E_ARG, "%s: bytes is NULL", who);
    if (tokens < 0 || tokens > DOPT_EMBED_MAX_TOKENS || vocab < 1 || vocab > INT32_MAX || cols < 1 || cols > DOPT_MAX_COLS)
        return dopt::fail(DOPT_E_ARG, "%s: tokens %lld, vocab %lld, cols %lld", who, static_cast<long long>(tokens),
                          static_cast<long long>(vocab), static_cast<long long>(cols));
    *bytes = most_space(tokens, vocab, cols);
    return DOPT_OK;
}

extern "C" int dopt_embed_grad(const void *ids, int32_t id_bytes, int64_t tokens, const void *d_out, dopt_dtype dtype,
                               int64_t cols, int64_t ld, int64_t vocab, float scale, void *grad, dopt_dtype grad_dtype,
                               int64_t grad_numel, int64_t grad_offset, uint32_t flags, void *workspace,
                               int64_t workspace_bytes, cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_embed_grad";
    OpRange range(who);
    int rc = check_ids(who, ids, id_bytes, tokens, vocab, cols);
    if (rc != DOPT_OK) return rc;
    if (!valid_dtype(dtype) || !valid_dtype(grad_dtype)) return fail(DOPT_E_ARG, "%s: unknown dtype", who);
    if (ld < cols)
        return fail(DOPT_E_ARG, "%s: row stride %lld for %lld columns", who, static_cast<long long>(ld),
                    static_cast<long long>(cols));
    if (flags & ~uint32_t(DOPT_EMBED_ACCUMULATE)) return fail(DOPT_E_ARG, "%s: unknown flags 0x%x", who, flags);
    if (!grad || (tokens > 0 && !d_out)) return fail(DOPT_E_ARG, "%s: NULL grad or d_out", who);
    if (grad_offset < 0 || grad_offset > grad_numel - vocab * cols)
        return fail(DOPT_E_ARG, "%s: %lld x %lld grads at %lld leave a buffer of %lld", who,
                    static_cast<long long>(vocab), static_cast<long long>(cols), static_cast<long long>(grad_offset),
                    static_cast<long long>(grad_numel));
    const size_t b = elem_bytes(dtype), gb = elem_bytes(grad_dtype);
    if (!aligned_to(d_out, b) || !aligned_to(grad, gb))
        return fail(DOPT_E_ALIGN, "%s: d_out or grad is not aligned to its elements", who);
    const EmbedSpace space(tokens, vocab, cols);
    if (!workspace || workspace_bytes < space.bytes)
        return fail(DOPT_E_ARG, "%s: workspace of %lld bytes, %lld are needed", who,
                    static_cast<long long>(workspace ? workspace_bytes : 0), static_cast<long long>(space.bytes));
    if (!aligned_to(workspace, 16)) return fail(DOPT_E_ALIGN, "%s: workspace is not 16-byte aligned", who);
    char *ws = static_cast<char *>(workspace);
    EmbedGradArgs a{};
    a.ids = ids;
    a.d_out = d_out;
    a.grad = static_cast<char *>(grad) + grad_offset * int64_t(gb);
    a.first = reinterpret_cast<int32_t *>(ws + space.first);
    a.token = reinterpret_cast<int32_t *>(ws + space.token);
    a.row = reinterpret_cast<int32_t *>(ws + space.row);
    a.list = reinterpret_cast<int2 *>(ws + space.list);
    a.arrived = reinterpret_cast<int32_t *>(ws + space.arrived);
    a.partial = reinterpret_cast<float *>(ws + space.partial);
    a.ld = ld;
    a.tokens = tokens;
    a.vocab = vocab;
    a.part_ld = space.part_ld;
    a.cols = int32_t(cols);
    a.pieces = int32_t(space.pieces);
    a.chunks = int32_t(space.chunks);
    a.share = space.share;
    a.vec = (address_bits(d_out) | uint64_t(ld) * b) % 16 == 0;
    a.vec_grad = (address_bits(a.grad) | uint64_t(cols) * gb) % 16 == 0;
    a.accumulate = (flags & DOPT_EMBED_ACCUMULATE) != 0;
    a.scale = scale;
    a.range = space.range;
    a.shift = space.shift;
    a.ranges = 1 << space.shift;
    const size_t smem = sort_smem(a.range);
    a.grad_bytes = int32_t(gb);
    if (int64_t(a.chunks) * a.pieces + vocab / (kZeroRows * kWarps) + 1 > INT32_MAX)
        return fail(DOPT_E_ARG, "%s: %lld tokens of %lld columns are too many for one call", who,
                    static_cast<long long>(tokens), static_cast<long long>(cols));
    if ((rc = set_up_sort(who)) != DOPT_OK) return rc;
    auto sort = id_bytes == 8 ? dopt_embed_sort_kernel<int64_t> : dopt_embed_sort_kernel<int32_t>;
    // Zeros are written beside the sort (64 KB a block, up to two blocks an SM),
    // which is bound by latencies, and a quarter of them after the sums' blocks,
    // for the same reason.  All beside the sort, three quarters, half, in a loop:
    // 16384 x 768 into 50257 rows bf16 28.4, 26.1, 27.1 us, fp32 42.2, 39.4, 38.0;
    // 8192 x 2048 into 32000 bf16 37.3, 38.0, 33.4; 16384 x 4096 into 32000 bf16
    // 87, 83, 79; 4096 x 1024 into 8192 and smaller ones no difference.
    a.zeroed = a.accumulate ? 0 : tokens > 0 ? vocab - vocab / 4 : vocab;
    const int64_t zero_blocks = std::min<int64_t>(304, (a.zeroed * cols * int64_t(gb) + 65535) / 65536);
    rc = launch_op(who, sort, dim3(unsigned(a.ranges + zero_blocks)), dim3(kSortThreads), smem, stream, a);
    if (rc != DOPT_OK || tokens == 0) return rc;
    switch (dtype) {
        case DOPT_BF16: return launch_grad<__nv_bfloat16>(who, grad_dtype, a, stream);
        case DOPT_FP16: return launch_grad<__half>(who, grad_dtype, a, stream);
        default: return launch_grad<float>(who, grad_dtype, a, stream);
    }
}
