// The cross entropy of a language model's output matrix (dopt_head_loss) and
// its gradients (dopt_head_loss_grad) without the logits; dopt.h states the
// contracts.
#include <mutex>
#include <type_traits>

#include "f32x2.cuh"
#include "pairs.cuh"
#include "rows.cuh"

namespace {

// All products are tcgen05.mma.cta_group::2 of a pair of CTAs (a cluster of
// two, one CTA an SM): M = 256, N = 256, K in steps of 64, operands by TMA with
// the 128-byte swizzle, each CTA 128 of the M and half of the N.
//
//   logits     M = tokens, N = the vocabulary, K = the width; both operands with
//              K contiguous.  A lane of tensor memory is a token, so a thread
//              goes through its token's logits alone: their maximum and sum of
//              exponentials, or their gradients in 16 bits.
//   d_x, d_w   M = the width, N = tokens or the vocabulary, K the other one.
//              Lanes lie along the width, which is contiguous in both results,
//              so a warp's stores are contiguous whatever the alignment.
//
// Long products are bound by the tensor cores (active 96-98 % of the cycles) and
// then by the card's power: 16384 tokens x 768 x 50257, bf16, loss 618-647 us in
// short runs (1.96-2.05 PFLOP/s), 706-728 under the power cap (1.74-1.79);
// gradients 2070-2180 and 2350-2450 us (1.83 and 1.55-1.62 PFLOP/s).  The logits'
// gradients are stored as they are made, 1.6 GB, which keeps the tensor cores at
// 83 % there; in pieces that stay in L2 d_x's fp32 sums would move more.  Few
// tokens: 24 x 2048 x 32000, loss 32 us (19 at the copy rate), 20 for the
// matrix, 7 of two launches, 4 until the first steps are there; its 125 tiles are
// two waves on 76 pairs, the second of 49.
constexpr int kM = 256, kN = 256, kK = 64;  // of a pair's tile, and of a step
constexpr int kSlab = 64 * 128;             // 64 rows of 128 bytes
constexpr int kOperand = 2 * kSlab;         // a CTA's share of one operand in a step
constexpr int kStage = 2 * kOperand;
constexpr int kTmemCols = 512;
constexpr int kMostSplit = 16, kMostSlots = 304;

constexpr int kLogitWarps = 8;  // that go through logits
constexpr int kLogitThreads = 32 * (kLogitWarps + 2);
// What a logit kernel keeps: nothing of the logits (the loss), or their
// gradients in one or two parts of 16 bits, a buffer of 4 KB a part and warp.
__host__ __device__ constexpr int logit_ring(int planes) { return planes == 2 ? 5 : 6; }
constexpr int kOutBuffer = 32 * 128;  // 32 tokens x 64 logits of 16 bits
constexpr int kStoreWarps = 8;  // two to 32 lanes, half of the columns each
constexpr int kProductThreads = 32 * (kStoreWarps + 2);
constexpr int kProductRing = 6;

struct HeadBarriers {
    unsigned long long full[6], empty[6];
    unsigned long long sum_full[2], sum_empty[2];
    uint32_t tmem;
    int32_t failed;
};
__host__ __device__ constexpr size_t logit_smem(int planes) {
    return logit_ring(planes) * size_t(kStage) + planes * kLogitWarps * size_t(kOutBuffer) + sizeof(HeadBarriers);
}
constexpr size_t kProductSmem = kProductRing * size_t(kStage) + sizeof(HeadBarriers);
static_assert(logit_smem(1) <= 232448 && logit_smem(2) <= 232448 && kProductSmem <= 232448, "a CTA's 227 KB");

// CTAs with a wait that ran past its limit (a copy or product that never
// completed).  Such a pair ends its work; what it has not written becomes NaN.
__device__ unsigned int g_head_timeouts;
constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s
constexpr uint32_t kNanBits = 0x7fffffffu;

#ifdef DOPT_DEVICE_CHECKS
// Test build only: the first pair of each launch issues the products of so many
// of its items (-1: of all), so that the waits for the next one's run out
// (dopt_head_wait_test).
__device__ int g_head_items = -1;
__device__ __forceinline__ bool products_withheld(int round) {
    return blockIdx.x == 0 && g_head_items >= 0 && round >= g_head_items;
}
#else
__device__ __forceinline__ bool products_withheld(int) { return false; }
#endif

// Wait for a phase of a barrier that threads of the cluster arrive on; false
// once any wait of this CTA has run out of time.  Both CTAs of a pair arrive
// on the leader's barriers and products of both read and write either one's
// memory, so arrivals release and waits acquire at the cluster's scope (an
// instruction without a scope orders the memory of its own CTA's threads only).
__device__ __forceinline__ bool try_phase(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
template <int SLEEP_NS>
__device__ __noinline__ bool wait_long(HeadBarriers &b, uint32_t bar, uint32_t parity) {
    unsigned long long t0, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (;;) {
        for (int i = 0; i < 64; ++i) {
            if (try_phase(bar, parity)) return true;
            if (SLEEP_NS > 0) __nanosleep(SLEEP_NS);
        }
        if (*static_cast<volatile int32_t *>(&b.failed)) return false;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (now - t0 > kWaitNs) {
            if (atomicExch(&b.failed, 1) == 0) atomicAdd(&g_head_timeouts, 1u);
            return false;
        }
    }
}
// (by a whole warp)
template <int SLEEP_NS = 0>
__device__ __forceinline__ bool wait_phase(HeadBarriers &b, unsigned long long &bar, uint32_t parity) {
    const uint32_t at = smem_of(&bar);
    bool ok = false;
    for (int i = 0; i < (SLEEP_NS > 0 ? 1 : 16) && !ok; ++i) ok = try_phase(at, parity);
    if (!ok) ok = wait_long<SLEEP_NS>(b, at, parity);
    return __all_sync(kFull, ok);
}

// An arrival on the leader's barrier once a warp has read its sums: what it
// waited for are loads from tensor memory, ordered by the fence before.
__device__ __forceinline__ void release_sums(HeadBarriers &b, int buffer, int lane) {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    if (lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         leader_address(smem_of(&b.sum_empty[buffer])))
                     : "memory");
}

// Descriptors of an operand in shared memory, 128-byte swizzle, 1024 bytes
// from 8 rows to the next 8.  K contiguous: 128 rows of 64 k; 16 k on are 32
// bytes on.  M or N contiguous: two slabs of 64 columns x 64 rows of k; 16 k on
// are 2048 bytes on.
constexpr uint64_t kRows8 = uint64_t(1024 >> 4) << 32, kSwizzle = (uint64_t(1) << 46) | (uint64_t(2) << 61);
__device__ __forceinline__ uint64_t k_descriptor(uint32_t address) {
    return (uint64_t(address & 0x3ffff) >> 4) | (uint64_t(1) << 16) | kRows8 | kSwizzle;
}
__device__ __forceinline__ uint64_t mn_descriptor(uint32_t address) {
    return (uint64_t(address & 0x3ffff) >> 4) | (uint64_t(kSlab >> 4) << 16) | kRows8 | kSwizzle;
}
template <typename T>
__host__ __device__ constexpr uint32_t instruction(bool a_mn, bool b_mn) {
    const uint32_t format = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    return (1u << 4) | (format << 7) | (format << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
           (uint32_t(kN >> 3) << 17) | (uint32_t(kM >> 4) << 24);
}

__device__ __forceinline__ void load_box(uint32_t to, const CUtensorMap *map, int x, int y, uint32_t barrier) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(to),
        "l"(map), "r"(x), "r"(y), "r"(barrier)
        : "memory");
}
// Written once and read once or twice much later: the first to leave L2, where
// the operands of the products stay (gradients of 16384 x 768 x 50257 2280 ->
// 2222 us).
__device__ __forceinline__ void store_box(const CUtensorMap *map, int x, int y, uint32_t from) {
    asm volatile(
        "{\n\t.reg .b64 policy;\n\t"
        "createpolicy.fractional.L2::evict_first.b64 policy, 1.0;\n\t"
        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%1, %2}], [%3], policy;\n\t}" ::"l"(map),
        "r"(x), "r"(y), "r"(from)
        : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t barrier, int bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(barrier), "r"(bytes) : "memory");
}
// To both CTAs' barriers, once the products issued so far are done.
__device__ __forceinline__ void commit(unsigned long long &bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_of(&bar)),
        "h"(uint16_t(3))
        : "memory");
}
__device__ __forceinline__ void product(uint32_t sums, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(sums),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
        : "memory");
}

// The start and the end of a pair's kernel.
__device__ __forceinline__ uint32_t pair_begin(HeadBarriers &b, int ring, int sum_readers, bool allocates) {
    let_dependents_start();
    if (threadIdx.x == 0) {
        auto init = [](unsigned long long &bar, int count) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(&bar)), "r"(count) : "memory");
        };
        for (int i = 0; i < ring; ++i) init(b.full[i], 1), init(b.empty[i], 1);
        for (int i = 0; i < 2; ++i) init(b.sum_full[i], 1), init(b.sum_empty[i], 2 * sum_readers);
        b.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (allocates) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&b.tmem)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    wait_for_grids_before();
    return b.tmem;
}
__device__ __forceinline__ void pair_end(HeadBarriers &b, uint32_t tmem, bool allocated) {
    __syncthreads();
    if (b.failed && threadIdx.x == 0) {  // copies still in flight get as long again
        unsigned long long t0, now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        do {
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        } while (now - t0 < kWaitNs);
    }
    __syncwarp();
    cluster_sync();  // the peer's barriers and operands stay until both are done
    if (allocated) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
    }
}
// Wait for the last of `uses` uses of each slot of the ring.
__device__ __forceinline__ void drain(HeadBarriers &b, int ring, int uses) {
    for (int s = 0; s < ring && s < uses; ++s)
        if (!wait_phase(b, b.empty[s], uint32_t((uses - 1 - s) / ring) & 1)) return;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    return rank;
}

// ---------------------------------------------------------------------------
// Logits
// ---------------------------------------------------------------------------

// Types whose range is so short that rows of d_x may need factors of their own.
template <typename T>
constexpr bool kHasRows = std::is_same<T, __half>::value;

struct LogitArgs {
    CUtensorMap x_map, w_map;
    CUtensorMap d_map[2];       // gradients: their 16 bits, and what those leave (fp32 grads)
    const void *targets;
    const float *lse, *d_loss, *d_lse;
    const float *factor;        // gradients: what they are multiplied by, what takes it back, and if rows have their own
    const float *row_back;      // gradients for d_x: what takes each row's own back, or NULL
    float2 *partial;            // loss: [2 * tiles_n][rows] (reference, sum), powers of two
    float *at_target;           // loss: [rows] the target's logit
    int64_t first, vocab;       // this launch's first column of the vocabulary; all of them
    int32_t rows, cols;         // tokens, columns of this launch
    int32_t steps, chunk, tiles_m, tiles_n, items;  // chunk: steps of one sum
    int32_t group;              // blocks of tokens that go through the vocabulary together
    int32_t x_ctas, step_bytes; // CTAs of a pair that have tokens; bytes of a pair's step
    int32_t wide;
    int32_t for_rows;           // 1: nothing is done unless rows have their own factors
};

struct Tile {
    int m0, n0;
};
// Items go through `group` blocks of 256 tokens for one block of the
// vocabulary before the next: the pairs at work share both operands in L2.
__device__ __forceinline__ Tile tile_of(const LogitArgs &a, int item) {
    const int per_group = a.group * a.tiles_n, g = item / per_group;
    const int left = item - g * per_group, blocks = min(a.group, a.tiles_m - g * a.group);
    const int n = left / blocks;
    return {(g * a.group + left - n * blocks) * kM, n * kN};
}

__device__ __forceinline__ int64_t target_of(const LogitArgs &a, int row) {
    return (a.wide ? static_cast<const int64_t *>(a.targets)[row] : int64_t(static_cast<const int32_t *>(a.targets)[row])) - a.first;
}

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504088896340736f;

// A token's part of a tile: (c, s) with sum of exp(logit) = exp(c) * s, c the
// largest logit so far, taken as it is (a rounded product of it would be off by
// more than exponents reach where logits are in the billions: masked ones) and
// into fp32's finite range, so that no two infinities are ever subtracted: logits
// of -inf add exp2(-inf) = 0, those of +inf make s infinite, NaN makes it NaN.
// Differences go two an instruction: the loss of 16384 x 768 x 50257 takes 673 us
// in a loop so, 683 one at a time, 670 with a product that is taken off fused.
constexpr float kLargest = 3.402823466e38f;
struct Running {
    float c = -kLargest, s = 0.0f;
    __device__ __forceinline__ void add(const float (&l)[32], int there) {
        float top[4] = {-kLargest, -kLargest, -kLargest, -kLargest};
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < there) top[j & 3] = fmaxf(top[j & 3], l[j]);
        const float reach = fminf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), kLargest);
        if (reach > c) {
            s *= exp2_of((c - reach) * kLog2e);
            c = reach;
        }
        float sum[4] = {};
        const F2 less(-c), by(kLog2e);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            float x, y;
            ((F2(l[j], l[j + 1]) + less) * by).get(x, y);
            if (j < there) sum[j & 3] += exp2_of(x);
            if (j + 1 < there) sum[(j + 1) & 3] += exp2_of(y);
        }
        s += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return uint32_t(__builtin_bit_cast(uint16_t, from_f32<T>(a))) | uint32_t(__builtin_bit_cast(uint16_t, from_f32<T>(b))) << 16;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// What 16 bits leave of a value.
template <typename T>
__device__ __forceinline__ float rest_of(float f) {
    return f - to_f32(from_f32<T>(f));
}

// PLANES: 0, the loss; 1 or 2, the parts of the logits' gradients.
template <typename T, int PLANES>
__global__ void __launch_bounds__(kLogitThreads, 1) __cluster_dims__(2, 1, 1)
    dopt_head_logit_kernel(const __grid_constant__ LogitArgs a) {
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr bool GRAD = PLANES > 0;
    constexpr int kRing = logit_ring(PLANES);
    constexpr int kMmaWarp = kLogitWarps, kLoadWarp = kLogitWarps + 1;
    if (GRAD && kHasRows<T> && a.for_rows) {
        wait_for_grids_before();
        if (a.factor[2] == 0.0f) return;
    }
    unsigned char *out_buffers = smem + kRing * kStage;
    HeadBarriers &b = *reinterpret_cast<HeadBarriers *>(out_buffers + PLANES * kLogitWarps * kOutBuffer);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pairs = int(gridDim.x >> 1), pair = int(blockIdx.x >> 1);
    const uint32_t tmem = pair_begin(b, kRing, kLogitWarps, warp == kMmaWarp);

    if (warp == kLoadWarp) {
        int n = 0;
        bool ok = true;
        for (int item = pair; ok && item < a.items; item += pairs) {
            const Tile t = tile_of(a, item);
            for (int i = 0; i < a.steps; ++i, ++n) {
                const int s = n % kRing;
                if (n >= kRing) ok = wait_phase<64>(b, b.empty[s], uint32_t(n / kRing - 1) & 1);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t full = smem_of(&b.full[s]), to = smem_of(smem + s * kStage);
                    if (rank == 0) expect_bytes(full, a.step_bytes);
                    if (int(rank) < a.x_ctas)
                        load_box(to, &a.x_map, i * kK, t.m0 + int(rank) * (kM / 2), leader_address(full));
                    load_box(to + kOperand, &a.w_map, i * kK, t.n0 + int(rank) * (kN / 2), leader_address(full));
                }
                __syncwarp();
            }
        }
        if (ok) drain(b, kRing, n);
    } else if (warp == kMmaWarp) {
        if (rank == 0) {
            constexpr uint32_t kIdesc = instruction<T>(false, false);
            const uint32_t base = uniform(tmem);
            const uint64_t first = k_descriptor(smem_of(smem));
            int n = 0, t = 0;
            bool ok = true;
            for (int item = pair, round = 0; ok && item < a.items; item += pairs, ++round) {
                if (products_withheld(round)) break;
                int left = 0, buffer = 0;  // steps left of the sum
                for (int i = 0; i < a.steps && ok; ++i, ++n, --left) {
                    const bool fresh = left == 0;
                    if (fresh) {
                        buffer = t & 1;
                        if (t >= 2) ok = wait_phase(b, b.sum_empty[buffer], uint32_t(t / 2 - 1) & 1);
                        ++t;
                        left = min(a.chunk, a.steps - i);
                        if (!ok) break;
                    }
                    const int s = n % kRing;
                    ok = wait_phase(b, b.full[s], uint32_t(n / kRing) & 1);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t sums = base + uint32_t(buffer * kN);
                    const uint64_t da = first + uint64_t(s * (kStage >> 4)), db = da + (kOperand >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) product(sums, da + 2 * k, db + 2 * k, kIdesc, !fresh || k > 0);
                        commit(b.empty[s]);
                        if (left == 1) commit(b.sum_full[buffer]);
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // warp w: tokens 32 (w % 4) on, 128 columns from 128 (w / 4) on
        const int half = warp >> 2;
        const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16) + uint32_t(half * 128);
        unsigned char *out = out_buffers + warp * PLANES * kOutBuffer;
        int t = 0;
        bool ok = true;
        for (int item = pair; item < a.items; item += pairs) {
            const Tile tile = tile_of(a, item);
            const int row0 = tile.m0 + int(rank) * (kM / 2) + (warp & 3) * 32, row = row0 + lane;
            const int c0 = tile.n0 + half * 128, there = a.cols - c0;
            const bool mine = row < a.rows;
            const int64_t target = mine ? target_of(a, row) : -1;
            float by_p = 0.0f, by_target = 0.0f, lse = 0.0f;
            if (GRAD && mine) {
                // (a target outside the vocabulary: of the launch that holds it, or of none)
                const int64_t whole = target + a.first;
                by_target = whole >= 0 && whole < a.vocab ? a.d_loss[row] : 0.0f;
                by_p = by_target + (a.d_lse ? a.d_lse[row] : 0.0f);
                lse = a.lse[row];
                const float factor = kHasRows<T> && a.row_back && a.factor[2] != 0.0f ? 1.0f / a.row_back[row] : a.factor[0];
                by_p *= factor, by_target *= factor;
            }
            // the logits of 128 columns: their sums' parts, added as they come
            float all[4][32];
            for (int i = 0; i < a.steps; i += a.chunk, ++t) {
                if (ok) ok = wait_phase<100>(b, b.sum_full[t & 1], uint32_t(t / 2) & 1);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t sums = lanes + uint32_t((t & 1) * kN);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t lo[16], hi[16];
                    load_sums(sums + 32 * k, lo);
                    load_sums(sums + 32 * k + 16, hi);
                    wait_sums(lo);
                    wait_sums(hi);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float f = __uint_as_float(lo[j]), g = __uint_as_float(hi[j]);
                        all[k][j] = i == 0 ? f : all[k][j] + f;
                        all[k][16 + j] = i == 0 ? g : all[k][16 + j] + g;
                    }
                }
                release_sums(b, t & 1, lane);
            }
            Running running;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float(&l)[32] = all[k];
                if (!ok) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) l[j] = __uint_as_float(kNanBits);
                }
                const int at = int(target - (c0 + 32 * k));
                const bool has_target = mine && target - (c0 + 32 * k) >= 0 && target - (c0 + 32 * k) < 32;
                if (!GRAD) {
                    if (there >= 32 * (k + 1)) running.add(l, 32);
                    else if (there > 32 * k) running.add(l, there - 32 * k);
                    if (has_target) {
                        float f = l[0];
#pragma unroll
                        for (int j = 1; j < 32; ++j)
                            if (at == j) f = l[j];
                        a.at_target[row] = f;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) l[j] = by_p * exp2_of((l[j] - lse) * kLog2e);
                    if (by_p == 0.0f && by_target == 0.0f && ok) {  // nothing, were its logits infinite
#pragma unroll
                        for (int j = 0; j < 32; ++j) l[j] = 0.0f;
                    }
                    if (has_target) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (at == j) l[j] -= by_target;
                    }
                    if ((k & 1) == 0) {  // the copies last made from the buffers have read them
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        __syncwarp();
                    }
#pragma unroll
                    for (int plane = 0; plane < PLANES; ++plane) {
                        unsigned char *to = out + plane * kOutBuffer + lane * 128;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint4 v;
                            v.x = pack2<T>(l[8 * q], l[8 * q + 1]), v.y = pack2<T>(l[8 * q + 2], l[8 * q + 3]);
                            v.z = pack2<T>(l[8 * q + 4], l[8 * q + 5]), v.w = pack2<T>(l[8 * q + 6], l[8 * q + 7]);
                            *reinterpret_cast<uint4 *>(to + ((((k & 1) * 4 + q) ^ (lane & 7)) << 4)) = v;
                        }
                        if (plane + 1 < PLANES) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) l[j] = rest_of<T>(l[j]);
                        }
                    }
                    if (k & 1) {
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        const int c = c0 + 32 * (k - 1);
                        if (lane == 0) {
                            if (c < a.cols && row0 < a.rows)
#pragma unroll
                                for (int plane = 0; plane < PLANES; ++plane)
                                    store_box(&a.d_map[plane], c, row0, smem_of(out + plane * kOutBuffer));
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                    }
                }
            }
            if (!GRAD && mine) a.partial[int64_t(2 * (tile.n0 / kN) + half) * a.rows + row] = make_float2(running.c, running.s);
        }
        if (GRAD && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    pair_end(b, tmem, warp == kMmaWarp);
}

// The parts of each row's sum joined: lse, and the loss.  A block: 32 rows, by
// WARPS warps' shares of the parts (32 where there are few rows, 8 where there
// is a block an SM: 16384 rows of 394 parts 21 us instead of 27), eight parts at
// a time under one reference.
struct JoinLossArgs {
    const float2 *partial;
    const float *at_target;
    const void *targets;
    float *loss, *lse;
    int64_t vocab;
    int32_t parts, rows, wide;
};
template <int N>
__device__ __forceinline__ void join_sums(float &c, float &s, const float2 (&v)[N]) {
    float top = c;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, v[i].x);
    s *= exp2_of((c - top) * kLog2e);  // (references are finite)
#pragma unroll
    for (int i = 0; i < N; ++i) s += v[i].y * exp2_of((v[i].x - top) * kLog2e);
    c = top;
}
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) dopt_head_join_kernel(const __grid_constant__ JoinLossArgs a) {
    __shared__ float2 part[WARPS][33];
    let_dependents_start();
    wait_for_grids_before();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = int(blockIdx.x) * 32 + lane;
    const float2 none = make_float2(-kLargest, 0.0f);
    float c = none.x, s = 0.0f;
    if (row < a.rows)
        for (int p = warp; p < a.parts; p += 8 * WARPS) {
            float2 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = p + i * WARPS < a.parts ? __ldcs(a.partial + int64_t(p + i * WARPS) * a.rows + row) : none;
            join_sums(c, s, v);
        }
    part[warp][lane] = make_float2(c, s);
    __syncthreads();
    // a warp joins rows w, w + WARPS, ...: a lane a part, then halves
    for (int r = warp; r < 32; r += WARPS) {
        const int mine = int(blockIdx.x) * 32 + r;
        if (mine >= a.rows) break;
        const float2 own = lane < WARPS ? part[lane][r] : none;
        c = own.x, s = own.y;
#pragma unroll
        for (int d = WARPS / 2; d > 0; d >>= 1) {
            const float2 v[1] = {make_float2(__shfl_down_sync(kFull, c, d), __shfl_down_sync(kFull, s, d))};
            join_sums(c, s, v);
        }
        if (lane > 0) continue;
        const double lse = double(c) + double(log2f(s)) * 0.69314718055994530942;
        const int64_t target = a.wide ? static_cast<const int64_t *>(a.targets)[mine]
                                      : int64_t(static_cast<const int32_t *>(a.targets)[mine]);
        a.lse[mine] = float(lse);
        a.loss[mine] = target >= 0 && target < a.vocab ? float(lse - double(a.at_target[mine])) : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// Products with the logits' gradients
// ---------------------------------------------------------------------------

struct ProductArgs {
    CUtensorMap a_map;          // [k][cols]: x or the output matrix
    CUtensorMap b_map[2];       // the logits' gradients
    void *out;                  // [outs][cols], row stride ld
    const float *add;           // fp32 [outs][cols] added to the sums, or NULL
    const float *back;          // factor of the result (then: if rows have their own), or NULL
    const float *row_back;      // d_x: each row's own
    float *partial;             // [slot][n][m] parts of split tiles
    int64_t ld;
    int32_t cols, outs, steps;  // steps of 64 k a plane
    int32_t planes;
    int32_t tiles_m, items, whole, split, chunk;
    int32_t accumulate, out_dtype;
};
// What a launch makes: d_x, for which k is contiguous in the logits' gradients;
// d_w, for which n is; or both, where all their tiles fit the card at once
// (all gradients of 1001 x 512 x 5003 bf16 33 us where two launches take 43, of 512
// x 768 x 4096 28 and 38, of 700 x 1024 x 2048 fp16 30 and 38; where there are more
// tiles, the choice at each costs more).
enum Which { kDx = 0, kDw = 1, kBoth = 2, kDxRows = 3 };  // kDxRows: d_x of rows that may have their own factors
struct Products {
    ProductArgs p[2];
    int32_t first, items;       // items of p[0], and of both
    int32_t joined;             // split tiles of p[0]
    const float *for_rows;      // not NULL: whether rows have their own factors, and nothing is done
    int32_t unless;             // where they have none (0) or have some (1)
};
__device__ __forceinline__ bool not_for_these(const Products &w) {
    return w.for_rows && (*w.for_rows != 0.0f) == (w.unless != 0);
}
struct Item {
    int m0, n0, from, steps, slot;
};
__device__ __forceinline__ Item item_of(const ProductArgs &a, int item) {
    Item it;
    int tile = item, part = 0, parts = 1;
    it.slot = -1;
    if (item >= a.whole) {
        parts = a.split;
        tile = a.whole + (item - a.whole) / parts;
        part = (item - a.whole) % parts;
        if (parts > 1) it.slot = item - a.whole;
    }
    it.m0 = tile % a.tiles_m * kM;
    it.n0 = tile / a.tiles_m * kN;
    const int64_t all = int64_t(a.steps) * a.planes;
    it.from = int(all * part / parts);
    it.steps = int(all * (part + 1) / parts) - it.from;
    return it;
}

template <Which WHICH>
__device__ __forceinline__ bool is_dx(const Products &w, int item) {
    return WHICH == kDx || WHICH == kDxRows || (WHICH == kBoth && item < w.first);
}
template <Which WHICH>
__device__ __forceinline__ const ProductArgs &product_of(const Products &w, int item) {
    return WHICH == kBoth && item >= w.first ? w.p[1] : w.p[0];
}
template <Which WHICH>
__device__ __forceinline__ Item item_of(const Products &w, int item) {
    return item_of(product_of<WHICH>(w, item), WHICH == kBoth && item >= w.first ? item - w.first : item);
}

// The factor of a product's results: one, or each row's own.
struct Back {
    float all = 1.0f;
    const float *rows = nullptr;
};
__device__ __forceinline__ Back back_of(const ProductArgs &a, bool rows) {
    Back back;
    if (!a.back) return back;
    if (rows && a.back[1] != 0.0f) back.rows = a.row_back;
    else back.all = *a.back;
    return back;
}

// 16 sums of one column, of which `there` are outputs, to the rows from p on
// (n: the first one's number); `add`: the sums so far.
template <typename G, bool ALL, bool ROWS>
__device__ __forceinline__ void store_sums(const ProductArgs &a, G *p, const float *add, int there, int n, const Back &back,
                                           float (&v)[16]) {
    if (add) {
        float more[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (ALL || j < there) more[j] = add[int64_t(j) * a.cols];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (ALL || j < there) v[j] += more[j];
    }
    if (ROWS && back.rows) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (ALL || j < there) v[j] *= back.rows[n + j];
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= back.all;
    }
    if (a.accumulate) {
        G old[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (ALL || j < there) old[j] = p[j * a.ld];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (ALL || j < there) v[j] += to_f32(old[j]);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j, p += a.ld)
        if (ALL || j < there) *p = from_f32<G>(v[j]);
}
template <typename G, bool ROWS>
__device__ __forceinline__ void store_column(const ProductArgs &a, int m, int n, const Back &back, float (&v)[16]) {
    if (m >= a.cols || n >= a.outs) return;
    G *p = static_cast<G *>(a.out) + n * a.ld + m;
    const float *add = a.add ? a.add + int64_t(n) * a.cols + m : nullptr;
    if (a.outs - n >= 16) store_sums<G, true, ROWS>(a, p, add, 16, n, back, v);
    else store_sums<G, false, ROWS>(a, p, add, a.outs - n, n, back, v);
}
// A warp's half of a tile's columns, from column n on, at `sums` in tensor
// memory, 32 at a time; NaN instead where there are none.
template <typename G, bool ROWS>
__device__ __forceinline__ void store_tile(const ProductArgs &a, int m, int n, const Back &back, uint32_t sums, bool there_are) {
    for (int o = 0; o < kN / 2; o += 32) {
        uint32_t r[2][16];
#pragma unroll
        for (int q = 0; q < 16; ++q) r[0][q] = r[1][q] = kNanBits;
        if (there_are) {
            load_sums(sums + uint32_t(o), r[0]);
            load_sums(sums + uint32_t(o + 16), r[1]);
            wait_sums(r[0]);
            wait_sums(r[1]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = __uint_as_float(r[h][q]);
            store_column<G, ROWS>(a, m, n + o + 16 * h, back, v);
        }
    }
}

template <typename T, Which WHICH>
__global__ void __launch_bounds__(kProductThreads, 1) __cluster_dims__(2, 1, 1)
    dopt_head_product_kernel(const __grid_constant__ Products w) {
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr int kRing = kProductRing, kMmaWarp = kStoreWarps, kLoadWarp = kStoreWarps + 1;
    constexpr bool ROWS = WHICH == kDxRows;
    if (kHasRows<T> && (WHICH == kDx || ROWS) && w.for_rows) {
        wait_for_grids_before();
        if (not_for_these(w)) return;
    }
    HeadBarriers &b = *reinterpret_cast<HeadBarriers *>(smem + kRing * kStage);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pairs = int(gridDim.x >> 1), pair = int(blockIdx.x >> 1);
    const uint32_t tmem = pair_begin(b, kRing, kStoreWarps, warp == kMmaWarp);

    if (warp == kLoadWarp) {
        int n = 0;
        bool ok = true;
        for (int item = pair; ok && item < w.items; item += pairs) {
            const ProductArgs &a = product_of<WHICH>(w, item);
            const Item it = item_of<WHICH>(w, item);
            for (int i = it.from; i < it.from + it.steps; ++i, ++n) {
                const int s = n % kRing;
                if (n >= kRing) ok = wait_phase<64>(b, b.empty[s], uint32_t(n / kRing - 1) & 1);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t full = smem_of(&b.full[s]), to = smem_of(smem + s * kStage), bar = leader_address(full);
                    const int plane = i >= a.steps, k = (plane ? i - a.steps : i) * kK;
                    const int m = it.m0 + int(rank) * (kM / 2), o = it.n0 + int(rank) * (kN / 2);
                    if (rank == 0) expect_bytes(full, 2 * kStage);
                    load_box(to, &a.a_map, m, k, bar);
                    load_box(to + kSlab, &a.a_map, m + 64, k, bar);
                    if (is_dx<WHICH>(w, item)) {
                        load_box(to + kOperand, &a.b_map[plane], k, o, bar);
                    } else {
                        load_box(to + kOperand, &a.b_map[plane], o, k, bar);
                        load_box(to + kOperand + kSlab, &a.b_map[plane], o + 64, k, bar);
                    }
                }
                __syncwarp();
            }
        }
        if (ok) drain(b, kRing, n);
    } else if (warp == kMmaWarp) {
        if (rank == 0) {
            const uint32_t base = uniform(tmem);
            const uint64_t a0 = mn_descriptor(smem_of(smem));
            int n = 0, t = 0;
            uint32_t used = 0, odd = 0;  // bit per buffer: used before, an odd number of times
            bool ok = true;
            for (int item = pair; ok && item < w.items; item += pairs, ++t) {
                if (products_withheld(t)) break;
                const ProductArgs &a = product_of<WHICH>(w, item);
                const Item it = item_of<WHICH>(w, item);
                const bool b_k = is_dx<WHICH>(w, item);
                const uint32_t idesc = b_k ? instruction<T>(true, false) : instruction<T>(true, true);
                const uint64_t b0 = b_k ? k_descriptor(smem_of(smem + kOperand)) : mn_descriptor(smem_of(smem + kOperand));
                const uint64_t b_step = b_k ? 2 : 128;  // 16 k on
                int buffer = t & 1, left = 0;  // steps left of the sum
                uint32_t sums = base;
                for (int i = 0; i < it.steps && ok; ++i, ++n, --left) {
                    const int s = n % kRing;
                    const bool fresh = left == 0;
                    if (fresh) {  // the tile's first sum, or the next one, in the other buffer
                        if (i > 0) buffer = ~t & 1;
                        if (used >> buffer & 1) ok = wait_phase(b, b.sum_empty[buffer], ~(odd >> buffer) & 1);
                        used |= 1u << buffer, odd ^= 1u << buffer;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        sums = base + uint32_t(buffer * kN);
                        left = min(a.chunk, it.steps - i);
                        if (!ok) break;
                    }
                    ok = wait_phase(b, b.full[s], uint32_t(n / kRing) & 1);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint64_t da = a0 + uint64_t(s * (kStage >> 4)), db = b0 + uint64_t(s * (kStage >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            product(sums, da + 128 * k, db + b_step * k, idesc, !fresh || k > 0);
                        commit(b.empty[s]);
                        if (left == 1) commit(b.sum_full[buffer]);
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        const int m_in = int(rank) * (kM / 2) + (warp & 3) * 32 + lane, half = (warp >> 2) * (kN / 2);
        const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16) + uint32_t(half);
        int t = 0;
        uint32_t odd = 0;
        bool ok = true;
        for (int item = pair; item < w.items; item += pairs, ++t) {
            const ProductArgs &a = product_of<WHICH>(w, item);
            const Item it = item_of<WHICH>(w, item);
            const Back back = back_of(a, ROWS);
            const int buffer = t & 1, m = it.m0 + m_in;
            const uint32_t sums = lanes + uint32_t(buffer * kN);
            for (int i = 0; ok && i < it.steps; i += a.chunk) {
                const int from = i > 0 ? buffer ^ 1 : buffer;
                ok = wait_phase<100>(b, b.sum_full[from], odd >> from & 1);
                if (!ok) break;
                odd ^= 1u << from;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (i > 0) {
                    add_tile(sums, lanes + uint32_t(from * kN), kN / 2);
                    release_sums(b, from, lane);
                }
            }
            if (it.slot >= 0) {
                float *p = a.partial + (int64_t(it.slot) * kN + half) * kM + m_in;
                for (int o = 0; o < kN / 2; o += 16) {
                    uint32_t r[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) r[q] = kNanBits;
                    if (ok) load_sums(sums + uint32_t(o), r), wait_sums(r);
#pragma unroll
                    for (int q = 0; q < 16; ++q, p += kM) *p = __uint_as_float(r[q]);
                }
            } else if (a.out_dtype == DOPT_FP32) {
                store_tile<float, ROWS>(a, m, it.n0 + half, back, sums, ok);
            } else if (a.out_dtype == DOPT_BF16) {
                store_tile<__nv_bfloat16, ROWS>(a, m, it.n0 + half, back, sums, ok);
            } else {
                store_tile<__half, ROWS>(a, m, it.n0 + half, back, sums, ok);
            }
            if (ok) release_sums(b, buffer, lane);
        }
    }
    pair_end(b, tmem, warp == kMmaWarp);
}

// The split tiles' parts, added in order and written.  blockIdx.x: tile,
// blockIdx.y: 16 of its outputs; a thread: one column.
__global__ void __launch_bounds__(kM) dopt_head_parts_kernel(const __grid_constant__ Products w) {
    let_dependents_start();
    wait_for_grids_before();
    if (not_for_these(w)) return;
    const int second = int(blockIdx.x) >= w.joined;
    const ProductArgs &a = w.p[second];
    const Item it = item_of(a, a.whole + (int(blockIdx.x) - second * w.joined) * a.split);
    const int o = int(blockIdx.y) * 16;
    if (it.n0 + o >= a.outs) return;
    float f[16] = {};
    for (int s = 0; s < a.split; ++s) {
        const float *p = a.partial + (int64_t(it.slot + s) * kN + o) * kM + threadIdx.x;
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = __ldcs(p + q * kM);
#pragma unroll
        for (int q = 0; q < 16; ++q) f[q] += v[q];
    }
    const Back back = back_of(a, a.row_back != nullptr);
    const int m = it.m0 + int(threadIdx.x);
    if (a.out_dtype == DOPT_FP32) store_column<float, true>(a, m, it.n0 + o, back, f);
    else if (a.out_dtype == DOPT_BF16) store_column<__nv_bfloat16, true>(a, m, it.n0 + o, back, f);
    else store_column<__half, true>(a, m, it.n0 + o, back, f);
}

// What comes before the products, in one launch.  Matrices whose rows are not
// 16-byte aligned go into rows that are (`ld`, a multiple of 8; zeros past the
// columns), 16 rows and 256 columns a block.  The first block finds the factor
// of the logits' gradients (factor[0]) and what takes it back (factor[1]): one
// over the largest d_loss, so that a mean's equal weights become ones and a
// target's -(1 - p) is rounded by what p is, not by what 1 / rows happens to be
// (the same way in every row: gradients were up to 2^-9 too large or small
// throughout), and for fp16 times 2^13, to stay in its normal range.  A d_loss
// that is not finite is no measure of the others.
// fp16 reaches no further than 2^-38 of the largest so.  Rows of d_x have nothing
// to do with one another: where a row's weight is less than a 16th of the
// largest, all have a factor of their own for d_x (row_back takes it back, and
// factor[2] says so); the output matrix's grads are sums over rows of one factor.
struct ReadyArgs {
    const void *from[2];
    void *to[2];
    int64_t from_ld[2], rows[2];
    int64_t blocks[2];  // of each matrix, after the factor's
    int64_t ld;
    int32_t cols, across;
    const float *d_loss, *d_lse;
    const void *targets;
    float *factor;      // or NULL
    float *row_back;    // fp16: each row's own, or NULL
    int64_t vocab;
    int32_t wide, half;
    int32_t tokens;
};
constexpr int kReadyThreads = 512, kReadyRows = kReadyThreads / 32;
// The measure of weights of which d_loss's largest is `top`, d_loss + d_lse's `top_p`.
// (a gradient is then at most 5 times as large; where d_lse is far larger, twice)
__device__ __forceinline__ float measure(float top, float top_p) { return top_p <= 4.0f * top ? top : top_p; }
// (nothing to scale by: zeros, infinities, and what has no normal inverse)
__device__ __forceinline__ bool has_factor(float top) { return top >= 1e-34f && top <= 1e34f; }
template <bool ROWS>
__device__ __forceinline__ void find_factor(const ReadyArgs &a) {
    __shared__ float tops[3][kReadyRows];
    constexpr int kAhead = 8;
    const float most = a.half ? 8192.0f : 1.0f;
    float top = 0.0f, top_p = 0.0f;  // of d_loss, and of d_loss + d_lse
    float least = kLargest;          // of the rows' own measures, if they count at all
    for (int r0 = threadIdx.x; r0 < a.tokens; r0 += kAhead * kReadyThreads) {
        int64_t t[kAhead];
        float loss[kAhead], lse[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + i * kReadyThreads;
            const bool there = r < a.tokens;
            t[i] = !there ? -1 : a.wide ? static_cast<const int64_t *>(a.targets)[r] : int64_t(static_cast<const int32_t *>(a.targets)[r]);
            loss[i] = there ? a.d_loss[r] : 0.0f;
            lse[i] = there && a.d_lse ? a.d_lse[r] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + i * kReadyThreads;
            const float by_target = t[i] >= 0 && t[i] < a.vocab ? loss[i] : 0.0f;
            const float l = fabsf(by_target), p = fabsf(by_target + lse[i]);
            if (l <= kLargest) top = fmaxf(top, l);
            if (p <= kLargest) top_p = fmaxf(top_p, p);
            if (ROWS && a.row_back) {
                const float own = measure(l, p);
                if (own > 0.0f) least = fminf(least, own);
                if (r < a.tokens) a.row_back[r] = has_factor(own) ? own / most : 1.0f;
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
        top_p = fmaxf(top_p, __shfl_xor_sync(kFull, top_p, d));
        if (ROWS) least = fminf(least, __shfl_xor_sync(kFull, least, d));
    }
    if ((threadIdx.x & 31) == 0)
        tops[0][threadIdx.x >> 5] = top, tops[1][threadIdx.x >> 5] = top_p, tops[2][threadIdx.x >> 5] = least;
    __syncthreads();
    if (threadIdx.x > 0) return;
    for (int w = 1; w < kReadyRows; ++w)
        top = fmaxf(top, tops[0][w]), top_p = fmaxf(top_p, tops[1][w]), least = fminf(least, tops[2][w]);
    top = measure(top, top_p);
    const bool fine = has_factor(top);
    a.factor[0] = fine ? most / top : 1.0f;
    a.factor[1] = fine ? top / most : 1.0f;
    a.factor[2] = ROWS && a.row_back && top > 16.0f * least ? 1.0f : 0.0f;
}
template <typename T>
__global__ void __launch_bounds__(kReadyThreads) dopt_head_ready_kernel(const __grid_constant__ ReadyArgs a) {
    let_dependents_start();
    wait_for_grids_before();
    int64_t block = blockIdx.x;
    if (a.factor) {
        if (block == 0) {
            find_factor<kHasRows<T>>(a);
            return;
        }
        --block;
    }
    const int which = block >= a.blocks[0];
    if (which) block -= a.blocks[0];
    const int lane = threadIdx.x & 31, c = int(block % a.across * 32 + lane) * 8;
    const int64_t r = block / a.across * kReadyRows + (threadIdx.x >> 5);
    if (r >= a.rows[which]) return;  // (a warp's rows are one)
    Values<T, 8> v;
    v.load(static_cast<const T *>(a.from[which]) + r * a.from_ld[which], c, a.cols, false, lane, 32);
    if (c < a.ld) *reinterpret_cast<uint4 *>(static_cast<T *>(a.to[which]) + r * a.ld + c) = v.raw[0];
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

int64_t up_to(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }

std::mutex g_head_mutex;
EncodeTiled g_encode = nullptr;
int g_head_pairs[64] = {};  // pairs of SMs of a device, once its kernels are set up

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}
template <typename T>
cudaError_t allow_all() {
    cudaError_t e = allow_smem(dopt_head_logit_kernel<T, 0>, logit_smem(0));
    if (e == cudaSuccess) e = allow_smem(dopt_head_logit_kernel<T, 1>, logit_smem(1));
    if (e == cudaSuccess) e = allow_smem(dopt_head_logit_kernel<T, 2>, logit_smem(2));
    if (e == cudaSuccess) e = allow_smem(dopt_head_product_kernel<T, kDx>, kProductSmem);
    if (e == cudaSuccess) e = allow_smem(dopt_head_product_kernel<T, kDw>, kProductSmem);
    if (e == cudaSuccess) e = allow_smem(dopt_head_product_kernel<T, kBoth>, kProductSmem);
    if constexpr (kHasRows<T>)
        if (e == cudaSuccess) e = allow_smem(dopt_head_product_kernel<T, kDxRows>, kProductSmem);
    return e;
}

// The tensor-map encoder, the kernels' shared-memory limits and the device's
// number of SM pairs, looked up once per device.
int set_up(const char *who, EncodeTiled *encode, int *pairs) {
    using dopt::fail;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess && (device < 0 || device >= 64)) return fail(DOPT_E_ARG, "%s: device %d", who, device);
    std::lock_guard<std::mutex> lock(g_head_mutex);
    if (e == cudaSuccess && !g_encode) {
        bool none = false;
        e = find_encoder(&g_encode, &none);
        if (none) return fail(DOPT_E_CUDA, "%s: the driver has no tensor maps", who);
    }
    if (e == cudaSuccess && g_head_pairs[device] == 0) {
        int sms = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
        if (e == cudaSuccess) e = allow_all<__nv_bfloat16>();
        if (e == cudaSuccess) e = allow_all<__half>();
        if (e == cudaSuccess) g_head_pairs[device] = std::max(1, sms / 2);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(DOPT_E_CUDA, "%s: set-up: %s", who, cudaGetErrorString(e));
    }
    *encode = g_encode;
    *pairs = g_head_pairs[device];
    return DOPT_OK;
}

// A matrix of 16-bit rows (extent `cols`, stride `ld`) read or written in boxes.
int make_map(const char *who, EncodeTiled encode, CUtensorMap *map, dopt_dtype dtype, const void *base, int64_t cols,
             int64_t rows, int64_t ld, uint32_t box_cols, uint32_t box_rows) {
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
    const cuuint32_t box[2] = {box_cols, box_rows}, unit[2] = {1, 1};
    const CUresult r = encode(map, dtype == DOPT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                              2, const_cast<void *>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return dopt::fail(DOPT_E_CUDA, "%s: a tensor map of %lld x %lld, row stride %lld, was refused (%d)", who,
                          static_cast<long long>(rows), static_cast<long long>(cols), static_cast<long long>(ld), int(r));
    return DOPT_OK;
}

// How a product's tiles go over the pairs: whole waves tile by tile, the last
// partial wave's tiles split along k.  Chosen for the least estimated time in
// steps of 64 k: a tile's stores 4 (they run under the next tile's products),
// the join's launch 12 and a part's trip through memory 0.5 (fitted at 1001 x 515 x
// 5003; gradients without split tiles: 2048 x 768 x 5003 63 us for 56, 512 x 2048
// x 32000 256 for 162, 24 x 2048 x 32000 226 for 117).
struct Plan {
    int64_t whole, tail;
    int parts;
    double time;  // of all tiles
};
Plan plan_product(int64_t tiles, int64_t steps, int64_t pairs) {
    const int64_t tail = tiles % pairs;
    const double waves = double(tiles / pairs) * (double(steps) + 4);
    Plan best{tiles, 0, 1, waves};
    if (tail == 0) return best;
    double least = double(steps) + 4;
    best.time = waves + least;
    for (int parts = 2; parts <= kMostSplit; ++parts) {
        if (steps / parts < 4 || tail * parts > kMostSlots) break;
        const double t = double((tail * parts + pairs - 1) / pairs) * (double(steps) / parts + 4) + 12 + 0.5 * double(tail * parts);
        if (t < least) {
            least = t;
            best = Plan{tiles - tail, tail, parts, waves + t};
        }
    }
    return best;
}

// Steps of one sum: the tensor cores cut off what 24 bits do not hold, always
// toward zero, so that the error grows with the sum's length.  Logits and fp32
// results add sums of 1024 k (512 with fp16 factors) up in fp32, rounding to
// nearest (lse of width 2048 and 4096, bf16: 6.3e-7 and 1.29e-6 off in one sum,
// 3.0e-7 and 2.9e-7 so; an fp32 product's is 3e-8 off);
// 16-bit results lose less than an eighth of their own rounding in 131072
// (bf16) or 16384 (fp16).
int32_t sum_chunk(dopt_dtype factors, dopt_dtype out) {
    if (out == DOPT_FP32) return factors == DOPT_BF16 ? 1024 / kK : 512 / kK;
    return out == DOPT_FP16 ? 16384 / kK : 131072 / kK;
}

// What a call keeps where in its workspace.
struct HeadSpace {
    int64_t copy_ld, x_copy, w_copy, rest;
    // bytes of the copies that rows which are not aligned need
    HeadSpace(int64_t rows, int64_t width, int64_t vocab, bool copy_x, bool copy_w) {
        copy_ld = up_to(width, 8);
        x_copy = 0;
        w_copy = x_copy + (copy_x ? up_to(rows * copy_ld * 2, 256) : 0);
        rest = w_copy + (copy_w ? up_to(vocab * copy_ld * 2, 256) : 0);
    }
};
int64_t loss_rest(int64_t rows, int64_t vocab) {
    return up_to(rows * 4, 256) + 2 * ((vocab + kN - 1) / kN) * rows * int64_t(sizeof(float2));
}
// Parts of split tiles that a product of `outs` rows has at most.
int64_t most_slots(int64_t width, int64_t outs) {
    return std::min<int64_t>(kMostSlots, kMostSplit * ((width + kM - 1) / kM) * ((outs + kN - 1) / kN));
}
// The gradients' workspace after the copies: the factor, the rows' own, fp32 sums of d_x
// where the vocabulary goes in pieces, parts of split tiles, and a piece's
// gradients of the logits.
struct GradSpace {
    int64_t factor, row_back, sums, parts, logits, bytes;
    int64_t piece, piece_ld;  // columns of a piece, and of its rows
    GradSpace(int64_t rows, int64_t width, int64_t vocab, int planes, int64_t pieces) {
        piece = std::min(vocab, up_to((vocab + pieces - 1) / pieces, kN));
        piece_ld = up_to(piece, 64);
        factor = 0;
        row_back = 256;
        sums = row_back + up_to(rows * 4, 256);
        parts = sums + (piece < vocab ? up_to(rows * width * 4, 256) : 0);
        logits = parts + (most_slots(width, rows) + most_slots(width, piece)) * kM * kN * 4;
        bytes = logits + planes * up_to(rows * piece_ld * 2, 256);
    }
};
constexpr int64_t kMostPieces = 1 << 20;

int check_head(const char *who, const void *x, dopt_dtype dtype, int64_t rows, int64_t width, int64_t ld_x,
               const void *weight, int64_t vocab, int64_t ld_w, const void *targets, int32_t target_bytes) {
    using dopt::fail;
    if (rows < 0 || rows > DOPT_HEAD_MAX_ROWS || width < 1 || width > DOPT_MAX_COLS || vocab < 1 ||
        vocab > DOPT_HEAD_MAX_VOCAB)
        return fail(DOPT_E_ARG, "%s: %lld rows, width %lld, vocab %lld", who, static_cast<long long>(rows),
                    static_cast<long long>(width), static_cast<long long>(vocab));
    if (dtype != DOPT_BF16 && dtype != DOPT_FP16) return fail(DOPT_E_ARG, "%s: x and weight must be bf16 or fp16", who);
    if (ld_x < width || ld_w < width)
        return fail(DOPT_E_ARG, "%s: row strides %lld, %lld for a width of %lld", who, static_cast<long long>(ld_x),
                    static_cast<long long>(ld_w), static_cast<long long>(width));
    if (target_bytes != 4 && target_bytes != 8)
        return fail(DOPT_E_ARG, "%s: target_bytes %d (4 or 8)", who, target_bytes);
    if (!weight || (rows > 0 && (!x || !targets))) return fail(DOPT_E_ARG, "%s: NULL x, weight or targets", who);
    if (!aligned_to(x, 2) || !aligned_to(weight, 2) || !aligned_to(targets, size_t(target_bytes)))
        return fail(DOPT_E_ALIGN, "%s: x, weight or targets is not aligned to its elements", who);
    return DOPT_OK;
}
// (a tensor map's stride is below 2^40 bytes)
bool by_tma(const void *p, int64_t ld) { return aligned_to(p, 16) && ld % 8 == 0 && ld < (int64_t(1) << 38); }

// x and the output matrix as the kernels read them.
struct Operands {
    const void *x, *w;
    int64_t ld_x, ld_w;
};
template <typename T>
int make_ready(const char *who, Operands &o, const HeadSpace &space, char *ws, int64_t rows, int64_t width,
               int64_t vocab, ReadyArgs a, cudaStream_t stream) {
    const bool copy[2] = {!by_tma(o.x, o.ld_x), !by_tma(o.w, o.ld_w)};
    if (!copy[0] && !copy[1] && !a.factor) return DOPT_OK;
    a.ld = space.copy_ld;
    a.cols = int32_t(width);
    a.across = int32_t((a.ld + 255) / 256);
    a.from[0] = o.x, a.from_ld[0] = o.ld_x, a.rows[0] = rows, a.to[0] = ws + space.x_copy;
    a.from[1] = o.w, a.from_ld[1] = o.ld_w, a.rows[1] = vocab, a.to[1] = ws + space.w_copy;
    for (int i = 0; i < 2; ++i) a.blocks[i] = copy[i] ? (a.rows[i] + kReadyRows - 1) / kReadyRows * a.across : 0;
    if (copy[0]) o.x = a.to[0], o.ld_x = a.ld;
    if (copy[1]) o.w = a.to[1], o.ld_w = a.ld;
    const int64_t blocks = a.blocks[0] + a.blocks[1] + (a.factor ? 1 : 0);
    if (blocks > INT32_MAX) return dopt::fail(DOPT_E_ARG, "%s: the matrices are too large to be copied", who);
    return launch_op(who, dopt_head_ready_kernel<T>, dim3(unsigned(blocks)), dim3(kReadyThreads), 0, stream, a);
}

// Rows of x in a box: of few tokens, no more than there are.  The rest of the
// operand is then whatever shared memory held, which reaches rows of the
// logits alone that nothing reads; boxes of 128 rows for 24 tokens took 38 us
// where these take 31 (24 x 2048 x 32000).
uint32_t x_box_rows(int64_t rows) { return uint32_t(std::min<int64_t>(kM / 2, up_to(rows, 8))); }

int fill_tiles(LogitArgs &a, dopt_dtype dtype, int64_t rows, int64_t width, int64_t cols) {
    a.x_ctas = rows > kM / 2 ? 2 : 1;
    a.step_bytes = int32_t(a.x_ctas * x_box_rows(rows) * kK * 2 + 2 * kOperand);
    a.rows = int32_t(rows);
    a.cols = int32_t(cols);
    a.steps = int32_t((width + kK - 1) / kK);
    a.chunk = sum_chunk(dtype, DOPT_FP32);
    a.tiles_m = int32_t((rows + kM - 1) / kM);
    a.tiles_n = int32_t((cols + kN - 1) / kN);
    // (blocks of tokens whose rows stay in L2 while the vocabulary goes by: 32 MB of them)
    a.group = int32_t(std::min<int64_t>(a.tiles_m, std::max<int64_t>(8, (int64_t(32) << 20) / (width * 2 * kM))));
    const int64_t items = int64_t(a.tiles_m) * a.tiles_n;
    a.items = int32_t(std::min<int64_t>(items, INT32_MAX));
    return items <= INT32_MAX / 2;
}

int64_t tiles_of(const ProductArgs &a) { return int64_t(a.tiles_m) * ((a.outs + kN - 1) / kN); }
void use(ProductArgs &a, const Plan &plan) {
    a.whole = int32_t(plan.whole);
    a.split = plan.parts;
    a.items = int32_t(plan.whole + plan.tail * plan.parts);
}
template <typename T>
int launch_products(const char *who, Which which, Products &w, int64_t pairs, cudaStream_t stream) {
    int64_t joined[2] = {};
    for (int i = 0; i < (which == kBoth ? 2 : 1); ++i)
        if (w.p[i].split > 1) joined[i] = (w.p[i].items - w.p[i].whole) / w.p[i].split;
    w.first = w.p[0].items;
    w.items = w.first + (which == kBoth ? w.p[1].items : 0);
    w.joined = int32_t(joined[0]);
    auto kernel = which == kDx ? dopt_head_product_kernel<T, kDx>
                               : which == kDw ? dopt_head_product_kernel<T, kDw> : dopt_head_product_kernel<T, kBoth>;
    if constexpr (kHasRows<T>)
        if (which == kDxRows) kernel = dopt_head_product_kernel<T, kDxRows>;
    const int rc = launch_op(who, kernel, dim3(unsigned(2 * std::min<int64_t>(w.items, pairs))), dim3(kProductThreads),
                             kProductSmem, stream, w);
    if (rc != DOPT_OK || joined[0] + joined[1] == 0) return rc;
    return launch_op(who, dopt_head_parts_kernel, dim3(unsigned(joined[0] + joined[1]), kN / 16), dim3(kM), 0, stream, w);
}
// d_x and d_w, either or both of them: in one launch where all their tiles fit
// at once and the estimates, in the plan's units, say so: d_x's tiles, few and
// long, in as many parts as leave room for d_w's, against two plans of their own
// and a launch.  (How sums are divided depends on the sizes alone, not on what
// is wanted or on the grads' type.)  for_rows: d_x is made on its own here if
// these are the rows' factors and there are some, or if they are not and there
// are none.
template <typename T>
int run_products(const char *who, const ProductArgs &dx, const ProductArgs &dw, bool want_dx, bool want_dw,
                 const float *for_rows, int64_t pairs, cudaStream_t stream) {
    const int64_t tiles_x = tiles_of(dx), tiles_w = tiles_of(dw);
    Plan plan_x = plan_product(tiles_x, dx.steps, pairs);
    Plan plan_w = plan_product(tiles_w, int64_t(dw.steps) * dw.planes, pairs);
    bool together = tiles_x + tiles_w <= pairs;
    if (together) {
        const int parts = int(std::max<int64_t>(1, std::min({int64_t(kMostSplit), (pairs - tiles_w) / tiles_x, int64_t(dx.steps) / 4})));
        const double time = std::max(double(dx.steps) / parts, double(dw.steps)) + 4 +
                            (parts > 1 ? 12 + 0.5 * double(tiles_x * parts) : 0);
        together = time < plan_x.time + plan_product(tiles_w, dw.steps, pairs).time + 12;
        if (together) {
            plan_x = parts > 1 ? Plan{0, tiles_x, parts, 0} : Plan{tiles_x, 0, 1, 0};
            plan_w = Plan{tiles_w, 0, 1, 0};
        }
    }
    Products w{};
    if (together && want_dx && want_dw) {
        w.p[0] = dx, w.p[1] = dw;
        use(w.p[0], plan_x);
        use(w.p[1], plan_w);
        return launch_products<T>(who, kBoth, w, pairs, stream);
    }
    int rc = DOPT_OK;
    if (want_dx) {
        w.p[0] = dx;
        w.for_rows = for_rows;
        w.unless = !dx.row_back;
        use(w.p[0], plan_x);
        rc = launch_products<T>(who, dx.row_back ? kDxRows : kDx, w, pairs, stream);
        w.for_rows = nullptr;
    }
    if (rc == DOPT_OK && want_dw) {
        w.p[0] = dw;
        use(w.p[0], plan_w);
        rc = launch_products<T>(who, kDw, w, pairs, stream);
    }
    return rc;
}

struct GradCall {
    dopt_dtype dtype, grad_dtype;
    int64_t rows, width, vocab;
    const void *targets;
    int32_t target_bytes, planes;
    const float *lse, *d_loss, *d_lse;
    void *d_x;
    int64_t ld_d_x;
    char *grad;  // its first element
    bool accumulate;
};

// One pass over the vocabulary, piece by piece.
struct Pass {
    bool d_x, grad;       // what it makes
    int32_t planes;       // of the logits' gradients
    bool by_row;          // with the rows' own factors, if they have any
    bool if_rows;         // nothing is done unless they have
    bool two;             // (one of two such passes)
};

template <typename T>
int run_pass(const char *who, const GradCall &c, const Pass &pass, const Operands &o, const GradSpace &g, char *rest,
             EncodeTiled encode, int pairs, cudaStream_t stream) {
    float *factor = reinterpret_cast<float *>(rest + g.factor), *sums = reinterpret_cast<float *>(rest + g.sums);
    const float *row_back = pass.by_row ? reinterpret_cast<const float *>(rest + g.row_back) : nullptr;
    const int64_t plane = up_to(c.rows * g.piece_ld * 2, 256);
    for (int64_t v0 = 0; v0 < c.vocab; v0 += g.piece) {
        const int64_t cols = std::min(g.piece, c.vocab - v0);
        const char *w = static_cast<const char *>(o.w) + v0 * o.ld_w * 2;
        LogitArgs a{};
        if (!fill_tiles(a, c.dtype, c.rows, c.width, cols)) return dopt::fail(DOPT_E_ARG, "%s: too many tiles", who);
        a.targets = c.targets;
        a.lse = c.lse;
        a.d_loss = c.d_loss;
        a.d_lse = c.d_lse;
        a.factor = factor;
        a.row_back = row_back;
        a.for_rows = pass.if_rows;
        a.first = v0;
        a.vocab = c.vocab;
        a.wide = c.target_bytes == 8;
        int rc = make_map(who, encode, &a.x_map, c.dtype, o.x, c.width, c.rows, o.ld_x, 64, x_box_rows(c.rows));
        if (rc == DOPT_OK) rc = make_map(who, encode, &a.w_map, c.dtype, w, c.width, cols, o.ld_w, 64, 128);
        for (int p = 0; p < pass.planes && rc == DOPT_OK; ++p)
            rc = make_map(who, encode, &a.d_map[p], c.dtype, rest + g.logits + p * plane, cols, c.rows, g.piece_ld, 64, 32);
        if (rc != DOPT_OK) return rc;
        rc = launch_op(who, pass.planes == 2 ? dopt_head_logit_kernel<T, 2> : dopt_head_logit_kernel<T, 1>,
                       dim3(unsigned(2 * std::min<int64_t>(a.items, pairs))), dim3(kLogitThreads), logit_smem(pass.planes),
                       stream, a);
        if (rc != DOPT_OK) return rc;
        ProductArgs dx{}, dw{};
        float *partial = reinterpret_cast<float *>(rest + g.parts);
        dx.cols = dw.cols = int32_t(c.width);
        dx.tiles_m = dw.tiles_m = int32_t((c.width + kM - 1) / kM);
        dx.outs = int32_t(c.rows);
        dx.steps = int32_t((cols + kK - 1) / kK);
        dx.planes = 1;
        dx.chunk = sum_chunk(c.dtype, c.dtype);
        dx.partial = partial;
        dw.outs = int32_t(cols);
        dw.steps = int32_t((c.rows + kK - 1) / kK);
        dw.planes = c.planes;
        dw.chunk = sum_chunk(c.dtype, c.grad_dtype);
        dw.partial = partial + most_slots(c.width, c.rows) * kM * kN;
        if (pass.d_x) {
            const bool last = v0 + cols == c.vocab;
            rc = make_map(who, encode, &dx.a_map, c.dtype, w, c.width, cols, o.ld_w, 64, 64);
            if (rc == DOPT_OK)
                rc = make_map(who, encode, &dx.b_map[0], c.dtype, rest + g.logits, cols, c.rows, g.piece_ld, 64, 128);
            if (rc != DOPT_OK) return rc;
            dx.out = last ? c.d_x : sums;
            dx.ld = last ? c.ld_d_x : c.width;
            dx.add = v0 > 0 ? sums : nullptr;
            dx.back = last ? factor + 1 : nullptr;
            dx.row_back = row_back;
            dx.out_dtype = last ? c.dtype : DOPT_FP32;
        }
        if (pass.grad) {
            rc = make_map(who, encode, &dw.a_map, c.dtype, o.x, c.width, c.rows, o.ld_x, 64, 64);
            for (int q = 0; q < pass.planes && rc == DOPT_OK; ++q)
                rc = make_map(who, encode, &dw.b_map[q], c.dtype, rest + g.logits + q * plane, cols, c.rows, g.piece_ld, 64, 64);
            if (rc != DOPT_OK) return rc;
            dw.out = c.grad + v0 * c.width * int64_t(elem_bytes(c.grad_dtype));
            dw.ld = c.width;
            dw.back = factor + 1;
            dw.out_dtype = c.grad_dtype;
            dw.accumulate = c.accumulate;
        }
        if ((rc = run_products<T>(who, dx, dw, pass.d_x, pass.grad, pass.two ? factor + 2 : nullptr, pairs, stream)) != DOPT_OK)
            return rc;
    }
    return DOPT_OK;
}

// With fp16, d_x alone takes the rows' own factors at once.  Where the matrix's
// grads are wanted too, whose sums need one factor, a second pass makes d_x from
// logits' gradients with the rows' own if weights are that far apart (the device
// knows): the logits' product a third time, 16384 x 768 x 50257 2.6 -> 3.55 ms;
// else two or three launches that end at once, 1001 x 512 x 5003 35 -> 40 us.
template <typename T>
int run_grad(const char *who, const GradCall &c, Operands o, const HeadSpace &space, const GradSpace &g, char *ws,
             EncodeTiled encode, int pairs, cudaStream_t stream) {
    char *rest = ws + space.rest;
    constexpr bool half = kHasRows<T>;
    const bool by_row = half && c.d_x && !c.grad;
    ReadyArgs ready{};
    ready.d_loss = c.d_loss;
    ready.d_lse = c.d_lse;
    ready.targets = c.targets;
    ready.factor = reinterpret_cast<float *>(rest + g.factor);
    ready.row_back = half && c.d_x ? reinterpret_cast<float *>(rest + g.row_back) : nullptr;
    ready.half = half;
    ready.vocab = c.vocab;
    ready.wide = c.target_bytes == 8;
    ready.tokens = int32_t(c.rows);
    int rc = make_ready<T>(who, o, space, ws, c.rows, c.width, c.vocab, ready, stream);
    const bool two = half && c.d_x && c.grad;
    if (rc == DOPT_OK)
        rc = run_pass<T>(who, c, Pass{c.d_x != nullptr, c.grad != nullptr, c.planes, by_row, false, two}, o, g, rest, encode,
                         pairs, stream);
    if (rc == DOPT_OK && two) rc = run_pass<T>(who, c, Pass{true, false, 1, true, true, true}, o, g, rest, encode, pairs, stream);
    return rc;
}

// The grads of a call without rows.
template <typename G>
__global__ void __launch_bounds__(256) dopt_head_zero_kernel(G *p, int64_t n) {
    let_dependents_start();
    wait_for_grids_before();
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) p[i] = from_f32<G>(0.0f);
}

bool sizes_ok(int64_t rows, int64_t width, int64_t vocab) {
    return rows >= 0 && rows <= DOPT_HEAD_MAX_ROWS && width >= 1 && width <= DOPT_MAX_COLS && vocab >= 1 &&
           vocab <= DOPT_HEAD_MAX_VOCAB;
}

}  // namespace

extern "C" int dopt_head_loss_workspace(int64_t rows, int64_t width, int64_t vocab, int32_t aligned, int64_t *bytes) {
    dopt::clear_error();
    const char *who = "dopt_head_loss_workspace";
    if (!bytes) return dopt::fail(DOPT_E_ARG, "%s: bytes is NULL", who);
    if (!sizes_ok(rows, width, vocab))
        return dopt::fail(DOPT_E_ARG, "%s: %lld rows, width %lld, vocab %lld", who, static_cast<long long>(rows),
                          static_cast<long long>(width), static_cast<long long>(vocab));
    const bool copy = !aligned || width % 8 != 0;
    *bytes = HeadSpace(rows, width, vocab, copy, copy).rest + loss_rest(rows, vocab);
    return DOPT_OK;
}

extern "C" int dopt_head_loss(const void *x, dopt_dtype dtype, int64_t rows, int64_t width, int64_t ld_x,
                              const void *weight, int64_t vocab, int64_t ld_w, const void *targets, int32_t target_bytes,
                              float *loss, float *lse, void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_head_loss";
    OpRange range(who);
    int rc = check_head(who, x, dtype, rows, width, ld_x, weight, vocab, ld_w, targets, target_bytes);
    if (rc != DOPT_OK) return rc;
    if (rows > 0 && (!loss || !lse)) return fail(DOPT_E_ARG, "%s: NULL loss or lse", who);
    if (!aligned_to(loss, 4) || !aligned_to(lse, 4)) return fail(DOPT_E_ALIGN, "%s: loss or lse is not 4-byte aligned", who);
    if (!aligned_to(workspace, 16)) return fail(DOPT_E_ALIGN, "%s: workspace is not 16-byte aligned", who);
    const HeadSpace space(rows, width, vocab, !by_tma(x, ld_x), !by_tma(weight, ld_w));
    const int64_t need = space.rest + loss_rest(rows, vocab);
    if (rows > 0 && (!workspace || workspace_bytes < need))
        return fail(DOPT_E_ARG, "%s: workspace of %lld bytes, %lld are needed", who,
                    static_cast<long long>(workspace ? workspace_bytes : 0), static_cast<long long>(need));
    if (rows == 0) return DOPT_OK;
    EncodeTiled encode = nullptr;
    int pairs = 0;
    if ((rc = set_up(who, &encode, &pairs)) != DOPT_OK) return rc;
    LogitArgs a{};
    if (!fill_tiles(a, dtype, rows, width, vocab)) return fail(DOPT_E_ARG, "%s: too many tiles", who);
    char *ws = static_cast<char *>(workspace), *rest = ws + space.rest;
    Operands o{x, weight, ld_x, ld_w};
    rc = dtype == DOPT_BF16 ? make_ready<__nv_bfloat16>(who, o, space, ws, rows, width, vocab, ReadyArgs{}, stream)
                            : make_ready<__half>(who, o, space, ws, rows, width, vocab, ReadyArgs{}, stream);
    if (rc == DOPT_OK) rc = make_map(who, encode, &a.x_map, dtype, o.x, width, rows, o.ld_x, 64, x_box_rows(rows));
    if (rc == DOPT_OK) rc = make_map(who, encode, &a.w_map, dtype, o.w, width, vocab, o.ld_w, 64, 128);
    if (rc != DOPT_OK) return rc;
    a.targets = targets;
    a.wide = target_bytes == 8;
    a.vocab = vocab;
    a.at_target = reinterpret_cast<float *>(rest);
    a.partial = reinterpret_cast<float2 *>(rest + up_to(rows * 4, 256));
    const dim3 grid(unsigned(2 * std::min<int64_t>(a.items, pairs)));
    rc = dtype == DOPT_BF16
             ? launch_op(who, dopt_head_logit_kernel<__nv_bfloat16, 0>, grid, dim3(kLogitThreads), logit_smem(0), stream, a)
             : launch_op(who, dopt_head_logit_kernel<__half, 0>, grid, dim3(kLogitThreads), logit_smem(0), stream, a);
    if (rc != DOPT_OK) return rc;
    JoinLossArgs j{a.partial, a.at_target, targets, loss, lse, vocab, 2 * a.tiles_n, a.rows, a.wide};
    const dim3 blocks(unsigned((rows + 31) / 32));
    return blocks.x >= 152 ? launch_op(who, dopt_head_join_kernel<8>, blocks, dim3(32 * 8), 0, stream, j)
                           : launch_op(who, dopt_head_join_kernel<32>, blocks, dim3(32 * 32), 0, stream, j);
}

extern "C" int dopt_head_loss_grad_workspace(int64_t rows, int64_t width, int64_t vocab, dopt_dtype grad_dtype,
                                             int64_t pieces, int32_t aligned, int64_t *bytes) {
    dopt::clear_error();
    const char *who = "dopt_head_loss_grad_workspace";
    if (!bytes) return dopt::fail(DOPT_E_ARG, "%s: bytes is NULL", who);
    if (!sizes_ok(rows, width, vocab) || pieces < 1 || pieces > kMostPieces)
        return dopt::fail(DOPT_E_ARG, "%s: %lld rows, width %lld, vocab %lld in %lld pieces", who,
                          static_cast<long long>(rows), static_cast<long long>(width), static_cast<long long>(vocab),
                          static_cast<long long>(pieces));
    if (!valid_dtype(grad_dtype)) return dopt::fail(DOPT_E_ARG, "%s: unknown dtype %d", who, int(grad_dtype));
    const bool copy = !aligned || width % 8 != 0;
    *bytes = HeadSpace(rows, width, vocab, copy, copy).rest +
             GradSpace(rows, width, vocab, grad_dtype == DOPT_FP32 ? 2 : 1, pieces).bytes;
    return DOPT_OK;
}

extern "C" int dopt_head_loss_grad(const void *x, dopt_dtype dtype, int64_t rows, int64_t width, int64_t ld_x,
                                   const void *weight, int64_t vocab, int64_t ld_w, const void *targets,
                                   int32_t target_bytes, const float *lse, const float *d_loss, const float *d_lse,
                                   void *d_x, int64_t ld_d_x, void *grad, dopt_dtype grad_dtype, int64_t grad_numel,
                                   int64_t grad_offset, uint32_t flags, void *workspace, int64_t workspace_bytes,
                                   cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_head_loss_grad";
    OpRange range(who);
    int rc = check_head(who, x, dtype, rows, width, ld_x, weight, vocab, ld_w, targets, target_bytes);
    if (rc != DOPT_OK) return rc;
    if (rows > 0 && (!lse || !d_loss)) return fail(DOPT_E_ARG, "%s: NULL lse or d_loss", who);
    if (!aligned_to(lse, 4) || !aligned_to(d_loss, 4) || !aligned_to(d_lse, 4))
        return fail(DOPT_E_ALIGN, "%s: lse, d_loss or d_lse is not 4-byte aligned", who);
    if (flags & ~uint32_t(DOPT_HEAD_ACCUMULATE)) return fail(DOPT_E_ARG, "%s: unknown flags 0x%x", who, flags);
    if (!d_x && !grad && rows > 0) return fail(DOPT_E_ARG, "%s: neither d_x nor grad is wanted", who);
    if (d_x && ld_d_x < width)
        return fail(DOPT_E_ARG, "%s: d_x has row stride %lld for a width of %lld", who, static_cast<long long>(ld_d_x),
                    static_cast<long long>(width));
    if (!aligned_to(d_x, 2)) return fail(DOPT_E_ALIGN, "%s: d_x is not aligned to its elements", who);
    GradCall c{};
    if (grad) {
        if (!valid_dtype(grad_dtype)) return fail(DOPT_E_ARG, "%s: unknown dtype %d", who, int(grad_dtype));
        if (!aligned_to(grad, elem_bytes(grad_dtype)))
            return fail(DOPT_E_ALIGN, "%s: grad is not aligned to its elements", who);
        if (grad_offset < 0 || grad_offset > grad_numel - vocab * width)
            return fail(DOPT_E_ARG, "%s: %lld x %lld grads at %lld leave a buffer of %lld", who,
                        static_cast<long long>(vocab), static_cast<long long>(width),
                        static_cast<long long>(grad_offset), static_cast<long long>(grad_numel));
        c.grad = static_cast<char *>(grad) + grad_offset * int64_t(elem_bytes(grad_dtype));
        c.grad_dtype = grad_dtype;
    }
    if (!aligned_to(workspace, 16)) return fail(DOPT_E_ALIGN, "%s: workspace is not 16-byte aligned", who);
    c.planes = grad && grad_dtype == DOPT_FP32 ? 2 : 1;
    const HeadSpace space(rows, width, vocab, !by_tma(x, ld_x), !by_tma(weight, ld_w));
    // the fewest pieces that the workspace has room for
    const int64_t most = (vocab + kN - 1) / kN;
    const int64_t room = workspace ? workspace_bytes - space.rest : -1;
    int64_t pieces = 1;
    while (pieces < most && GradSpace(rows, width, vocab, c.planes, pieces).bytes > room) ++pieces;
    const GradSpace g(rows, width, vocab, c.planes, pieces);
    if (rows > 0 && g.bytes > room)
        return fail(DOPT_E_ARG, "%s: workspace of %lld bytes, at least %lld are needed", who,
                    static_cast<long long>(workspace ? workspace_bytes : 0), static_cast<long long>(space.rest + g.bytes));
    if (rows == 0) {
        if (!grad || flags & DOPT_HEAD_ACCUMULATE) return DOPT_OK;
        const int64_t n = vocab * width;
        const dim3 blocks(unsigned(std::min<int64_t>((n + 255) / 256, 152 * 8)));
        if (grad_dtype == DOPT_FP32)
            return launch_op(who, dopt_head_zero_kernel<float>, blocks, dim3(256), 0, stream, reinterpret_cast<float *>(c.grad), n);
        if (grad_dtype == DOPT_BF16)
            return launch_op(who, dopt_head_zero_kernel<__nv_bfloat16>, blocks, dim3(256), 0, stream,
                             reinterpret_cast<__nv_bfloat16 *>(c.grad), n);
        return launch_op(who, dopt_head_zero_kernel<__half>, blocks, dim3(256), 0, stream, reinterpret_cast<__half *>(c.grad), n);
    }
    EncodeTiled encode = nullptr;
    int pairs = 0;
    if ((rc = set_up(who, &encode, &pairs)) != DOPT_OK) return rc;
    c.dtype = dtype;
    c.rows = rows, c.width = width, c.vocab = vocab;
    c.targets = targets, c.target_bytes = target_bytes;
    c.lse = lse, c.d_loss = d_loss, c.d_lse = d_lse;
    c.d_x = d_x, c.ld_d_x = ld_d_x;
    c.accumulate = (flags & DOPT_HEAD_ACCUMULATE) != 0;
    const Operands o{x, weight, ld_x, ld_w};
    char *ws = static_cast<char *>(workspace);
    return dtype == DOPT_BF16 ? run_grad<__nv_bfloat16>(who, c, o, space, g, ws, encode, pairs, stream)
                              : run_grad<__half>(who, c, o, space, g, ws, encode, pairs, stream);
}

extern "C" int dopt_head_timeouts(int reset, uint32_t *count) {
    using dopt::fail;
    dopt::clear_error();
    if (!count) return fail(DOPT_E_ARG, "dopt_head_timeouts: NULL output");
    unsigned int c = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&c, g_head_timeouts, sizeof c);
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_head_timeouts, &zero, sizeof zero);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(DOPT_E_CUDA, "dopt_head_timeouts: %s", cudaGetErrorString(e));
    }
    *count = c;
    return DOPT_OK;
}

extern "C" int dopt_head_wait_test(int32_t items) {
    using dopt::fail;
    dopt::clear_error();
#ifdef DOPT_DEVICE_CHECKS
    if (items < -1) return fail(DOPT_E_ARG, "dopt_head_wait_test: %d items", items);
    const int v = items;
    const cudaError_t e = cudaMemcpyToSymbol(g_head_items, &v, sizeof v);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(DOPT_E_CUDA, "dopt_head_wait_test: %s", cudaGetErrorString(e));
    }
    return DOPT_OK;
#else
    (void)items;
    return fail(DOPT_E_STATE, "dopt_head_wait_test: this library was built without DOPT_DEVICE_CHECKS");
#endif
}
