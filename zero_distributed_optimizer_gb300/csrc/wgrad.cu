// The weight gradients of a linear layer, or of a layer's experts, from the
// 8-bit checkpoint of its input, written into the flat grad buffer
// (dopt_ckpt_wgrad; dopt.h states the contract).
#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "op_common.cuh"

namespace {

// A pair of CTAs (a cluster of two, on two SMs) computes a tile of 256
// columns c by up to 256 outputs o of one group's gradient with
// tcgen05.mma.cta_group::2: M = c, N = o, K = the group's rows in steps of
// 64.  Each CTA keeps 128 of the c (operand A) and half of the o (operand B)
// in shared memory, both as they lie in memory, rows of K with M or N
// contiguous, in slabs of 64 columns x 64 rows with the 128-byte swizzle.
//
//   dy  bf16 / fp16, by TMA (a ring of 4 steps); by plain loads in a group's
//       last step, whose rows past the group must read as zeros whatever the
//       next group holds there, and where rows are not 16-byte aligned
//   x   two warps copy a step's 64 rows of 128 codes to shared memory
//       (16-byte asynchronous copies, from wherever the row's token is) with
//       their exponent bytes, 3 steps ahead; 8 warps widen them (exactly) and store them
//       swizzled (a ring of 2 steps).  These warps keep no load of their own
//       in flight: the fence before a product would wait for it (codes loaded
//       ahead into registers ran at 581 TFLOP/s, a third of the warps'
//       time in that fence).  A row that counts as zeros has exponent bytes 0.
//
// The sums are fp32 in tensor memory (128 lanes x 256 columns a CTA: half of
// it, so two CTAs share an SM and one's stores run under the other's
// products).  With lanes along c the stores of a warp are contiguous.
constexpr int kTileC = 256;          // of a pair
constexpr int kTileO = 256;
constexpr int kK = 64;               // rows a step
constexpr int kDyRing = 3;
constexpr int kXRing = 2;
constexpr int kRawRing = 3;
constexpr int kSlab = kK * 128;      // 64 columns x 64 rows of 16 bits
constexpr int kStage = 2 * kSlab;    // a CTA's 128 columns
constexpr int kWorkers = 256;        // threads that widen and store
constexpr int kWgradThreads = kWorkers + 128;
constexpr int kMmaWarp = kWorkers / 32, kDyWarp = kMmaWarp + 1, kRawWarp = kMmaWarp + 2;  // and the next
constexpr int kGroup = kWorkers / kXRing;  // threads that fill one stage of the x ring
constexpr int kTmemCols = 256;
constexpr int kRawCodes = kK * 128;  // a CTA's codes of a step, then 4 exponent bytes a row
constexpr int kRaw = kRawCodes + kK * 4;
constexpr int kMaxSplit = 16;
constexpr int64_t kSlotBytes = int64_t(kTileC) * kTileO * 4;

struct WgradBarriers {
    unsigned long long dy_full[kDyRing], dy_empty[kDyRing], x_full[kXRing], x_empty[kXRing];
    unsigned long long raw_full[kRawRing], raw_empty[kRawRing], done;
    uint32_t tmem;
    int32_t failed;
};
constexpr size_t kWgradSmem = (kDyRing + kXRing) * size_t(kStage) + kRawRing * size_t(kRaw) + sizeof(WgradBarriers);
static_assert(kWgradSmem <= 115712, "two CTAs share an SM's 228 KB");

struct WgradArgs {
    CUtensorMap dy_map;        // with `tma`
    const uint8_t *codes, *scales;
    const int32_t *row_token;  // or NULL: row r reads checkpoint row r
    const void *dy;
    const int32_t *offsets;    // or NULL: one group of all rows
    void *grad;
    float *partial;            // fp32 sums of the split tiles, [slot][o][c]
    int64_t x_rows, cols, pitch;
    int64_t dy_rows, outs, dy_ld;
    int32_t tiles_c, tiles_o;
    int32_t whole;             // tiles before the split ones
    int32_t split;             // parts of a split tile
    int32_t accumulate;
    int32_t tma, vec;          // dy by TMA; dy's rows are 16-byte aligned
    int32_t grad_dtype;
    int64_t grad_offset[DOPT_MAX_GROUPS];
};

// Waits that ran past their limit (a copy or product that never completed);
// the pair then left its tile alone.
__device__ unsigned int g_wgrad_timeouts;
constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s

__device__ __forceinline__ uint32_t smem_of(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Wait for a phase of a barrier that threads of the cluster arrive on; false
// once any wait of this CTA has run out of time.
__device__ __forceinline__ bool wait_phase(WgradBarriers &b, unsigned long long &bar, uint32_t parity) {
    const uint32_t at = smem_of(&bar);
    unsigned long long t0 = 0;
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(at), "r"(parity), "r"(1000000u)  // sleeps up to 1 ms a try
            : "memory");
        if (done) return true;
        if (*static_cast<volatile int32_t *>(&b.failed)) return false;
        unsigned long long now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitNs) {
            if (atomicExch(&b.failed, 1) == 0) atomicAdd(&g_wgrad_timeouts, 1u);
            return false;
        }
    }
}

// Wait for the last use of each slot of a ring.
__device__ __forceinline__ void drain(WgradBarriers &b, unsigned long long *empty, int ring, int steps) {
    for (int s = 0; s < ring && s < steps; ++s)
        if (!wait_phase(b, empty[s], uint32_t((steps - 1 - s) / ring) & 1)) return;
}

__device__ __forceinline__ uint32_t leader_address(uint32_t own) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(own));
    return r;
}
__device__ __forceinline__ void arrive_remote(uint32_t cluster_address) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_address) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// An asynchronous copy of N bytes to shared memory; zeros unless `there`
// (then nothing is read).
template <int N>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(N), "r"(there ? N : 0)
                 : "memory");
}

// Descriptor of an operand slab pair: 128-byte swizzle, 1024 bytes from 8
// rows to the next 8, one slab from 64 columns to the next 64.
__device__ __forceinline__ uint64_t slab_descriptor(uint32_t address) {
    return (uint64_t(address & 0x3ffff) >> 4) | (uint64_t(kSlab >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// The 16-byte chunk q (of 16) of row k in a stage, swizzled.
__device__ __forceinline__ uint32_t stage_chunk(int k, int q) {
    return uint32_t((q >> 3) * kSlab + k * 128 + (((q & 7) ^ (k & 7)) << 4));
}

// Rows of operand A are columns c in the order 0 2 1 3, 4 6 5 7, ...: the
// bytes 0 and 2 of a word of codes, and 1 and 3, are then its pairs, without
// a permutation of bytes.
__device__ __forceinline__ int column_of(int m) { return (m & ~3) | ((m & 1) << 1) | ((m >> 1) & 1); }

// 8 codes to 8 values of 16 bits, exactly: code * 2^k has 7 significant
// bits.  bf16: with m a code's low 7 bits and s its sign bit, 128 + m and
// 128 (1 + s) are bf16 whose bits are those of the code and 0x4300, and the
// code is their difference.  fp16: 1024 + (code + 128) likewise, less 1152.
// (Codes of a block with exponent 255 are 0: times infinity, NaN.)
__device__ __forceinline__ uint4 widen(__nv_bfloat16, const uint2 &w, uint32_t byte) {
    const uint32_t step = byte * 0x00800080u;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = (i < 2 ? w.x : w.y) >> (i & 1 ? 8 : 0);
        const uint32_t m = (pair & 0x007f007fu) | 0x43004300u, s = (pair & 0x00800080u) | 0x43004300u;
        const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&m),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&s));
        const __nv_bfloat162 v = __hmul2(q, *reinterpret_cast<const __nv_bfloat162 *>(&step));
        o[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 widen(__half, const uint2 &w, uint32_t byte) {
    const __half2 step = __float2half2_rn(__uint_as_float(byte << 23));
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = (((i < 2 ? w.x : w.y) >> (i & 1 ? 8 : 0)) & 0x00ff00ffu) ^ 0x64806480u;
        const __half2 q = __hsub2(*reinterpret_cast<const __half2 *>(&pair), __float2half2_rn(1152.0f));
        const __half2 v = __hmul2(q, step);
        o[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The part of the work that one pair does.
struct WgradItem {
    int64_t lo, hi;    // rows
    int64_t c0, o0;    // of the pair's tile
    int32_t group, slot;  // slot < 0: the whole sum, written to the grads
    int32_t n;         // outputs of the product (a multiple of 32)
};

__device__ __forceinline__ WgradItem item_of(const WgradArgs &a, int item) {
    WgradItem it;
    int tile = item, part = 0, parts = 1;
    it.slot = -1;
    if (item >= a.whole) {
        parts = a.split;
        tile = a.whole + (item - a.whole) / parts;
        part = (item - a.whole) % parts;
        if (parts > 1) it.slot = item - a.whole;
    }
    const int per_group = a.tiles_c * a.tiles_o;
    it.group = tile / per_group;
    tile %= per_group;
    it.c0 = int64_t(tile % a.tiles_c) * kTileC;
    it.o0 = int64_t(tile / a.tiles_c) * kTileO;
    it.n = int(min(int64_t(kTileO), (a.outs - it.o0 + 31) / 32 * 32));
    it.lo = 0;
    it.hi = a.dy_rows;
    if (a.offsets) {
        it.lo = min(max(int64_t(a.offsets[it.group]), int64_t(0)), a.dy_rows);
        it.hi = min(max(int64_t(a.offsets[it.group + 1]), it.lo), a.dy_rows);
    }
    if (parts > 1) {
        const int64_t steps = (it.hi - it.lo + kK - 1) / kK;
        const int64_t end = it.hi;
        it.hi = min(end, it.lo + steps * (part + 1) / parts * kK);
        it.lo = min(end, it.lo + steps * part / parts * kK);
    }
    return it;
}

// A CTA's half of 64 rows of dy by plain loads, zeros past the rows and
// columns there are.
template <typename T>
__device__ __forceinline__ void stage_dy(const WgradArgs &a, int64_t r0, int64_t hi, int64_t o0, int n_half,
                                         unsigned char *stage) {
    const T *dy = static_cast<const T *>(a.dy);
    const int chunks = (n_half + 7) / 8;
    for (int i = threadIdx.x % kGroup; i < kK * 16; i += kGroup) {
        const int k = i >> 4, q = i & 15;
        if (q >= chunks) continue;
        const int64_t r = r0 + k, o = o0 + q * 8;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (r < hi && o < a.outs) {
            const T *p = dy + r * a.dy_ld + o;
            if (a.vec && o + 8 <= a.outs) {
                raw = *reinterpret_cast<const uint4 *>(p);
            } else {
                uint16_t e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    e[j] = o + j < a.outs ? reinterpret_cast<const uint16_t *>(p)[j] : uint16_t(0);
                memcpy(&raw, e, sizeof raw);
            }
        }
        *reinterpret_cast<uint4 *>(stage + stage_chunk(k, q)) = raw;
    }
}

// 32 lanes x 16 columns of a CTA's sums to the grads; `any` false: zeros.
template <typename G>
__device__ __forceinline__ void store_sums(const WgradArgs &a, const WgradItem &it, int64_t c, int64_t o,
                                           const float (&f)[16]) {
    if (c >= a.cols) return;
    G *p = static_cast<G *>(a.grad) + a.grad_offset[it.group] + o * a.cols + c;
    if (a.accumulate) {
        G old[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (o + j < a.outs) old[j] = p[j * a.cols];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (o + j < a.outs) p[j * a.cols] = from_f32<G>(to_f32(old[j]) + f[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (o + j < a.outs) p[j * a.cols] = from_f32<G>(f[j]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kWgradThreads, 2) __cluster_dims__(2, 1, 1)
    dopt_ckpt_wgrad_kernel(const __grid_constant__ WgradArgs a) {
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *dy_ring = smem, *x_ring = smem + kDyRing * kStage, *raw_ring = x_ring + kXRing * kStage;
    WgradBarriers &b = *reinterpret_cast<WgradBarriers *>(raw_ring + kRawRing * kRaw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

    let_dependents_start();
    if (threadIdx.x == 0) {
        auto init = [](unsigned long long &bar, int count) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(&bar)), "r"(count) : "memory");
        };
        for (int i = 0; i < kDyRing; ++i) init(b.dy_full[i], 1), init(b.dy_empty[i], 1);
        for (int i = 0; i < kXRing; ++i) init(b.x_full[i], 2 * kGroup / 32), init(b.x_empty[i], 1);
        for (int i = 0; i < kRawRing; ++i) init(b.raw_full[i], 64), init(b.raw_empty[i], kGroup / 32);
        init(b.done, 1);
        b.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {  // all of the pair's CTAs allocate; freed before they end
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&b.tmem)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    wait_for_grids_before();
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = b.tmem;

    const WgradItem it = item_of(a, int(blockIdx.x >> 1));
    const int rows = int(it.hi - it.lo);
    const int steps = (rows + kK - 1) / kK;
    const int tma_steps = a.tma ? rows / kK : 0;
    const int n_half = it.n / 2;
    const int64_t my_o = it.o0 + int64_t(rank) * n_half;
    const int64_t my_c = it.c0 + int64_t(rank) * (kTileC / 2);

    if (warp == kMmaWarp) {
        if (lane == 0 && rank == 0 && steps > 0) {  // the pair's products
            constexpr uint32_t kFormat = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
            const uint32_t idesc = (1u << 4) | (kFormat << 7) | (kFormat << 10) | (1u << 15) | (1u << 16) |
                                   (uint32_t(it.n >> 3) << 17) | (uint32_t(kTileC >> 4) << 24);
            bool ok = true;
            for (int i = 0; i < steps && ok; ++i) {
                const int sd = i % kDyRing, sx = i % kXRing;
                ok = wait_phase(b, b.x_full[sx], uint32_t(i / kXRing) & 1);
                if (ok && i < tma_steps) ok = wait_phase(b, b.dy_full[sd], uint32_t(i / kDyRing) & 1);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const int subs = (min(kK, rows - i * kK) + 15) / 16;
                for (int k = 0; k < subs; ++k) {
                    const uint64_t da = slab_descriptor(smem_of(x_ring + sx * kStage) + k * 2048);
                    const uint64_t db = slab_descriptor(smem_of(dy_ring + sd * kStage) + k * 2048);
                    asm volatile(
                        "{\n\t.reg .pred p;\n\t"
                        "setp.ne.u32 p, %4, 0;\n\t"
                        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
                        "l"(da), "l"(db), "r"(idesc), "r"(uint32_t(i > 0 || k > 0))
                        : "memory");
                }
                auto commit = [](unsigned long long &bar) {  // to both CTAs' barriers
                    asm volatile(
                        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
                        " [%0], %1;" ::"r"(smem_of(&bar)),
                        "h"(uint16_t(3))
                        : "memory");
                };
                commit(b.x_empty[sx]);
                commit(b.dy_empty[sd]);
                if (i == steps - 1) commit(b.done);
            }
        }
    } else if (warp == kDyWarp) {
        if (lane == 0) {  // dy, by TMA into both CTAs, counted on the leader's barriers
            const int boxes = (n_half + 63) / 64;
            for (int i = 0; i < tma_steps; ++i) {
                const int s = i % kDyRing;
                if (i >= kDyRing && !wait_phase(b, b.dy_empty[s], uint32_t(i / kDyRing - 1) & 1)) break;
                const uint32_t full = smem_of(&b.dy_full[s]);
                if (rank == 0)
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full),
                                 "r"(2 * boxes * kSlab)
                                 : "memory");
                for (int x = 0; x < boxes; ++x)
                    asm volatile(
                        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_of(dy_ring + s * kStage + x * kSlab)),
                        "l"(&a.dy_map), "r"(int(my_o) + 64 * x), "r"(int(it.lo) + i * kK), "r"(leader_address(full))
                        : "memory");
            }
            // every arrival on this CTA's barriers has happened before it ends
            drain(b, b.dy_empty, kDyRing, steps);
            drain(b, b.x_empty, kXRing, steps);
        }
    } else if (warp >= kRawWarp) {
        // x: two warps, 32 rows of a step each; lane l has the l-th row's
        // token, loaded for four steps at a time and four steps ahead (looked
        // at only when it is used, so that nothing waits)
        const int row0 = 32 * (warp - kRawWarp);
        const bool any = my_c < a.pitch && a.x_rows > 0;
        const unsigned char *codes = a.codes + my_c + (lane & 7) * 16;
        const unsigned char *scales = a.scales + my_c / kBlock;
        const uint32_t pitch = uint32_t(a.pitch);
        auto token = [&](int i) -> int {
            const int64_t r = it.lo + int64_t(i) * kK + row0 + lane;
            if (r >= it.hi) return -1;
            return a.row_token ? a.row_token[r] : int(r);
        };
        int now[4], next[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) now[u] = token(u);
        bool ok = true;
        for (int i0 = 0; i0 < steps && ok; i0 += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) next[u] = token(i0 + 4 + u);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u;
                if (i >= steps) break;
                const int s = i % kRawRing;
                if (i >= kRawRing) ok = wait_phase(b, b.raw_empty[s], uint32_t(i / kRawRing - 1) & 1);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                const bool there = any && now[u] >= 0 && now[u] < a.x_rows;
                const uint32_t t = there ? uint32_t(now[u]) : 0u;
                // a row that counts as zeros has whatever codes, and exponent bytes 0
                unsigned char *raw = raw_ring + s * kRaw + row0 * 128, *exps = raw_ring + s * kRaw + kRawCodes + (row0 + lane) * 4;
                if (any) {
                    const uint32_t to = smem_of(raw) + lane * 16;
#pragma unroll
                    for (int n = 0; n < 8; ++n)  // 4 rows at a time, 8 lanes a row
                        copy_async<16>(to + n * 512, codes + uint64_t(__shfl_sync(kFull, t, 4 * n + (lane >> 3))) * pitch,
                                       true);
                    copy_async<4>(smem_of(exps), scales + uint64_t(t) * (pitch / kBlock), there);
                } else {
                    *reinterpret_cast<uint32_t *>(exps) = 0;
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_of(&b.raw_full[s]))
                             : "memory");
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) now[u] = next[u];
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // x: half of these warps fill the even steps' stage of the ring, half
        // the odd steps', so that one half's waits, stores and fence run under
        // the other's conversions.  A warp takes two rows at a time, a thread
        // 8 columns: chunk q of rows 2 w + lane / 16 + 8 h.
        const int half = warp / (kGroup / 32), w = warp % (kGroup / 32);
        const int q = lane & 15, k0 = 2 * w + (lane >> 4);
        const uint32_t full = leader_address(smem_of(&b.x_full[half]));
        // 8 rows on: 1024 bytes on, and the swizzle is the same
        unsigned char *stage = x_ring + half * kStage + stage_chunk(k0, q);
        const unsigned char *my_raw = raw_ring + k0 * 128 + q * 8;
        const unsigned char *my_exp = raw_ring + kRawCodes + k0 * 4 + (q >> 2);
        bool ok = true;
        uint32_t phase = 1;  // of the stage (a new barrier passes a wait for phase 1)
        for (int i = half; i < steps; i += kXRing, phase ^= 1) {
            const int sr = i % kRawRing;
            // the other half is done with this slot: only then is the parity of
            // its phase this step's (a ring of 3 alternates between the halves)
            ok = i < kRawRing || wait_phase(b, b.raw_empty[sr], uint32_t(i / kRawRing - 1) & 1);
            ok = ok && wait_phase(b, b.raw_full[sr], uint32_t(i / kRawRing) & 1);
            const unsigned char *raw = my_raw + sr * kRaw, *exp = my_exp + sr * kRaw;
            uint4 v[4];
#pragma unroll
            for (int h = 0; h < 4; ++h)
                v[h] = widen(T(), *reinterpret_cast<const uint2 *>(raw + h * 1024), exp[h * 32]);
            ok = wait_phase(b, b.x_empty[half], phase) && ok;
            if (i >= tma_steps && i >= kDyRing && ok)
                ok = wait_phase(b, b.dy_empty[i % kDyRing], uint32_t(i / kDyRing - 1) & 1);
            if (!__all_sync(kFull, ok)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) *reinterpret_cast<uint4 *>(stage + h * 1024) = v[h];
#pragma unroll
            for (int h = 4; h < 8; ++h)
                *reinterpret_cast<uint4 *>(stage + h * 1024) =
                    widen(T(), *reinterpret_cast<const uint2 *>(raw + h * 1024), exp[h * 32]);
            if (i >= tma_steps)
                stage_dy<T>(a, it.lo + int64_t(i) * kK, it.hi, my_o, n_half, dy_ring + (i % kDyRing) * kStage);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_of(&b.raw_empty[sr])) : "memory");
                arrive_remote(full);
            }
        }
        // the sums: warp w reads the 32 lanes that are its own (w % 4) and half of the columns
        if (steps > 0) {
            ok = ok && wait_phase(b, b.done, 0);
            ok = __all_sync(kFull, ok);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        }
        if (ok) {
            const int quad = warp & 3;
            const int m = int(rank) * (kTileC / 2) + quad * 32 + lane;
            const int cols = it.n / 2;
            for (int o = (warp >> 2) * cols; o < ((warp >> 2) + 1) * cols; o += 16) {
                float f[16] = {};
                if (steps > 0) {
                    uint32_t r[16];
                    asm volatile(
                        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
                        "%12, %13, %14, %15}, [%16];"
                        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
                          "=r"(r[14]), "=r"(r[15])
                        : "r"(tmem + (uint32_t(quad * 32) << 16) + uint32_t(o)));
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int q = 0; q < 16; ++q) f[q] = __uint_as_float(r[q]);
                }
                if (it.slot >= 0) {
                    float *p = a.partial + it.slot * (kSlotBytes / 4) + int64_t(o) * kTileC + m;
#pragma unroll
                    for (int q = 0; q < 16; ++q) p[q * kTileC] = f[q];
                } else if (a.grad_dtype == DOPT_FP32) {
                    store_sums<float>(a, it, it.c0 + column_of(m), it.o0 + o, f);
                } else if (a.grad_dtype == DOPT_BF16) {
                    store_sums<__nv_bfloat16>(a, it, it.c0 + column_of(m), it.o0 + o, f);
                } else {
                    store_sums<__half>(a, it, it.c0 + column_of(m), it.o0 + o, f);
                }
            }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
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
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
    }
}

// The split tiles' parts, added in the order of the rows and written.
// blockIdx.x: tile, blockIdx.y: 16 of its outputs; a thread: one column.
template <typename G>
__global__ void __launch_bounds__(kTileC) dopt_ckpt_wgrad_join_kernel(const __grid_constant__ WgradArgs a) {
    let_dependents_start();
    wait_for_grids_before();
    const WgradItem it = item_of(a, a.whole + int(blockIdx.x) * a.split);
    const int o = int(blockIdx.y) * 16;
    if (o >= it.n) return;
    float f[16] = {};
    for (int s = 0; s < a.split; ++s) {
        const float *p = a.partial + (it.slot + s) * (kSlotBytes / 4) + int64_t(o) * kTileC + threadIdx.x;
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = __ldcs(p + q * kTileC);
#pragma unroll
        for (int q = 0; q < 16; ++q) f[q] += v[q];
    }
    store_sums<G>(a, it, it.c0 + column_of(threadIdx.x), it.o0 + o, f);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// How the tiles go over `pairs` pairs of SMs.  Whole waves of tiles are done
// tile by tile; the last, partial wave's tiles are split along the rows into
// the number of parts whose estimated time is least, in steps of 64 rows: a
// wave of parts is steps / parts, the join's launch takes about as long as 11
// steps and a part's trip through memory 0.2.
struct Split {
    int64_t whole, tail;
    int parts;
};
Split plan_split(int64_t tiles, int64_t steps, int64_t pairs, int64_t workspace_bytes) {
    Split best{tiles, 0, 1};
    const int64_t tail = tiles % pairs;
    if (tail == 0) return best;
    double least = double(steps);
    for (int s = 2; s <= kMaxSplit && steps / s >= 4; ++s) {
        if (tail * s * kSlotBytes > workspace_bytes) break;
        const double t = double((tail * s + pairs - 1) / pairs) * double(steps) / s + 11.0 + 0.2 * double(tail * s);
        if (t < least) {
            least = t;
            best = Split{tiles - tail, tail, s};
        }
    }
    return best;
}

int64_t tiles_of(int64_t outs, int64_t cols, int n_groups) {
    return (outs + kTileO - 1) / kTileO * ((cols + kTileC - 1) / kTileC) * n_groups;
}
int64_t steps_of(int64_t dy_rows, int n_groups) { return (dy_rows / n_groups + kK - 1) / kK; }

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::mutex g_wgrad_mutex;
EncodeTiled g_encode = nullptr;
int g_pairs[64] = {};  // pairs of SMs of a device, once its kernels are set up

// The tensor-map encoder, the kernels' shared-memory limit and the device's
// number of SM pairs, looked up once per device.
int set_up(const char *who, EncodeTiled *encode, int *pairs) {
    using dopt::fail;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess && (device < 0 || device >= 64)) return fail(DOPT_E_ARG, "%s: device %d", who, device);
    std::lock_guard<std::mutex> lock(g_wgrad_mutex);
    if (e == cudaSuccess && !g_encode) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found{};
        e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        if (e == cudaSuccess && (found != cudaDriverEntryPointSuccess || !f))
            return fail(DOPT_E_CUDA, "%s: the driver has no tensor maps", who);
        if (e == cudaSuccess) g_encode = reinterpret_cast<EncodeTiled>(f);
    }
    if (e == cudaSuccess && g_pairs[device] == 0) {
        int sms = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(dopt_ckpt_wgrad_kernel<__nv_bfloat16>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, int(kWgradSmem));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(dopt_ckpt_wgrad_kernel<__half>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     int(kWgradSmem));
        if (e == cudaSuccess) g_pairs[device] = std::max(1, sms / 2);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(DOPT_E_CUDA, "%s: set-up: %s", who, cudaGetErrorString(e));
    }
    *encode = g_encode;
    *pairs = g_pairs[device];
    return DOPT_OK;
}

template <typename T>
int launch_wgrad(const char *who, const WgradArgs &a, int64_t items, int64_t tail, cudaStream_t stream) {
    int rc = launch_op(who, dopt_ckpt_wgrad_kernel<T>, dim3(unsigned(2 * items)), dim3(kWgradThreads), kWgradSmem,
                       stream, a);
    if (rc != DOPT_OK || a.split == 1) return rc;
    const dim3 grid(unsigned(tail), kTileO / 16);
    switch (a.grad_dtype) {
        case DOPT_BF16: return launch_op(who, dopt_ckpt_wgrad_join_kernel<__nv_bfloat16>, grid, dim3(kTileC), 0, stream, a);
        case DOPT_FP16: return launch_op(who, dopt_ckpt_wgrad_join_kernel<__half>, grid, dim3(kTileC), 0, stream, a);
        default: return launch_op(who, dopt_ckpt_wgrad_join_kernel<float>, grid, dim3(kTileC), 0, stream, a);
    }
}

// Whether the groups' stretches of n grads do not overlap.
bool apart(const int64_t *offsets, int n_groups, int64_t n) {
    bool rising = true;
    for (int g = 1; g < n_groups && rising; ++g) rising = offsets[g] >= offsets[g - 1] + n;
    if (rising) return true;
    int64_t sorted[DOPT_MAX_GROUPS];
    std::copy(offsets, offsets + n_groups, sorted);
    std::sort(sorted, sorted + n_groups);
    for (int g = 1; g < n_groups; ++g)
        if (sorted[g] < sorted[g - 1] + n) return false;
    return true;
}

}  // namespace

extern "C" int dopt_ckpt_wgrad(const void *ckpt, dopt_dtype ckpt_dtype, int64_t x_rows, int64_t cols,
                               const int32_t *row_token, const void *dy, dopt_dtype dy_dtype,
                               int64_t dy_rows, int64_t outs, int64_t dy_ld, const int32_t *offsets,
                               int32_t n_groups, const int64_t *grad_offsets, void *grad,
                               dopt_dtype grad_dtype, int64_t grad_numel, uint32_t flags,
                               void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_ckpt_wgrad";
    OpRange range(who);
    if (x_rows < 0 || x_rows > INT32_MAX || cols < 1 || cols > DOPT_MAX_COLS || dy_rows < 0 ||
        dy_rows > INT32_MAX || outs < 1 || outs > DOPT_MAX_COLS || dy_ld < outs)
        return fail(DOPT_E_ARG, "%s: checkpoint %lld x %lld, dy %lld x %lld, row stride %lld", who,
                    static_cast<long long>(x_rows), static_cast<long long>(cols),
                    static_cast<long long>(dy_rows), static_cast<long long>(outs),
                    static_cast<long long>(dy_ld));
    if (!valid_dtype(ckpt_dtype) || !valid_dtype(grad_dtype))
        return fail(DOPT_E_ARG, "%s: unknown dtype", who);
    if (dy_dtype != DOPT_BF16 && dy_dtype != DOPT_FP16)
        return fail(DOPT_E_ARG, "%s: dy must be bf16 or fp16", who);
    if (dy_dtype == DOPT_FP16 && ckpt_dtype != DOPT_FP16)
        return fail(DOPT_E_ARG, "%s: fp16 dy needs a checkpoint of fp16 values", who);
    if (flags & ~uint32_t(DOPT_WGRAD_ACCUMULATE))
        return fail(DOPT_E_ARG, "%s: unknown flags 0x%x", who, flags);
    if (n_groups < 1 || n_groups > DOPT_MAX_GROUPS || (!offsets && n_groups != 1))
        return fail(DOPT_E_ARG, "%s: n_groups %d (1..%d, 1 without offsets)", who, n_groups, DOPT_MAX_GROUPS);
    if (!row_token && dy_rows > x_rows)
        return fail(DOPT_E_ARG, "%s: %lld rows of dy for %lld of the checkpoint and no row_token", who,
                    static_cast<long long>(dy_rows), static_cast<long long>(x_rows));
    if (!grad_offsets || !grad) return fail(DOPT_E_ARG, "%s: NULL grad or grad_offsets", who);
    if ((x_rows > 0 && !ckpt) || (dy_rows > 0 && !dy))
        return fail(DOPT_E_ARG, "%s: NULL checkpoint or dy", who);
    if (!aligned_to(ckpt, 16)) return fail(DOPT_E_ALIGN, "%s: checkpoint is not 16-byte aligned", who);
    if (!aligned_to(dy, 2) || !aligned_to(grad, elem_bytes(grad_dtype)) || !aligned_to(offsets, 4) ||
        !aligned_to(row_token, 4))
        return fail(DOPT_E_ALIGN, "%s: dy, grad, offsets or row_token is not aligned to its elements", who);
    if (workspace_bytes < 0 || (workspace_bytes > 0 && !workspace))
        return fail(DOPT_E_ARG, "%s: NULL workspace of %lld bytes", who, static_cast<long long>(workspace_bytes));
    if (!aligned_to(workspace, 16)) return fail(DOPT_E_ALIGN, "%s: workspace is not 16-byte aligned", who);
    const int64_t n = outs * cols;  // below 2^44
    WgradArgs a{};
    for (int g = 0; g < n_groups; ++g) {
        if (grad_offsets[g] < 0 || grad_offsets[g] > grad_numel - n)
            return fail(DOPT_E_ARG, "%s: group %d's %lld grads at %lld leave a buffer of %lld", who, g,
                        static_cast<long long>(n), static_cast<long long>(grad_offsets[g]),
                        static_cast<long long>(grad_numel));
        a.grad_offset[g] = grad_offsets[g];
    }
    if (!apart(grad_offsets, n_groups, n))
        return fail(DOPT_E_ARG, "%s: two groups' grads overlap", who);
    a.pitch = ckpt_pitch(cols);
    a.codes = static_cast<const uint8_t *>(ckpt);
    a.scales = a.codes + x_rows * a.pitch;
    a.row_token = row_token;
    a.dy = dy;
    a.offsets = offsets;
    a.grad = grad;
    a.x_rows = x_rows;
    a.cols = cols;
    a.dy_rows = dy_rows;
    a.outs = outs;
    a.dy_ld = dy_ld;
    a.accumulate = (flags & DOPT_WGRAD_ACCUMULATE) != 0;
    a.vec = aligned_to(dy, 16) && dy_ld * 2 % 16 == 0;
    a.grad_dtype = grad_dtype;
    EncodeTiled encode = nullptr;
    int pairs = 0;
    int rc = set_up(who, &encode, &pairs);
    if (rc != DOPT_OK) return rc;
    if (a.vec && dy_rows > 0) {  // 16-byte aligned rows go by TMA
        const cuuint64_t dims[2] = {cuuint64_t(outs), cuuint64_t(dy_rows)};
        const cuuint64_t strides[1] = {cuuint64_t(dy_ld) * 2};
        const cuuint32_t box[2] = {64, kK}, unit[2] = {1, 1};
        const CUresult r = encode(&a.dy_map,
                                  dy_dtype == DOPT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                  2, const_cast<void *>(dy), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        a.tma = r == CUDA_SUCCESS;  // a stride past the map's limit: plain loads
    }
    const int64_t tiles = tiles_of(outs, cols, n_groups);
    const Split split = plan_split(tiles, steps_of(dy_rows, n_groups), pairs, workspace_bytes);
    const int64_t items = split.whole + split.tail * split.parts;
    if (items > INT32_MAX / 2) return fail(DOPT_E_ARG, "%s: %lld tiles", who, static_cast<long long>(tiles));
    a.tiles_c = int32_t((cols + kTileC - 1) / kTileC);
    a.tiles_o = int32_t((outs + kTileO - 1) / kTileO);
    a.whole = int32_t(split.whole);
    a.split = split.parts;
    a.partial = static_cast<float *>(workspace);
    if (dy_dtype == DOPT_BF16) return launch_wgrad<__nv_bfloat16>(who, a, items, split.tail, stream);
    return launch_wgrad<__half>(who, a, items, split.tail, stream);
}

extern "C" int dopt_ckpt_wgrad_workspace(int64_t dy_rows, int64_t outs, int64_t cols,
                                         int32_t n_groups, int64_t *bytes) {
    dopt::clear_error();
    const char *who = "dopt_ckpt_wgrad_workspace";
    if (!bytes) return dopt::fail(DOPT_E_ARG, "%s: bytes is NULL", who);
    if (dy_rows < 0 || dy_rows > INT32_MAX || outs < 1 || outs > DOPT_MAX_COLS || cols < 1 ||
        cols > DOPT_MAX_COLS || n_groups < 1 || n_groups > DOPT_MAX_GROUPS)
        return dopt::fail(DOPT_E_ARG, "%s: %lld rows, %lld x %lld, %d groups", who,
                          static_cast<long long>(dy_rows), static_cast<long long>(outs),
                          static_cast<long long>(cols), n_groups);
    // for a device of 76 pairs of SMs; a call takes what it is given
    const Split split = plan_split(tiles_of(outs, cols, n_groups), steps_of(dy_rows, n_groups), 76, INT64_MAX);
    *bytes = split.parts > 1 ? split.tail * split.parts * kSlotBytes : 0;
    return DOPT_OK;
}

extern "C" int dopt_wgrad_timeouts(int reset, uint32_t *count) {
    using dopt::fail;
    dopt::clear_error();
    if (!count) return fail(DOPT_E_ARG, "dopt_wgrad_timeouts: NULL output");
    unsigned int c = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&c, g_wgrad_timeouts, sizeof c);
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_wgrad_timeouts, &zero, sizeof zero);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(DOPT_E_CUDA, "dopt_wgrad_timeouts: %s", cudaGetErrorString(e));
    }
    *count = c;
    return DOPT_OK;
}
