// The weight gradients of a linear layer, or of a layer's experts, from the
// 8-bit checkpoint of its input, written into the flat grad buffer
// (dopt_ckpt_wgrad; dopt.h states the contract).
#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "rows.cuh"

namespace {

// A pair of CTAs (a cluster of two, one CTA an SM) goes through tiles of 256
// columns c by NB * 256 outputs o of one group's gradient, with
// tcgen05.mma.cta_group::2: M = c, N = o, K = the group's rows in steps of
// 64.  Each CTA keeps 128 of the c (operand A) and half of the o (operand B)
// in shared memory, both as they lie in memory, rows of K with M or N
// contiguous, in slabs of 64 columns x 64 rows with the 128-byte swizzle.
//
//   dy  bf16 / fp16, by TMA (a ring of 8 blocks of 256 o); by the warps that
//       widen codes in a group's last step, whose rows past the group must read
//       as zeros whatever the next group holds there (copies of 16 bytes, in
//       flight under the conversions), and where rows are not 16-byte aligned
//       (plain loads)
//   x   16 warps load 16 codes a thread and row into registers, widen them to
//       16 bits (exactly) and store them swizzled (a ring of 4 steps).  Four
//       warps take a step, so that one step's waits, stores and fence run
//       under another's conversions; a warp loads its next step's codes after
//       the fence that ends a step and finds them there four steps later.  A
//       row that counts as zeros has exponent bytes 0.
//
// The sums are fp32 in tensor memory, 128 lanes x 512 columns a CTA: NB = 1
// uses it for two tiles in turn, four warps storing one while the other is
// summed; NB = 2 for one tile of twice the outputs, so that codes are widened
// once for two products, and its stores are waited for.  With lanes along c
// the stores of a warp are contiguous.
//
// The tensor cores add 16 rows' products to a sum at a time and cut off what
// its 24 bits do not hold, always toward zero: the error of one long sum grows
// as its rows do (fp32 grads of 16384 rows were 1.1e-5 off with bf16 dy, 1.8e-5
// with fp16, where fp32 additions that round are off by 2-4e-7).  So a sum takes
// `chunk` steps; the four storing warps then add it to the tile's first sum,
// rounding to nearest, and it starts anew.  Both are in tensor memory, with
// NB = 1: the other buffer, once the tile before is stored.  sum_chunk has
// the rows and why.  16384 rows x 5632 columns x 2048 outputs with fp32 grads
// take 254 us so (195 in one sum of NB = 2).
//
// Long sums are bound by the tensor cores: 16384 rows x 5632 columns x 2048
// outputs, bf16, take 200-204 us (1.89 PFLOP/s; 222-227 us, 1.68, where the
// card's power limits it).  Many short groups are bound by the steps' latency (codes
// of a step's rows arrive, are widened and fenced, 4 steps at a time) and by
// the stores, together: 64 experts of about 1024 rows x 512 columns x 1408
// outputs, fp32 grads, take 99-101 us (0.95 PFLOP/s, 3.8 TB/s; 93 in one sum).
// Adding to old grads is bound by their loads, 4 in flight a thread: 449 us there.
constexpr int kTileC = 256;          // of a pair
constexpr int kTileO = 256;          // of a product; a tile has NB of them
constexpr int kK = 64;               // rows a step
constexpr int kDyRing = 8;
constexpr int kXRing = 4;
constexpr int kSlab = kK * 128;      // 64 columns x 64 rows of 16 bits
constexpr int kStage = 2 * kSlab;    // a CTA's 128 columns
constexpr int kGroups = 4;           // of warps that widen codes
constexpr int kGroup = 128;          // threads of one
constexpr int kWorkers = kGroups * kGroup;
constexpr int kStoreWarp = kWorkers / 32, kMmaWarp = kStoreWarp + 4, kDyWarp = kMmaWarp + 1;
constexpr int kWgradThreads = 32 * (kDyWarp + 1);
constexpr int kTmemCols = 512;
constexpr int kMaxSplit = 16;
static_assert(kStoreWarp % 4 == 0, "a warp reads the tensor-memory lanes of its place in four");

struct WgradBarriers {
    unsigned long long dy_full[kDyRing], dy_empty[kDyRing], x_full[kXRing], x_empty[kXRing];
    unsigned long long sum_full[2], sum_empty[2];
    uint32_t tmem;
    int32_t failed;
};
// The groups' first rows and, with several groups, the groups from the one
// with the most rows down.
struct WgradGroups {
    int32_t first[DOPT_MAX_GROUPS + 1];
    int32_t order[DOPT_MAX_GROUPS];
};
constexpr size_t kWgradSmem =
    (kDyRing + kXRing) * size_t(kStage) + sizeof(WgradBarriers) + sizeof(WgradGroups);
static_assert(kWgradSmem <= 232448, "a CTA's 227 KB");

__host__ __device__ constexpr int64_t slot_floats(int nb) { return int64_t(kTileC) * kTileO * nb; }

struct WgradArgs {
    CUtensorMap dy_map;        // with `tma`
    const uint8_t *codes, *scales;
    const int32_t *row_token;  // or NULL: row r reads checkpoint row r
    const void *dy;
    const int32_t *offsets;    // or NULL: one group of all rows
    void *grad;
    float *partial;            // fp32 sums of the split tiles, [slot][o][c]
    int64_t cols, pitch, dy_ld;
    int32_t x_rows, dy_rows, outs, groups;
    int32_t tiles_c, tiles_o;
    int32_t items;             // tiles and parts of tiles
    int32_t whole;             // tiles before the split ones
    int32_t split;             // parts of a split tile
    int32_t chunk;             // steps of a sum
    int32_t accumulate;
    int32_t tma, vec;          // dy by TMA; dy's rows are 16-byte aligned
    int32_t grad_dtype;
    int64_t grad_offset[DOPT_MAX_GROUPS];
};

// CTAs with a wait that ran past its limit (a copy or product that never
// completed).  Such a pair ends its work; the grads that it has not written
// become NaN, parts of split sums too, which carry it into theirs.
__device__ unsigned int g_wgrad_timeouts;
constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s
constexpr uint32_t kNanBits = 0x7fffffffu;

#ifdef DOPT_DEVICE_CHECKS
// Test build only: the first pair issues the products of so many of its items
// (-1: of all), so that the waits for the next one's run out
// (dopt_wgrad_wait_test).
__device__ int g_wgrad_items = -1;
__device__ __forceinline__ bool products_withheld(int round) {
    return blockIdx.x == 0 && g_wgrad_items >= 0 && round >= g_wgrad_items;
}
#else
__device__ __forceinline__ bool products_withheld(int) { return false; }
#endif

__device__ __forceinline__ uint32_t smem_of(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

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
// (Warps that poll take issue slots from those that work: where a wait is
// long and its end not urgent, they sleep between two tries.)
template <int SLEEP_NS>
__device__ __noinline__ bool wait_long(WgradBarriers &b, uint32_t bar, uint32_t parity) {
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
            if (atomicExch(&b.failed, 1) == 0) atomicAdd(&g_wgrad_timeouts, 1u);
            return false;
        }
    }
}
template <int SLEEP_NS = 0>
__device__ __forceinline__ bool wait_phase(WgradBarriers &b, unsigned long long &bar, uint32_t parity) {
    const uint32_t at = smem_of(&bar);
    for (int i = 0; i < (SLEEP_NS > 0 ? 1 : 16); ++i)
        if (try_phase(at, parity)) return true;
    return wait_long<SLEEP_NS>(b, at, parity);
}

// Wait for the last of `uses` uses of each slot of a ring.
__device__ __forceinline__ void drain(WgradBarriers &b, unsigned long long *empty, int ring, int uses) {
    for (int s = 0; s < ring && s < uses; ++s)
        if (!wait_phase(b, empty[s], uint32_t((uses - 1 - s) / ring) & 1)) return;
}

// A value that is the same in all lanes, and known to be.
template <typename V>
__device__ __forceinline__ V uniform(V v) {
    return __shfl_sync(kFull, v, 0);
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t leader_address(uint32_t own) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(own));
    return r;
}
// An arrival on the leader's barrier that releases, at the cluster's scope, what
// this warp stored in shared memory before; that is all that its waiter reads
// (sums leave tensor memory before tcgen05.fence::before_thread_sync).  A
// release of all memory would wait for the grads' stores and a trip to L2 at
// every step: 220 us where this takes 200 (16384 rows x 5632 x 2048), 118 and 94
// for 64 experts.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_address) {
    asm volatile(
        "fence.release.sync_restrict::shared::cta.cluster;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_address)
        : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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
// bytes 0 and 2 of a word of codes, and 1 and 3, are then its pairs.
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
        const uint32_t pair = __byte_perm(i < 2 ? w.x : w.y, 0x43434343u, i & 1 ? 0x4341 : 0x4240);
        const uint32_t m = pair & 0xff7fff7fu, s = pair & 0xff80ff80u;
        uint32_t code;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(code) : "r"(s), "r"(0xbf80bf80u), "r"(m));      // m - s
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o[i]) : "r"(code), "r"(step), "r"(0x80008000u));  // times step
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 widen(__half, const uint2 &w, uint32_t byte) {
    const __half2 step = __float2half2_rn(__uint_as_float(byte << 23));
    const uint2 u = make_uint2(w.x ^ 0x80808080u, w.y ^ 0x80808080u);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = __byte_perm(i < 2 ? u.x : u.y, 0x64646464u, i & 1 ? 0x4341 : 0x4240);
        const __half2 q = __hsub2(*reinterpret_cast<const __half2 *>(&pair), __float2half2_rn(1152.0f));
        const __half2 v = __hmul2(q, step);
        o[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A tile, or a part of one.
struct WgradItem {
    int32_t lo, rows;     // rows of dy
    int32_t c0, o0;
    int32_t group, slot;  // slot < 0: the whole sum, written to the grads
    int32_t steps, full;  // of 64 rows, and those that are full
    int32_t blocks;       // products of up to 256 outputs
};

// The item that pair p of `pairs` takes in round k: the rounds' order turns
// back and forth, which, with the groups in order of falling length, gives
// the pairs nearly equal shares (1.07 times the mean for 64 experts of 30 to
// 3000 rows, where rounds in one order gave 1.33).  Negative: none is left.
__device__ __forceinline__ int item_number(const WgradArgs &a, int k) {
    const int pairs = int(gridDim.x >> 1), p = int(blockIdx.x >> 1);
    const int item = k * pairs + (k & 1 ? pairs - 1 - p : p);
    return item < a.items ? item : -1;
}

template <int NB>
__device__ __forceinline__ WgradItem item_of(const WgradArgs &a, const WgradGroups &g, int item) {
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
    it.group = g.order[tile / per_group];
    tile %= per_group;
    it.c0 = tile % a.tiles_c * kTileC;
    it.o0 = tile / a.tiles_c * (kTileO * NB);
    it.blocks = a.outs - it.o0 > kTileO ? NB : 1;
    it.lo = g.first[it.group];
    it.rows = max(0, g.first[it.group + 1] - it.lo);
    if (parts > 1) {
        const int steps = (it.rows + kK - 1) / kK;
        const int from = int(int64_t(steps) * part / parts * kK), to = int(int64_t(steps) * (part + 1) / parts * kK);
        it.lo += from;
        it.rows = min(it.rows, to) - from;
    }
    it.steps = (it.rows + kK - 1) / kK;
    it.full = it.rows / kK;
    return it;
}

// The groups' tables, by all threads of the CTA.
__device__ __forceinline__ void fill_groups(const WgradArgs &a, WgradGroups &g) {
    for (int e = threadIdx.x; e <= a.groups; e += blockDim.x)
        g.first[e] = a.offsets ? min(max(a.offsets[e], 0), a.dy_rows) : e * a.dy_rows;
    __syncthreads();
    for (int e = threadIdx.x; e < a.groups; e += blockDim.x) {
        const int rows = g.first[e + 1] - g.first[e];
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) {
            const int other = g.first[o + 1] - g.first[o];
            rank += other > rows || (other == rows && o < e);
        }
        g.order[rank] = e;
    }
}

// Outputs of a tile's product nb: a multiple of 32.
__device__ __forceinline__ int block_outs(const WgradArgs &a, const WgradItem &it, int nb) {
    return min(kTileO, (a.outs - it.o0 - nb * kTileO + 31) / 32 * 32);
}

// A CTA's half of 64 rows of dy, zeros past the rows and columns there are, by
// a group's threads: aligned rows by asynchronous copies of 16 bytes, all in
// flight until copies_done, others by plain loads.
template <typename T>
__device__ __forceinline__ void stage_dy(const WgradArgs &a, int r0, int rows, int o0, int n_half,
                                         unsigned char *stage) {
    const T *dy = static_cast<const T *>(a.dy);
    const int chunks = (n_half + 7) / 8;
    for (int i = threadIdx.x % kGroup; i < kK * 16; i += kGroup) {
        const int k = i >> 4, q = i & 15;
        if (q >= chunks) continue;
        const int o = o0 + q * 8, n = k < rows ? min(8, max(0, a.outs - o)) : 0;
        const T *p = n > 0 ? dy + (r0 + k) * a.dy_ld + o : dy;
        if (a.vec) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_of(stage + stage_chunk(k, q))),
                         "l"(p), "r"(2 * n)
                         : "memory");
            continue;
        }
        uint16_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = j < n ? reinterpret_cast<const uint16_t *>(p)[j] : uint16_t(0);
        uint4 raw;
        memcpy(&raw, e, sizeof raw);
        *reinterpret_cast<uint4 *>(stage + stage_chunk(k, q)) = raw;
    }
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The dy of step i of the item of round k, block u of all on, into slots
// whose last products are done.
template <typename T, int NB>
__device__ __forceinline__ bool stage_step(const WgradArgs &a, const WgradGroups &g, WgradBarriers &b,
                                        unsigned char *dy_ring, int k, int i, int u, uint32_t rank) {
    const WgradItem it = item_of<NB>(a, g, item_number(a, k));
    bool ok = true;
    for (int nb = 0; nb < it.blocks; ++nb, ++u) {
        const int n_half = block_outs(a, it, nb) / 2;
        if (u >= kDyRing) ok = wait_phase(b, b.dy_empty[u % kDyRing], uint32_t(u / kDyRing - 1) & 1);
        if (!__all_sync(kFull, ok)) return false;
        stage_dy<T>(a, it.lo + i * kK, it.rows - i * kK, it.o0 + nb * kTileO + int(rank) * n_half, n_half,
                    dy_ring + (u % kDyRing) * kStage);
    }
    return true;
}

// 16 outputs' sums of one column, of which `n` are outputs, to the grads from p on.
template <typename G>
__device__ __forceinline__ void store_sums(const WgradArgs &a, G *p, int n, const float (&f)[16]) {
    if (a.accumulate) {
#pragma unroll
        for (int j0 = 0; j0 < 16; j0 += 4) {
            G old[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j0 + j < n) old[j] = p[j * a.cols];
#pragma unroll
            for (int j = 0; j < 4; ++j, p += a.cols)
                if (j0 + j < n) *p = from_f32<G>(to_f32(old[j]) + f[j0 + j]);
        }
    } else if (n >= 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j, p += a.cols) *p = from_f32<G>(f[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j, p += a.cols)
            if (j < n) *p = from_f32<G>(f[j]);
    }
}

// The grad of column c and the tile's first output.
template <typename G>
__device__ __forceinline__ G *grad_at(const WgradArgs &a, const WgradItem &it, int c) {
    return static_cast<G *>(a.grad) + a.grad_offset[it.group] + it.o0 * a.cols + c;
}

// 32 lanes x 16 columns of tensor memory, in flight until wait_sums.
__device__ __forceinline__ void load_sums(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
__device__ __forceinline__ void wait_sums(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// 16 columns back to tensor memory, in flight until tcgen05.wait::st.
__device__ __forceinline__ void put_sums(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// A warp's 32 lanes of the sums at `from` added to those at `into`.
__device__ __forceinline__ void add_tile(uint32_t into, uint32_t from, int outs) {
    for (int o = 0; o < outs; o += 16) {  // (outs is a multiple of 32)
        uint32_t r[16], more[16];
        load_sums(into + uint32_t(o), r);
        load_sums(from + uint32_t(o), more);
        wait_sums(r);
        wait_sums(more);
#pragma unroll
        for (int q = 0; q < 16; ++q) r[q] = __float_as_uint(__uint_as_float(r[q]) + __uint_as_float(more[q]));
        put_sums(into + uint32_t(o), r);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A tile's sums of a warp's 32 columns, at `sums` in tensor memory, to the
// grads; `fill` instead of them where there are none.
template <typename G>
__device__ __forceinline__ void store_tile(const WgradArgs &a, const WgradItem &it, int c, int outs, uint32_t sums,
                                           bool there_are, uint32_t fill) {
    G *p = grad_at<G>(a, it, c);
    const int there = c < a.cols ? a.outs - it.o0 : 0;
    for (int o = 0; o < outs; o += 32) {  // (outs is a multiple of 32)
        uint32_t r[2][16];
#pragma unroll
        for (int q = 0; q < 16; ++q) r[0][q] = r[1][q] = fill;
        if (there_are) {
            load_sums(sums + uint32_t(o), r[0]);
            load_sums(sums + uint32_t(o + 16), r[1]);
            wait_sums(r[0]);
            wait_sums(r[1]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h, p += 16 * a.cols) {
            float f[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) f[q] = __uint_as_float(r[h][q]);
            store_sums(a, p, there - o - 16 * h, f);
        }
    }
}

template <typename T, int NB>
__global__ void __launch_bounds__(kWgradThreads, 1) __cluster_dims__(2, 1, 1)
    dopt_ckpt_wgrad_kernel(const __grid_constant__ WgradArgs a) {
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *dy_ring = smem, *x_ring = smem + kDyRing * kStage;
    WgradBarriers &b = *reinterpret_cast<WgradBarriers *>(x_ring + kXRing * kStage);
    WgradGroups &groups = *reinterpret_cast<WgradGroups *>(&b + 1);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

    let_dependents_start();
    if (threadIdx.x == 0) {
        auto init = [](unsigned long long &bar, int count) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(&bar)), "r"(count) : "memory");
        };
        for (int i = 0; i < kDyRing; ++i) init(b.dy_full[i], 1), init(b.dy_empty[i], 1);
        for (int i = 0; i < kXRing; ++i) init(b.x_full[i], 2 * kGroup / 32), init(b.x_empty[i], 1);
        for (int i = 0; i < 2; ++i) init(b.sum_full[i], 1), init(b.sum_empty[i], 2 * 4);
        b.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {  // both of the pair's CTAs allocate; freed before they end
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&b.tmem)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    wait_for_grids_before();
    fill_groups(a, groups);
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = b.tmem;

    // Every role walks the same items.  n counts steps, u blocks of dy and t
    // tiles that have rows: a ring's slot and phase follow from them.
    if (warp == kDyWarp) {
        // dy, by TMA into both CTAs, counted on the leader's barriers
        int n = 0, u = 0;
        bool ok = true;
        for (int k = 0, item; ok && (item = item_number(a, k)) >= 0; ++k) {
            const WgradItem it = item_of<NB>(a, groups, item);
            const int steps = uniform(it.steps), full_steps = a.tma ? uniform(it.full) : 0;
            const int blocks = it.blocks;  // (of the item's number alone)
            const int outs[2] = {block_outs(a, it, 0), blocks > 1 ? block_outs(a, it, 1) : 0};
            int row = uniform(it.lo);
            for (int i = 0; i < steps && ok; ++i, ++n, row += kK) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if (nb >= blocks) break;
                    const int s = u % kDyRing;
                    if (u >= kDyRing) ok = __all_sync(kFull, wait_phase<64>(b, b.dy_empty[s], uint32_t(u / kDyRing - 1) & 1));
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t full = smem_of(&b.dy_full[s]);
                        // the steps that are not full are stored by the widening warps
                        const int boxes = i < full_steps ? (outs[nb] / 2 + 63) / 64 : 0;
                        if (rank == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full),
                                         "r"(2 * boxes * kSlab)
                                         : "memory");
                        for (int x = 0; x < boxes; ++x)
                            asm volatile(
                                "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::"
                                "bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_of(dy_ring + s * kStage + x * kSlab)),
                                "l"(&a.dy_map), "r"(it.o0 + nb * kTileO + int(rank) * (outs[nb] / 2) + 64 * x),
                                "r"(row), "r"(leader_address(full))
                                : "memory");
                    }
                    __syncwarp();
                    ++u;
                }
            }
        }
        // every arrival on this CTA's barriers has happened before it ends
        if (ok) drain(b, b.dy_empty, kDyRing, u), drain(b, b.x_empty, kXRing, n);
    } else if (warp == kMmaWarp) {
        // The pair's products.  The whole warp walks the steps and one lane
        // issues: operands that are the same in all lanes go to a product
        // without the loop that a lane of its own would need (the products of
        // a step then took 1180 cycles to issue and 512 to compute).
        if (rank == 0) {
            constexpr uint32_t kFormat = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
            constexpr uint32_t kInstruction = (1u << 4) | (kFormat << 7) | (kFormat << 10) | (1u << 15) | (1u << 16) |
                                              (uint32_t(kTileC >> 4) << 24);
            auto commit = [](unsigned long long &bar) {  // to both CTAs' barriers, once the products are done
                asm volatile(
                    "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
                    " [%0], %1;" ::"r"(smem_of(&bar)),
                    "h"(uint16_t(3))
                    : "memory");
            };
            auto product = [](uint32_t sums, uint64_t da, uint64_t db, uint32_t idesc, bool add) {
                asm volatile(
                    "{\n\t.reg .pred p;\n\t"
                    "setp.ne.u32 p, %4, 0;\n\t"
                    "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(sums),
                    "l"(da), "l"(db), "r"(idesc), "r"(uint32_t(add))
                    : "memory");
            };
            const uint32_t base = uniform(tmem);
            const uint64_t x0 = slab_descriptor(smem_of(x_ring)), dy0 = slab_descriptor(smem_of(dy_ring));
            int n = 0, u = 0, t = 0;
            uint32_t used = 0, odd = 0;  // bit per buffer: used before, an odd number of times
            bool ok = true;
            for (int round = 0, item; ok && (item = item_number(a, round)) >= 0; ++round) {
                if (products_withheld(round)) break;
                const WgradItem it = item_of<NB>(a, groups, item);
                const int steps = uniform(it.steps), full_steps = uniform(it.full);
                const int rest = (uniform(it.rows) - full_steps * kK + 15) / 16;  // products of the last step
                if (steps == 0) continue;
                const int blocks = it.blocks;
                const uint32_t idesc[2] = {kInstruction | (uint32_t(block_outs(a, it, 0) >> 3) << 17),
                                           kInstruction | (uint32_t(blocks > 1 ? block_outs(a, it, 1) >> 3 : 0) << 17)};
                int buffer = NB == 1 ? t & 1 : 0, left = 0;  // steps left of the sum
                uint32_t sums = base;
                for (int i = 0; i < steps && ok; ++i, ++n, --left) {
                    const int sx = n % kXRing;
                    const bool fresh = left == 0;
                    if (fresh) {  // the tile's first sum, or the next one, in the other buffer
                        if (NB == 1 && i > 0) buffer = ~t & 1;
                        if (used >> buffer & 1)
                            ok = __all_sync(kFull, wait_phase(b, b.sum_empty[buffer], ~(odd >> buffer) & 1));
                        used |= 1u << buffer, odd ^= 1u << buffer;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        sums = base + uint32_t(buffer * kTileO);
                        left = min(a.chunk, steps - i);
                        if (!ok) break;
                    }
                    ok = __all_sync(kFull, wait_phase(b, b.x_full[sx], uint32_t(n / kXRing) & 1));
                    const uint64_t da = x0 + uint64_t(sx * (kStage >> 4));
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        if (nb >= blocks || !ok) break;
                        const int sd = u % kDyRing;
                        ok = __all_sync(kFull, wait_phase(b, b.dy_full[sd], uint32_t(u / kDyRing) & 1));
                        if (!ok) break;
                        ++u;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint64_t db = dy0 + uint64_t(sd * (kStage >> 4));
                        if (elect_one()) {  // 16 rows on: 2048 bytes on
                            if (i < full_steps) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    product(sums + uint32_t(nb * kTileO), da + uint64_t(k * 128), db + uint64_t(k * 128),
                                            idesc[nb], !fresh || k > 0);
                            } else {
                                for (int k = 0; k < rest; ++k)
                                    product(sums + uint32_t(nb * kTileO), da + uint64_t(k * 128), db + uint64_t(k * 128),
                                            idesc[nb], !fresh || k > 0);
                            }
                            commit(b.dy_empty[sd]);
                            if (nb == blocks - 1) commit(b.x_empty[sx]);
                            if (nb == blocks - 1 && left == 1) commit(b.sum_full[buffer]);
                        }
                        __syncwarp();
                    }
                }
                ++t;
            }
        }
    } else if (warp >= kStoreWarp) {
        // the sums to the grads: warp w reads the 32 lanes that are its own
        const int m = int(rank) * (kTileC / 2) + (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
        int t = 0;
        uint32_t odd = 0;  // bit per buffer: used an odd number of times
        bool ok = true;
        auto release = [&](int buffer) {
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_remote(leader_address(smem_of(&b.sum_empty[buffer])));
        };
        for (int k = 0, item; (item = item_number(a, k)) >= 0; ++k) {
            const WgradItem it = item_of<NB>(a, groups, item);
            const int c = it.c0 + column_of(m);
            const int outs = (it.blocks - 1) * kTileO + block_outs(a, it, it.blocks - 1);
            const int buffer = NB == 1 ? t & 1 : 0;
            const uint32_t sums = lanes + uint32_t(buffer * kTileO);
            for (int i = 0; ok && i < it.steps; i += a.chunk) {
                const int from = NB == 1 && i > 0 ? buffer ^ 1 : buffer;
                ok = __all_sync(kFull, wait_phase<200>(b, b.sum_full[from], odd >> from & 1));
                if (!ok) break;
                odd ^= 1u << from;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (i > 0) {
                    add_tile(sums, lanes + uint32_t(from * kTileO), outs);
                    release(from);
                }
            }
            // once a wait has run out, the items that have rows are lost
            const bool there_are = ok && it.steps > 0;
            const uint32_t fill = ok || it.steps == 0 ? 0 : kNanBits;
            if (it.slot >= 0) {
                float *p = a.partial + it.slot * slot_floats(NB) + m;
                for (int o = 0; o < outs; o += 16) {
                    uint32_t r[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) r[q] = fill;
                    if (there_are) load_sums(sums + uint32_t(o), r), wait_sums(r);
#pragma unroll
                    for (int q = 0; q < 16; ++q, p += kTileC) *p = __uint_as_float(r[q]);
                }
            } else if (a.accumulate && it.steps == 0) {
                // nothing is added: the grads stay as they are
            } else if (a.grad_dtype == DOPT_FP32) {
                store_tile<float>(a, it, c, outs, sums, there_are, fill);
            } else if (a.grad_dtype == DOPT_BF16) {
                store_tile<__nv_bfloat16>(a, it, c, outs, sums, there_are, fill);
            } else {
                store_tile<__half>(a, it, c, outs, sums, there_are, fill);
            }
            if (there_are) {
                release(buffer);
                ++t;
            }
        }
    } else {
        // x: group g takes steps g, g + 4, ... of all the pair's steps; a warp 16
        // rows of a step, a thread 16 columns of four of them: rows 4 w + r +
        // 16 h, columns c16 on.  Eight lanes' chunks, of two neighbouring rows
        // in one slab, fall into different banks.
        const int w = warp & 3, r = ((lane >> 2) & 1) + 2 * (lane >> 4);
        const int c16 = 64 * ((lane >> 3) & 1) + 16 * (lane & 3);
        struct {
            int k, i, n, u;  // the round, the step in its item; the step and block of dy of all
            int lo, rows, c, blocks;
        } at;
        at.k = at.i = at.n = at.u = 0;
        auto enter = [&](int item) {
            const WgradItem it = item_of<NB>(a, groups, item);
            at.lo = it.lo, at.rows = it.rows, at.blocks = NB == 1 ? 1 : it.blocks;
            at.c = it.c0 + int(rank) * (kTileC / 2);
        };
        // on by so many steps, over items; false past the last
        auto advance = [&](int by) -> bool {
            at.i += by;
            at.n += by;
            at.u += by * at.blocks;
            for (int steps; at.i >= (steps = (at.rows + kK - 1) / kK);) {
                at.u -= (at.i - steps) * at.blocks;
                at.i -= steps;
                const int item = item_number(a, ++at.k);
                if (item < 0) return false;
                enter(item);
                at.u += at.i * at.blocks;
            }
            return true;
        };
        // whether the step's dy comes from here
        auto own = [&]() { return !a.tma || at.i >= at.rows / kK; };
        uint4 code[4];
        uint32_t exp[4];
        int tokens = -1;
        uint32_t absent = 0;  // bit r + 4 h: that row counts as zeros
        // the token of row 4 w + (l & 3) + 16 (l / 4) of the step, in lane l
        auto load_tokens = [&]() {
            const int k = at.i * kK + 4 * w + (lane & 3) + 4 * (lane & 12);
            tokens = -1;
            if (k < at.rows && lane < 16) tokens = a.row_token ? a.row_token[at.lo + k] : at.lo + k;
        };
        const uint32_t pitch = uint32_t(a.pitch);
        auto load_codes = [&]() {
            const int c = at.c;
            if (c >= a.pitch || a.x_rows <= 0) {  // no such columns, or no rows: zeros
#pragma unroll
                for (int h = 0; h < 4; ++h) code[h] = make_uint4(0, 0, 0, 0);
                absent = 0xffff;
                return;
            }
            const unsigned char *codes = a.codes + (c + c16), *scales = a.scales + (c + c16) / kBlock;
            const bool there = uint32_t(tokens) < uint32_t(a.x_rows);
            absent = __ballot_sync(kFull, !there);
            const uint32_t mine = there ? uint32_t(tokens) : 0;  // (an absent row reads row 0)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint64_t row = __shfl_sync(kFull, mine, r + 4 * h);
                code[h] = __ldg(reinterpret_cast<const uint4 *>(codes + row * pitch));
                exp[h] = __ldg(scales + row * (pitch / kBlock));
            }
        };
        enter(item_number(a, 0));
        bool more = advance(warp >> 2);
        if (more) load_tokens(), load_codes();
        // 16 rows on: 2048 bytes on, and the swizzle is the same
        const uint32_t chunk0 = stage_chunk(4 * w + r, c16 / 8), chunk1 = stage_chunk(4 * w + r, c16 / 8 + 1);
        bool ok = true;
        while (more) {
            const int n = at.n, s = n % kXRing;
            unsigned char *stage = x_ring + s * kStage;
            const bool own_dy = own();
            if (own_dy) ok = stage_step<T, NB>(a, groups, b, dy_ring, at.k, at.i, at.u, rank);
            if (absent & 0xffff) {
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    if (absent >> (r + 4 * h) & 1) exp[h] = 0;
            }
            uint4 v[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[2 * h] = widen(T(), make_uint2(code[h].x, code[h].y), exp[h]);
                v[2 * h + 1] = widen(T(), make_uint2(code[h].z, code[h].w), exp[h]);
            }
            if (n >= kXRing) ok = wait_phase<32>(b, b.x_empty[s], uint32_t(n / kXRing - 1) & 1) && ok;
            if (!__all_sync(kFull, ok)) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                *reinterpret_cast<uint4 *>(stage + chunk0 + h * 2048) = v[2 * h];
                *reinterpret_cast<uint4 *>(stage + chunk1 + h * 2048) = v[2 * h + 1];
            }
#pragma unroll
            for (int h = 2; h < 4; ++h) {
                *reinterpret_cast<uint4 *>(stage + chunk0 + h * 2048) =
                    widen(T(), make_uint2(code[h].x, code[h].y), exp[h]);
                *reinterpret_cast<uint4 *>(stage + chunk1 + h * 2048) =
                    widen(T(), make_uint2(code[h].z, code[h].w), exp[h]);
            }
            if (own_dy) copies_done();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_remote(leader_address(smem_of(&b.x_full[s])));
            more = advance(kGroups);
            if (more) {
                load_tokens();
                load_codes();
            }
        }
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
template <typename G, int NB>
__global__ void __launch_bounds__(kTileC) dopt_ckpt_wgrad_join_kernel(const __grid_constant__ WgradArgs a) {
    let_dependents_start();
    wait_for_grids_before();
    __shared__ WgradGroups groups;
    fill_groups(a, groups);
    __syncthreads();
    const WgradItem it = item_of<NB>(a, groups, a.whole + int(blockIdx.x) * a.split);
    const int o = int(blockIdx.y) * 16;
    if (it.o0 + o >= a.outs || (a.accumulate && groups.first[it.group + 1] <= groups.first[it.group])) return;
    float f[16] = {};
    for (int s = 0; s < a.split; ++s) {
        const float *p = a.partial + (it.slot + s) * slot_floats(NB) + int64_t(o) * kTileC + threadIdx.x;
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = __ldcs(p + q * kTileC);
#pragma unroll
        for (int q = 0; q < 16; ++q) f[q] += v[q];
    }
    const int c = it.c0 + column_of(threadIdx.x);
    if (c < a.cols) store_sums(a, grad_at<G>(a, it, c) + o * a.cols, a.outs - it.o0 - o, f);
}

// dy with rows that are not 16-byte aligned, into rows that are (`ld`, a
// multiple of 8, zeros past the outputs): one pass, which 16384 x 5631 rows
// repay seven times over.
template <typename T>
__global__ void __launch_bounds__(256) dopt_ckpt_wgrad_align_kernel(const T *dy, int64_t dy_ld, int rows, int outs,
                                                                   T *copy, int64_t ld) {
    let_dependents_start();
    wait_for_grids_before();
    const int lane = threadIdx.x, c = (blockIdx.x * 32 + lane) * 8;
    for (uint32_t r0 = blockIdx.y * 8; r0 < uint32_t(rows); r0 += gridDim.y * 8) {
        const uint32_t r = r0 + threadIdx.y;
        const bool here = r < uint32_t(rows);
        Values<T, 8> v;
        v.load(dy + (here ? int64_t(r) * dy_ld : 0), c, here ? outs : 0, false, lane, 32);
        if (here && c < ld) *reinterpret_cast<uint4 *>(copy + int64_t(r) * ld + c) = v.raw[0];
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// How the work goes over `pairs` pairs of SMs: tiles of nb * 256 outputs,
// whole waves of them tile by tile and the last, partial wave's tiles split
// along the rows into parts.  Chosen for the least estimated time, in units
// of one product of 64 rows (0.295 us): a step takes 1.25 with nb = 1 (codes
// are widened for one product) and 2.0 with nb = 2, a tile's stores 10 a block
// (with nb = 1 they run under the next tile's products but slow them), the
// join's launch 12 and a part's trip through memory 0.2 a block.  In us, with
// nb = 1 and 2: 16384 rows x 5632 columns x 2048 outputs 224 and 199, 2048 x
// 5632 x 2048 41.4 and 46.3, 4096 x 768 x 768 18.8 and 22.8, 8 experts of 4096
// rows x 1024 x 4096 191 and 165, 64 of 1024 x 512 x 1408 94.4 and 93.1, 128 of
// 1024 x 2048 x 768 348 and 353 (all in one sum a tile).
// A tile whose sum takes several chunks has nb = 1 (nb = 2 leaves no
// tensor memory to start another sum in); adding one up stops the products for
// 2.5.
struct Plan {
    int nb, parts;
    int64_t whole, tail;
};
Plan plan_wgrad(int64_t outs, int64_t cols, int n_groups, int64_t dy_rows, int64_t chunk, int64_t pairs,
                int64_t workspace_bytes) {
    const double steps = double(dy_rows / n_groups + kK - 1) / kK;
    // (of several groups, one may have all the rows)
    const int64_t longest = (dy_rows + kK - 1) / kK;
    Plan best{};
    double least = -1;
    for (int nb = 1; nb <= 2; ++nb) {
        const int64_t tiles = (outs + kTileO * nb - 1) / (kTileO * nb) * ((cols + kTileC - 1) / kTileC) * n_groups;
        const int64_t tail = tiles % pairs;
        const double step = nb == 1 ? 1.25 + 2.5 / double(chunk) : 2.0, each = steps * step + 10.0 * nb;
        const double waves = double(tiles / pairs) * each;
        for (int parts = 1; parts <= kMaxSplit; ++parts) {
            // (groups go from long to short: the tail's tiles are the shortest)
            if (parts > 1 && (tail == 0 || (n_groups > 1 && tiles > pairs) || steps / parts < 4 || tail * parts * slot_floats(nb) * 4 > workspace_bytes))
                break;
            // (a tail's parts are shorter than the whole tiles that there are besides)
            if (nb == 2 && longest > chunk * (n_groups > 1 || tiles > tail ? 1 : parts)) continue;
            double t = waves + double((tail * parts + pairs - 1) / pairs) * (each - steps * step + steps * step / parts);
            if (parts > 1) t += 12.0 + 0.2 * nb * double(tail * parts);
            if (least < 0 || t < least) {
                least = t;
                best = parts > 1 ? Plan{nb, parts, tiles - tail, tail} : Plan{nb, 1, tiles, 0};
            }
        }
    }
    return best;
}

// Rows of one sum, in steps of 64.  fp32 grads: 1024 with bf16 dy and 512 with
// fp16, whose products have more bits to lose; errors are then 3.2e-7 and
// 4.2e-7 of the grads' size at any number of rows (random signs), and no more
// than 64 * 2^-23 of the sum of magnitudes in a chunk.  16-bit grads take as
// many rows as lose an eighth of their rounding: fp16 16384 (1.8e-5), bf16
// 131072.
int64_t sum_chunk(dopt_dtype dy, dopt_dtype grad) {
    if (grad == DOPT_FP32) return dy == DOPT_BF16 ? 1024 / kK : 512 / kK;
    return grad == DOPT_FP16 ? 16384 / kK : 131072 / kK;
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::mutex g_wgrad_mutex;
EncodeTiled g_encode = nullptr;
int g_pairs[64] = {};  // pairs of SMs of a device, once its kernels are set up

cudaError_t allow_smem(void (*kernel)(WgradArgs)) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kWgradSmem));
}

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
            e = allow_smem(dopt_ckpt_wgrad_kernel<__nv_bfloat16, 1>);
        if (e == cudaSuccess) e = allow_smem(dopt_ckpt_wgrad_kernel<__nv_bfloat16, 2>);
        if (e == cudaSuccess) e = allow_smem(dopt_ckpt_wgrad_kernel<__half, 1>);
        if (e == cudaSuccess) e = allow_smem(dopt_ckpt_wgrad_kernel<__half, 2>);
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

// Rows in whole steps stay below 2^31: the kernel counts them in 32 bits.
constexpr int64_t kMostRows = int64_t(INT32_MAX) / kK * kK;
static_assert(kMostRows == DOPT_WGRAD_MAX_ROWS, "the limit that dopt.h states");

// Row length, in elements, and bytes of the aligned copy of dy.
int64_t copy_ld(int64_t outs) { return (outs + 7) / 8 * 8; }
int64_t copy_bytes(int64_t dy_rows, int64_t outs) { return (dy_rows * copy_ld(outs) * 2 + 15) / 16 * 16; }

template <typename T>
int align_dy(const char *who, const void *dy, int64_t dy_ld, int64_t dy_rows, int64_t outs, void *copy,
             cudaStream_t stream) {
    const dim3 grid(unsigned((copy_ld(outs) + 255) / 256), unsigned(std::min<int64_t>((dy_rows + 7) / 8, 65535)));
    return launch_op(who, dopt_ckpt_wgrad_align_kernel<T>, grid, dim3(32, 8), 0, stream, static_cast<const T *>(dy),
                     dy_ld, int(dy_rows), int(outs), static_cast<T *>(copy), copy_ld(outs));
}

template <typename T, int NB>
int launch_wgrad(const char *who, const WgradArgs &a, int64_t pairs, int64_t tail, cudaStream_t stream) {
    int rc = launch_op(who, dopt_ckpt_wgrad_kernel<T, NB>, dim3(unsigned(2 * std::min<int64_t>(a.items, pairs))),
                       dim3(kWgradThreads), kWgradSmem, stream, a);
    if (rc != DOPT_OK || a.split == 1) return rc;
    const dim3 grid(unsigned(tail), kTileO * NB / 16);
    switch (a.grad_dtype) {
        case DOPT_BF16:
            return launch_op(who, dopt_ckpt_wgrad_join_kernel<__nv_bfloat16, NB>, grid, dim3(kTileC), 0, stream, a);
        case DOPT_FP16:
            return launch_op(who, dopt_ckpt_wgrad_join_kernel<__half, NB>, grid, dim3(kTileC), 0, stream, a);
        default: return launch_op(who, dopt_ckpt_wgrad_join_kernel<float, NB>, grid, dim3(kTileC), 0, stream, a);
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
        dy_rows > kMostRows || outs < 1 || outs > DOPT_MAX_COLS || dy_ld < outs)
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
    a.x_rows = int32_t(x_rows);
    a.cols = cols;
    a.dy_rows = int32_t(dy_rows);
    a.outs = int32_t(outs);
    a.groups = n_groups;
    a.dy_ld = dy_ld;
    a.accumulate = (flags & DOPT_WGRAD_ACCUMULATE) != 0;
    a.vec = aligned_to(dy, 16) && dy_ld * 2 % 16 == 0;
    const int64_t copied = copy_bytes(dy_rows, outs);
    const bool copy = !a.vec && dy_rows > 0 && workspace_bytes >= copied;
    a.grad_dtype = grad_dtype;
    EncodeTiled encode = nullptr;
    int pairs = 0;
    int rc = set_up(who, &encode, &pairs);
    if (rc != DOPT_OK) return rc;
    if (copy) {
        rc = dy_dtype == DOPT_BF16 ? align_dy<__nv_bfloat16>(who, dy, dy_ld, dy_rows, outs, workspace, stream)
                                   : align_dy<__half>(who, dy, dy_ld, dy_rows, outs, workspace, stream);
        if (rc != DOPT_OK) return rc;
        dy = a.dy = workspace;
        dy_ld = a.dy_ld = copy_ld(outs);
        a.vec = 1;
        workspace = static_cast<char *>(workspace) + copied;
        workspace_bytes -= copied;
    }
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
    a.chunk = int32_t(sum_chunk(dy_dtype, grad_dtype));
    const Plan plan = plan_wgrad(outs, cols, n_groups, dy_rows, a.chunk, pairs, workspace_bytes);
    const int64_t items = plan.whole + plan.tail * plan.parts;
    if (items > INT32_MAX / 2) return fail(DOPT_E_ARG, "%s: %lld tiles", who, static_cast<long long>(items));
    a.tiles_c = int32_t((cols + kTileC - 1) / kTileC);
    a.tiles_o = int32_t((outs + kTileO * plan.nb - 1) / (kTileO * plan.nb));
    a.items = int32_t(items);
    a.whole = int32_t(plan.whole);
    a.split = plan.parts;
    a.partial = static_cast<float *>(workspace);
    if (dy_dtype == DOPT_BF16)
        return plan.nb == 1 ? launch_wgrad<__nv_bfloat16, 1>(who, a, pairs, plan.tail, stream)
                            : launch_wgrad<__nv_bfloat16, 2>(who, a, pairs, plan.tail, stream);
    return plan.nb == 1 ? launch_wgrad<__half, 1>(who, a, pairs, plan.tail, stream)
                        : launch_wgrad<__half, 2>(who, a, pairs, plan.tail, stream);
}

extern "C" int dopt_ckpt_wgrad_workspace(int64_t dy_rows, int64_t outs, int64_t cols,
                                         int32_t n_groups, int64_t *bytes) {
    dopt::clear_error();
    const char *who = "dopt_ckpt_wgrad_workspace";
    if (!bytes) return dopt::fail(DOPT_E_ARG, "%s: bytes is NULL", who);
    if (dy_rows < 0 || dy_rows > kMostRows || outs < 1 || outs > DOPT_MAX_COLS || cols < 1 ||
        cols > DOPT_MAX_COLS || n_groups < 1 || n_groups > DOPT_MAX_GROUPS)
        return dopt::fail(DOPT_E_ARG, "%s: %lld rows, %lld x %lld, %d groups", who,
                          static_cast<long long>(dy_rows), static_cast<long long>(outs),
                          static_cast<long long>(cols), n_groups);
    // for a device of 76 pairs of SMs and the types that take most; a call takes what it is given
    int64_t most = 0;
    for (dopt_dtype dy : {DOPT_BF16, DOPT_FP16})
        for (dopt_dtype grad : {DOPT_BF16, DOPT_FP16, DOPT_FP32}) {
            const Plan plan = plan_wgrad(outs, cols, n_groups, dy_rows, sum_chunk(dy, grad), 76, INT64_MAX);
            most = std::max(most, plan.tail * plan.parts * slot_floats(plan.nb) * int64_t(sizeof(float)));
        }
    *bytes = most + (outs % 8 != 0 ? copy_bytes(dy_rows, outs) : 0);
    return DOPT_OK;
}

extern "C" int dopt_ckpt_wgrad_plan(int64_t dy_rows, int64_t outs, int64_t cols, int32_t n_groups,
                                    dopt_dtype dy_dtype, dopt_dtype grad_dtype, int64_t workspace_bytes,
                                    int64_t plan[4]) {
    dopt::clear_error();
    const char *who = "dopt_ckpt_wgrad_plan";
    if (!plan) return dopt::fail(DOPT_E_ARG, "%s: plan is NULL", who);
    if (dy_rows < 0 || dy_rows > kMostRows || outs < 1 || outs > DOPT_MAX_COLS || cols < 1 || cols > DOPT_MAX_COLS ||
        n_groups < 1 || n_groups > DOPT_MAX_GROUPS || workspace_bytes < 0)
        return dopt::fail(DOPT_E_ARG, "%s: %lld rows, %lld x %lld, %d groups, workspace of %lld bytes", who,
                          static_cast<long long>(dy_rows), static_cast<long long>(outs), static_cast<long long>(cols),
                          n_groups, static_cast<long long>(workspace_bytes));
    if ((dy_dtype != DOPT_BF16 && dy_dtype != DOPT_FP16) || !valid_dtype(grad_dtype))
        return dopt::fail(DOPT_E_ARG, "%s: dtypes %d, %d", who, int(dy_dtype), int(grad_dtype));
    const Plan p = plan_wgrad(outs, cols, n_groups, dy_rows, sum_chunk(dy_dtype, grad_dtype), 76, workspace_bytes);
    plan[0] = p.nb;
    plan[1] = p.whole;
    plan[2] = p.tail;
    plan[3] = p.parts;
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

extern "C" int dopt_wgrad_wait_test(int32_t items) {
    using dopt::fail;
    dopt::clear_error();
#ifdef DOPT_DEVICE_CHECKS
    if (items < -1) return fail(DOPT_E_ARG, "dopt_wgrad_wait_test: %d items", items);
    const int v = items;
    const cudaError_t e = cudaMemcpyToSymbol(g_wgrad_items, &v, sizeof v);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(DOPT_E_CUDA, "dopt_wgrad_wait_test: %s", cudaGetErrorString(e));
    }
    return DOPT_OK;
#else
    (void)items;
    return fail(DOPT_E_STATE, "dopt_wgrad_wait_test: this library was built without DOPT_DEVICE_CHECKS");
#endif
}
