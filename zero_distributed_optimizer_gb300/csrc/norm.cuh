#pragma once
// What the norms around a block (norm.cu) and their gradients (norm_grad.cu)
// share: a row's values and sums, how rows are given to threads, and what both
// refuse.
#include "f32x2.cuh"
#include "rows.cuh"

namespace {

constexpr int kCols = 8;      // columns of one access group of a thread
constexpr int kMostRow = 512;  // threads of a row
constexpr int kMostSums = 4;
constexpr int kParts = 1024;  // groups of rows whose column sums are kept apart

struct NormArgs {
    const void *x, *y, *d_n, *d_h;  // backward: x is the residual h
    void *h, *n;                    // backward: d_x, d_y
    const void *weight, *bias, *post_weight, *post_bias, *gate;
    const float *row_gate;
    float *d_row_gate;
    float *partial;                 // [groups][sums][part_ld]
    int64_t ld_x, ld_y, ld_h, ld_n, ld_d_n, ld_d_h, part_ld;
    int64_t rows;
    int32_t cols;
    int32_t vec, vec_params;        // rows, params are 16-byte aligned
    int32_t post;
    float scale, eps;
};

// ---------------------------------------------------------------------------
// Sums over a row, by the threads (threadIdx.x) of its group (threadIdx.y)
// ---------------------------------------------------------------------------

// f becomes the sums over the row's threads with few shuffles: in a warp, the
// values are first shared out over the lanes (a lane keeps the half of its
// values that its number says, and adds the other lane's), then added; the
// warps' sums, up to 8 a value and lane, are read by one load and added
// likewise.  Two buffers in turn: a thread that writes one has passed the
// barrier after the last reads of it.
struct RowSums {
    float v[2][kMostSums][kMostRow / 32];
};
template <int K>
__device__ __forceinline__ void row_sums(RowSums &s, int &turn, float (&f)[K]) {
    static_assert(K == 1 || K == 2 || K == 4, "values are shared out by halves");
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float mine = f[0];
    if constexpr (K == 4) {
        const bool up = lane & 16;
        float a = up ? f[2] : f[0], b = up ? f[3] : f[1];
        a += __shfl_xor_sync(kFull, up ? f[0] : f[2], 16);
        b += __shfl_xor_sync(kFull, up ? f[1] : f[3], 16);
        mine = (lane & 8 ? b : a) + __shfl_xor_sync(kFull, lane & 8 ? a : b, 8);
    } else if constexpr (K == 2) {
        mine = (lane & 16 ? f[1] : f[0]) + __shfl_xor_sync(kFull, lane & 16 ? f[0] : f[1], 16);
    }
    // value k is now in the lanes from k * (32 / K) on
#pragma unroll
    for (int d = 16 / K; d > 0; d >>= 1) mine += __shfl_xor_sync(kFull, mine, d);
    if (warps > 1) {
        float(&v)[kMostSums][kMostRow / 32] = s.v[turn];
        turn ^= 1;
        if (lane % (32 / K) == 0) v[lane / (32 / K)][threadIdx.x >> 5] = mine;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
        // lanes 8 k + w: value k of warps w and w + 8
        const int k = lane >> 3, w = lane & 7;
        mine = k < K && w < warps ? v[k][w] : 0.0f;
        if (warps > 8 && k < K && w + 8 < warps) mine += v[k][w + 8];
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) mine += __shfl_xor_sync(kFull, mine, d);
#pragma unroll
        for (int i = 0; i < K; ++i) f[i] = __shfl_sync(kFull, mine, 8 * i);
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i) f[i] = __shfl_sync(kFull, mine, i * (32 / K));
    }
}

// All threads of a row have read what they will (rows that are not aligned are
// read by neighbours too, and may be written in place).
__device__ __forceinline__ void row_read() {
    if (blockDim.x > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
}

// Column of a thread's values i.
__device__ __forceinline__ int column(int i) { return int(i * blockDim.x + threadIdx.x) * kCols; }

template <typename T, int NV>
struct RowValues {
    Values<T, kCols> v[NV];
    __device__ __forceinline__ void load(const T *row, int cols, bool vec) {
        typename Values<T, kCols>::Ahead ahead[NV];
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < NV; ++i) Values<T, kCols>::fetch(ahead[i], row, column(i), cols, vec, lane, 32);
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i].take(ahead[i], vec, lane, 32);
    }
    __device__ __forceinline__ void store(T *row, int cols, bool vec) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i].store(row, column(i), cols, vec, threadIdx.x & 31, 32);
    }
};

// A param's values, `none` where there is no such param.
template <typename T, int NV>
struct Param {
    RowValues<T, NV> p;
    bool there;
    __device__ __forceinline__ void load(const void *at, int cols, bool vec) {
        there = at != nullptr;
        if (there) p.load(static_cast<const T *>(at), cols, vec);
    }
    __device__ __forceinline__ void get(int i, float none, float (&f)[kCols]) const {
#pragma unroll
        for (int q = 0; q < kCols; ++q) f[q] = none;
        if (there) p.v[i].get(f);
    }
};

// The mean (layer norm) and the factor of a row's values.
template <int NV, bool LAYER>
__device__ __forceinline__ void standard(RowSums &s, int &turn, const float (&f)[NV][kCols], int cols, float eps,
                                         float &mean, float &factor) {
    mean = 0.0f;
    if constexpr (LAYER) {
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < kCols; ++q) sum[0] += f[i][q];
        row_sums(s, turn, sum);
        mean = sum[0] / float(cols);
    }
    float square[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = column(i);
#pragma unroll
        for (int q = 0; q < kCols; ++q) {
            const float v = !LAYER || c + q < cols ? f[i][q] - mean : 0.0f;
            square[0] = fmaf(v, v, square[0]);
        }
    }
    row_sums(s, turn, square);
    factor = 1.0f / sqrtf(square[0] / float(cols) + eps);
}

// ---------------------------------------------------------------------------
// Rows and params that are 16-byte aligned, of a multiple of 8 columns
// ---------------------------------------------------------------------------

// 8 values of a thread, as pairs.
constexpr int kPairs = kCols / 2;
__device__ __forceinline__ F2 widen2(__nv_bfloat16, uint32_t w) { return F2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ F2 widen2(__half, uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return F2(f.x, f.y);
}
__device__ __forceinline__ uint32_t narrow2(__nv_bfloat16, F2 v) {
    float a, b;
    v.get(a, b);
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t narrow2(__half, F2 v) {
    float a, b;
    v.get(a, b);
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
template <typename T>
struct Eight {
    static constexpr int kPieces = kCols * int(sizeof(T)) / 16;
    uint4 raw[kPieces];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) raw[i] = make_uint4(0, 0, 0, 0);
    }
    // (left as they are where they are not there)
    __device__ __forceinline__ void load(const T *p, bool there) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (there) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void get(F2 (&f)[kPairs]) const {
        if constexpr (sizeof(T) == 2) {
            f[0] = widen2(T(), raw[0].x), f[1] = widen2(T(), raw[0].y), f[2] = widen2(T(), raw[0].z), f[3] = widen2(T(), raw[0].w);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[2 * i] = F2(__uint_as_float(raw[i].x), __uint_as_float(raw[i].y));
                f[2 * i + 1] = F2(__uint_as_float(raw[i].z), __uint_as_float(raw[i].w));
            }
        }
    }
    static __device__ __forceinline__ void put(T *p, const F2 (&f)[kPairs], bool there) {
        if (!there) return;
        if constexpr (sizeof(T) == 2) {
            __stcs(reinterpret_cast<uint4 *>(p),
                   make_uint4(narrow2(T(), f[0]), narrow2(T(), f[1]), narrow2(T(), f[2]), narrow2(T(), f[3])));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float4 v;
                f[2 * i].get(v.x, v.y), f[2 * i + 1].get(v.z, v.w);
                __stcs(reinterpret_cast<float4 *>(p) + i, v);
            }
        }
    }
};
// 8 values of a param, which stays in L1 (nothing is kept of it from row to row).
template <typename T>
__device__ __forceinline__ void param_values(const void *param, int c, bool there, float none, F2 (&f)[kPairs]) {
#pragma unroll
    for (int q = 0; q < kPairs; ++q) f[q] = F2(none);
    if (param && there) {
        Eight<T> v;
#pragma unroll
        for (int i = 0; i < Eight<T>::kPieces; ++i)
            v.raw[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(param) + c) + i);
        v.get(f);
    }
}
__device__ __forceinline__ float both(F2 v) {
    float a, b;
    v.get(a, b);
    return a + b;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// How rows are given to threads: nv groups of 8 columns a thread; short rows
// share a block.  A row's sums cost a thread the same whatever it holds, so the
// forward pass, with few values to hold, takes two groups from 1024 columns on;
// the gradients, which hold four times as many, take them from 2048 on.
struct NormShape {
    int nv;
    dim3 block;
    NormShape(int64_t cols, bool backward) {
        nv = cols <= (backward ? 2048 : 1024) ? 1 : cols <= (backward ? 8192 : 4096) ? 2 : 4;
        const unsigned threads = unsigned((cols + 32 * kCols * nv - 1) / (32 * kCols * nv) * 32);
        block = dim3(threads, std::min(8u, std::max(1u, 256 / threads)));
    }
};

int64_t norm_part_ld(int64_t cols) { return (cols + kCols - 1) / kCols * kCols; }

// What both directions refuse, and the params.
int check_norm(const char *who, const dopt_norm_cfg *cfg, const dopt_norm_params *params, dopt_dtype dtype,
               int64_t rows, int64_t cols, const void *y) {
    using dopt::fail;
    if (!cfg || !params) return fail(DOPT_E_ARG, "%s: NULL configuration or params", who);
    if (cfg->kind != DOPT_NORM_RMS && cfg->kind != DOPT_NORM_LAYER)
        return fail(DOPT_E_ARG, "%s: unknown kind %d", who, int(cfg->kind));
    if (cfg->post != 0 && cfg->post != 1) return fail(DOPT_E_ARG, "%s: post %d (0 or 1)", who, cfg->post);
    if (!(cfg->eps >= 0.0f)) return fail(DOPT_E_ARG, "%s: eps %g", who, double(cfg->eps));
    if (!valid_dtype(dtype)) return fail(DOPT_E_ARG, "%s: unknown dtype %d", who, int(dtype));
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > DOPT_NORM_MAX_COLS)
        return fail(DOPT_E_ARG, "%s: %lld rows of %lld columns (1..%d)", who, static_cast<long long>(rows),
                    static_cast<long long>(cols), DOPT_NORM_MAX_COLS);
    if (cfg->kind == DOPT_NORM_RMS && (params->bias || params->post_bias))
        return fail(DOPT_E_ARG, "%s: an RMS norm has no bias", who);
    // (an empty matrix may have no address)
    if (rows > 0 && !y && (cfg->post || params->post_weight || params->post_bias || params->gate || params->row_gate))
        return fail(DOPT_E_ARG, "%s: a norm after the block or a gate without y", who);
    if (!cfg->post && (params->post_weight || params->post_bias))
        return fail(DOPT_E_ARG, "%s: post_weight or post_bias without post", who);
    const size_t b = elem_bytes(dtype);
    for (const void *p : {params->weight, params->bias, params->post_weight, params->post_bias, params->gate})
        if (!aligned_to(p, b)) return fail(DOPT_E_ALIGN, "%s: a param is not aligned to its elements", who);
    if (!aligned_to(params->row_gate, 4)) return fail(DOPT_E_ALIGN, "%s: row_gate is not 4-byte aligned", who);
    return DOPT_OK;
}

NormArgs norm_args(const dopt_norm_cfg &cfg, const dopt_norm_params &params, int64_t rows, int64_t cols) {
    NormArgs a{};
    a.weight = params.weight;
    a.bias = params.bias;
    a.post_weight = params.post_weight;
    a.post_bias = params.post_bias;
    a.gate = params.gate;
    a.row_gate = params.row_gate;
    a.rows = rows;
    a.cols = int32_t(cols);
    a.post = cfg.post;
    a.scale = cfg.scale;
    a.eps = cfg.eps;
    uint64_t bits = 0;
    for (const void *p : {a.weight, a.bias, a.post_weight, a.post_bias, a.gate}) bits |= address_bits(p);
    a.vec_params = bits % 16 == 0;
    return a;
}

// A matrix of rows: its pointer and stride, refused or added to `bits`.
int check_rows(const char *who, const char *name, const void *p, int64_t ld, int64_t cols, size_t elem, uint64_t &bits) {
    using dopt::fail;
    if (!p) return DOPT_OK;
    if (ld < cols)
        return fail(DOPT_E_ARG, "%s: %s has row stride %lld for %lld columns", who, name, static_cast<long long>(ld),
                    static_cast<long long>(cols));
    if (!aligned_to(p, elem)) return fail(DOPT_E_ALIGN, "%s: %s is not aligned to its elements", who, name);
    bits |= address_bits(p) | uint64_t(ld) * elem;
    return DOPT_OK;
}

}  // namespace
