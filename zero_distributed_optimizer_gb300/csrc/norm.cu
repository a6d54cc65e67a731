// The norms around a block, with the residual add, the block's gates and its
// scale (dopt_norm), and their gradients (dopt_norm_grad); dopt.h states the
// contracts.
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

struct RowSums {
    float v[2][kMostRow / 32][kMostSums];
};

// f becomes the sums over the row's threads.  Two buffers in turn: a thread
// that writes one has passed the barrier after the last reads of it.
template <int K>
__device__ __forceinline__ void row_sums(RowSums &s, int &turn, float (&f)[K]) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) f[k] += __shfl_xor_sync(kFull, f[k], d);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    float(&v)[kMostRow / 32][kMostSums] = s.v[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) v[threadIdx.x >> 5][k] = f[k];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) f[k] = 0.0f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k) f[k] += v[w][k];
}

// All threads of a row have read what they will (rows that are not aligned are
// read by neighbours too, and may be written in place).
__device__ __forceinline__ void row_read() {
    if (blockDim.x > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
}

template <typename T, int NV>
struct RowValues {
    Values<T, kCols> v[NV];
    // Column of a thread's values i.
    static __device__ __forceinline__ int column(int i) { return int(i * blockDim.x + threadIdx.x) * kCols; }
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
        const int c = RowValues<float, NV>::column(i);
#pragma unroll
        for (int q = 0; q < kCols; ++q) {
            const float v = !LAYER || c + q < cols ? f[i][q] - mean : 0.0f;
            square[0] = fmaf(v, v, square[0]);
        }
    }
    row_sums(s, turn, square);
    factor = 1.0f / sqrtf(square[0] / float(cols) + eps);
}

template <typename T, int NV, bool LAYER>
__global__ void __launch_bounds__(kMostRow) dopt_norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ RowSums sums[8];
    let_dependents_start();
    wait_for_grids_before();
    RowSums &s = sums[threadIdx.y];
    int turn = 0;
    Param<T, NV> weight, bias, post_weight, post_bias, gate;
    weight.load(a.weight, a.cols, a.vec_params);
    bias.load(a.bias, a.cols, a.vec_params);
    post_weight.load(a.post_weight, a.cols, a.vec_params);
    post_bias.load(a.post_bias, a.cols, a.vec_params);
    gate.load(a.gate, a.cols, a.vec_params);
    for (int64_t r = int64_t(blockIdx.x) * blockDim.y + threadIdx.y; r < a.rows; r += int64_t(gridDim.x) * blockDim.y) {
        RowValues<T, NV> x;
        x.load(static_cast<const T *>(a.x) + r * a.ld_x, a.cols, a.vec);
        float h[NV][kCols];
#pragma unroll
        for (int i = 0; i < NV; ++i) x.v[i].get(h[i]);
        if (a.y) {
            RowValues<T, NV> y;
            y.load(static_cast<const T *>(a.y) + r * a.ld_y, a.cols, a.vec);
            const float by = a.row_gate ? a.scale * a.row_gate[r] : a.scale;
            float u[NV][kCols];
#pragma unroll
            for (int i = 0; i < NV; ++i) y.v[i].get(u[i]);
            if (!a.vec) row_read();
            if (a.post) {
                float mean, factor;
                standard<NV, LAYER>(s, turn, u, a.cols, a.eps, mean, factor);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float w[kCols], b[kCols];
                    post_weight.get(i, 1.0f, w);
                    post_bias.get(i, 0.0f, b);
#pragma unroll
                    for (int q = 0; q < kCols; ++q) u[i][q] = fmaf((u[i][q] - mean) * factor, w[q], b[q]);
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float g[kCols];
                gate.get(i, 1.0f, g);
                const int c = RowValues<T, NV>::column(i);
#pragma unroll
                for (int q = 0; q < kCols; ++q)  // (a mean was taken off the values past the row too)
                    h[i][q] = c + q < a.cols ? fmaf(u[i][q], by * g[q], h[i][q]) : 0.0f;
                x.v[i].set(h[i]);
            }
            if (a.h) x.store(static_cast<T *>(a.h) + r * a.ld_h, a.cols, a.vec);
        }
        if (a.n) {
            float mean, factor;
            standard<NV, LAYER>(s, turn, h, a.cols, a.eps, mean, factor);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float w[kCols], b[kCols];
                weight.get(i, 1.0f, w);
                bias.get(i, 0.0f, b);
#pragma unroll
                for (int q = 0; q < kCols; ++q) h[i][q] = fmaf((h[i][q] - mean) * factor, w[q], b[q]);
                x.v[i].set(h[i]);
            }
            x.store(static_cast<T *>(a.n) + r * a.ld_n, a.cols, a.vec);
        }
    }
}

// The gradients of a group's rows and, per group, the sums over its rows
// that the params' gradients are made of:
//   0  d_n * hat(h)                    1  d_n  (layer norm)
//   2  scale * row_gate * d_x * hat(y)  3  scale * row_gate * d_x  (layer norm)
// (RMS norm: 0 and 2 alone; without a norm after the block, hat(y) is y.)
template <typename T, int NV, bool LAYER>
__global__ void __launch_bounds__(kMostRow) dopt_norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kSums = LAYER ? 4 : 2;
    constexpr int kPost = LAYER ? 2 : 1;  // the first sum of the block's side
    __shared__ RowSums sums[8];
    let_dependents_start();
    wait_for_grids_before();
    RowSums &s = sums[threadIdx.y];
    int turn = 0;
    const float cols = float(a.cols);
    Param<T, NV> weight, post_weight, post_bias, gate;
    weight.load(a.weight, a.cols, a.vec_params);
    post_weight.load(a.post_weight, a.cols, a.vec_params);
    post_bias.load(a.post_bias, a.cols, a.vec_params);
    gate.load(a.gate, a.cols, a.vec_params);
    float acc[kSums][NV][kCols] = {};
    for (int64_t r = int64_t(blockIdx.x) * blockDim.y + threadIdx.y; r < a.rows; r += int64_t(gridDim.x) * blockDim.y) {
        RowValues<T, NV> raw;
        float dx[NV][kCols] = {}, u[NV][kCols] = {};
        if (a.d_h) {
            raw.load(static_cast<const T *>(a.d_h) + r * a.ld_d_h, a.cols, a.vec);
#pragma unroll
            for (int i = 0; i < NV; ++i) raw.v[i].get(dx[i]);
        }
        if (a.y) {
            raw.load(static_cast<const T *>(a.y) + r * a.ld_y, a.cols, a.vec);
#pragma unroll
            for (int i = 0; i < NV; ++i) raw.v[i].get(u[i]);
        }
        if (a.d_n) {
            float h[NV][kCols], d[NV][kCols];
            raw.load(static_cast<const T *>(a.x) + r * a.ld_x, a.cols, a.vec);
#pragma unroll
            for (int i = 0; i < NV; ++i) raw.v[i].get(h[i]);
            raw.load(static_cast<const T *>(a.d_n) + r * a.ld_d_n, a.cols, a.vec);
#pragma unroll
            for (int i = 0; i < NV; ++i) raw.v[i].get(d[i]);
            float mean, factor;
            standard<NV, LAYER>(s, turn, h, a.cols, a.eps, mean, factor);
            float dot[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float w[kCols];
                weight.get(i, 1.0f, w);
#pragma unroll
                for (int q = 0; q < kCols; ++q) {
                    h[i][q] = (h[i][q] - mean) * factor;
                    acc[0][i][q] = fmaf(d[i][q], h[i][q], acc[0][i][q]);
                    if constexpr (LAYER) acc[1][i][q] += d[i][q];
                    d[i][q] *= w[q];
                    dot[0] = fmaf(d[i][q], h[i][q], dot[0]);
                    if constexpr (LAYER) dot[1] += d[i][q];
                }
            }
            row_sums(s, turn, dot);
            const float along = dot[0] / cols, level = LAYER ? dot[1] / cols : 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < kCols; ++q)
                    dx[i][q] = fmaf(factor, d[i][q] - level - h[i][q] * along, dx[i][q]);
        }
        if (!a.vec) row_read();
        if (a.h) {
#pragma unroll
            for (int i = 0; i < NV; ++i) raw.v[i].set(dx[i]);
            raw.store(static_cast<T *>(a.h) + r * a.ld_h, a.cols, a.vec);
        }
        if (!a.y) continue;
        const float by = a.row_gate ? a.scale * a.row_gate[r] : a.scale;
        float mean = 0.0f, factor = 1.0f;
        if (a.post) standard<NV, LAYER>(s, turn, u, a.cols, a.eps, mean, factor);
        float dot[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = RowValues<T, NV>::column(i);
            float w[kCols], b[kCols], g[kCols];
            post_weight.get(i, 1.0f, w);
            post_bias.get(i, 0.0f, b);
            gate.get(i, 1.0f, g);
#pragma unroll
            for (int q = 0; q < kCols; ++q) {
                const float d = c + q < a.cols ? dx[i][q] : 0.0f;
                u[i][q] = (u[i][q] - mean) * factor;
                dot[2] = fmaf(d * g[q], fmaf(u[i][q], w[q], b[q]), dot[2]);
                const float v = by * d;
                acc[kPost][i][q] = fmaf(v, u[i][q], acc[kPost][i][q]);
                if constexpr (LAYER) acc[kPost + 1][i][q] += v;
                dx[i][q] = v * g[q] * w[q];  // of hat(y)
                dot[0] = fmaf(dx[i][q], u[i][q], dot[0]);
                dot[1] += dx[i][q];
            }
        }
        if (a.post || a.d_row_gate) row_sums(s, turn, dot);
        if (a.d_row_gate && threadIdx.x == 0) a.d_row_gate[r] = a.scale * dot[2];
        if (!a.n) continue;
        const float along = a.post ? dot[0] / cols : 0.0f, level = LAYER && a.post ? dot[1] / cols : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int q = 0; q < kCols; ++q) dx[i][q] = factor * (dx[i][q] - level - u[i][q] * along);
            raw.v[i].set(dx[i]);
        }
        raw.store(static_cast<T *>(a.n) + r * a.ld_n, a.cols, a.vec);
    }
    const int64_t group = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
#pragma unroll
    for (int k = 0; k < kSums; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = RowValues<T, NV>::column(i);
            if (c >= a.cols) continue;  // (part_ld is a multiple of 8)
            float4 *p = reinterpret_cast<float4 *>(a.partial + (group * kSums + k) * a.part_ld + c);
            p[0] = make_float4(acc[k][i][0], acc[k][i][1], acc[k][i][2], acc[k][i][3]);
            p[1] = make_float4(acc[k][i][4], acc[k][i][5], acc[k][i][6], acc[k][i][7]);
        }
}

// ---------------------------------------------------------------------------
// Rows and params that are 16-byte aligned, of a multiple of 8 columns
// ---------------------------------------------------------------------------

// f becomes the sums over the row's threads, with few shuffles: in a warp, the
// values are first shared out over the lanes (a lane keeps the half of its
// values that its number says, and adds the other lane's), then added; the
// warps' sums, up to 8 a value and lane, are read by one load and added
// likewise.
struct LaneSums {
    float v[2][kMostSums][kMostRow / 32];
};
template <int K>
__device__ __forceinline__ void row_sums(LaneSums &s, int &turn, float (&f)[K]) {
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

// 8 values of a thread.
template <typename T>
struct Eight {
    static constexpr int kPieces = kCols * int(sizeof(T)) / 16;
    uint4 raw[kPieces];
    __device__ __forceinline__ void load(const T *p, bool there) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            raw[i] = there ? __ldcs(reinterpret_cast<const uint4 *>(p) + i) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&f)[kCols]) const {
        constexpr int kPer = 16 / int(sizeof(T));
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float g[kPer];
            unpack<T, 16>(raw[i], g);
#pragma unroll
            for (int q = 0; q < kPer; ++q) f[i * kPer + q] = g[q];
        }
    }
    static __device__ __forceinline__ void put(T *p, const float (&f)[kCols], bool there) {
        constexpr int kPer = 16 / int(sizeof(T));
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float g[kPer];
#pragma unroll
            for (int q = 0; q < kPer; ++q) g[q] = f[i * kPer + q];
            if (there) __stcs(reinterpret_cast<uint4 *>(p) + i, pack<T, 16>(g));
        }
    }
};
// 8 values of a param, which stays in L1 (nothing is kept of it from row to row).
template <typename T>
__device__ __forceinline__ void param_values(const void *param, int c, bool there, float none, float (&f)[kCols]) {
#pragma unroll
    for (int q = 0; q < kCols; ++q) f[q] = none;
    if (param && there) {
        Eight<T> v;
#pragma unroll
        for (int i = 0; i < Eight<T>::kPieces; ++i)
            v.raw[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(param) + c) + i);
        v.get(f);
    }
}

// The next row's loads are in flight under a row's sums: they go to the
// registers that this row's values came in.
template <typename T, int NV, bool LAYER>
__global__ void __launch_bounds__(NV == 4 ? kMostRow : 256, NV == 1 ? 4 : NV == 2 ? 2 : 1)
    dopt_norm_whole_kernel(const __grid_constant__ NormArgs a) {
    __shared__ LaneSums sums[8];
    let_dependents_start();
    wait_for_grids_before();
    LaneSums &s = sums[threadIdx.y];
    int turn = 0;
    const float per_col = 1.0f / float(a.cols);
    int col[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) col[i] = RowValues<T, NV>::column(i), in[i] = col[i] < a.cols;
    const int64_t step = int64_t(gridDim.x) * blockDim.y;
    int64_t r = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    Eight<T> x[NV], y[NV];
    float row_gate = 1.0f;
    const T *x_at = static_cast<const T *>(a.x) + r * a.ld_x, *y_at = static_cast<const T *>(a.y) + r * a.ld_y;
    const bool with_y = a.y != nullptr;
    auto fetch = [&](int64_t row) {
        const bool there = row < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i].load(x_at + col[i], there && in[i]);
            y[i].load(y_at + col[i], there && in[i] && with_y);
        }
        x_at += step * a.ld_x, y_at += step * a.ld_y;
        if (a.row_gate && there) row_gate = a.row_gate[row];
    };
    fetch(r);
    for (; r < a.rows; r += step) {
        float h[NV][kCols], u[NV][kCols];
        const float by = a.scale * row_gate;
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i].get(h[i]), y[i].get(u[i]);
        fetch(r + step);
        if (a.y) {
            if (a.post) {
                float mean = 0.0f;
                if constexpr (LAYER) {
                    float sum[1] = {0.0f};
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int q = 0; q < kCols; ++q) sum[0] += u[i][q];
                    row_sums(s, turn, sum);
                    mean = sum[0] * per_col;
                }
                float square[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (!LAYER || in[i])
#pragma unroll
                        for (int q = 0; q < kCols; ++q) {
                            if constexpr (LAYER) u[i][q] -= mean;
                            square[0] = fmaf(u[i][q], u[i][q], square[0]);
                        }
                row_sums(s, turn, square);
                const float factor = rsqrtf(fmaf(square[0], per_col, a.eps));
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float w[kCols];
                    param_values<T>(a.post_weight, col[i], in[i], 1.0f, w);
#pragma unroll
                    for (int q = 0; q < kCols; ++q) u[i][q] *= factor * w[q];
                    if (LAYER && a.post_bias) {
                        param_values<T>(a.post_bias, col[i], in[i], 0.0f, w);
#pragma unroll
                        for (int q = 0; q < kCols; ++q) u[i][q] += w[q];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float g[kCols];
                param_values<T>(a.gate, col[i], in[i], 1.0f, g);
#pragma unroll
                for (int q = 0; q < kCols; ++q) h[i][q] = fmaf(u[i][q], by * g[q], h[i][q]);
                if (a.h) Eight<T>::put(static_cast<T *>(a.h) + r * a.ld_h + col[i], h[i], in[i]);
            }
        }
        if (!a.n) continue;
        float mean = 0.0f;
        if constexpr (LAYER) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i])
#pragma unroll
                    for (int q = 0; q < kCols; ++q) sum[0] += h[i][q];
            row_sums(s, turn, sum);
            mean = sum[0] * per_col;
        }
        float square[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i])
#pragma unroll
                for (int q = 0; q < kCols; ++q) {
                    if constexpr (LAYER) h[i][q] -= mean;
                    square[0] = fmaf(h[i][q], h[i][q], square[0]);
                }
        row_sums(s, turn, square);
        const float factor = rsqrtf(fmaf(square[0], per_col, a.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float w[kCols];
            param_values<T>(a.weight, col[i], in[i], 1.0f, w);
#pragma unroll
            for (int q = 0; q < kCols; ++q) h[i][q] *= factor * w[q];
            if (LAYER && a.bias) {
                param_values<T>(a.bias, col[i], in[i], 0.0f, w);
#pragma unroll
                for (int q = 0; q < kCols; ++q) h[i][q] += w[q];
            }
            Eight<T>::put(static_cast<T *>(a.n) + r * a.ld_n + col[i], h[i], in[i]);
        }
    }
}

// The gradients as dopt_norm_grad_kernel has them.  The sums of a row that do
// not wait for one another go together: an RMS norm takes two rounds of them
// (h's, y's and d_n's; then d_x's), a layer norm three.
template <typename T, int NV, bool LAYER>
__global__ void __launch_bounds__(NV == 1 ? 256 : kMostRow, NV == 1 ? 2 : 1)
    dopt_norm_grad_whole_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kSums = LAYER ? 4 : 2;
    constexpr int kPost = LAYER ? 2 : 1;
    __shared__ LaneSums sums[8];
    let_dependents_start();
    wait_for_grids_before();
    LaneSums &s = sums[threadIdx.y];
    int turn = 0;
    const float per_col = 1.0f / float(a.cols);
    int col[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) col[i] = RowValues<T, NV>::column(i), in[i] = col[i] < a.cols;
    const int64_t step = int64_t(gridDim.x) * blockDim.y;
    int64_t r = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    Eight<T> raw_h[NV], raw_y[NV], raw_dn[NV], raw_dh[NV];
    float row_gate = 1.0f;
    const bool with_n = a.d_n != nullptr, with_y = a.y != nullptr, with_h = a.d_h != nullptr;
    auto fetch = [&](int64_t row) {
        const bool there = row < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool here = there && in[i];
            raw_h[i].load(static_cast<const T *>(a.x) + row * a.ld_x + col[i], here && with_n);
            raw_dn[i].load(static_cast<const T *>(a.d_n) + row * a.ld_d_n + col[i], here && with_n);
            raw_y[i].load(static_cast<const T *>(a.y) + row * a.ld_y + col[i], here && with_y);
            raw_dh[i].load(static_cast<const T *>(a.d_h) + row * a.ld_d_h + col[i], here && with_h);
        }
        if (a.row_gate && there) row_gate = a.row_gate[row];
    };
    float acc[kSums][NV][kCols] = {};
    fetch(r);
    for (; r < a.rows; r += step) {
        float h[NV][kCols], d[NV][kCols], u[NV][kCols], dx[NV][kCols];
        const float by = a.scale * row_gate;
#pragma unroll
        for (int i = 0; i < NV; ++i) raw_h[i].get(h[i]), raw_dn[i].get(d[i]), raw_y[i].get(u[i]), raw_dh[i].get(dx[i]);
        fetch(r + step);
        float h_mean = 0.0f, y_mean = 0.0f;
        if constexpr (LAYER) {
            float f[2] = {};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < kCols; ++q) f[0] += h[i][q], f[1] += u[i][q];
            row_sums(s, turn, f);
            h_mean = f[0] * per_col, y_mean = a.post ? f[1] * per_col : 0.0f;
        }
        float f[4] = {};  // of (h - mean)^2, (y - mean)^2, d_n w (h - mean), d_n w
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float w[kCols];
            param_values<T>(a.weight, col[i], in[i], 1.0f, w);
            if (in[i])
#pragma unroll
                for (int q = 0; q < kCols; ++q) {
                    if constexpr (LAYER) h[i][q] -= h_mean, u[i][q] -= y_mean;
                    const float g = d[i][q] * w[q];
                    f[0] = fmaf(h[i][q], h[i][q], f[0]);
                    f[1] = fmaf(u[i][q], u[i][q], f[1]);
                    f[2] = fmaf(g, h[i][q], f[2]);
                    if constexpr (LAYER) f[3] += g;
                }
        }
        row_sums(s, turn, f);
        const float h_factor = a.d_n ? rsqrtf(fmaf(f[0], per_col, a.eps)) : 0.0f;
        const float y_factor = a.post ? rsqrtf(fmaf(f[1], per_col, a.eps)) : 1.0f;
        const float along = f[2] * h_factor * per_col, level = f[3] * per_col;
        float dot[4] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float w[kCols];
            param_values<T>(a.weight, col[i], in[i], 1.0f, w);
#pragma unroll
            for (int q = 0; q < kCols; ++q) {
                h[i][q] *= h_factor;
                acc[0][i][q] = fmaf(d[i][q], h[i][q], acc[0][i][q]);
                if constexpr (LAYER) acc[1][i][q] += d[i][q];
                float g = d[i][q] * w[q];
                if constexpr (LAYER) g -= level;
                dx[i][q] = fmaf(h_factor, fmaf(-h[i][q], along, g), dx[i][q]);
            }
            if (a.h) Eight<T>::put(static_cast<T *>(a.h) + r * a.ld_h + col[i], dx[i], in[i]);
            if (!in[i])
#pragma unroll
                for (int q = 0; q < kCols; ++q) dx[i][q] = 0.0f;
        }
        if (!a.y) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float w[kCols], g[kCols];
            param_values<T>(a.post_weight, col[i], in[i], 1.0f, w);
            param_values<T>(a.gate, col[i], in[i], 1.0f, g);
            if (a.d_row_gate) {
                float b[kCols];
                param_values<T>(a.post_bias, col[i], in[i], 0.0f, b);
#pragma unroll
                for (int q = 0; q < kCols; ++q) dot[2] = fmaf(dx[i][q] * g[q], fmaf(u[i][q] * y_factor, w[q], b[q]), dot[2]);
            }
#pragma unroll
            for (int q = 0; q < kCols; ++q) {
                u[i][q] *= y_factor;
                const float v = by * dx[i][q];
                acc[kPost][i][q] = fmaf(v, u[i][q], acc[kPost][i][q]);
                if constexpr (LAYER) acc[kPost + 1][i][q] += v;
                dx[i][q] = v * (g[q] * w[q]);  // of hat(y)
                dot[0] = fmaf(dx[i][q], u[i][q], dot[0]);
                if constexpr (LAYER) dot[1] += dx[i][q];
            }
        }
        if (LAYER || a.d_row_gate) {
            if (a.post || a.d_row_gate) row_sums(s, turn, dot);
        } else if (a.post) {
            float one[1] = {dot[0]};
            row_sums(s, turn, one);
            dot[0] = one[0];
        }
        if (a.d_row_gate && threadIdx.x == 0) a.d_row_gate[r] = a.scale * dot[2];
        if (!a.n) continue;
        const float y_along = a.post ? dot[0] * per_col : 0.0f, y_level = LAYER && a.post ? dot[1] * per_col : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int q = 0; q < kCols; ++q) {
                float v = dx[i][q];
                if constexpr (LAYER) v -= y_level;
                dx[i][q] = y_factor * fmaf(-u[i][q], y_along, v);
            }
            Eight<T>::put(static_cast<T *>(a.n) + r * a.ld_n + col[i], dx[i], in[i]);
        }
    }
    const int64_t group = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
#pragma unroll
    for (int k = 0; k < kSums; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i]) continue;
            float4 *p = reinterpret_cast<float4 *>(a.partial + (group * kSums + k) * a.part_ld + col[i]);
            p[0] = make_float4(acc[k][i][0], acc[k][i][1], acc[k][i][2], acc[k][i][3]);
            p[1] = make_float4(acc[k][i][4], acc[k][i][5], acc[k][i][6], acc[k][i][7]);
        }
}

struct ParamGradArgs {
    const float *partial;
    const void *post_weight, *post_bias, *gate;
    void *grad;
    int64_t at[5];       // weight, bias, post_weight, post_bias, gate: where in grad, or -1
    int64_t part_ld;
    int32_t groups, cols, layer, post, accumulate;
};

// The groups' sums added, in an order of their numbers alone, and the params'
// gradients made of them.  A block: 32 columns, by 32 warps.
template <typename T, typename G, bool LAYER>
__global__ void __launch_bounds__(1024) dopt_norm_param_kernel(const __grid_constant__ ParamGradArgs a) {
    __shared__ float part[32][4][33];
    let_dependents_start();
    wait_for_grids_before();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = int(blockIdx.x) * 32 + lane;
    constexpr int kSums = LAYER ? 4 : 2, kAhead = 16 / kSums;
    float f[4] = {};
    if (c < a.cols)
        for (int g0 = warp; g0 < a.groups; g0 += 32 * kAhead) {
            float v[kAhead][kSums];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int k = 0; k < kSums; ++k) {
                    const int g = g0 + 32 * j;
                    v[j][k] = g < a.groups ? __ldcs(a.partial + (int64_t(g) * kSums + k) * a.part_ld + c) : 0.0f;
                }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int k = 0; k < kSums; ++k) f[k] += v[j][k];
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) part[warp][k][lane] = f[k];
    __syncthreads();
    if (warp > 0 || c >= a.cols) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[k] = 0.0f;
        for (int w = 0; w < 32; ++w) f[k] += part[w][k][lane];
    }
    const float d_weight = f[0], d_bias = f[1], along = LAYER ? f[2] : f[1], level = f[3];
    auto value = [&](const void *p, float none) { return p ? to_f32(static_cast<const T *>(p)[c]) : none; };
    const float gate = value(a.gate, 1.0f);
    const float found[5] = {d_weight, d_bias, gate * along, gate * level,
                            fmaf(value(a.post_weight, 1.0f), along, LAYER ? value(a.post_bias, 0.0f) * level : 0.0f)};
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        if (a.at[i] < 0) continue;
        G *p = static_cast<G *>(a.grad) + a.at[i] + c;
        *p = from_f32<G>(a.accumulate ? to_f32(*p) + found[i] : found[i]);
    }
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

template <typename T, int NV, bool LAYER>
int launch_norm(const char *who, const NormArgs &a, bool backward, int64_t blocks, dim3 block, cudaStream_t stream) {
    const dim3 grid{unsigned(blocks)};
    if (a.vec && a.vec_params && a.cols % kCols == 0)
        return backward ? launch_op(who, dopt_norm_grad_whole_kernel<T, NV, LAYER>, grid, block, 0, stream, a)
                        : launch_op(who, dopt_norm_whole_kernel<T, NV, LAYER>, grid, block, 0, stream, a);
    return backward ? launch_op(who, dopt_norm_grad_kernel<T, NV, LAYER>, grid, block, 0, stream, a)
                    : launch_op(who, dopt_norm_kernel<T, NV, LAYER>, grid, block, 0, stream, a);
}
template <typename T, bool LAYER>
int launch_norm(const char *who, const NormArgs &a, bool backward, int64_t blocks, const NormShape &shape,
                cudaStream_t stream) {
    switch (shape.nv) {
        case 1: return launch_norm<T, 1, LAYER>(who, a, backward, blocks, shape.block, stream);
        case 2: return launch_norm<T, 2, LAYER>(who, a, backward, blocks, shape.block, stream);
        default: return launch_norm<T, 4, LAYER>(who, a, backward, blocks, shape.block, stream);
    }
}
int launch_norm(const char *who, dopt_dtype dtype, bool layer, const NormArgs &a, bool backward, int64_t blocks,
                const NormShape &shape, cudaStream_t stream) {
    switch (dtype) {
        case DOPT_BF16:
            return layer ? launch_norm<__nv_bfloat16, true>(who, a, backward, blocks, shape, stream)
                         : launch_norm<__nv_bfloat16, false>(who, a, backward, blocks, shape, stream);
        case DOPT_FP16:
            return layer ? launch_norm<__half, true>(who, a, backward, blocks, shape, stream)
                         : launch_norm<__half, false>(who, a, backward, blocks, shape, stream);
        default:
            return layer ? launch_norm<float, true>(who, a, backward, blocks, shape, stream)
                         : launch_norm<float, false>(who, a, backward, blocks, shape, stream);
    }
}

template <typename T, typename G>
int launch_params(const char *who, const ParamGradArgs &a, cudaStream_t stream) {
    const dim3 grid(unsigned((a.cols + 31) / 32));
    return a.layer ? launch_op(who, dopt_norm_param_kernel<T, G, true>, grid, dim3(1024), 0, stream, a)
                   : launch_op(who, dopt_norm_param_kernel<T, G, false>, grid, dim3(1024), 0, stream, a);
}
template <typename T>
int launch_params(const char *who, dopt_dtype grad, const ParamGradArgs &a, cudaStream_t stream) {
    switch (grad) {
        case DOPT_BF16: return launch_params<T, __nv_bfloat16>(who, a, stream);
        case DOPT_FP16: return launch_params<T, __half>(who, a, stream);
        default: return launch_params<T, float>(who, a, stream);
    }
}

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

extern "C" int dopt_norm(const dopt_norm_cfg *cfg, const dopt_norm_params *params, dopt_dtype dtype, int64_t rows,
                         int64_t cols, const void *x, int64_t ld_x, const void *y, int64_t ld_y, void *h, int64_t ld_h,
                         void *n, int64_t ld_n, cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_norm";
    OpRange range(who);
    int rc = check_norm(who, cfg, params, dtype, rows, cols, y);
    if (rc != DOPT_OK) return rc;
    if (rows > 0 && !x) return fail(DOPT_E_ARG, "%s: x is NULL", who);
    if (!n && !h && rows > 0) return fail(DOPT_E_ARG, "%s: neither n nor h is wanted", who);
    if (rows > 0 && h && !y) return fail(DOPT_E_ARG, "%s: h without y is x", who);
    const size_t b = elem_bytes(dtype);
    uint64_t bits = 0;
    if ((rc = check_rows(who, "x", x, ld_x, cols, b, bits)) != DOPT_OK ||
        (rc = check_rows(who, "y", y, ld_y, cols, b, bits)) != DOPT_OK ||
        (rc = check_rows(who, "h", h, ld_h, cols, b, bits)) != DOPT_OK ||
        (rc = check_rows(who, "n", n, ld_n, cols, b, bits)) != DOPT_OK)
        return rc;
    if (rows == 0) return DOPT_OK;
    NormArgs a = norm_args(*cfg, *params, rows, cols);
    a.x = x, a.ld_x = ld_x;
    a.y = y, a.ld_y = ld_y;
    a.h = h, a.ld_h = ld_h;
    a.n = n, a.ld_n = ld_n;
    a.vec = bits % 16 == 0;
    const NormShape shape(cols, false);
    const int64_t blocks = std::min<int64_t>((rows + shape.block.y - 1) / shape.block.y, 152 * 4);
    return launch_norm(who, dtype, cfg->kind == DOPT_NORM_LAYER, a, false, blocks, shape, stream);
}

extern "C" int dopt_norm_workspace(int64_t rows, int64_t cols, int64_t *bytes) {
    dopt::clear_error();
    const char *who = "dopt_norm_workspace";
    if (!bytes) return dopt::fail(DOPT_E_ARG, "%s: bytes is NULL", who);
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > DOPT_NORM_MAX_COLS)
        return dopt::fail(DOPT_E_ARG, "%s: %lld rows of %lld columns", who, static_cast<long long>(rows),
                          static_cast<long long>(cols));
    // (groups of a block's rows that there are not have sums too)
    *bytes = std::min<int64_t>(kParts, (rows + 7) / 8 * 8) * 4 * norm_part_ld(cols) * int64_t(sizeof(float));
    return DOPT_OK;
}

extern "C" int dopt_norm_grad(const dopt_norm_cfg *cfg, const dopt_norm_params *params, dopt_dtype dtype, int64_t rows,
                              int64_t cols, const void *h, int64_t ld_h, const void *y, int64_t ld_y, const void *d_n,
                              int64_t ld_d_n, const void *d_h, int64_t ld_d_h, void *d_x, int64_t ld_d_x, void *d_y,
                              int64_t ld_d_y, float *d_row_gate, void *grad, dopt_dtype grad_dtype, int64_t grad_numel,
                              const int64_t grad_offsets[5], uint32_t flags, void *workspace, int64_t workspace_bytes,
                              cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_norm_grad";
    OpRange range(who);
    int rc = check_norm(who, cfg, params, dtype, rows, cols, y);
    if (rc != DOPT_OK) return rc;
    if (flags & ~uint32_t(DOPT_NORM_ACCUMULATE)) return fail(DOPT_E_ARG, "%s: unknown flags 0x%x", who, flags);
    if (rows > 0 && d_n && !h) return fail(DOPT_E_ARG, "%s: d_n without h", who);
    if (rows > 0 && !d_n && !d_h) return fail(DOPT_E_ARG, "%s: neither d_n nor d_h", who);
    if (rows > 0 && d_y && !y) return fail(DOPT_E_ARG, "%s: d_y without y", who);
    if (rows > 0 && d_row_gate && !params->row_gate) return fail(DOPT_E_ARG, "%s: d_row_gate without row_gate", who);
    if (!aligned_to(d_row_gate, 4)) return fail(DOPT_E_ALIGN, "%s: d_row_gate is not 4-byte aligned", who);
    const size_t b = elem_bytes(dtype);
    uint64_t bits = 0;
    if ((rc = check_rows(who, "h", h, ld_h, cols, b, bits)) != DOPT_OK ||
        (rc = check_rows(who, "y", y, ld_y, cols, b, bits)) != DOPT_OK ||
        (rc = check_rows(who, "d_n", d_n, ld_d_n, cols, b, bits)) != DOPT_OK ||
        (rc = check_rows(who, "d_h", d_h, ld_d_h, cols, b, bits)) != DOPT_OK ||
        (rc = check_rows(who, "d_x", d_x, ld_d_x, cols, b, bits)) != DOPT_OK ||
        (rc = check_rows(who, "d_y", d_y, ld_d_y, cols, b, bits)) != DOPT_OK)
        return rc;
    ParamGradArgs p{};
    bool wanted = false;
    if (grad_offsets) {
        const bool layer = cfg->kind == DOPT_NORM_LAYER;
        const bool in_norm = rows == 0 || d_n, in_block = rows == 0 || y;
        const bool there[5] = {in_norm, layer && in_norm, in_block && cfg->post, layer && in_block && cfg->post, in_block};
        for (int i = 0; i < 5; ++i) {
            const int64_t at = grad_offsets[i];
            p.at[i] = at;
            if (at == -1) continue;
            wanted = true;
            if (!there[i]) return fail(DOPT_E_ARG, "%s: the gradient of a param that takes no part (%d)", who, i);
            if (at < 0 || at > grad_numel - cols)
                return fail(DOPT_E_ARG, "%s: %lld grads at %lld leave a buffer of %lld", who,
                            static_cast<long long>(cols), static_cast<long long>(at), static_cast<long long>(grad_numel));
            for (int j = 0; j < i; ++j)
                if (p.at[j] >= 0 && at < p.at[j] + cols && p.at[j] < at + cols)
                    return fail(DOPT_E_ARG, "%s: two params' grads overlap", who);
        }
    }
    if (wanted) {
        if (!grad || !valid_dtype(grad_dtype)) return fail(DOPT_E_ARG, "%s: NULL grad or unknown dtype", who);
        if (!aligned_to(grad, elem_bytes(grad_dtype)))
            return fail(DOPT_E_ALIGN, "%s: grad is not aligned to its elements", who);
    }
    int64_t need = 0;
    if ((rc = dopt_norm_workspace(rows, cols, &need)) != DOPT_OK) return rc;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(DOPT_E_ARG, "%s: workspace of %lld bytes, %lld are needed", who,
                    static_cast<long long>(workspace ? workspace_bytes : 0), static_cast<long long>(need));
    if (!aligned_to(workspace, 16)) return fail(DOPT_E_ALIGN, "%s: workspace is not 16-byte aligned", who);
    const bool layer = cfg->kind == DOPT_NORM_LAYER;
    int64_t groups = 0;
    if (rows > 0) {
        NormArgs a = norm_args(*cfg, *params, rows, cols);
        a.x = h, a.ld_x = ld_h;
        a.y = y, a.ld_y = ld_y;
        a.d_n = d_n, a.ld_d_n = ld_d_n;
        a.d_h = d_h, a.ld_d_h = ld_d_h;
        a.h = d_x, a.ld_h = ld_d_x;
        a.n = d_y, a.ld_n = ld_d_y;
        a.d_row_gate = d_row_gate;
        a.partial = static_cast<float *>(workspace);
        a.part_ld = norm_part_ld(cols);
        a.vec = bits % 16 == 0;
        const NormShape shape(cols, true);
        const int64_t blocks = std::min<int64_t>((rows + shape.block.y - 1) / shape.block.y,
                                                 std::min<int64_t>(152 * 2, kParts / shape.block.y));
        groups = blocks * shape.block.y;
        if ((rc = launch_norm(who, dtype, layer, a, true, blocks, shape, stream)) != DOPT_OK) return rc;
    }
    if (!wanted || (rows == 0 && flags & DOPT_NORM_ACCUMULATE)) return DOPT_OK;
    p.partial = static_cast<const float *>(workspace);
    p.post_weight = params->post_weight;
    p.post_bias = params->post_bias;
    p.gate = params->gate;
    p.grad = grad;
    p.part_ld = norm_part_ld(cols);
    p.groups = int32_t(groups);
    p.cols = int32_t(cols);
    p.layer = layer;
    p.accumulate = (flags & DOPT_NORM_ACCUMULATE) != 0;
    switch (dtype) {
        case DOPT_BF16: return launch_params<__nv_bfloat16>(who, grad_dtype, p, stream);
        case DOPT_FP16: return launch_params<__half>(who, grad_dtype, p, stream);
        default: return launch_params<float>(who, grad_dtype, p, stream);
    }
}
