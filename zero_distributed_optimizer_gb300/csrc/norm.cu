// The norms around a block, with the residual add, the block's gates and its
// scale (dopt_norm); dopt.h states the contract.
//
// One pass over the rows, each row's values in the registers of its threads:
// x and y are read once, h and n written once.  What bounds it, with memory, is
// instructions, of which a row's sums have many: threads hold 16 columns from
// 1024 columns on (norm.cuh).  16384 x 2048 bf16 with a norm before and after
// and a gate: 46 us, 5.9 TB/s (146 us with a row's loads waited for, 63 with
// the next row's in flight, 47 with few shuffles a sum); layer norms, of two more
// sums a row, 65.  As many bytes in rows of 4096 columns 48 and 68 us; above those
// a thread holds 32 and spills 48-92 bytes (fp32 up to 424): of 8192 57 and 103,
// of 16384 65 and 110.  Rows of 2047 columns, whose loads are waited for, 160 and
// 192 (16-bit ones spill from 4097 columns on, bf16 layer norms a little and fp32
// ones from 1025).
#include "norm.cuh"

namespace {

// Rows of any alignment and width.
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
                const int c = column(i);
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

// Rows and params that are 16-byte aligned, of a multiple of 8 columns.
// The next row's loads are in flight under a row's sums: they go to the
// registers that this row's values came in.
template <typename T, int NV, bool LAYER>
__global__ void __launch_bounds__(NV == 4 ? kMostRow : 256, NV == 1 ? 4 : NV == 2 ? 2 : 1)
    dopt_norm_whole_kernel(const __grid_constant__ NormArgs a) {
    __shared__ RowSums sums[8];
    let_dependents_start();
    wait_for_grids_before();
    RowSums &s = sums[threadIdx.y];
    int turn = 0;
    const float per_col = 1.0f / float(a.cols);
    int col[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) col[i] = column(i), in[i] = col[i] < a.cols;
    Eight<T> x[NV], y[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i].zero(), y[i].zero();
    const int64_t step = int64_t(gridDim.x) * blockDim.y;
    int64_t r = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
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
    // v less its mean (layer norm; values past the row stay 0), and its factor
    auto standard = [&](F2(&v)[NV][kPairs]) {
        if constexpr (LAYER) {
            F2 sum(0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < kPairs; ++q) sum = sum + v[i][q];
            float f[1] = {both(sum)};
            row_sums(s, turn, f);
            const F2 less(-f[0] / float(a.cols));  // (divided: so many times a rounded 1 / cols leaves constant rows a residue)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i])
#pragma unroll
                    for (int q = 0; q < kPairs; ++q) v[i][q] = v[i][q] + less;
        }
        F2 square(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < kPairs; ++q) square = fma2(v[i][q], v[i][q], square);
        float f[1] = {both(square)};
        row_sums(s, turn, f);
        return rsqrtf(fmaf(f[0], per_col, a.eps));
    };
    // v * factor * weight + bias
    auto affine = [&](F2(&v)[NV][kPairs], float factor, const void *weight, const void *bias) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F2 w[kPairs] = {F2(1.0f), F2(1.0f), F2(1.0f), F2(1.0f)}, b[kPairs] = {F2(0.0f), F2(0.0f), F2(0.0f), F2(0.0f)};
            param_values<T>(weight, col[i], in[i], 1.0f, w);
            if (LAYER) param_values<T>(bias, col[i], in[i], 0.0f, b);
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                v[i][q] = v[i][q] * F2(factor);
                v[i][q] = LAYER ? fma2(v[i][q], w[q], b[q]) : v[i][q] * w[q];
            }
        }
    };
    fetch(r);
    for (; r < a.rows; r += step) {
        F2 h[NV][kPairs] = {}, u[NV][kPairs] = {};
        const float by = a.scale * row_gate;
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i].get(h[i]), y[i].get(u[i]);
        fetch(r + step);
        if (with_y) {
            if (a.post) {
                const float factor = standard(u);
                affine(u, factor, a.post_weight, a.post_bias);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                F2 g[kPairs] = {};
                param_values<T>(a.gate, col[i], in[i], 1.0f, g);
                if (in[i])
#pragma unroll
                    for (int q = 0; q < kPairs; ++q) h[i][q] = fma2(u[i][q], g[q] * F2(by), h[i][q]);
                if (a.h) Eight<T>::put(static_cast<T *>(a.h) + r * a.ld_h + col[i], h[i], in[i]);
            }
        }
        if (!a.n) continue;
        const float factor = standard(h);
        affine(h, factor, a.weight, a.bias);
#pragma unroll
        for (int i = 0; i < NV; ++i) Eight<T>::put(static_cast<T *>(a.n) + r * a.ld_n + col[i], h[i], in[i]);
    }
}

template <typename T, int NV, bool LAYER>
int launch_norm(const char *who, const NormArgs &a, int64_t blocks, dim3 block, cudaStream_t stream) {
    const bool whole = a.vec && a.vec_params && a.cols % kCols == 0;
    return launch_op(who, whole ? dopt_norm_whole_kernel<T, NV, LAYER> : dopt_norm_kernel<T, NV, LAYER>, dim3(unsigned(blocks)), block,
                     0, stream, a);
}
template <typename T, bool LAYER>
int launch_norm(const char *who, const NormArgs &a, int64_t blocks, const NormShape &shape, cudaStream_t stream) {
    switch (shape.nv) {
        case 1: return launch_norm<T, 1, LAYER>(who, a, blocks, shape.block, stream);
        case 2: return launch_norm<T, 2, LAYER>(who, a, blocks, shape.block, stream);
        default: return launch_norm<T, 4, LAYER>(who, a, blocks, shape.block, stream);
    }
}
int launch_norm(const char *who, dopt_dtype dtype, bool layer, const NormArgs &a, int64_t blocks, const NormShape &shape,
                cudaStream_t stream) {
    switch (dtype) {
        case DOPT_BF16:
            return layer ? launch_norm<__nv_bfloat16, true>(who, a, blocks, shape, stream)
                         : launch_norm<__nv_bfloat16, false>(who, a, blocks, shape, stream);
        case DOPT_FP16:
            return layer ? launch_norm<__half, true>(who, a, blocks, shape, stream)
                         : launch_norm<__half, false>(who, a, blocks, shape, stream);
        default:
            return layer ? launch_norm<float, true>(who, a, blocks, shape, stream)
                         : launch_norm<float, false>(who, a, blocks, shape, stream);
    }
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
    return launch_norm(who, dtype, cfg->kind == DOPT_NORM_LAYER, a, blocks, shape, stream);
}
