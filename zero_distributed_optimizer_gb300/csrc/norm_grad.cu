// The gradients of the norms around a block (dopt_norm_grad); dopt.h states the
// contract.
//
// One pass over the rows, which reads h, y and both gradients once and writes
// d_x and d_y; a thread keeps the sums over its rows that the params' gradients
// are made of, and a second launch adds the groups' sums.  Four streams in and
// two out need few instructions a value: sums of a row that do not wait for one
// another go together, arithmetic is two columns an instruction.  16384 x 2048
// bf16 with a norm before and after and a gate: 91 us, 4.4 TB/s, instructions in
// 60 % of the issue slots at two blocks an SM (three spill: 150 us); 259 us
// with a row's loads waited for, 143 with the next row's in flight, 100 with
// few shuffles a sum, 94 with two columns an instruction; layer norms 138.
// Rows of more than 2048 columns take two groups of columns a thread, of more than
// 8192 four, and spill: 460-960 bytes a thread and 1560-2672 (fp32 the most; of
// up to 2048 columns fp32 layer norms alone, 108).  As many bytes in rows of 4096
// columns 147 us (layer 173), of 8192 175 (205), of 16384 329 (468).  Rows of 2047
// columns, whose loads are waited for, 308 (350).
#include "norm.cuh"

namespace {

// Rows of any alignment and width.
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
        float dot[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i);
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
            const int c = column(i);
            if (c >= a.cols) continue;  // (part_ld is a multiple of 8)
            float4 *p = reinterpret_cast<float4 *>(a.partial + (group * kSums + k) * a.part_ld + c);
            p[0] = make_float4(acc[k][i][0], acc[k][i][1], acc[k][i][2], acc[k][i][3]);
            p[1] = make_float4(acc[k][i][4], acc[k][i][5], acc[k][i][6], acc[k][i][7]);
        }
}

// Rows and params that are 16-byte aligned, of a multiple of 8 columns.
// The gradients as dopt_norm_grad_kernel has them.  The sums of a row that do
// not wait for one another go together: an RMS norm takes two rounds of them
// (h's, y's and d_n's; then d_x's), a layer norm three.
template <typename T, int NV, bool LAYER>
__global__ void __launch_bounds__(NV == 1 ? 256 : kMostRow, NV == 1 ? 2 : 1)
    dopt_norm_grad_whole_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kSums = LAYER ? 4 : 2;
    constexpr int kPost = LAYER ? 2 : 1;
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
    const int64_t step = int64_t(gridDim.x) * blockDim.y;
    int64_t r = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    Eight<T> raw_h[NV], raw_y[NV], raw_dn[NV], raw_dh[NV];
    F2 branch[NV][kPairs] = {};  // gate * post_weight
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        raw_h[i].zero(), raw_y[i].zero(), raw_dn[i].zero(), raw_dh[i].zero();
        F2 w[kPairs] = {}, g[kPairs] = {};
        param_values<T>(a.post_weight, col[i], in[i], 1.0f, w);
        param_values<T>(a.gate, col[i], in[i], 1.0f, g);
#pragma unroll
        for (int q = 0; q < kPairs; ++q) branch[i][q] = g[q] * w[q];
    }
    float row_gate = 1.0f;
    const T *h_at = static_cast<const T *>(a.x) + r * a.ld_x, *y_at = static_cast<const T *>(a.y) + r * a.ld_y;
    const T *dn_at = static_cast<const T *>(a.d_n) + r * a.ld_d_n, *dh_at = static_cast<const T *>(a.d_h) + r * a.ld_d_h;
    const bool with_n = a.d_n != nullptr, with_y = a.y != nullptr, with_h = a.d_h != nullptr;
    auto fetch = [&](int64_t row) {
        const bool there = row < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool here = there && in[i];
            raw_h[i].load(h_at + col[i], here && with_n);
            raw_dn[i].load(dn_at + col[i], here && with_n);
            raw_y[i].load(y_at + col[i], here && with_y);
            raw_dh[i].load(dh_at + col[i], here && with_h);
        }
        h_at += step * a.ld_x, dn_at += step * a.ld_d_n, y_at += step * a.ld_y, dh_at += step * a.ld_d_h;
        if (a.row_gate && there) row_gate = a.row_gate[row];
    };
    F2 acc[kSums][NV][kPairs] = {};
    fetch(r);
    for (; r < a.rows; r += step) {
        F2 h[NV][kPairs] = {}, d[NV][kPairs] = {}, u[NV][kPairs] = {}, dx[NV][kPairs] = {};
        const float by = a.scale * row_gate;
#pragma unroll
        for (int i = 0; i < NV; ++i) raw_h[i].get(h[i]), raw_dn[i].get(d[i]), raw_y[i].get(u[i]), raw_dh[i].get(dx[i]);
        fetch(r + step);
        if constexpr (LAYER) {
            F2 sum[2] = {F2(0.0f), F2(0.0f)};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < kPairs; ++q) sum[0] = sum[0] + h[i][q], sum[1] = sum[1] + u[i][q];
            float f[2] = {both(sum[0]), both(sum[1])};
            row_sums(s, turn, f);
            // (divided: so many times a rounded 1 / cols leaves constant rows a residue)
            const F2 h_less(-f[0] / float(a.cols)), y_less(a.post ? -f[1] / float(a.cols) : 0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i])
#pragma unroll
                    for (int q = 0; q < kPairs; ++q) h[i][q] = h[i][q] + h_less, u[i][q] = u[i][q] + y_less;
        }
        float f[4];  // of (h - mean)^2, (y - mean)^2, d_n w (h - mean), d_n w
        {
            F2 sum[4] = {F2(0.0f), F2(0.0f), F2(0.0f), F2(0.0f)};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                F2 w[kPairs] = {};
                param_values<T>(a.weight, col[i], in[i], 1.0f, w);
#pragma unroll
                for (int q = 0; q < kPairs; ++q) {
                    const F2 g = d[i][q] * w[q];
                    sum[0] = fma2(h[i][q], h[i][q], sum[0]);
                    sum[1] = fma2(u[i][q], u[i][q], sum[1]);
                    sum[2] = fma2(g, h[i][q], sum[2]);
                    if constexpr (LAYER) sum[3] = sum[3] + g;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = both(sum[k]);
        }
        row_sums(s, turn, f);
        const float h_factor = with_n ? rsqrtf(fmaf(f[0], per_col, a.eps)) : 0.0f;
        const float y_factor = a.post ? rsqrtf(fmaf(f[1], per_col, a.eps)) : 1.0f;
        // d_x = d_h + factor (d_n w - mean(d_n w) - hat mean(d_n w hat))
        const F2 less_along(-f[2] * h_factor * per_col), less_level(-f[3] * per_col), by2(by), hf(h_factor), yf(y_factor);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F2 w[kPairs] = {};
            param_values<T>(a.weight, col[i], in[i], 1.0f, w);
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                const F2 hat = h[i][q] * hf;
                acc[0][i][q] = fma2(d[i][q], hat, acc[0][i][q]);
                if constexpr (LAYER) acc[1][i][q] = acc[1][i][q] + d[i][q];
                const F2 g = LAYER ? fma2(d[i][q], w[q], less_level) : d[i][q] * w[q];
                dx[i][q] = fma2(fma2(hat, less_along, g), hf, dx[i][q]);
            }
            if (a.h) Eight<T>::put(static_cast<T *>(a.h) + r * a.ld_h + col[i], dx[i], in[i]);
        }
        if (!with_y) continue;
        F2 dot[3] = {F2(0.0f), F2(0.0f), F2(0.0f)};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i]) continue;  // (a layer norm's level was taken off the values past the row too)
            if (a.d_row_gate) {  // u * gate = hat(y) * branch + post_bias * gate
                F2 b[kPairs] = {}, g[kPairs] = {};
                param_values<T>(LAYER ? a.post_bias : nullptr, col[i], in[i], 0.0f, b);
                param_values<T>(a.gate, col[i], in[i], 1.0f, g);
#pragma unroll
                for (int q = 0; q < kPairs; ++q)
                    dot[2] = fma2(dx[i][q], fma2(u[i][q] * yf, branch[i][q], b[q] * g[q]), dot[2]);
            }
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                u[i][q] = u[i][q] * yf;
                const F2 v = dx[i][q] * by2;
                acc[kPost][i][q] = fma2(v, u[i][q], acc[kPost][i][q]);
                if constexpr (LAYER) acc[kPost + 1][i][q] = acc[kPost + 1][i][q] + v;
                dx[i][q] = v * branch[i][q];  // of hat(y)
                dot[0] = fma2(dx[i][q], u[i][q], dot[0]);
                if constexpr (LAYER) dot[1] = dot[1] + dx[i][q];
            }
        }
        float t[4] = {both(dot[0]), both(dot[1]), both(dot[2]), 0.0f};
        if (LAYER || a.d_row_gate) {
            if (a.post || a.d_row_gate) row_sums(s, turn, t);
        } else if (a.post) {
            float one[1] = {t[0]};
            row_sums(s, turn, one);
            t[0] = one[0];
        }
        if (a.d_row_gate && threadIdx.x == 0) a.d_row_gate[r] = a.scale * t[2];
        if (!a.n) continue;
        const F2 y_along(a.post ? -t[0] * per_col : 0.0f), y_level(LAYER && a.post ? -t[1] * per_col : 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                const F2 v = LAYER ? dx[i][q] + y_level : dx[i][q];
                dx[i][q] = fma2(u[i][q], y_along, v) * yf;
            }
            Eight<T>::put(static_cast<T *>(a.n) + r * a.ld_n + col[i], dx[i], in[i]);
        }
    }
    const int64_t group = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
#pragma unroll
    for (int k = 0; k < kSums; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) Eight<float>::put(a.partial + (group * kSums + k) * a.part_ld + col[i], acc[k][i], true);
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

template <typename T, int NV, bool LAYER>
int launch_norm(const char *who, const NormArgs &a, int64_t blocks, dim3 block, cudaStream_t stream) {
    const bool whole = a.vec && a.vec_params && a.cols % kCols == 0;
    return launch_op(who, whole ? dopt_norm_grad_whole_kernel<T, NV, LAYER> : dopt_norm_grad_kernel<T, NV, LAYER>, dim3(unsigned(blocks)), block,
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

}  // namespace

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
        if ((rc = launch_norm(who, dtype, layer, a, blocks, shape, stream)) != DOPT_OK) return rc;
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
