// The weight gradients of a linear layer, or of a layer's experts, from the
// 8-bit checkpoint of its input, written into the flat grad buffer
// (dopt_ckpt_wgrad; dopt.h states the contract).
#include "op_common.cuh"

namespace {

struct WgradArgs {
    const uint8_t *codes, *scales;
    const int32_t *row_token;  // or NULL: row r reads checkpoint row r
    const void *dy;
    const int32_t *offsets;    // or NULL: one group of all rows
    void *grad;
    int64_t x_rows, cols, pitch;
    int64_t dy_rows, outs, dy_ld;
    int32_t accumulate;
    int64_t grad_offset[DOPT_MAX_GROUPS];
};

constexpr int kTile = 64;
constexpr int kStep = 16;

// A CTA takes 64 x 64 values of one group's gradient and goes through the
// group's rows 16 at a time.
template <typename T, typename G>
__global__ void __launch_bounds__(256) dopt_ckpt_wgrad_kernel(const __grid_constant__ WgradArgs a) {
    __shared__ float ys[kStep][kTile], xs[kStep][kTile];
    let_dependents_start();
    wait_for_grids_before();
    const int g = blockIdx.z;
    const int64_t o0 = int64_t(blockIdx.y) * kTile, c0 = int64_t(blockIdx.x) * kTile;
    int64_t lo = 0, hi = a.dy_rows;
    if (a.offsets) {
        lo = min(max(int64_t(a.offsets[g]), int64_t(0)), a.dy_rows);
        hi = min(max(int64_t(a.offsets[g + 1]), lo), a.dy_rows);
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t r0 = lo; r0 < hi; r0 += kStep) {
        for (int i = threadIdx.x; i < kStep * kTile; i += 256) {
            const int q = i / kTile, e = i % kTile;
            const int64_t r = r0 + q;
            float y = 0.0f, x = 0.0f;
            if (r < hi) {
                if (o0 + e < a.outs) y = to_f32(static_cast<const T *>(a.dy)[r * a.dy_ld + o0 + e]);
                const int64_t t = a.row_token ? a.row_token[r] : r;
                if (t >= 0 && t < a.x_rows && c0 + e < a.cols) {
                    const int64_t at = t * a.pitch + c0 + e;
                    x = float(int8_t(a.codes[at])) * ckpt_step(a.scales[at / kBlock]);
                }
            }
            ys[q][e] = y;
            xs[q][e] = x;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kStep; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ys[q][ty * 4 + i], xs[q][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    G *grad = static_cast<G *>(a.grad) + a.grad_offset[g];
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t o = o0 + ty * 4 + i, c = c0 + tx + 16 * j;
            if (o >= a.outs || c >= a.cols) continue;
            G *p = grad + o * a.cols + c;
            *p = from_f32<G>(a.accumulate ? to_f32(*p) + acc[i][j] : acc[i][j]);
        }
}

template <typename T, typename G>
int launch_wgrad(const char *who, const WgradArgs &a, int n_groups, cudaStream_t stream) {
    const dim3 grid(unsigned((a.cols + kTile - 1) / kTile), unsigned((a.outs + kTile - 1) / kTile),
                    unsigned(n_groups));
    return launch_op(who, dopt_ckpt_wgrad_kernel<T, G>, grid, dim3(256), 0, stream, a);
}

template <typename T>
int pick_wgrad(const char *who, const WgradArgs &a, int n_groups, dopt_dtype grad_dtype,
               cudaStream_t stream) {
    switch (grad_dtype) {
        case DOPT_BF16: return launch_wgrad<T, __nv_bfloat16>(who, a, n_groups, stream);
        case DOPT_FP16: return launch_wgrad<T, __half>(who, a, n_groups, stream);
        default: return launch_wgrad<T, float>(who, a, n_groups, stream);
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
    if (dy_dtype == DOPT_BF16) return pick_wgrad<__nv_bfloat16>(who, a, n_groups, grad_dtype, stream);
    return pick_wgrad<__half>(who, a, n_groups, grad_dtype, stream);
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
    *bytes = 0;
    return DOPT_OK;
}
