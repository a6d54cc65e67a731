// Activations kept in 8 bits: saving (dopt_ckpt_save), reading back
// (dopt_ckpt_load) and an activation function's backward pass from its kept
// input (dopt_ckpt_act_grad).  dopt.h states the format.
//
// Every kernel gives a thread 16 columns of a row: half a block of 32, one
// 16-byte load or store of codes, two (four for fp32) of values.  A thread
// block covers bx threads' columns of `by` rows and strides over the rows,
// so no index is divided.
#include "op_common.cuh"

namespace {

constexpr int kCols = 16;  // columns a thread takes
constexpr int kCkptThreads = 256;

struct CkptArgs {
    const void *x;        // save: values; activation gradient: d_out
    void *out;            // load: values; activation gradient: d_in
    uint8_t *codes;       // [rows][pitch], the exponent bytes after them
    uint8_t *scales;      // [rows][pitch / 32]
    const int32_t *index; // load: row of each output row, or NULL
    int64_t rows;         // rows of the checkpoint
    int64_t n_out;        // rows the launch goes through
    int64_t cols, pitch;
    int64_t ld, ld_out;
    int64_t half;         // gated: columns of the output (cols / 2)
    int32_t min_exp;      // least exponent byte
    int32_t vec;          // rows are 16-byte aligned
};

// 16 values of a row from column c on; columns at or past `cols` are 0.
template <typename T>
__device__ __forceinline__ void load_vals(const T *row, int64_t c, int64_t cols, bool vec,
                                          float (&f)[kCols]) {
    constexpr int N = 16 / int(sizeof(T));
    if (vec && c + kCols <= cols) {
        uint4 raw[kCols / N];
#pragma unroll
        for (int i = 0; i < kCols / N; ++i) raw[i] = reinterpret_cast<const uint4 *>(row + c)[i];
#pragma unroll
        for (int i = 0; i < kCols / N; ++i) {
            float g[N];
            unpack<T, 16>(raw[i], g);
#pragma unroll
            for (int q = 0; q < N; ++q) f[i * N + q] = g[q];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) f[i] = c + i < cols ? to_f32(row[c + i]) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store_vals(T *row, int64_t c, int64_t cols, bool vec,
                                           const float (&f)[kCols]) {
    constexpr int N = 16 / int(sizeof(T));
    if (vec && c + kCols <= cols) {
#pragma unroll
        for (int i = 0; i < kCols / N; ++i) {
            float g[N];
#pragma unroll
            for (int q = 0; q < N; ++q) g[q] = f[i * N + q];
            reinterpret_cast<uint4 *>(row + c)[i] = pack<T, 16>(g);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i)
            if (c + i < cols) row[c + i] = from_f32<T>(f[i]);
    }
}

// The 16 kept values from column c (a multiple of 16) of row r on.
__device__ __forceinline__ void load_kept(const CkptArgs &a, int64_t r, int64_t c, float (&f)[kCols]) {
    const uint4 raw = *reinterpret_cast<const uint4 *>(a.codes + r * a.pitch + c);
    const float step = ckpt_step(a.scales[(r * a.pitch + c) / kBlock]);
    int8_t q[kCols];
    memcpy(q, &raw, sizeof q);
#pragma unroll
    for (int i = 0; i < kCols; ++i) f[i] = float(q[i]) * step;
}

// The kept values from any column on, one at a time.
__device__ __forceinline__ void load_kept_any(const CkptArgs &a, int64_t r, int64_t c, int64_t end,
                                              float (&f)[kCols]) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        f[i] = 0.0f;
        if (c + i < end) {
            const int64_t at = r * a.pitch + c + i;
            f[i] = float(int8_t(a.codes[at])) * ckpt_step(a.scales[at / kBlock]);
        }
    }
}

// A block of 32 columns is two neighbouring threads.  The step is the power
// of two 2^k with the largest magnitude in [64, 128) steps (k no less than
// the type's least); codes are round-to-nearest-even of value / step,
// clamped to 127.  Multiplying by a power of two is exact, so a code is one
// rounding of the value; and code * step has at most 7 significant bits, so
// the products of the backward pass read it in 16 bits without a second
// rounding.  The comparison of magnitudes as integers puts Inf and NaN above
// every finite value.
template <typename T>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_save_kernel(const CkptArgs a) {
    let_dependents_start();
    wait_for_grids_before();
    const int64_t c = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * kCols;
    if (c >= a.pitch) return;  // both threads of a block: the pitch is a multiple of 32
    // a block's two lanes of the warp (bx is 8, 16 or 32: a warp may hold several rows)
    const unsigned pair = 3u << ((threadIdx.y * blockDim.x + threadIdx.x) & 30);
    for (int64_t r = int64_t(blockIdx.y) * blockDim.y + threadIdx.y; r < a.rows;
         r += int64_t(gridDim.y) * blockDim.y) {
        float f[kCols];
        load_vals(static_cast<const T *>(a.x) + r * a.ld, c, a.cols, a.vec, f);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kCols; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(pair, top, 1));
        const bool finite = top < 0x7f800000u;
        const int byte = max(int(top >> 23) - 6, a.min_exp);
        const float inv = __uint_as_float(uint32_t(254 - byte) << 23);
        uint8_t q[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            const float v = fminf(fmaxf(f[i] * inv, -127.0f), 127.0f);
            q[i] = finite ? uint8_t(int8_t(__float2int_rn(v))) : 0;
        }
        uint4 raw;
        memcpy(&raw, q, sizeof raw);
        *reinterpret_cast<uint4 *>(a.codes + r * a.pitch + c) = raw;
        if ((threadIdx.x & 1) == 0)
            a.scales[(r * a.pitch + c) / kBlock] = uint8_t(finite ? byte : kNanByte);
    }
}

template <typename T>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_load_kernel(const CkptArgs a) {
    let_dependents_start();
    wait_for_grids_before();
    const int64_t c = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * kCols;
    if (c >= a.cols) return;
    for (int64_t o = int64_t(blockIdx.y) * blockDim.y + threadIdx.y; o < a.n_out;
         o += int64_t(gridDim.y) * blockDim.y) {
        const int64_t r = a.index ? a.index[o] : o;
        float f[kCols] = {};
        if (r >= 0 && r < a.rows) load_kept(a, r, c, f);
        store_vals(static_cast<T *>(a.out) + o * a.ld_out, c, a.cols, a.vec, f);
    }
}

// 1 / (1 + e^-x) and 1 - that, each with small relative error for |x| <= 87
// (further out e^-x leaves fp32's normal range).  Results that are rounded
// to 16 bits take the hardware's exponential and division (at most 2 +
// 1.173 |x| units in the last place of fp32, below 2^-16 over that range),
// fp32 ones the library's.
template <typename T>
__device__ __forceinline__ void sigmoid(float x, float &s, float &one_minus) {
    const float e = sizeof(T) == 4 ? expf(-x) : __expf(-x);
    s = sizeof(T) == 4 ? 1.0f / (1.0f + e) : __fdividef(1.0f, 1.0f + e);
    one_minus = e * s;
}
__device__ __forceinline__ float clamp_nan(float x, float b) {  // NaN stays NaN
    return x < -b ? -b : x > b ? b : x;
}

// silu'(h) = s (1 + h (1 - s)) and silu(h) = h s, s = sigmoid(h).  Below -87
// both are 0 to within 2e-36; above 87 they are 1 and h (and h (1 - s) must
// not become Inf * 0).
template <typename T>
__device__ __forceinline__ float silu_slope(float h, float &silu) {
    const float x = clamp_nan(h, 87.0f);
    float s, m;
    sigmoid<T>(x, s, m);
    silu = h < -87.0f ? 0.0f : h * s;
    return h < -87.0f ? 0.0f : s * fmaf(x, m, 1.0f);
}

// GELU in its tanh form is h p with p = (1 + tanh u) / 2 = sigmoid(2u),
// u = c (h + a h^3); its slope p + h 2 p (1 - p) c (1 + 3 a h^2).  Beyond
// |h| = 9.9 (2u = 85) it is 0 or 1 to within 1e-34.
template <typename T>
__device__ __forceinline__ float gelu_slope(float h) {
    constexpr float kC = 0.79788456080286536f, kA = 0.044715f;
    const float x = clamp_nan(h, 9.9f);
    const float x2 = x * x;
    float p, m;
    sigmoid<T>(2.0f * kC * x * fmaf(kA, x2, 1.0f), p, m);
    return h < -9.9f ? 0.0f : fmaf(2.0f * kC * x * fmaf(3.0f * kA, x2, 1.0f), p * m, p);
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_act_grad_kernel(const CkptArgs a) {
    let_dependents_start();
    wait_for_grids_before();
    const int64_t c = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * kCols;
    const int64_t width = ACT == DOPT_ACT_SWIGLU ? a.half : a.cols;
    if (c >= width) return;
    for (int64_t r = int64_t(blockIdx.y) * blockDim.y + threadIdx.y; r < a.rows;
         r += int64_t(gridDim.y) * blockDim.y) {
        float d[kCols], h[kCols];
        load_vals(static_cast<const T *>(a.x) + r * a.ld, c, width, a.vec, d);
        load_kept(a, r, c, h);
        T *out = static_cast<T *>(a.out) + r * a.ld_out;
        if constexpr (ACT == DOPT_ACT_SWIGLU) {
            float u[kCols];
            if (width % kBlock == 0)
                load_kept(a, r, width + c, u);
            else
                load_kept_any(a, r, width + c, a.cols, u);
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
                float silu;
                const float slope = silu_slope<T>(h[i], silu);
                h[i] = d[i] * u[i] * slope;
                u[i] = d[i] * silu;
            }
            store_vals(out, c, width, a.vec, h);
            store_vals(out + width, c, width, a.vec, u);
        } else {
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
                float silu;
                d[i] *= ACT == DOPT_ACT_SILU ? silu_slope<T>(h[i], silu) : gelu_slope<T>(h[i]);
            }
            store_vals(out, c, width, a.vec, d);
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

int check_ckpt(const char *who, const void *ckpt, int64_t rows, int64_t cols) {
    using dopt::fail;
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > DOPT_MAX_COLS)
        return fail(DOPT_E_ARG, "%s: rows %lld, cols %lld (rows below 2^31, cols in 1..%d)", who,
                    static_cast<long long>(rows), static_cast<long long>(cols), DOPT_MAX_COLS);
    if (rows > 0 && !ckpt) return fail(DOPT_E_ARG, "%s: checkpoint is NULL", who);
    if (!aligned_to(ckpt, 16)) return fail(DOPT_E_ALIGN, "%s: checkpoint is not 16-byte aligned", who);
    return DOPT_OK;
}

int check_values(const char *who, const char *name, const void *p, dopt_dtype dtype, int64_t cols,
                 int64_t ld) {
    using dopt::fail;
    if (!valid_dtype(dtype)) return fail(DOPT_E_ARG, "%s: unknown dtype %d", who, int(dtype));
    if (ld < cols)
        return fail(DOPT_E_ARG, "%s: %s has row stride %lld for %lld columns", who, name,
                    static_cast<long long>(ld), static_cast<long long>(cols));
    if (!p) return fail(DOPT_E_ARG, "%s: %s is NULL", who, name);
    if (!aligned_to(p, elem_bytes(dtype)))
        return fail(DOPT_E_ALIGN, "%s: %s is not aligned to its elements", who, name);
    return DOPT_OK;
}

bool vec_rows(const void *p, dopt_dtype dtype, int64_t ld) {
    return aligned_to(p, 16) && ld * int64_t(elem_bytes(dtype)) % 16 == 0;
}

CkptArgs ckpt_args(const void *ckpt, int64_t rows, int64_t cols) {
    CkptArgs a{};
    a.rows = rows;
    a.cols = cols;
    a.pitch = ckpt_pitch(cols);
    a.codes = static_cast<uint8_t *>(const_cast<void *>(ckpt));
    a.scales = a.codes + rows * a.pitch;
    return a;
}

// Blocks of bx threads along the columns and 256 / bx rows.
template <typename Kernel>
int launch_rows(const char *who, Kernel kernel, const CkptArgs &a, int64_t cols, int64_t rows,
                cudaStream_t stream) {
    const int64_t groups = (cols + kCols - 1) / kCols;
    const int bx = groups > 16 ? 32 : groups > 8 ? 16 : 8;
    const int by = kCkptThreads / bx;
    const dim3 grid(unsigned((groups + bx - 1) / bx),
                    unsigned(std::min<int64_t>((rows + by - 1) / by, 65535)));
    return launch_op(who, kernel, grid, dim3(bx, by), 0, stream, a);
}

template <typename T>
int launch_act(const char *who, dopt_act act, const CkptArgs &a, int64_t width, cudaStream_t stream) {
    switch (act) {
        case DOPT_ACT_SILU:
            return launch_rows(who, dopt_ckpt_act_grad_kernel<T, DOPT_ACT_SILU>, a, width, a.rows, stream);
        case DOPT_ACT_GELU:
            return launch_rows(who, dopt_ckpt_act_grad_kernel<T, DOPT_ACT_GELU>, a, width, a.rows, stream);
        default:
            return launch_rows(who, dopt_ckpt_act_grad_kernel<T, DOPT_ACT_SWIGLU>, a, width, a.rows, stream);
    }
}

}  // namespace

extern "C" int dopt_ckpt_bytes(int64_t rows, int64_t cols, int64_t *bytes) {
    dopt::clear_error();
    const char *who = "dopt_ckpt_bytes";
    if (!bytes) return dopt::fail(DOPT_E_ARG, "%s: bytes is NULL", who);
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > DOPT_MAX_COLS)
        return dopt::fail(DOPT_E_ARG, "%s: rows %lld, cols %lld (rows below 2^31, cols in 1..%d)", who,
                          static_cast<long long>(rows), static_cast<long long>(cols), DOPT_MAX_COLS);
    const int64_t pitch = ckpt_pitch(cols);
    *bytes = rows * (pitch + pitch / kBlock);
    return DOPT_OK;
}

extern "C" int dopt_ckpt_save(const void *x, dopt_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                              void *ckpt, cudaStream_t stream) {
    dopt::clear_error();
    const char *who = "dopt_ckpt_save";
    OpRange range(who);
    int rc = check_ckpt(who, ckpt, rows, cols);
    if (rc != DOPT_OK) return rc;
    if (rows == 0) return valid_dtype(dtype) ? DOPT_OK : dopt::fail(DOPT_E_ARG, "%s: unknown dtype %d", who, int(dtype));
    if ((rc = check_values(who, "x", x, dtype, cols, ld)) != DOPT_OK) return rc;
    CkptArgs a = ckpt_args(ckpt, rows, cols);
    a.x = x;
    a.ld = ld;
    a.vec = vec_rows(x, dtype, ld);
    a.min_exp = dtype == DOPT_FP16 ? 127 - 24 : 1;
    switch (dtype) {
        case DOPT_BF16: return launch_rows(who, dopt_ckpt_save_kernel<__nv_bfloat16>, a, a.pitch, rows, stream);
        case DOPT_FP16: return launch_rows(who, dopt_ckpt_save_kernel<__half>, a, a.pitch, rows, stream);
        default: return launch_rows(who, dopt_ckpt_save_kernel<float>, a, a.pitch, rows, stream);
    }
}

extern "C" int dopt_ckpt_load(const void *ckpt, int64_t rows, int64_t cols, const int32_t *row_index,
                              int64_t n_out, void *out, dopt_dtype dtype, int64_t ld,
                              cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_ckpt_load";
    OpRange range(who);
    int rc = check_ckpt(who, ckpt, rows, cols);
    if (rc != DOPT_OK) return rc;
    if (n_out < 0 || n_out > INT32_MAX || (!row_index && n_out != rows && n_out != 0))
        return fail(DOPT_E_ARG, "%s: %lld output rows of a checkpoint of %lld", who,
                    static_cast<long long>(n_out), static_cast<long long>(rows));
    if (row_index && !aligned_to(row_index, 4))
        return fail(DOPT_E_ALIGN, "%s: row_index is not aligned to its elements", who);
    if (n_out == 0) return valid_dtype(dtype) ? DOPT_OK : fail(DOPT_E_ARG, "%s: unknown dtype %d", who, int(dtype));
    if ((rc = check_values(who, "out", out, dtype, cols, ld)) != DOPT_OK) return rc;
    CkptArgs a = ckpt_args(ckpt, rows, cols);
    a.out = out;
    a.ld_out = ld;
    a.index = row_index;
    a.n_out = n_out;
    a.vec = vec_rows(out, dtype, ld);
    switch (dtype) {
        case DOPT_BF16: return launch_rows(who, dopt_ckpt_load_kernel<__nv_bfloat16>, a, cols, n_out, stream);
        case DOPT_FP16: return launch_rows(who, dopt_ckpt_load_kernel<__half>, a, cols, n_out, stream);
        default: return launch_rows(who, dopt_ckpt_load_kernel<float>, a, cols, n_out, stream);
    }
}

extern "C" int dopt_ckpt_act_grad(const void *ckpt, int64_t rows, int64_t cols, dopt_act act,
                                  const void *d_out, int64_t ld, dopt_dtype dtype, void *d_in,
                                  int64_t ld_in, cudaStream_t stream) {
    using dopt::fail;
    dopt::clear_error();
    const char *who = "dopt_ckpt_act_grad";
    OpRange range(who);
    int rc = check_ckpt(who, ckpt, rows, cols);
    if (rc != DOPT_OK) return rc;
    if (act != DOPT_ACT_SILU && act != DOPT_ACT_GELU && act != DOPT_ACT_SWIGLU)
        return fail(DOPT_E_ARG, "%s: unknown activation %d", who, int(act));
    if (act == DOPT_ACT_SWIGLU && cols % 2 != 0)
        return fail(DOPT_E_ARG, "%s: %lld columns have no two halves", who, static_cast<long long>(cols));
    if (rows == 0) return valid_dtype(dtype) ? DOPT_OK : fail(DOPT_E_ARG, "%s: unknown dtype %d", who, int(dtype));
    const int64_t width = act == DOPT_ACT_SWIGLU ? cols / 2 : cols;
    if ((rc = check_values(who, "d_out", d_out, dtype, width, ld)) != DOPT_OK) return rc;
    if ((rc = check_values(who, "d_in", d_in, dtype, cols, ld_in)) != DOPT_OK) return rc;
    CkptArgs a = ckpt_args(ckpt, rows, cols);
    a.x = d_out;
    a.out = d_in;
    a.ld = ld;
    a.ld_out = ld_in;
    a.half = width;
    a.vec = vec_rows(d_out, dtype, ld) && vec_rows(d_in, dtype, ld_in) &&
            (act != DOPT_ACT_SWIGLU || width * int64_t(elem_bytes(dtype)) % 16 == 0);
    switch (dtype) {
        case DOPT_BF16: return launch_act<__nv_bfloat16>(who, act, a, width, stream);
        case DOPT_FP16: return launch_act<__half>(who, act, a, width, stream);
        default: return launch_act<float>(who, act, a, width, stream);
    }
}
