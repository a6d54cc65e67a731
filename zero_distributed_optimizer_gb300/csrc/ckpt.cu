// Activations kept in 8 bits: saving (dopt_ckpt_save), reading back
// (dopt_ckpt_load) and an activation function's backward pass from its kept
// input (dopt_ckpt_act_grad).  dopt.h states the format.
//
// Saving and reading back give a thread 32 bytes of a row's values (16 columns
// of 16 bits, 8 of fp32), the activation gradients 8 columns: few enough
// registers that the threads of an SM keep enough loads in flight for
// memory's rate, enough columns that indexes cost little.  A thread block
// covers bx threads' columns of 256 / bx rows and strides over
// the rows, so no index is divided.
//
// Codes are always aligned (a row's pitch is a multiple of 128); rows of
// values that are not go in aligned pieces all the same (rows.cuh): 16384 x
// 5631 bf16, kept and read back, took 585 us one element at a time.
#include "rows.cuh"

namespace {

constexpr int kCkptThreads = 256;

struct CkptArgs {
    const void *x;        // save: values; activation gradient: d_out
    void *out;            // load: values; activation gradient: d_in
    uint8_t *codes;       // [rows][pitch], the exponent bytes after them
    uint8_t *scales;      // [rows][pitch / 32]
    const int32_t *index; // load: row of each output row, or NULL
    int64_t ld, ld_out;
    int32_t rows;         // rows of the checkpoint
    int32_t n_out;        // rows the launch goes through
    int32_t cols, pitch;
    int32_t half;         // gated: columns of the output (cols / 2)
    int32_t min_exp;      // least exponent byte
    int32_t vec;          // rows are 16-byte aligned
};

// ---------------------------------------------------------------------------
// Codes
// ---------------------------------------------------------------------------

// 4 codes times a step (of exponent byte `byte`) as fp32: with the byte of
// code + 128 in the low bits of 2^23, that number less 2^23 + 128.  Both
// products with the step are exact, so one fused operation gives the value,
// unless 2^23 steps leave fp32's range.
__device__ __forceinline__ void code_values(uint32_t w, uint32_t byte, float *f) {
    const float step = ckpt_step(byte);
    w ^= 0x80808080u;
    if (byte < 230 || byte == kNanByte) {
        const float less = step * -8388736.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = fmaf(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440u + i)), step, less);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440u + i)) - 8388736.0f) * step;
    }
}

__device__ __forceinline__ uint64_t kept_at(const CkptArgs &a, uint32_t r, int c) {
    return uint64_t(r) * uint32_t(a.pitch) + uint32_t(c);
}

// The COLS (8 or 16) kept values from column c (a multiple of COLS) of row r on.
template <int COLS>
__device__ __forceinline__ void load_kept(const CkptArgs &a, uint32_t r, int c, float (&f)[COLS]) {
    const uint64_t at = kept_at(a, r, c);
    uint32_t w[COLS / 4];
    if constexpr (COLS == 16) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(a.codes + at));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(a.codes + at));
        w[0] = v.x, w[1] = v.y;
    }
    const uint32_t byte = a.scales[at / kBlock];
#pragma unroll
    for (int i = 0; i < COLS / 4; ++i) code_values(w[i], byte, f + 4 * i);
}

// The 8 kept values from any column on (the gated half of an odd width):
// codes from the aligned 8 bytes around them, exponents of up to two blocks.
// Nothing past the row's pitch is read.
__device__ __forceinline__ void load_kept_any(const CkptArgs &a, uint32_t r, int c, float (&f)[8]) {
    const uint64_t at = kept_at(a, r, c & ~7);
    const uint32_t bytes = c & 7;
    const uint2 lo = __ldcs(reinterpret_cast<const uint2 *>(a.codes + at));
    uint2 hi = make_uint2(0, 0);
    if (bytes && (c & ~7) + 8 < a.pitch) hi = __ldcs(reinterpret_cast<const uint2 *>(a.codes + at + 8));
    const uint4 w = shift_down(make_uint4(lo.x, lo.y, hi.x, hi.y), make_uint4(0, 0, 0, 0), bytes);
    const uint64_t block = kept_at(a, r, c) / kBlock;
    const uint32_t first = a.scales[block];
    const int in_first = kBlock - (c & (kBlock - 1));
    code_values(w.x, first, f);
    code_values(w.y, first, f + 4);
    if (in_first < 8 && c + in_first < a.pitch) {
        float g[8];
        const uint32_t second = a.scales[block + 1];
        code_values(w.x, second, g);
        code_values(w.y, second, g + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= in_first) f[i] = g[i];
    }
}

// A block of 32 columns is 32 / COLS neighbouring threads.  The step is the
// power of two 2^k with the largest magnitude in [64, 128) steps (k no less
// than the type's least); codes are round-to-nearest-even of value / step,
// clamped to 127.  Multiplying by a power of two is exact, so a code is one
// rounding of the value (done by adding 1.5 * 2^23, whose last bit weighs 1);
// and code * step has at most 7 significant bits, so the products of the
// backward pass read it in 16 bits without a second rounding.  The comparison
// of magnitudes as integers puts Inf and NaN above every finite value.
template <typename T>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_save_kernel(const __grid_constant__ CkptArgs a) {
    constexpr int COLS = 32 / int(sizeof(T));
    let_dependents_start();
    wait_for_grids_before();
    const int bx = blockDim.x, lane = threadIdx.x;
    const int c = (blockIdx.x * bx + lane) * COLS;
    for (uint32_t r0 = blockIdx.y * blockDim.y; r0 < uint32_t(a.rows); r0 += gridDim.y * blockDim.y) {
        const uint32_t r = r0 + threadIdx.y;
        const bool here = r < uint32_t(a.rows);
        Values<T, COLS> x;
        x.load(static_cast<const T *>(a.x) + (here ? int64_t(r) * a.ld : 0), c, here ? a.cols : 0, a.vec, lane, bx);
        float f[COLS];
        x.get(f);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < COLS; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        if constexpr (COLS == 8) top = max(top, __shfl_xor_sync(kFull, top, 2));
        const bool finite = top < 0x7f800000u;
        const int byte = max(int(top >> 23) - 6, a.min_exp);
        const float inv = __uint_as_float(uint32_t(254 - byte) << 23);
        uint32_t q[COLS], w[COLS / 4];
#pragma unroll
        for (int i = 0; i < COLS; ++i)
            q[i] = __float_as_uint(fminf(fmaxf(f[i] * inv, -127.0f), 127.0f) + 12582912.0f);
#pragma unroll
        for (int i = 0; i < COLS / 4; ++i) {
            w[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040),
                               __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
            if (!finite) w[i] = 0;
        }
        if (here && c < a.pitch) {
            const uint64_t at = kept_at(a, r, c);
            if constexpr (COLS == 16)
                *reinterpret_cast<uint4 *>(a.codes + at) = make_uint4(w[0], w[1], w[2], w[3]);
            else
                *reinterpret_cast<uint2 *>(a.codes + at) = make_uint2(w[0], w[1]);
            if (c % kBlock == 0) a.scales[at / kBlock] = uint8_t(finite ? byte : kNanByte);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_load_kernel(const __grid_constant__ CkptArgs a) {
    constexpr int COLS = 32 / int(sizeof(T));
    let_dependents_start();
    wait_for_grids_before();
    const int bx = blockDim.x, lane = threadIdx.x;
    const int c = (blockIdx.x * bx + lane) * COLS;
    for (uint32_t r0 = blockIdx.y * blockDim.y; r0 < uint32_t(a.n_out); r0 += gridDim.y * blockDim.y) {
        const uint32_t o = r0 + threadIdx.y;
        const bool here = o < uint32_t(a.n_out);
        float f[COLS] = {};
        if (here && c < a.cols) {
            const uint32_t r = a.index ? uint32_t(a.index[o]) : o;
            if (r < uint32_t(a.rows)) load_kept<COLS>(a, r, c, f);
        }
        Values<T, COLS> y;
        y.set(f);
        y.store(static_cast<T *>(a.out) + (here ? int64_t(o) * a.ld_out : 0), c, here ? a.cols : 0, a.vec, lane, bx);
    }
}

// ---------------------------------------------------------------------------
// Activation functions
// ---------------------------------------------------------------------------

// s = 1 / (1 + e^-x) and 1 - s = e^-x s, each with small relative error for
// x >= -87 (below, e^-x leaves fp32's normal range).  Results that are rounded
// to 16 bits take the hardware's powers of two and reciprocal, each off by at
// most 2^-22 of its result, the power also by the rounding of -x / ln 2 (in
// all below (2 + 1.2 |x|) 2^-23); fp32 ones take the library's functions.
template <typename T>
__device__ __forceinline__ void sigmoid(float x, float &s, float &rest) {
    float e;
    if constexpr (sizeof(T) == 4) {
        e = expf(-x);
        s = 1.0f / (1.0f + e);
    } else {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    }
    rest = e * s;
}
__device__ __forceinline__ float at_least(float x, float b) {  // NaN stays NaN
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(b));
    return y;
}
__device__ __forceinline__ float at_most(float x, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(b));
    return y;
}

// silu'(h) = s (1 + h (1 - s)) and silu(h) = h s, s = sigmoid(h).  Below -87
// both are within 2e-36 of what they are there, 0 in effect.
template <typename T>
__device__ __forceinline__ float silu_slope(float h, float &silu) {
    const float x = at_least(h, -87.0f);
    float s, rest;
    sigmoid<T>(x, s, rest);
    silu = x * s;
    return s * fmaf(x, rest, 1.0f);
}

// GELU in its tanh form is h p with p = (1 + tanh u) / 2 = sigmoid(2u),
// u = c (h + a h^3); its slope p + h 2 p (1 - p) c (1 + 3 a h^2).  Beyond
// |h| = 9.9 (2u = 85) it is 0 or 1 to within 1e-34.
template <typename T>
__device__ __forceinline__ float gelu_slope(float h) {
    constexpr float kC = 0.79788456080286536f, kA = 0.044715f;
    const float x = at_most(at_least(h, -9.9f), 9.9f);
    const float x2 = x * x;
    float p, rest;
    sigmoid<T>(2.0f * kC * x * fmaf(kA, x2, 1.0f), p, rest);
    return fmaf(2.0f * kC * x * fmaf(3.0f * kA, x2, 1.0f), p * rest, p);
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_act_grad_kernel(const __grid_constant__ CkptArgs a) {
    constexpr int COLS = 8;
    let_dependents_start();
    wait_for_grids_before();
    const int bx = blockDim.x, lane = threadIdx.x;
    const int c = (blockIdx.x * bx + lane) * COLS;
    const int width = ACT == DOPT_ACT_SWIGLU ? a.half : a.cols;
    for (uint32_t r0 = blockIdx.y * blockDim.y; r0 < uint32_t(a.rows); r0 += gridDim.y * blockDim.y) {
        const uint32_t r = r0 + threadIdx.y;
        const bool here = r < uint32_t(a.rows);
        Values<T, COLS> x;
        x.load(static_cast<const T *>(a.x) + (here ? int64_t(r) * a.ld : 0), c, here ? width : 0, a.vec, lane, bx);
        float h[COLS] = {}, u[COLS] = {};
        if (here && c < width) {
            load_kept<COLS>(a, r, c, h);
            if constexpr (ACT == DOPT_ACT_SWIGLU) {
                if (width % kBlock == 0)
                    load_kept<COLS>(a, r, width + c, u);
                else
                    load_kept_any(a, r, width + c, u);
            }
        }
        float d[COLS];
        x.get(d);
        T *out = static_cast<T *>(a.out) + (here ? int64_t(r) * a.ld_out : 0);
#pragma unroll
        for (int i = 0; i < COLS; ++i) {
            float silu;
            if constexpr (ACT == DOPT_ACT_SWIGLU) {
                const float slope = silu_slope<T>(h[i], silu);
                h[i] = d[i] * u[i] * slope;
                u[i] = d[i] * silu;
            } else {
                h[i] = d[i] * (ACT == DOPT_ACT_SILU ? silu_slope<T>(h[i], silu) : gelu_slope<T>(h[i]));
            }
        }
        Values<T, COLS> y;
        y.set(h);
        y.store(out, c, here ? width : 0, a.vec, lane, bx);
        if constexpr (ACT == DOPT_ACT_SWIGLU) {
            y.set(u);
            y.store(out + width, c, here ? width : 0, a.vec, lane, bx);
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
    a.rows = int32_t(rows);
    a.cols = int32_t(cols);
    a.pitch = int32_t(ckpt_pitch(cols));
    a.codes = static_cast<uint8_t *>(const_cast<void *>(ckpt));
    a.scales = a.codes + rows * a.pitch;
    return a;
}

// Blocks of bx threads along the columns, `each` columns a thread, and
// 256 / bx rows.
template <typename Kernel>
int launch_rows(const char *who, Kernel kernel, const CkptArgs &a, int64_t cols, int each, int64_t rows,
                cudaStream_t stream) {
    const int64_t groups = (cols + each - 1) / each;
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
            return launch_rows(who, dopt_ckpt_act_grad_kernel<T, DOPT_ACT_SILU>, a, width, 8, a.rows, stream);
        case DOPT_ACT_GELU:
            return launch_rows(who, dopt_ckpt_act_grad_kernel<T, DOPT_ACT_GELU>, a, width, 8, a.rows, stream);
        default:
            return launch_rows(who, dopt_ckpt_act_grad_kernel<T, DOPT_ACT_SWIGLU>, a, width, 8, a.rows, stream);
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
        case DOPT_BF16: return launch_rows(who, dopt_ckpt_save_kernel<__nv_bfloat16>, a, a.pitch, 16, rows, stream);
        case DOPT_FP16: return launch_rows(who, dopt_ckpt_save_kernel<__half>, a, a.pitch, 16, rows, stream);
        default: return launch_rows(who, dopt_ckpt_save_kernel<float>, a, a.pitch, 8, rows, stream);
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
    a.n_out = int32_t(n_out);
    a.vec = vec_rows(out, dtype, ld);
    switch (dtype) {
        case DOPT_BF16: return launch_rows(who, dopt_ckpt_load_kernel<__nv_bfloat16>, a, cols, 16, n_out, stream);
        case DOPT_FP16: return launch_rows(who, dopt_ckpt_load_kernel<__half>, a, cols, 16, n_out, stream);
        default: return launch_rows(who, dopt_ckpt_load_kernel<float>, a, cols, 8, n_out, stream);
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
    a.half = int32_t(width);
    a.vec = vec_rows(d_out, dtype, ld) && vec_rows(d_in, dtype, ld_in) &&
            (act != DOPT_ACT_SWIGLU || width * int64_t(elem_bytes(dtype)) % 16 == 0);
    switch (dtype) {
        case DOPT_BF16: return launch_act<__nv_bfloat16>(who, act, a, width, stream);
        case DOPT_FP16: return launch_act<__half>(who, act, a, width, stream);
        default: return launch_act<float>(who, act, a, width, stream);
    }
}
