// Activations kept in 8 bits: saving (dopt_ckpt_save), reading back
// (dopt_ckpt_load) and an activation function's backward pass from its kept
// input (dopt_ckpt_act_grad).  dopt.h states the format.
//
// All three are bound by memory.  Saving and reading back give a thread 32
// bytes of a row's values (16 columns of 16 bits, 8 of fp32), the activation
// gradients 8 columns: few enough registers that the threads of an SM keep
// enough loads in flight for memory's rate, enough columns that indexes cost
// little.  A thread block covers bx threads' columns of 256 / bx rows, so no
// index is divided, and goes on to the next rows where that pays
// (launch_rows); the next rows' loads are then in flight under the
// arithmetic.  16384 x 5632 bf16, kept and read back: 86 us (6.5 TB/s); the
// gated gradient of 16384 x 2 * 5632: 122 us (6.1 TB/s), of which its
// instructions are some 60 us.
//
// Codes are always aligned (a row's pitch is a multiple of 128).  Rows of
// whole, aligned groups have kernels without the checks for any others (94 us
// with them).  Rows that are not go in aligned pieces all the same
// (rows.cuh): 16384 x 5631 bf16, kept and read back, 113 us (585 us one
// element at a time).
#include "f32x2.cuh"
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
    int32_t turns;        // times a block takes its number of rows
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
        const F2 less = step * -8388736.0f;
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            fma2(F2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440u + i)),
                    __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441u + i))), step, less).get(f[i], f[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440u + i)) - 8388736.0f) * step;
    }
}

__device__ __forceinline__ uint64_t kept_at(const CkptArgs &a, uint32_t r, int c) {
    return uint64_t(r) * uint32_t(a.pitch) + uint32_t(c);
}

// The COLS (8 or 16) kept values from column c (a multiple of COLS) of row r
// on; 0 where the checkpoint has no such row.
template <int COLS>
struct Kept {
    uint32_t w[COLS / 4], byte;
    __device__ __forceinline__ void load(const CkptArgs &a, uint32_t r, int c) {
#pragma unroll
        for (int i = 0; i < COLS / 4; ++i) w[i] = 0;
        byte = 1;
        if (r >= uint32_t(a.rows)) return;
        const uint64_t at = kept_at(a, r, c);
        if constexpr (COLS == 16) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(a.codes + at));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(a.codes + at));
            w[0] = v.x, w[1] = v.y;
        }
        byte = a.scales[at / kBlock];
    }
    __device__ __forceinline__ void get(float (&f)[COLS]) const {
#pragma unroll
        for (int i = 0; i < COLS / 4; ++i) code_values(w[i], byte, f + 4 * i);
    }
};

// The 8 kept values from any column on (the gated half of an odd width):
// codes from the aligned 8 bytes around them, exponents of up to two blocks.
// Nothing past the row's pitch is read.
struct KeptAny {
    uint2 lo, hi;
    uint32_t first, second, bytes, in_first;
    __device__ __forceinline__ void load(const CkptArgs &a, uint32_t r, int c, bool some) {
        bytes = c & 7;
        in_first = kBlock - (c & (kBlock - 1));
        lo = hi = make_uint2(0, 0);
        first = second = 1;
        if (!some) return;
        const uint64_t at = kept_at(a, r, c & ~7), block = kept_at(a, r, c) / kBlock;
        lo = __ldcs(reinterpret_cast<const uint2 *>(a.codes + at));
        if (bytes && (c & ~7) + 8 < a.pitch) hi = __ldcs(reinterpret_cast<const uint2 *>(a.codes + at + 8));
        first = a.scales[block];
        if (in_first < 8 && c + int(in_first) < a.pitch) second = a.scales[block + 1];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint4 w = shift_down(make_uint4(lo.x, lo.y, hi.x, hi.y), make_uint4(0, 0, 0, 0), bytes);
        code_values(w.x, first, f);
        code_values(w.y, first, f + 4);
        if (in_first < 8) {
            float g[8];
            code_values(w.x, second, g);
            code_values(w.y, second, g + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= int(in_first)) f[i] = g[i];
        }
    }
};

// A block of 32 columns is 32 / COLS neighbouring threads.  The step is the
// power of two 2^k with the largest magnitude in [64, 128) steps (k no less
// than the type's least); codes are round-to-nearest-even of value / step,
// clamped to 127.  Multiplying by a power of two is exact, so a code is one
// rounding of the value (done by adding 1.5 * 2^23, whose last bit weighs 1);
// and code * step has at most 7 significant bits, so the products of the
// backward pass read it in 16 bits without a second rounding.  The comparison
// of magnitudes as integers puts Inf and NaN above every finite value.
// WHOLE: rows of whole, aligned groups of COLS columns.  The next row's loads
// are in flight under a row's arithmetic.
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_save_kernel(const __grid_constant__ CkptArgs a) {
    constexpr int COLS = 32 / int(sizeof(T));
    let_dependents_start();
    wait_for_grids_before();
    const int bx = blockDim.x, lane = threadIdx.x;
    const int c = (blockIdx.x * bx + lane) * COLS;
    const uint32_t step = blockDim.y, first = blockIdx.y * step * a.turns;
    const uint32_t end = min(first + step * a.turns, uint32_t(a.rows));
    Values<T, COLS> x;
    typename Values<T, COLS>::Ahead ahead;
    auto load = [&](uint32_t r) {
        const bool here = r < uint32_t(a.rows);
        const T *row = static_cast<const T *>(a.x) + (here ? int64_t(r) * a.ld : 0);
        if constexpr (WHOLE)
            x.load_whole(row, c, here && c < a.cols);
        else
            x.fetch(ahead, row, c, here ? a.cols : 0, a.vec, lane, bx);
    };
    load(first + threadIdx.y);
    for (uint32_t r0 = first; r0 < end; r0 += step) {
        const uint32_t r = r0 + threadIdx.y;
        const bool here = r < uint32_t(a.rows);
        float f[COLS];
        if constexpr (!WHOLE) x.take(ahead, a.vec, lane, bx);
        x.get(f);
        if (r0 + step < end) load(r + step);
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

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_load_kernel(const __grid_constant__ CkptArgs a) {
    constexpr int COLS = 32 / int(sizeof(T));
    let_dependents_start();
    wait_for_grids_before();
    const int bx = blockDim.x, lane = threadIdx.x;
    const int c = (blockIdx.x * bx + lane) * COLS;
    const uint32_t step = blockDim.y, first = blockIdx.y * step * a.turns;
    const uint32_t n = min(first + step * a.turns, uint32_t(a.n_out));
    // the checkpoint's row of output row o
    auto row_of = [&](uint32_t o) { return o >= n || c >= a.cols ? ~0u : a.index ? uint32_t(a.index[o]) : o; };
    Kept<COLS> kept;
    kept.load(a, row_of(first + threadIdx.y), c);
    uint32_t next = row_of(first + threadIdx.y + step);
    for (uint32_t r0 = first; r0 < n; r0 += step) {
        const uint32_t o = r0 + threadIdx.y;
        float f[COLS];
        kept.get(f);
        kept.load(a, next, c);
        next = row_of(o + 2 * step);
        Values<T, COLS> y;
        y.set(f);
        const bool here = o < n;
        T *row = static_cast<T *>(a.out) + (here ? int64_t(o) * a.ld_out : 0);
        if constexpr (WHOLE)
            y.store_whole(row, c, here && c < a.cols);
        else
            y.store(row, c, here ? a.cols : 0, a.vec, lane, bx);
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
__device__ __forceinline__ void sigmoid(F2 x, F2 &s, F2 &rest) {
    float x0, x1, e0, e1, d0, d1;
    if constexpr (sizeof(T) == 4) {
        x.get(x0, x1);
        e0 = expf(-x0), e1 = expf(-x1);
        s = F2(1.0f / (1.0f + e0), 1.0f / (1.0f + e1));
    } else {
        (x * -1.44269504f).get(x0, x1);
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(x0));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(x1));
        (F2(e0, e1) + 1.0f).get(d0, d1);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d0) : "f"(d0));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d1) : "f"(d1));
        s = F2(d0, d1);
    }
    rest = F2(e0, e1) * s;
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
__device__ __forceinline__ F2 silu_slope(float h0, float h1, F2 &silu) {
    const F2 x(at_least(h0, -87.0f), at_least(h1, -87.0f));
    F2 s = 0.0f, rest = 0.0f;
    sigmoid<T>(x, s, rest);
    silu = x * s;
    return s * fma2(x, rest, 1.0f);
}

// GELU in its tanh form is h p with p = (1 + tanh u) / 2 = sigmoid(2u),
// u = c (h + a h^3); its slope p + h 2 p (1 - p) c (1 + 3 a h^2).  Beyond
// |h| = 9.9 (2u = 85) it is 0 or 1 to within 1e-34.
template <typename T>
__device__ __forceinline__ F2 gelu_slope(float h0, float h1) {
    constexpr float kC = 0.79788456080286536f, kA = 0.044715f;
    const F2 x(at_most(at_least(h0, -9.9f), 9.9f), at_most(at_least(h1, -9.9f), 9.9f));
    const F2 x2 = x * x, cx = x * (2.0f * kC);
    F2 p = 0.0f, rest = 0.0f;
    sigmoid<T>(cx * fma2(kA, x2, 1.0f), p, rest);
    return fma2(cx * fma2(3.0f * kA, x2, 1.0f), p * rest, p);
}

template <typename T, int ACT>
__device__ __forceinline__ void act_grad(const float (&d)[8], float (&h)[8], float (&u)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const F2 dd(d[i], d[i + 1]);
        F2 silu = 0.0f;
        if constexpr (ACT == DOPT_ACT_SWIGLU) {
            const F2 slope = silu_slope<T>(h[i], h[i + 1], silu);
            (dd * F2(u[i], u[i + 1]) * slope).get(h[i], h[i + 1]);
            (dd * silu).get(u[i], u[i + 1]);
        } else if constexpr (ACT == DOPT_ACT_SILU) {
            (dd * silu_slope<T>(h[i], h[i + 1], silu)).get(h[i], h[i + 1]);
        } else {
            (dd * gelu_slope<T>(h[i], h[i + 1])).get(h[i], h[i + 1]);
        }
    }
}

// Rows of whole, aligned groups of 8 columns: the next row's loads are in
// flight under a row's arithmetic.
template <typename T, int ACT>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_act_grad_whole_kernel(const __grid_constant__ CkptArgs a) {
    constexpr bool kGated = ACT == DOPT_ACT_SWIGLU;
    const int width = kGated ? a.half : a.cols;
    const int c = int(blockIdx.x * blockDim.x + threadIdx.x) * 8;
    const uint32_t step = blockDim.y, first = blockIdx.y * step * a.turns;
    const uint32_t end = min(first + step * a.turns, uint32_t(a.rows));
    uint32_t r = first + threadIdx.y;
    let_dependents_start();
    wait_for_grids_before();
    if (c >= width || r >= end) return;
    Values<T, 8> x;
    Kept<8> kept_h, kept_u;
    auto load = [&](uint32_t row) {
        x.load_whole(static_cast<const T *>(a.x) + int64_t(row) * a.ld, c, true);
        kept_h.load(a, row, c);
        if constexpr (kGated) kept_u.load(a, row, width + c);
    };
    load(r);
    for (; r < end; r += step) {
        float d[8], h[8], u[8];
        x.get(d);
        kept_h.get(h);
        if constexpr (kGated) kept_u.get(u);
        if (r + step < end) load(r + step);
        act_grad<T, ACT>(d, h, u);
        T *out = static_cast<T *>(a.out) + int64_t(r) * a.ld_out;
        Values<T, 8> y;
        y.set(h);
        y.store_whole(out, c, true);
        if constexpr (kGated) {
            y.set(u);
            y.store_whole(out, width + c, true);
        }
    }
}

// Rows of any width and alignment.
template <typename T, int ACT>
__global__ void __launch_bounds__(kCkptThreads) dopt_ckpt_act_grad_kernel(const __grid_constant__ CkptArgs a) {
    constexpr int COLS = 8;
    let_dependents_start();
    wait_for_grids_before();
    const int bx = blockDim.x, lane = threadIdx.x;
    const int c = (blockIdx.x * bx + lane) * COLS;
    const int width = ACT == DOPT_ACT_SWIGLU ? a.half : a.cols;
    const uint32_t step = blockDim.y, first = blockIdx.y * step * a.turns;
    const uint32_t end = min(first + step * a.turns, uint32_t(a.rows));
    Values<T, COLS> x;
    typename Values<T, COLS>::Ahead ahead;
    Kept<COLS> kept_h;
    KeptAny kept_u;
    auto load = [&](uint32_t r) {
        const bool here = r < uint32_t(a.rows), some = here && c < width;
        x.fetch(ahead, static_cast<const T *>(a.x) + (here ? int64_t(r) * a.ld : 0), c, here ? width : 0, a.vec, lane, bx);
        kept_h.load(a, some ? r : ~0u, c);
        if constexpr (ACT == DOPT_ACT_SWIGLU) kept_u.load(a, r, width + c, some);
    };
    load(first + threadIdx.y);
    for (uint32_t r0 = first; r0 < end; r0 += step) {
        const uint32_t r = r0 + threadIdx.y;
        const bool here = r < uint32_t(a.rows);
        float d[COLS], h[COLS], u[COLS];
        x.take(ahead, a.vec, lane, bx);
        x.get(d);
        kept_h.get(h);
        if constexpr (ACT == DOPT_ACT_SWIGLU) kept_u.get(u);
        if (r0 + step < end) load(r + step);
        T *out = static_cast<T *>(a.out) + (here ? int64_t(r) * a.ld_out : 0);
        act_grad<T, ACT>(d, h, u);
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
// 256 / bx rows at a time, for up to `turns` times, where that leaves 5 blocks
// an SM.  Whole rows are saved and read back in one turn (16384 x 5632 bf16:
// 86 us; 87 in two turns, 92 in four); there is arithmetic to hide the next
// loads under in the others: the gated gradient takes 135, 125, 122.5 and 124
// us in 1, 2, 4 and 8 turns, 16384 x 5631 saved and read back 130, 116, 113
// and 116.
template <typename Kernel>
int launch_rows(const char *who, Kernel kernel, CkptArgs a, int64_t cols, int each, int64_t rows, int turns,
                cudaStream_t stream) {
    const int64_t groups = (cols + each - 1) / each;
    const int bx = groups > 16 ? 32 : groups > 8 ? 16 : 8;
    const int by = kCkptThreads / bx;
    const int64_t across = (groups + bx - 1) / bx, down = (rows + by - 1) / by;
    a.turns = int(std::max<int64_t>(1, std::min<int64_t>(turns, across * down / (152 * 5))));
    while ((down + a.turns - 1) / a.turns > 65535) a.turns *= 2;  // the grid's limit
    const dim3 grid(unsigned(across), unsigned((down + a.turns - 1) / a.turns));
    return launch_op(who, kernel, grid, dim3(bx, by), 0, stream, a);
}

template <typename T>
int launch_save(const char *who, const CkptArgs &a, cudaStream_t stream) {
    constexpr int kEach = 32 / int(sizeof(T));
    return a.vec && a.cols % kEach == 0
               ? launch_rows(who, dopt_ckpt_save_kernel<T, true>, a, a.pitch, kEach, a.rows, 1, stream)
               : launch_rows(who, dopt_ckpt_save_kernel<T, false>, a, a.pitch, kEach, a.rows, 4, stream);
}

template <typename T>
int launch_load(const char *who, const CkptArgs &a, cudaStream_t stream) {
    constexpr int kEach = 32 / int(sizeof(T));
    return a.vec && a.cols % kEach == 0
               ? launch_rows(who, dopt_ckpt_load_kernel<T, true>, a, a.cols, kEach, a.n_out, 1, stream)
               : launch_rows(who, dopt_ckpt_load_kernel<T, false>, a, a.cols, kEach, a.n_out, 4, stream);
}

template <typename T, int ACT>
int launch_act_as(const char *who, const CkptArgs &a, int64_t width, cudaStream_t stream) {
    return a.vec && width % 8 == 0
               ? launch_rows(who, dopt_ckpt_act_grad_whole_kernel<T, ACT>, a, width, 8, a.rows, 4, stream)
               : launch_rows(who, dopt_ckpt_act_grad_kernel<T, ACT>, a, width, 8, a.rows, 4, stream);
}

template <typename T>
int launch_act(const char *who, dopt_act act, const CkptArgs &a, int64_t width, cudaStream_t stream) {
    switch (act) {
        case DOPT_ACT_SILU: return launch_act_as<T, DOPT_ACT_SILU>(who, a, width, stream);
        case DOPT_ACT_GELU: return launch_act_as<T, DOPT_ACT_GELU>(who, a, width, stream);
        default: return launch_act_as<T, DOPT_ACT_SWIGLU>(who, a, width, stream);
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
        case DOPT_BF16: return launch_save<__nv_bfloat16>(who, a, stream);
        case DOPT_FP16: return launch_save<__half>(who, a, stream);
        default: return launch_save<float>(who, a, stream);
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
        case DOPT_BF16: return launch_load<__nv_bfloat16>(who, a, stream);
        case DOPT_FP16: return launch_load<__half>(who, a, stream);
        default: return launch_load<float>(who, a, stream);
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
