#pragma once
// 16-byte accesses to rows of any alignment.  Rows that are not 16-byte
// aligned are read and written in the aligned pieces around them: the threads
// of a row hold neighbouring pieces, take the part that is missing from their
// neighbour and shift.  Only pieces that reach over the ends of the row
// (reading) or of the threads' stretch of it (writing) go element by element.
#include "op_common.cuh"

namespace {

// A 16-byte piece and its successor, shifted down by `bytes` (0..15): the 4
// words from that byte on.
__device__ __forceinline__ uint4 shift_down(const uint4 &lo, const uint4 &hi, uint32_t bytes) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (bytes & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (bytes & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = (bytes & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}
__device__ __forceinline__ uint4 shuffle_down(const uint4 &v, int width) {
    return make_uint4(__shfl_down_sync(kFull, v.x, 1, width), __shfl_down_sync(kFull, v.y, 1, width),
                      __shfl_down_sync(kFull, v.z, 1, width), __shfl_down_sync(kFull, v.w, 1, width));
}
__device__ __forceinline__ uint4 shuffle_up(const uint4 &v, int width) {
    return make_uint4(__shfl_up_sync(kFull, v.x, 1, width), __shfl_up_sync(kFull, v.y, 1, width),
                      __shfl_up_sync(kFull, v.z, 1, width), __shfl_up_sync(kFull, v.w, 1, width));
}

// The 16 bytes at elements [e, e + 16 / sizeof(T)) of a row of `cols`; those
// before or past the row are not read (0).
template <typename T>
__device__ __forceinline__ uint4 load_piece(const T *row, int e, int cols) {
    constexpr int N = 16 / int(sizeof(T));
    if (e >= 0 && e + N <= cols) return __ldcs(reinterpret_cast<const uint4 *>(row + e));
    using E = typename Raw<int(sizeof(T))>::type;
    E v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = e + i >= 0 && e + i < cols ? reinterpret_cast<const E *>(row)[e + i] : E(0);
    uint4 raw;
    memcpy(&raw, v, sizeof raw);
    return raw;
}
// The same to elements [e, ...) of which those in [from, to) are written.
template <typename T>
__device__ __forceinline__ void store_piece(T *row, int e, int from, int to, const uint4 &raw) {
    constexpr int N = 16 / int(sizeof(T));
    if (e >= from && e + N <= to) {
        __stcs(reinterpret_cast<uint4 *>(row + e), raw);
        return;
    }
    using E = typename Raw<int(sizeof(T))>::type;
    E v[N];
    memcpy(v, &raw, sizeof raw);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (e + i >= from && e + i < to) reinterpret_cast<E *>(row)[e + i] = v[i];
}

// ---------------------------------------------------------------------------
// COLS values of a row.  All threads of a warp call these together; `lane` is
// the thread's place among the bx of its row.
// ---------------------------------------------------------------------------

template <typename T, int COLS>
struct Values {
    static constexpr int kPer = 16 / int(sizeof(T));  // elements a piece
    static constexpr int kPieces = COLS / kPer;
    uint4 raw[kPieces];

    // What is read for them, in flight until take(): the pieces around the
    // values, and the one after them where no neighbour has it.
    struct Ahead {
        uint4 raw[kPieces], last;
        uint32_t off;  // bytes from the first piece to the first value
    };

    // Values from column c on; those at or past `cols` (0 where there is no row) are 0.
    static __device__ __forceinline__ void fetch(Ahead &a, const T *row, int c, int cols, bool vec, int lane, int bx) {
        a.off = vec ? 0 : uint32_t(reinterpret_cast<uintptr_t>(row + c) & 15);
        const int e = c - int(a.off / sizeof(T));
#pragma unroll
        for (int i = 0; i < kPieces; ++i) a.raw[i] = load_piece(row, e + i * kPer, cols);
        a.last = make_uint4(0, 0, 0, 0);
        if (!vec && lane == bx - 1) a.last = load_piece(row, e + COLS, cols);
    }
    __device__ __forceinline__ void take(const Ahead &a, bool vec, int lane, int bx) {
        if (vec) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) raw[i] = a.raw[i];
        } else {
            uint4 next = shuffle_down(a.raw[0], bx);
            if (lane == bx - 1) next = a.last;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) raw[i] = shift_down(a.raw[i], i + 1 < kPieces ? a.raw[i + 1] : next, a.off);
        }
    }
    __device__ __forceinline__ void load(const T *row, int c, int cols, bool vec, int lane, int bx) {
        Ahead a;
        fetch(a, row, c, cols, vec, lane, bx);
        take(a, vec, lane, bx);
    }
    // The same where c and the row are aligned and all COLS values are there (or none: `some` false).
    __device__ __forceinline__ void load_whole(const T *row, int c, bool some) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            raw[i] = some ? __ldcs(reinterpret_cast<const uint4 *>(row + c) + i) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void store_whole(T *row, int c, bool some) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (some) __stcs(reinterpret_cast<uint4 *>(row + c) + i, raw[i]);
    }

    __device__ __forceinline__ void get(float (&f)[COLS]) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float g[kPer];
            unpack<T, 16>(raw[i], g);
#pragma unroll
            for (int q = 0; q < kPer; ++q) f[i * kPer + q] = g[q];
        }
    }
    __device__ __forceinline__ void set(const float (&f)[COLS]) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float g[kPer];
#pragma unroll
            for (int q = 0; q < kPer; ++q) g[q] = f[i * kPer + q];
            raw[i] = pack<T, 16>(g);
        }
    }

    // Values to column c on, those before `cols`.
    __device__ __forceinline__ void store(T *row, int c, int cols, bool vec, int lane, int bx) const {
        if (vec) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) store_piece(row, c + i * kPer, c, cols, raw[i]);
        } else {
            const int from = c - lane * COLS, to = min(cols, from + bx * COLS);  // what the row's threads hold
            const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(row + c) & 15);
            const int e = c - int(off / sizeof(T));
            const uint4 before = shuffle_up(raw[kPieces - 1], bx);
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                store_piece(row, e + i * kPer, from, to,
                            off ? shift_down(i ? raw[i - 1] : before, raw[i], 16 - off) : raw[i]);
            if (lane == bx - 1 && off)  // the rest of the last thread's values
                store_piece(row, e + COLS, from, to,
                            shift_down(raw[kPieces - 1], make_uint4(0, 0, 0, 0), 16 - off));
        }
    }
};

}  // namespace
