#pragma once
// What the routing and checkpoint operators share: conversions between the
// three element types and fp32, accesses of 2 to 16 bytes, the layout of a
// checkpoint, and launches.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "dopt_internal.h"

namespace {

// A named range around each entry point for timeline profilers.
struct OpRange {
    explicit OpRange(const char *name) { nvtxRangePushA(name); }
    ~OpRange() { nvtxRangePop(); }
};

constexpr unsigned kFull = 0xffffffffu;

// ---------------------------------------------------------------------------
// Elements
// ---------------------------------------------------------------------------

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
    return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// VB bytes moved by one access.
template <int VB>
struct Raw;
template <>
struct Raw<2> {
    using type = uint16_t;
};
template <>
struct Raw<4> {
    using type = uint32_t;
};
template <>
struct Raw<8> {
    using type = uint2;
};
template <>
struct Raw<16> {
    using type = uint4;
};

// The VB / sizeof(T) elements of one access, as fp32 and back.
template <typename T, int VB>
__device__ __forceinline__ void unpack(const typename Raw<VB>::type &raw,
                                       float (&f)[VB / sizeof(T)]) {
    T e[VB / sizeof(T)];
    memcpy(e, &raw, VB);
#pragma unroll
    for (int i = 0; i < int(VB / sizeof(T)); ++i) f[i] = to_f32(e[i]);
}
template <typename T, int VB>
__device__ __forceinline__ typename Raw<VB>::type pack(const float (&f)[VB / sizeof(T)]) {
    T e[VB / sizeof(T)];
#pragma unroll
    for (int i = 0; i < int(VB / sizeof(T)); ++i) e[i] = from_f32<T>(f[i]);
    typename Raw<VB>::type raw;
    memcpy(&raw, e, VB);
    return raw;
}

// ---------------------------------------------------------------------------
// Checkpoints: rows x pitch int8 codes, then rows x pitch / 32 exponent bytes
// (dopt.h states the format).
// ---------------------------------------------------------------------------

constexpr int kBlock = DOPT_CKPT_BLOCK;
constexpr int kNanByte = 255;

__host__ __device__ inline int64_t ckpt_pitch(int64_t cols) {
    return (cols + DOPT_CKPT_PITCH - 1) / DOPT_CKPT_PITCH * DOPT_CKPT_PITCH;
}

// 2^(byte - 127) for byte 1..254; NaN for 255.
__device__ __forceinline__ float ckpt_step(uint32_t byte) {
    return __uint_as_float(byte == kNanByte ? 0x7fffffffu : byte << 23);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

inline size_t elem_bytes(dopt_dtype t) { return t == DOPT_FP32 ? 4 : 2; }
inline bool valid_dtype(int t) { return t == DOPT_BF16 || t == DOPT_FP32 || t == DOPT_FP16; }
inline bool aligned_to(const void *p, size_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// The widest of 16, 8, 4 and 2 bytes on which `address bits` (the OR of
// pointers and byte strides) are aligned.
inline int access_bytes(uint64_t bits) {
    return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
}
inline uint64_t address_bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }

// A launch as a programmatic dependent of the kernel before it on the stream:
// the kernels launched this way execute griddepcontrol.wait before their
// first access to memory.
template <typename... KArgs, typename... Args>
int launch_cluster(const char *who, void (*kernel)(KArgs...), dim3 grid, unsigned cluster, dim3 block, size_t smem,
                   cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = cluster > 0 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&lc, kernel, KArgs(args)...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return dopt::fail(DOPT_E_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    }
    return DOPT_OK;
}
// (cluster 0: as the kernel was compiled)
template <typename... KArgs, typename... Args>
int launch_op(const char *who, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
              const Args &...args) {
    return launch_cluster(who, kernel, grid, 0, block, smem, stream, args...);
}

__device__ __forceinline__ void wait_for_grids_before() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_dependents_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace
