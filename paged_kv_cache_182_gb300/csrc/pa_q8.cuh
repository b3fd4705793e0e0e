// pa_q8.cuh -- shared by the kernels of the cache in 8 bits (include/pa_q8.h):
// rounding to codes, codes to fp16, copies and checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_ptx.cuh"
#include "pa_q8.h"
#include "pa_vjp.cuh"

namespace pa {

constexpr unsigned kFullWarp = 0xffffffffu;
constexpr float kMinScale = PA_Q8_MIN_SCALE;

// What every kernel here begins with, in this order: a kernel that is let off may read
// its inputs before this one has ended (pa_opts.inputs_unchanged), and what the kernel
// ahead of this one writes may be among them.
__device__ __forceinline__ void grid_begin()
{
    grid_dependency_wait();
    grid_dependents_launch();
}

__device__ __forceinline__ void q8_report(int* status, int bit)
{
    if (status)
        atomicOr(status, bit);
}

// A block's scale for a largest magnitude: a / 127 rounded once (the remainder of
// a first quotient corrects it; compared with the division for every significand).
__device__ __forceinline__ float q8_scale_of(float a)
{
    constexpr float r = 1.f / 127.f;
    const float q = __fmul_rn(a, r);
    return fmaxf(__fmaf_rn(__fmaf_rn(-127.f, q, a), r, q), kMinScale);
}

// 1 / x of the hardware (a unit in the last place).
__device__ __forceinline__ float fast_rcp(float x)
{
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Largest of m and |x|, leaving out what is not finite.
__device__ __forceinline__ float q8_amax(float m, float x)
{
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? fmaxf(m, a) : m;
}

// Nearest integer to (x + e) / scale, ties to even, |.| <= 127 (inv = 1 / scale,
// |e| at most half a unit in the last place of x).  The product with inv may
// round across a half; the remainder x - r scale is exact in an fma (|x| <= 127.5
// scale, and r is within one of the quotient), so its distance to half a step
// tells.
__device__ __forceinline__ float q8_round(float x, float e, float scale, float inv)
{
    float r = rintf(x * inv);
    const float d = __fmaf_rn(-r, scale, x), half = 0.5f * scale;
    const bool odd = static_cast<int>(r) & 1;
    const float up = (d - half) + e, down = (d + half) + e;
    if (up > 0.f || (up == 0.f && odd))
        r += 1.f;
    else if (down < 0.f || (down == 0.f && odd))
        r -= 1.f;
    return fminf(fmaxf(r, -127.f), 127.f);
}

// Code of a new value: an infinity is the largest code, a NaN 0.
__device__ __forceinline__ int q8_code(float x, float scale, float inv)
{
    if (!(fabsf(x) <= 3.402823466e38f))
        return x != x ? 0 : x > 0.f ? 127 : -127;
    return static_cast<int>(q8_round(x, 0.f, scale, inv));
}

// Code of an earlier code under a larger scale: code * was in two parts, exact.
__device__ __forceinline__ int q8_again(int code, float was, float scale, float inv)
{
    const float c = static_cast<float>(code), x = c * was;
    return static_cast<int>(q8_round(x, __fmaf_rn(c, was, -x), scale, inv));
}

// 16 values of a row, from 16-byte aligned memory.
template <typename T>
__device__ __forceinline__ void q8_load16(float* f, const T* p)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
            f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 two;
                if constexpr (std::is_same_v<T, __half>)
                    two = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                else
                    two = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]));
                f[8 * i + 2 * j] = two.x;
                f[8 * i + 2 * j + 1] = two.y;
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void q8_store16(T* p, const float* f)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (std::is_same_v<T, __half>) {
                    const __half2 h = __floats2half2_rn(f[8 * i + 2 * j], f[8 * i + 2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[8 * i + 2 * j], f[8 * i + 2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
            reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

__device__ __forceinline__ void q8_copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void q8_copy4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Bytes at `pick` (two of code + 128) as two fp16 codes.
__device__ __forceinline__ uint32_t codes2(uint32_t biased, uint32_t pick)
{
    const uint32_t w = __byte_perm(biased, 0x64646464u, pick);
    const uint32_t off = 0x64806480u;  // 1152
    uint32_t r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(off));
    return r;
}

// Byte j of a word as a signed integer.
__device__ __forceinline__ int q8_byte(uint32_t w, int j) { return static_cast<int>(static_cast<int8_t>(w >> (8 * j))); }

inline bool q8_a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool q8_a4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

struct Q8Range {
    const void* x;
    size_t bytes;
    bool written;
};

// Whether a written range overlaps another one (NULL and empty ranges do not).
inline bool q8_overlap(const Q8Range* r, int n)
{
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < i; ++j) {
            if (!(r[i].written || r[j].written) || !r[i].x || !r[j].x || !r[i].bytes || !r[j].bytes)
                continue;
            const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].x), b = reinterpret_cast<uintptr_t>(r[j].x);
            if (a < b + r[j].bytes && b < a + r[i].bytes)
                return true;
        }
    return false;
}

// Sizes of the cache that every call refuses.
inline int q8_sizes(int B, int KV, int D, int BLOCK, int max_blocks, int num_blocks, int dtype)
{
    if (B < 0 || KV < 1 || D < 1 || BLOCK < 1 || max_blocks < 1 || num_blocks < 1 ||
        static_cast<long long>(max_blocks) * BLOCK >= (1ll << 30) || static_cast<long long>(num_blocks) * BLOCK >= (1ll << 31))
        return PA_ERR_BAD_DIMS;
    if ((D != 64 && D != 128) || (BLOCK != 8 && BLOCK != 16 && BLOCK != 32 && BLOCK != 64) ||
        (dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16) || B > kMaxBatch || KV > 1024)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// A launch that may begin before the kernel ahead of it on the stream has ended;
// the kernel waits for that one before it reads anything (grid_begin).
inline int q8_launch(const void* fn, dim3 grid, int threads, size_t smem, cudaStream_t st, void** args, int cluster = 1)
{
    if (smem > 40 * 1024 && !allow_shared_memory(fn))  // (48 KB with what a kernel has statically)
        return PA_ERR_CUDA;
    if (cluster > 8 && cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return PA_ERR_CUDA;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess)
        return PA_ERR_CUDA;
    count_launches(1);
    return PA_OK;
}

}  // namespace pa
