// pa_q8_store.cu -- new rows into the cache in 8 bits, and rows back out of it
// (include/pa_q8.h).
//
// pa_q8_append_kernel: a group of BLOCK * D / 32 threads owns one block of one
// sequence and KV head, its keys and its values; a thread holds two runs of 16
// elements of each in registers, so the rows are read once for their largest
// magnitude and their codes.  The largest magnitudes, and for keys the lowest and
// highest codes by channel, are joined by shuffles and through shared memory.  Earlier
// codes are read only where the scale grew, and for the bounds.
// Prompts (4 of 3080 rows, 8 heads of 128 channels, bounds): 16-bit rows 19.4 us, 4.0
// TB/s, float32 31.8 us, 4.0 TB/s (one of 65536 rows 80 us, 5.0, and 147, 4.6).  Neither
// memory nor arithmetic is full (29 % of the peak, half the issue slots): a CTA lives
// for one block, and little but the other CTAs covers its chain of length, table, rows,
// maximum, codes (41 us before ties were corrected in registers, 34 before own scales
// spared the check).  A step of one row a sequence is a launch and two dependent reads,
// 3.1 us back to back, 7.4 to 8.3 where every block's scale grows (12.7 with 31 of 32
// rows there): the earlier codes are then rounded again byte by byte.
//
// pa_q8_read_kernel: a thread takes runs of 16 codes, about four one after another,
// heads and columns innermost: whole lines both ways.  Memory bounds it: 201 MB in
// 34.4 us, 5.8 TB/s (the four runs' loads together 37.7; 8 or 16 tokens a CTA more,
// or all in one, 36 to 43).
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kStoreThreads = 256;

// Threads of an append CTA for a block's rows of so many elements.
__host__ __device__ constexpr int append_threads(int elements) { return elements / 32 < 64 ? 64 : elements / 32; }

struct AppendParams {
    int8_t* cache[2];  // K, V
    float* scale[2];
    const void* rows[2];
    long long stride[2][3];
    int8_t* bounds;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* counts;
    int* status;
    int KV, N, maxb, num_blocks, cap;
};

__device__ __forceinline__ int clamp_report(int x, int hi, int* status)
{
    if (x >= 0 && x <= hi)
        return x;
    q8_report(status, PA_STATUS_BAD_LENGTH);
    return x < 0 ? 0 : hi;
}

// 16 elements of a row as they are in memory.
template <typename T>
struct Run {
    static constexpr int kVectors = sizeof(T);
    uint4 v[kVectors];

    __device__ __forceinline__ uint32_t word(int i) const
    {
        const uint4 x = v[i >> 2];
        return (i & 3) == 0 ? x.x : (i & 3) == 1 ? x.y : (i & 3) == 2 ? x.z : x.w;
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(word(i));
        } else {
            const uint32_t w = word(i >> 1);
            if constexpr (std::is_same_v<T, __half>) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
                return i & 1 ? f.y : f.x;
            } else {
                return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
            }
        }
    }
    // Largest magnitude, NaN where an element is none (16-bit: two side by side).
    __device__ __forceinline__ uint32_t largest(uint32_t m) const
    {
#pragma unroll
        for (int i = 0; i < 4 * kVectors; ++i) {
            if constexpr (sizeof(T) == 4)
                asm("max.NaN.f32 %0, %0, %1;" : "+r"(m) : "r"(word(i) & 0x7fffffffu));
            else if constexpr (std::is_same_v<T, __half>)
                asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(word(i) & 0x7fff7fffu));
            else
                asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(word(i) & 0x7fff7fffu));
        }
        return m;
    }
};

// The magnitude of largest()'s word.
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t m)
{
    if constexpr (sizeof(T) == 4)
        return __uint_as_float(m);
    float2 f;
    if constexpr (std::is_same_v<T, __half>)
        f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    else
        f = make_float2(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    return f.x + f.y == f.x + f.y ? fmaxf(f.x, f.y) : f.x + f.y;
}

__device__ __forceinline__ float element(const float* p) { return *p; }
__device__ __forceinline__ float element(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float element(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// How a block's values become whole numbers: by one product with `inv` and one
// rounding (adding 1.5 2^23) where `sure`, else with a look at the remainder.
//
// 16-bit values under a scale made of their own largest magnitude a are sure.
// Values and a are whole multiples of a unit u, so that x / (a / 127) is a half or
// at least u / (254 x) >= 2^-19 of itself away from one; the scale is a / 127
// (1 - e) with |e| <= 2^-24, and all halves go the way of e.  So `inv` is 1 / scale
// times 1 +- 1.5 2^-22 in the direction of e (with the error of the reciprocal
// between 2^-23 and 2^-21): halves fall on their side, nothing else crosses.  With
// e = 0 the halves are ties, and with an earlier block's scale anything may lie next
// to a half: then the checked way.
struct Rounding {
    float scale, inv;
    bool sure;
};

template <typename T>
__device__ __forceinline__ Rounding rounding_of(float a, float scale)
{
    Rounding r{scale, fast_rcp(scale), false};
    if constexpr (sizeof(T) == 2) {
        const float e = __fmaf_rn(-127.f, scale, a);  // a - 127 scale: its sign is exact
        if (e != 0.f && scale == q8_scale_of(a) && scale > kMinScale) {
            r.inv = __fmaf_rn(r.inv, copysignf(1.5f / 4194304.f, e), r.inv);
            r.sure = true;
        }
    }
    return r;
}

// Stores the codes of 16 elements (also at `src`) and returns them.  The checked
// way: the product with 1 / scale is within 2^-16 of the quotient; only where that
// leaves the side of a half open is the remainder x - r scale (exact in an fma)
// compared with half a step.  What is not finite goes through a loop, to keep the
// code short.
template <typename T>
__device__ __forceinline__ uint4 run_codes(int8_t* dst, const Run<T>& r, const T* src, const Rounding& by, bool odd)
{
    constexpr float kWhole = 12582912.f;
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        t[i] = __fmaf_rn(r.get(i), by.inv, kWhole);
    if (!by.sure) {
        float worst = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            worst = fmaxf(worst, fabsf(__fmaf_rn(r.get(i), by.inv, -(t[i] - kWhole))));
        if (worst > 0.49995f) {
            const float half = 0.5f * by.scale;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float d = __fmaf_rn(-(t[i] - kWhole), by.scale, r.get(i));
                const bool uneven = __float_as_uint(t[i]) & 1u;
                if (d > half || (uneven && d == half))
                    t[i] += 1.f;
                else if (d < -half || (uneven && d == -half))
                    t[i] -= 1.f;
            }
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __byte_perm(__byte_perm(__float_as_uint(t[4 * i]), __float_as_uint(t[4 * i + 1]), 0x0040),
                           __byte_perm(__float_as_uint(t[4 * i + 2]), __float_as_uint(t[4 * i + 3]), 0x0040), 0x5410);
    uint4 codes = make_uint4(w[0], w[1], w[2], w[3]);
    if (odd) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            dst[i] = static_cast<int8_t>(q8_code(element(src + i), by.scale, by.inv));
        codes = *reinterpret_cast<const uint4*>(dst);
    } else {
        *reinterpret_cast<uint4*>(dst) = codes;
    }
    return codes;
}

// Lowest and highest of two fp16 codes each.
__device__ __forceinline__ uint32_t lowest2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t highest2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight words of two fp16 codes as bytes: code + 1152 has code + 128 in its low byte.
__device__ __forceinline__ uint4 pack_codes(const uint32_t* two)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm("add.f16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(two[i]), "r"(0x64806480u));
    return make_uint4(__byte_perm(w[0], w[1], 0x6420) ^ 0x80808080u, __byte_perm(w[2], w[3], 0x6420) ^ 0x80808080u,
                      __byte_perm(w[4], w[5], 0x6420) ^ 0x80808080u, __byte_perm(w[6], w[7], 0x6420) ^ 0x80808080u);
}

// grid (blocks a sequence's new rows may touch, ceil(KV / heads of a CTA), B)
// (16-bit rows in 96 registers: 21.0 us for 12,300 rows of 8 heads; 124 by
// themselves 22.5, 64 27.3)
template <typename T, int D, int BLOCK>
__global__ void __launch_bounds__(append_threads(BLOCK * D), sizeof(T) == 2 ? 672 / append_threads(BLOCK * D) : 1) pa_q8_append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int kGroup = BLOCK * D / 32;           // threads of a block and head
    constexpr int kThreads = append_threads(BLOCK * D);
    constexpr int kHeads = kThreads / kGroup;        // heads of a CTA
    constexpr int kRuns = D / 16, kRows = kGroup / kRuns;  // a thread's rows: r, r + kRows (= BLOCK / 2)
    __shared__ float part[2][kThreads / 32];
    __shared__ __align__(16) uint32_t ends[kThreads / 32][2][kRuns * 8];  // lowest, highest codes by warp
    grid_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.z;
    const int h = blockIdx.y * kHeads + tid / kGroup;
    const int me = tid % kGroup, run = me % kRuns, row0 = me / kRuns;
    const bool report = blockIdx.x == 0 && blockIdx.y == 0 && tid == 0;
    const int past = clamp_report(__ldg(p.lens + b), p.cap, report ? p.status : nullptr);
    const int want = p.counts ? clamp_report(__ldg(p.counts + b), p.N, report ? p.status : nullptr) : p.N;
    const int blk = past / BLOCK + blockIdx.x;  // of the sequence
    const int first = blk * BLOCK;
    if (want == 0 || first >= past + want)  // no new row; the same in every thread of the CTA
        return;
    int phys = -1;
    if (blk < p.maxb)
        phys = __ldg(p.table + static_cast<int64_t>(b) * p.maxb + blk);
    // the new rows are on their way while the block is looked up
    const bool head = h < p.KV;
    Run<T> x[2][2];  // keys, values
    bool fresh[2];
    uint32_t most[2] = {0, 0};
    const T* rows[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
        rows[kv] = static_cast<const T*>(p.rows[kv]) + b * p.stride[kv][0] + h * p.stride[kv][1] +
                   (first + row0 - past) * p.stride[kv][2] + run * 16;
    auto src_of = [&](int kv, int k) { return rows[kv] + (k ? kRows * p.stride[kv][2] : 0ll); };
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int token = first + row0 + k * kRows;
        fresh[k] = head && token >= past && token < past + want;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
            if (fresh[k]) {
                const T* src = src_of(kv, k);
#pragma unroll
                for (int i = 0; i < Run<T>::kVectors; ++i)
                    x[kv][k].v[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
            }
    }
    if (phys < 0 || phys >= p.num_blocks) {
        if (tid == 0)
            q8_report(p.status, PA_STATUS_BAD_SLOT);
        return;
    }
    const bool earlier = first < past;
    const int64_t at = static_cast<int64_t>(phys) * p.KV + h;
    const int64_t place = ((static_cast<int64_t>(phys) * BLOCK + row0) * p.KV + h) * D + run * 16;
    float was[2] = {0.f, 0.f}, a[2];
    bool odd = false;  // something is not finite
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        if (head && earlier)
            was[kv] = p.scale[kv][at];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (fresh[k])
                most[kv] = x[kv][k].largest(most[kv]);
        a[kv] = magnitude<T>(most[kv]);
        if (!(a[kv] <= 3.402823466e38f)) {
            odd = true;
            a[kv] = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (fresh[k])
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        a[kv] = q8_amax(a[kv], x[kv][k].get(i));
        }
#pragma unroll
        for (int o = 1; o < (kGroup < 32 ? kGroup : 32); o <<= 1)
            a[kv] = fmaxf(a[kv], __shfl_xor_sync(kFullWarp, a[kv], o));
    }
    if (odd)
        q8_report(p.status, PA_STATUS_NOT_FINITE);
    if constexpr (kGroup > 32) {
        if (lane == 0) {
            part[0][warp] = a[0];
            part[1][warp] = a[1];
        }
        __syncthreads();
        constexpr int kWarps = kGroup / 32;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
            for (int i = 0; i < kWarps; ++i)
                a[kv] = fmaxf(a[kv], part[kv][warp / kWarps * kWarps + i]);
    } else {
        __syncwarp();  // (all have read the earlier scales, one stores the new ones)
    }

    uint32_t lo[8], hi[8];  // of this thread's keys: lowest and highest code by channel, two a word
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = 0x57f057f0u;  // 127
        hi[i] = 0xd7f0d7f0u;  // -127
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const float scale = fmaxf(q8_scale_of(a[kv]), was[kv]);
        const Rounding by = rounding_of<T>(a[kv], scale);
        const bool grown = earlier && scale > was[kv], ranged = kv == 0 && p.bounds;
        if (head && me == 0 && (!earlier || grown))
            p.scale[kv][at] = scale;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = row0 + k * kRows;
            int8_t* dst = p.cache[kv] + place + (k ? kRows * p.KV * D : 0);
            const bool old = head && first + row < past && (grown || ranged);
            uint4 c = make_uint4(0u, 0u, 0u, 0u);
            if (fresh[k]) {
                c = run_codes(dst, x[kv][k], src_of(kv, k), by, odd);
            } else if (old) {
                if (grown) {
#pragma unroll 1
                    for (int i = 0; i < 16; ++i)
                        dst[i] = static_cast<int8_t>(q8_again(dst[i], was[kv], scale, by.inv));
                }
                c = *reinterpret_cast<const uint4*>(dst);
            }
            if (ranged && (fresh[k] || old)) {
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t two = codes2(w[i >> 1] ^ 0x80808080u, i & 1 ? 0x4342 : 0x4140);
                    lo[i] = lowest2(lo[i], two);
                    hi[i] = highest2(hi[i], two);
                }
            }
        }
    }

    if (p.bounds) {  // (the same in every thread)
        // lanes with the same columns, then warps
#pragma unroll
        for (int o = kRuns; o < (kGroup < 32 ? kGroup : 32); o <<= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo[i] = lowest2(lo[i], __shfl_xor_sync(kFullWarp, lo[i], o));
                hi[i] = highest2(hi[i], __shfl_xor_sync(kFullWarp, hi[i], o));
            }
        if constexpr (kGroup > 32) {
            if (lane < kRuns && me >= 32) {
                uint4* to = reinterpret_cast<uint4*>(&ends[warp][0][lane * 8]);
                to[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                to[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                to[kRuns * 2] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                to[kRuns * 2 + 1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
            }
            __syncthreads();
        }
        if (head && me < kRuns) {
            if constexpr (kGroup > 32) {
                constexpr int kWarps = kGroup / 32;
                const int base = warp / kWarps * kWarps;
#pragma unroll
                for (int v = 1; v < kWarps; ++v) {
                    const uint4* at = reinterpret_cast<const uint4*>(&ends[base + v][0][me * 8]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 x = at[i], y = at[kRuns * 2 + i];
                        lo[4 * i] = lowest2(lo[4 * i], x.x), lo[4 * i + 1] = lowest2(lo[4 * i + 1], x.y);
                        lo[4 * i + 2] = lowest2(lo[4 * i + 2], x.z), lo[4 * i + 3] = lowest2(lo[4 * i + 3], x.w);
                        hi[4 * i] = highest2(hi[4 * i], y.x), hi[4 * i + 1] = highest2(hi[4 * i + 1], y.y);
                        hi[4 * i + 2] = highest2(hi[4 * i + 2], y.z), hi[4 * i + 3] = highest2(hi[4 * i + 3], y.w);
                    }
                }
            }
            uint4* to = reinterpret_cast<uint4*>(p.bounds + at * 2 * D + me * 16);
            to[0] = pack_codes(lo);
            to[D / 16] = pack_codes(hi);
        }
    }
}

struct ReadParams {
    const int8_t* cache[2];
    const float* scale[2];
    void* out[2];
    const int32_t* table;
    const int32_t* starts;
    const int32_t* counts;
    int* status;
    int KV, N, BLOCK, shift, maxb, num_blocks, cap;
};

// grid (ranges of a sequence's rows, 2, B): runs of 16 codes, heads and columns
// innermost, as the cache has them.
template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) pa_q8_read_kernel(const __grid_constant__ ReadParams p, int rows_cta)
{
    grid_begin();
    constexpr int kRuns = D / 16;
    const int tid = threadIdx.x, b = blockIdx.z, kv = blockIdx.y;
    const bool lead = tid == 0 && blockIdx.x == 0 && kv == 0;
    const int start = clamp_report(__ldg(p.starts + b), p.cap, lead ? p.status : nullptr);
    int rows = p.counts ? clamp_report(__ldg(p.counts + b), p.N, lead ? p.status : nullptr) : p.N;
    rows = clamp_report(rows, p.cap - start, lead ? p.status : nullptr);
    const int r0 = blockIdx.x * rows_cta, r1 = min(r0 + rows_cta, rows);
    const int per = p.KV * kRuns;  // runs of a token
    const int total = max(r1 - r0, 0) * per;
    for (int i = tid; i < total; i += kStoreThreads) {
        const int r = r0 + i / per, hr = i % per, h = hr / kRuns, run = hr % kRuns;
        const int token = start + r, blk = token >> p.shift;
        const int phys = __ldg(p.table + static_cast<int64_t>(b) * p.maxb + blk);
        if (phys < 0 || phys >= p.num_blocks) {
            q8_report(p.status, PA_STATUS_BAD_BLOCK);
            continue;
        }
        const float scale = __ldg(p.scale[kv] + static_cast<int64_t>(phys) * p.KV + h);
        const uint4 c = __ldg(reinterpret_cast<const uint4*>(
            p.cache[kv] + ((static_cast<int64_t>(phys) * p.BLOCK + (token & (p.BLOCK - 1))) * p.KV + h) * D + run * 16));
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
            f[k] = static_cast<float>(q8_byte(w[k >> 2], k & 3)) * scale;
        q8_store16(static_cast<T*>(p.out[kv]) + ((static_cast<int64_t>(b) * p.KV + h) * p.N + r) * D + run * 16, f);
    }
}

template <typename T, int D>
const void* append_kernel(int BLOCK)
{
    return BLOCK == 8    ? reinterpret_cast<const void*>(pa_q8_append_kernel<T, D, 8>)
           : BLOCK == 16 ? reinterpret_cast<const void*>(pa_q8_append_kernel<T, D, 16>)
           : BLOCK == 32 ? reinterpret_cast<const void*>(pa_q8_append_kernel<T, D, 32>)
                         : reinterpret_cast<const void*>(pa_q8_append_kernel<T, D, 64>);
}

template <typename T>
const void* append_kernel(int D, int BLOCK)
{
    return D == 64 ? append_kernel<T, 64>(BLOCK) : append_kernel<T, 128>(BLOCK);
}

template <typename T>
const void* read_kernel(int D)
{
    return D == 64 ? reinterpret_cast<const void*>(pa_q8_read_kernel<T, 64>) : reinterpret_cast<const void*>(pa_q8_read_kernel<T, 128>);
}

// Elements from the first to behind the last of rows with these strides.
size_t span_of(int B, int KV, int N, int D, const long long* s)
{
    return static_cast<size_t>((B - 1) * s[0] + (KV - 1) * s[1] + (N - 1) * s[2] + D);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_q8_append(int8_t* k_cache, int8_t* v_cache, float* k_scale, float* v_scale, const void* k_new,
                            const void* v_new, const int32_t* block_table, const int32_t* seq_lens, int B, int KV, int D, int N,
                            int BLOCK, const pa_q8_append_opts* opts, void* stream)
{
    if (!opts)
        return PA_ERR_NULL_POINTER;
    const pa_q8_append_opts& o = *opts;
    const int rc = q8_sizes(B, KV, D, BLOCK, o.max_blocks, o.num_blocks, o.dtype);
    if (rc != PA_OK)
        return rc;
    if (N < 0)
        return PA_ERR_BAD_DIMS;
    if (N > PA_MAX_PREFILL)
        return PA_ERR_UNSUPPORTED;
    if (B == 0 || N == 0)
        return PA_OK;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !k_new || !v_new || !block_table || !seq_lens)
        return PA_ERR_NULL_POINTER;
    const int e = o.dtype == PA_F32 ? 4 : 2;
    if (!q8_a16(k_cache) || !q8_a16(v_cache) || !q8_a16(k_new) || !q8_a16(v_new) || !q8_a16(o.bounds) || !q8_a4(k_scale) ||
        !q8_a4(v_scale) || !q8_a4(block_table) || !q8_a4(seq_lens) || !q8_a4(o.counts) || !q8_a4(o.status))
        return PA_ERR_ALIGNMENT;
    for (int i = 0; i < 3; ++i) {
        if (o.k_strides[i] < 0 || o.v_strides[i] < 0 || (o.k_strides[i] * e) % 16 != 0 || (o.v_strides[i] * e) % 16 != 0)
            return PA_ERR_ALIGNMENT;
        if (o.k_strides[i] >= (1ll << 40) || o.v_strides[i] >= (1ll << 40))
            return PA_ERR_BAD_DIMS;
    }
    const size_t blocks = static_cast<size_t>(o.num_blocks) * KV, pool = blocks * BLOCK * D, b4 = static_cast<size_t>(B) * 4;
    const Q8Range r[] = {{k_cache, pool, true},        {v_cache, pool, true},
                         {k_scale, blocks * 4, true},  {v_scale, blocks * 4, true},
                         {o.bounds, blocks * 2 * D, true}, {o.status, 4, true},
                         {k_new, span_of(B, KV, N, D, o.k_strides) * e, false}, {v_new, span_of(B, KV, N, D, o.v_strides) * e, false},
                         {block_table, b4 * o.max_blocks, false}, {seq_lens, b4, false}, {o.counts, b4, false}};
    if (q8_overlap(r, 11))
        return PA_ERR_BAD_DIMS;
    AppendParams p{};
    p.cache[0] = k_cache, p.cache[1] = v_cache;
    p.scale[0] = k_scale, p.scale[1] = v_scale;
    p.rows[0] = k_new, p.rows[1] = v_new;
    for (int i = 0; i < 3; ++i)
        p.stride[0][i] = o.k_strides[i], p.stride[1][i] = o.v_strides[i];
    p.bounds = o.bounds;
    p.table = block_table;
    p.lens = seq_lens;
    p.counts = o.counts;
    p.status = o.status;
    p.KV = KV;
    p.N = N;
    p.maxb = o.max_blocks;
    p.num_blocks = o.num_blocks;
    p.cap = o.max_blocks * BLOCK;
    const int group = BLOCK * D / 32, threads = append_threads(BLOCK * D), heads = threads / group;
    const void* fn = o.dtype == PA_F32   ? append_kernel<float>(D, BLOCK)
                     : o.dtype == PA_F16 ? append_kernel<__half>(D, BLOCK)
                                         : append_kernel<__nv_bfloat16>(D, BLOCK);
    void* args[] = {&p};
    return q8_launch(fn, dim3((N + BLOCK - 2) / BLOCK + 1, (KV + heads - 1) / heads, B), threads, 0,
                     static_cast<cudaStream_t>(stream), args);
}

extern "C" int pa_q8_read(const int8_t* k_cache, const int8_t* v_cache, const float* k_scale, const float* v_scale,
                          const int32_t* block_table, const int32_t* starts, void* k_out, void* v_out, int B, int KV, int D, int N,
                          int BLOCK, const pa_q8_read_opts* opts, void* stream)
{
    if (!opts)
        return PA_ERR_NULL_POINTER;
    const pa_q8_read_opts& o = *opts;
    const int rc = q8_sizes(B, KV, D, BLOCK, o.max_blocks, o.num_blocks, o.dtype);
    if (rc != PA_OK)
        return rc;
    if (N < 0 || N >= (1 << 30))
        return PA_ERR_BAD_DIMS;
    if (B == 0 || N == 0)
        return PA_OK;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !k_out || !v_out || !block_table || !starts)
        return PA_ERR_NULL_POINTER;
    if (!q8_a16(k_cache) || !q8_a16(v_cache) || !q8_a16(k_out) || !q8_a16(v_out) || !q8_a4(k_scale) || !q8_a4(v_scale) ||
        !q8_a4(block_table) || !q8_a4(starts) || !q8_a4(o.counts) || !q8_a4(o.status))
        return PA_ERR_ALIGNMENT;
    const size_t blocks = static_cast<size_t>(o.num_blocks) * KV, pool = blocks * BLOCK * D, b4 = static_cast<size_t>(B) * 4;
    const size_t out = static_cast<size_t>(B) * KV * N * D * (o.dtype == PA_F32 ? 4 : 2);
    const Q8Range r[] = {{k_out, out, true},           {v_out, out, true},
                         {o.status, 4, true},          {k_cache, pool, false},
                         {v_cache, pool, false},       {k_scale, blocks * 4, false},
                         {v_scale, blocks * 4, false}, {block_table, b4 * o.max_blocks, false},
                         {starts, b4, false},          {o.counts, b4, false}};
    if (q8_overlap(r, 10))
        return PA_ERR_BAD_DIMS;
    ReadParams p{};
    p.cache[0] = k_cache, p.cache[1] = v_cache;
    p.scale[0] = k_scale, p.scale[1] = v_scale;
    p.out[0] = k_out, p.out[1] = v_out;
    p.table = block_table;
    p.starts = starts;
    p.counts = o.counts;
    p.status = o.status;
    p.KV = KV;
    p.N = N;
    p.BLOCK = BLOCK;
    p.shift = BLOCK == 8 ? 3 : BLOCK == 16 ? 4 : BLOCK == 32 ? 5 : 6;
    p.maxb = o.max_blocks;
    p.num_blocks = o.num_blocks;
    p.cap = o.max_blocks * BLOCK;
    const void* fn = o.dtype == PA_F32 ? read_kernel<float>(D) : o.dtype == PA_F16 ? read_kernel<__half>(D) : read_kernel<__nv_bfloat16>(D);
    // about four runs a thread
    int rows = 4 * kStoreThreads / (KV * (D / 16));
    rows = rows < 1 ? 1 : rows;
    void* args[] = {&p, &rows};
    return q8_launch(fn, dim3((N + rows - 1) / rows, 2, B), kStoreThreads, 0, static_cast<cudaStream_t>(stream), args);
}
