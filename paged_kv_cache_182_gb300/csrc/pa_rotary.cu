// pa_rotary.cu -- rotary positions (include/pa_rotary.h): queries and keys
// turned by their positions, forward and gradient, optionally with the store
// of the rotated keys and the values into the paged cache.
//
// Bound by memory: every row is read and written once (a cached row once
// more), three multiply-adds an element.  What it must not do is compute a
// cosine and a sine per element: the angle depends on the position and the
// pair alone, so a CTA takes a few positions of one sequence and all (or a
// share) of their heads.  Its threads compute the positions' cosines and sines
// together into shared memory; then each keeps those of its own 16 bytes of a
// row in registers and walks the heads with them.  The first heads' rows are in
// flight while the table is computed.
//
// What is left: with one or two heads a position's sines are the time (1 + 1
// heads, 4 x 16384 rows: 24.6 us for 10 of bytes); halves that are not whole
// vectors read their partners one element at a time ([4, 32 + 8, 2048] bf16:
// D = 72 halves 51.0 us, pairs 30.7; D = 80 with rot 36 50.8, rot 32 26.7); and
// every CTA of a store looks through the rest of its sequence for a later row
// with its slots, N^2 / 2 reads a head share (one sequence of 8192 rows, 32 + 8
// heads: 71 us, 33 without the store; of 65536: 2.0 ms, 0.23 without).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_rotary.h"
#include "pa_vjp.cuh"

namespace pa {
namespace {

constexpr int kRotThreads = 256;  // at most
constexpr int kRotHeads = 2;  // heads in flight per thread

struct RotaryParams {
    const void* x[3];       // q, k, v
    void* out[2];           // q_out, k_out (or NULL)
    void* cache[2];         // k_cache, v_cache (or NULL)
    long long st[3][3];     // strides of q, k, v: batch, head, row
    const int32_t* positions;
    const uint64_t* table;
    const int32_t* slots;
    int* status;
    int B, H, KV, N, D, rot;
    int heads;              // H + KV (+ KV value rows with a cache store)
    int rows_cta;           // positions of one sequence per CTA
    int head_cta;           // heads per CTA
    long long num_slots;
    float factor;
    int inverse;
};

// The angle's cosine and sine times the factor.  The phase is reduced to the
// nearest quarter turn as an integer, so that the float conversion of the rest
// (|rest| <= 1/8 turn) keeps 24 bits of it.
__device__ __forceinline__ float2 turn(int pos, uint64_t per, float factor, bool inverse)
{
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * per;
    const uint32_t hi = static_cast<uint32_t>((phase + 0x80000000u) >> 32);  // nearest 2^-32 turn
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(hi - (quarter << 30));
    float s, c;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    const float c1 = (quarter & 1) ? -s : c, s1 = (quarter & 1) ? c : s;
    const float sg = (quarter & 2) ? -factor : factor;
    return make_float2(c1 * sg, inverse ? -s1 * sg : s1 * sg);
}

template <typename T>
struct Vec;  // 16 bytes of T as floats
template <>
struct Vec<float> {
    static constexpr int n = 4;
    __device__ static void get(const uint4& u, float* f)
    {
        memcpy(f, &u, 16);
    }
    __device__ static uint4 put(const float* f)
    {
        uint4 u;
        memcpy(&u, f, 16);
        return u;
    }
};
template <>
struct Vec<__half> {
    static constexpr int n = 8;
    __device__ static void get(const uint4& u, float* f)
    {
        __half2 h[4];
        memcpy(h, &u, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(h[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    __device__ static uint4 put(const float* f)
    {
        __half2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        uint4 u;
        memcpy(&u, h, 16);
        return u;
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    __device__ static void get(const uint4& u, float* f)
    {
        __nv_bfloat162 h[4];
        memcpy(h, &u, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __bfloat1622float2(h[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    __device__ static uint4 put(const float* f)
    {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        uint4 u;
        memcpy(&u, h, 16);
        return u;
    }
};

// How the 16-byte vectors of a row meet their pairs:
//   kHalves  rot / 2 is whole vectors: a thread takes vector i of the first half
//            and the one rot / 2 columns on, or one of the untouched vectors
//   kSide    interleaved pairs: a thread takes one vector, its pairs inside it
//   kAny     halves of any other length: a thread takes one vector, its
//            elements' partners read one at a time (they are in the same row,
//            so in the lines that the vectors fetch)
enum { kHalves = 0, kSide = 1, kAny = 2 };

// Thread t of a CTA: unit t % units (row, vector), head group t / units.
template <typename T, int MODE>
__global__ void __launch_bounds__(kRotThreads) pa_rotary_kernel(const __grid_constant__ RotaryParams p)
{
    constexpr int V = Vec<T>::n;
    constexpr int NP = MODE == kSide ? V / 2 : V;  // pairs of a thread
    constexpr int U = kRotHeads;
    // a kernel launched after this one with programmatic launch may set up
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ float2 tab[];  // [rows_cta][rot / 2] (cos, sin)
    const int half = p.rot >> 1;
    const int chunks = (p.N + p.rows_cta - 1) / p.rows_cta;
    const int b = blockIdx.x / chunks;
    const int n0 = (blockIdx.x - b * chunks) * p.rows_cta;
    const int rows = min(p.rows_cta, p.N - n0);
    const int per_row = MODE == kHalves ? (p.D - half) / V : p.D / V;
    const int units = p.rows_cta * per_row;
    const int groups = static_cast<int>(blockDim.x) / units;
    const int unit = threadIdx.x % units, group = threadIdx.x / units;
    const int row = unit / per_row, v = unit - row * per_row;
    const bool live = group < groups && row < rows;
    const bool two = MODE == kHalves && v < half / V;
    const int col = MODE == kHalves && !two ? v * V + half : v * V;
    const int n = n0 + row;
    const int h1 = min(p.heads, (static_cast<int>(blockIdx.y) + 1) * p.head_cta);
    int h = blockIdx.y * p.head_cta + group;

    auto source = [&](int head) {
        const int t = head < p.H ? 0 : head < p.H + p.KV ? 1 : 2;
        const int hl = t == 0 ? head : t == 1 ? head - p.H : head - p.H - p.KV;
        return static_cast<const T*>(p.x[t]) + b * p.st[t][0] + hl * p.st[t][1] + n * p.st[t][2];
    };
    uint4 a[U], c[U];
    auto load = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int head = h + u * groups;
            if (live && head < h1) {
                const T* x = source(head) + col;
                a[u] = __ldg(reinterpret_cast<const uint4*>(x));
                if (two)
                    c[u] = __ldg(reinterpret_cast<const uint4*>(x + half));
            }
        }
    };
    load();
    for (int i = threadIdx.x; i < rows * half; i += static_cast<int>(blockDim.x)) {
        const int r = i / half;
        tab[i] = turn(__ldg(p.positions + static_cast<int64_t>(b) * p.N + n0 + r), __ldg(p.table + (i - r * half)), p.factor,
                      p.inverse);
    }
    // The rows' slots, -1 where nothing is stored: skipped, outside the pool, or
    // taken by a later row of the sequence, which the CTA's threads look for
    // together (a prompt of N rows asks N / 2 of them for each).
    const bool stores = p.slots && h1 > p.H;  // this CTA has keys or values
    int* slots = reinterpret_cast<int*>(tab + p.rows_cta * half);  // [rows_cta]
    if (stores) {
        const int32_t* sl = p.slots + static_cast<int64_t>(b) * p.N;
        for (int r = threadIdx.x; r < rows; r += static_cast<int>(blockDim.x)) {
            int s = __ldg(sl + n0 + r);
            if (s < -1 || s >= p.num_slots) {
                if (p.status)
                    atomicOr(p.status, PA_STATUS_BAD_SLOT);
                s = -1;
            }
            slots[r] = s;
        }
        __syncthreads();
        for (int r = 0; r < rows; ++r) {
            const int s = slots[r];
            bool later = false;
            if (s >= 0)
                for (int j = n0 + r + 1 + threadIdx.x; j < p.N; j += static_cast<int>(blockDim.x))
                    later |= __ldg(sl + j) == s;
            if (__syncthreads_or(later) && threadIdx.x == 0)
                slots[r] = -1;
        }
    }
    __syncthreads();
    const int slot = stores && live ? slots[row] : -1;
    float2 w[NP];
    if (live) {
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            int i = MODE == kSide ? (col >> 1) + e : col + e;
            if (MODE == kAny && i >= half)
                i -= half;
            // columns past rot: the identity, so that one loop serves all
            w[e] = i < half && (MODE != kHalves || two) ? tab[row * half + i] : make_float2(1.f, 0.f);
        }
    }
    for (; h < h1; h += U * groups) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int head = h + u * groups;
            if (!live || head >= h1)
                continue;
            const int t = head < p.H ? 0 : head < p.H + p.KV ? 1 : 2;
            const int hl = t == 0 ? head : t == 1 ? head - p.H : head - p.H - p.KV;
            if (t < 2) {
                if (two) {
                    float x[V], y[V];
                    Vec<T>::get(a[u], x);
                    Vec<T>::get(c[u], y);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float nx = x[e] * w[e].x - y[e] * w[e].y;
                        y[e] = fmaf(x[e], w[e].y, y[e] * w[e].x);
                        x[e] = nx;
                    }
                    a[u] = Vec<T>::put(x);
                    c[u] = Vec<T>::put(y);
                } else if (MODE == kSide && col < p.rot) {
                    float x[V];
                    Vec<T>::get(a[u], x);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e)
                        if (col + 2 * e < p.rot) {
                            const float nx = x[2 * e] * w[e].x - x[2 * e + 1] * w[e].y;
                            x[2 * e + 1] = fmaf(x[2 * e], w[e].y, x[2 * e + 1] * w[e].x);
                            x[2 * e] = nx;
                        }
                    a[u] = Vec<T>::put(x);
                } else if (MODE == kAny && col < p.rot) {
                    const T* xr = source(head);
                    float x[V];
                    Vec<T>::get(a[u], x);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int i = col + e;
                        if (i < half)
                            x[e] = x[e] * w[e].x - static_cast<float>(xr[i + half]) * w[e].y;
                        else if (i < p.rot)
                            x[e] = fmaf(static_cast<float>(xr[i - half]), w[e].y, x[e] * w[e].x);
                    }
                    a[u] = Vec<T>::put(x);
                }
                if (p.out[t]) {
                    T* o = static_cast<T*>(p.out[t]) +
                           ((static_cast<int64_t>(b) * (t == 0 ? p.H : p.KV) + hl) * p.N + n) * p.D + col;
                    *reinterpret_cast<uint4*>(o) = a[u];
                    if (two)
                        *reinterpret_cast<uint4*>(o + half) = c[u];
                }
            }
            if (t >= 1 && slot >= 0) {
                T* o = static_cast<T*>(p.cache[t - 1]) + (static_cast<int64_t>(slot) * p.KV + hl) * p.D + col;
                *reinterpret_cast<uint4*>(o) = a[u];
                if (two)
                    *reinterpret_cast<uint4*>(o + half) = c[u];
            }
        }
        if (h + U * groups < h1) {
            h += U * groups;
            load();
            h -= U * groups;
        }
    }
}

bool a16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; }

struct Range {
    uintptr_t lo, hi;
};

Range strided(const void* x, const long long* st, int B, int H, int N, int D, int es)
{
    const long long last = (B - 1) * st[0] + (H - 1) * st[1] + (N - 1) * st[2] + D;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(x);
    return {lo, lo + static_cast<uintptr_t>(last * es)};
}

using RotFn = void (*)(RotaryParams);

template <typename T>
RotFn pick_rotary(int mode)
{
    return mode == kHalves ? pa_rotary_kernel<T, kHalves> : mode == kSide ? pa_rotary_kernel<T, kSide> : pa_rotary_kernel<T, kAny>;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_rotary(const void* q, const void* k, const int32_t* positions, const uint64_t* table,
                         void* q_out, void* k_out, int B, int H, int KV, int N, int D, int rot,
                         const pa_rotary_opts* opts, void* stream)
{
    if (!opts)
        return PA_ERR_NULL_POINTER;
    const pa_rotary_opts& o = *opts;
    const bool store = o.slot_mapping != nullptr;
    if (B < 0 || H < 0 || KV < 0 || H + static_cast<long long>(KV) < 1 || N < 0 || D < 1 || rot < 2 || rot > D || (rot & 1) ||
        !std::isfinite(o.factor) || (store && (KV < 1 || o.BLOCK < 1 || o.num_blocks < 1)))
        return PA_ERR_BAD_DIMS;
    if (o.dtype != PA_F32 && o.dtype != PA_F16 && o.dtype != PA_BF16)
        return PA_ERR_UNSUPPORTED;
    const int es = o.dtype == PA_F32 ? 4 : 2;
    if (D > 1024 || D * es % 16 != 0 || (store && N > PA_MAX_PREFILL))
        return PA_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * N >= (1ll << 31) || H + 2ll * KV >= (1 << 16) ||
        (store && static_cast<long long>(o.num_blocks) * o.BLOCK >= (1ll << 31)))
        return PA_ERR_BAD_DIMS;
    if (B == 0 || N == 0)
        return PA_OK;
    if (!positions || !table || (H > 0 && (!q || !q_out)) || (KV > 0 && (!k || (!k_out && !store))) ||
        (store && (!o.v || !o.k_cache || !o.v_cache)))
        return PA_ERR_NULL_POINTER;
    if (!a16(q) || !a16(k) || !a16(q_out) || !a16(k_out) || (reinterpret_cast<uintptr_t>(positions) & 3) ||
        (reinterpret_cast<uintptr_t>(table) & 7) ||
        (store && (!a16(o.v) || !a16(o.k_cache) || !a16(o.v_cache) || (reinterpret_cast<uintptr_t>(o.slot_mapping) & 3))))
        return PA_ERR_ALIGNMENT;
    const int V = 16 / es;
    for (int i = 0; i < 3; ++i) {
        const long long sq = H > 0 ? o.q_strides[i] : 0, sk = KV > 0 ? o.k_strides[i] : 0, sv = store ? o.v_strides[i] : 0;
        for (long long s : {sq, sk, sv})
            if (s < 0 || s % V != 0)
                return PA_ERR_ALIGNMENT;
            else if (s >= (1ll << 40))
                return PA_ERR_BAD_DIMS;
    }
    // outputs apart from inputs
    const uintptr_t row = static_cast<uintptr_t>(D) * es;
    Range in[3] = {}, out[4] = {};
    if (H > 0) {
        in[0] = strided(q, o.q_strides, B, H, N, D, es);
        out[0] = {reinterpret_cast<uintptr_t>(q_out), reinterpret_cast<uintptr_t>(q_out) + row * H * B * N};
    }
    if (KV > 0) {
        in[1] = strided(k, o.k_strides, B, KV, N, D, es);
        if (k_out)
            out[1] = {reinterpret_cast<uintptr_t>(k_out), reinterpret_cast<uintptr_t>(k_out) + row * KV * B * N};
    }
    if (store) {
        in[2] = strided(o.v, o.v_strides, B, KV, N, D, es);
        const uintptr_t pool = row * KV * o.BLOCK * o.num_blocks;
        out[2] = {reinterpret_cast<uintptr_t>(o.k_cache), reinterpret_cast<uintptr_t>(o.k_cache) + pool};
        out[3] = {reinterpret_cast<uintptr_t>(o.v_cache), reinterpret_cast<uintptr_t>(o.v_cache) + pool};
    }
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : in)
            if (out[i].lo < r.hi && r.lo < out[i].hi)
                return PA_ERR_BAD_DIMS;
        for (int j = 0; j < i; ++j)
            if (out[i].lo < out[j].hi && out[j].lo < out[i].hi)
                return PA_ERR_BAD_DIMS;
    }

    RotaryParams p{};
    p.x[0] = q;
    p.x[1] = k;
    p.x[2] = o.v;
    p.out[0] = q_out;
    p.out[1] = KV > 0 ? k_out : nullptr;
    p.cache[0] = o.k_cache;
    p.cache[1] = o.v_cache;
    for (int i = 0; i < 3; ++i) {
        p.st[0][i] = o.q_strides[i];
        p.st[1][i] = o.k_strides[i];
        p.st[2][i] = o.v_strides[i];
    }
    p.positions = positions;
    p.table = table;
    p.slots = o.slot_mapping;
    p.status = o.status;
    p.B = B;
    p.H = H;
    p.KV = KV;
    p.N = N;
    p.D = D;
    p.rot = rot;
    p.heads = H + KV + (store ? KV : 0);
    p.num_slots = static_cast<long long>(o.num_blocks) * o.BLOCK;
    p.factor = o.factor;
    p.inverse = o.inverse ? 1 : 0;
    const int mode = o.interleaved ? kSide : (rot / 2) % V == 0 ? kHalves : kAny;
    // Small CTAs: 64 threads (more only where a row has more vectors).  With many
    // heads about 16 units of 16 or 32 bytes, so that four threads share a
    // unit's heads; with fewer than 20 heads a unit per thread, so that a
    // CTA still has enough to do; 32 KB of table at most; and as many heads as four rounds
    // of two take, fewer where the call would leave SMs idle.
    // us with 16 units / a unit per thread, bf16, D = 128, four sequences: 1 + 1
    // heads (16384 rows) 45.1 / 24.6, 4 + 1 (8192) 28.7 / 22.5, 8 + 2 (4096)
    // 22.1 / 21.4, 12 + 3 28.6 / 28.7, 16 + 4 (2048) 20.5 / 20.8, 24 + 6 27.8 /
    // 28.7, 32 + 8 32.8 (5.1 TB/s) / 36.6; f32, D = 64: [31, 8 + 2, 1492] 41.0 /
    // 42.6, [16, 16 + 4, 1492] 39.8 (6.1 TB/s) / 42.7.
    const int per_row = mode == kHalves ? (D - rot / 2) / V : D / V;
    const int threads = per_row > 128 ? 256 : per_row > 64 ? 128 : 64;
    int rows = p.heads >= 20 ? (15 + per_row) / per_row : threads / per_row;
    if (rows * per_row > threads)
        rows = threads / per_row;
    const int fit = 32768 / (rot / 2 * static_cast<int>(sizeof(float2)));
    rows = rows < 1 ? 1 : rows;
    rows = rows > fit ? fit : rows;
    rows = rows > N ? N : rows;
    const auto ctas = [&](int r) { return static_cast<long long>(B) * ((N + r - 1) / r); };
    while (rows > 1 && ctas(rows) < 304)
        --rows;
    p.rows_cta = rows;
    const int groups = threads / (rows * per_row);
    int rounds = 4;
    p.head_cta = groups * kRotHeads * rounds;
    while (p.head_cta > groups && ctas(rows) * ((p.heads + p.head_cta - 1) / p.head_cta) < 152)
        p.head_cta -= groups;
    const long long gx = static_cast<long long>(B) * ((N + p.rows_cta - 1) / p.rows_cta);
    const int gy = (p.heads + p.head_cta - 1) / p.head_cta;
    if (gx >= (1ll << 31))
        return PA_ERR_BAD_DIMS;
    const RotFn fn = o.dtype == PA_F32 ? pick_rotary<float>(mode) : o.dtype == PA_F16 ? pick_rotary<__half>(mode) : pick_rotary<__nv_bfloat16>(mode);
    const size_t smem = static_cast<size_t>(p.rows_cta) * (rot / 2 * sizeof(float2) + sizeof(int));
    fn<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), threads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    if (cudaGetLastError() != cudaSuccess)
        return PA_ERR_CUDA;
    count_launches(1);
    return PA_OK;
}
