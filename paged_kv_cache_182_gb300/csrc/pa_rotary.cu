// pa_rotary.cu -- rotary positions (include/pa_rotary.h): queries and keys
// turned by their positions, forward and gradient, optionally with the store
// of the rotated keys and the values into the paged cache.
//
// Bound by memory: every row is read and written once (a cached row once
// more), three multiply-adds an element.  What it must not do is compute a
// cosine and a sine per element: the angle depends on the position and the
// pair alone, so a CTA takes a few positions of one sequence and all (or a
// share) of their heads, and keeps the positions' cosines and sines in shared
// memory.  The rows are in flight while the table is computed.
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

constexpr int kRotThreads = 256;
constexpr int kRotItems = 4;  // items in flight per thread

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
//   kHalves  rot / 2 is whole vectors: an item is vector i of the first half
//            and the one rot / 2 columns on, then the untouched vectors, one
//            an item
//   kSide    interleaved pairs: an item is one vector, its pairs inside it
//   kAny     halves of any other length: an item is one vector, its elements'
//            partners read one at a time (they are in the same row, so in the
//            lines that the vectors fetch)
enum { kHalves = 0, kSide = 1, kAny = 2 };

template <typename T, int MODE>
__global__ void __launch_bounds__(kRotThreads) pa_rotary_kernel(const __grid_constant__ RotaryParams p)
{
    constexpr int V = Vec<T>::n;
    // a kernel launched after this one with programmatic launch may set up
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ float2 tab[];  // [rows_cta][rot / 2] (cos, sin)
    const int half = p.rot >> 1;
    const int chunks = (p.N + p.rows_cta - 1) / p.rows_cta;
    const int b = blockIdx.x / chunks;
    const int n0 = (blockIdx.x - b * chunks) * p.rows_cta;
    const int rows = min(p.rows_cta, p.N - n0);
    const int h0 = blockIdx.y * p.head_cta;
    const int nh = min(p.head_cta, p.heads - h0);
    const int per_row = MODE == kHalves ? (p.D - half) / V : p.D / V;  // items of one row of one head
    const int pairs = MODE == kHalves ? half / V : 0;                  // of them, two-vector items
    const int total = nh * rows * per_row;

    for (int base = 0; base < total; base += kRotThreads * kRotItems) {
        uint4 a[kRotItems], c[kRotItems];
        int tens[kRotItems], hh[kRotItems], rr[kRotItems], vv[kRotItems];
#pragma unroll
        for (int u = 0; u < kRotItems; ++u) {
            const int i = base + u * kRotThreads + static_cast<int>(threadIdx.x);
            tens[u] = -1;
            if (i < total) {
                const int hr = i / per_row;
                vv[u] = i - hr * per_row;
                const int hl = hr / rows;
                rr[u] = hr - hl * rows;
                int h = h0 + hl;
                tens[u] = 0;
                if (h >= p.H) {
                    h -= p.H;
                    tens[u] = 1;
                    if (h >= p.KV) {
                        h -= p.KV;
                        tens[u] = 2;
                    }
                }
                hh[u] = h;
                const T* row = static_cast<const T*>(p.x[tens[u]]) + b * p.st[tens[u]][0] + h * p.st[tens[u]][1] +
                               (n0 + rr[u]) * p.st[tens[u]][2];
                const int col = MODE == kHalves && vv[u] >= pairs ? vv[u] * V + half : vv[u] * V;
                a[u] = __ldg(reinterpret_cast<const uint4*>(row + col));
                if (MODE == kHalves && vv[u] < pairs)
                    c[u] = __ldg(reinterpret_cast<const uint4*>(row + col + half));
            }
        }
        if (base == 0) {
            // the positions' table, while the first rows are in flight
            for (int i = threadIdx.x; i < rows * half; i += kRotThreads) {
                const int r = i / half, j = i - r * half;
                tab[i] = turn(__ldg(p.positions + static_cast<long long>(b) * p.N + n0 + r), __ldg(p.table + j),
                              p.factor, p.inverse);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kRotItems; ++u) {
            if (tens[u] < 0)
                continue;
            const int col = MODE == kHalves && vv[u] >= pairs ? vv[u] * V + half : vv[u] * V;
            const bool two = MODE == kHalves && vv[u] < pairs;
            if (tens[u] < 2) {
                const float2* t = tab + rr[u] * half;
                if (two) {
                    float x[V], y[V];
                    Vec<T>::get(a[u], x);
                    Vec<T>::get(c[u], y);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float2 w = t[col + e];
                        const float nx = x[e] * w.x - y[e] * w.y;
                        y[e] = fmaf(x[e], w.y, y[e] * w.x);
                        x[e] = nx;
                    }
                    a[u] = Vec<T>::put(x);
                    c[u] = Vec<T>::put(y);
                } else if (MODE == kSide && col < p.rot) {
                    float x[V];
                    Vec<T>::get(a[u], x);
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        if (col + e < p.rot) {
                            const float2 w = t[(col + e) >> 1];
                            const float nx = x[e] * w.x - x[e + 1] * w.y;
                            x[e + 1] = fmaf(x[e], w.y, x[e + 1] * w.x);
                            x[e] = nx;
                        }
                    }
                    a[u] = Vec<T>::put(x);
                } else if (MODE == kAny && col < p.rot) {
                    const T* row = static_cast<const T*>(p.x[tens[u]]) + b * p.st[tens[u]][0] + hh[u] * p.st[tens[u]][1] +
                                   (n0 + rr[u]) * p.st[tens[u]][2];
                    float x[V];
                    Vec<T>::get(a[u], x);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int i = col + e;
                        if (i < half) {
                            const float2 w = t[i];
                            x[e] = x[e] * w.x - static_cast<float>(row[i + half]) * w.y;
                        } else if (i < p.rot) {
                            const float2 w = t[i - half];
                            x[e] = fmaf(static_cast<float>(row[i - half]), w.y, x[e] * w.x);
                        }
                    }
                    a[u] = Vec<T>::put(x);
                }
            }
            long long at = ((static_cast<long long>(b) * (tens[u] == 0 ? p.H : p.KV) + hh[u]) * p.N + n0 + rr[u]) * p.D + col;
            if (tens[u] < 2 && p.out[tens[u]]) {
                T* o = static_cast<T*>(p.out[tens[u]]) + at;
                *reinterpret_cast<uint4*>(o) = a[u];
                if (two)
                    *reinterpret_cast<uint4*>(o + half) = c[u];
            }
            if (tens[u] >= 1 && p.slots) {
                const int32_t* sl = p.slots + static_cast<long long>(b) * p.N;
                const int s = __ldg(sl + n0 + rr[u]);
                bool store = s >= 0 && s < p.num_slots;
                if (!store && s != -1 && p.status && tens[u] == 1 && hh[u] == 0 && vv[u] == 0)
                    atomicOr(p.status, PA_STATUS_BAD_SLOT);
                for (int j = n0 + rr[u] + 1; store && j < p.N; ++j)
                    store = __ldg(sl + j) != s;  // a later row of this sequence lands there
                if (store) {
                    T* o = static_cast<T*>(p.cache[tens[u] - 1]) + (static_cast<long long>(s) * p.KV + hh[u]) * p.D + col;
                    *reinterpret_cast<uint4*>(o) = a[u];
                    if (two)
                        *reinterpret_cast<uint4*>(o + half) = c[u];
                }
            }
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
    // A CTA takes about two passes of its threads' items (1024 a pass) over
    // consecutive positions; a short call spreads over the SMs instead, its
    // heads split so that a CTA still fills its threads once.
    const int per_row = mode == kHalves ? (D - rot / 2) / V : D / V;
    const long long row_items = static_cast<long long>(p.heads) * per_row;
    const long long want = (2 * kRotThreads * kRotItems + row_items - 1) / row_items;
    p.rows_cta = static_cast<int>(want < 1 ? 1 : want > 16 ? 16 : want);
    const int fit = 32768 / (rot / 2 * static_cast<int>(sizeof(float2)));  // 32 KB of table at most
    if (p.rows_cta > fit)
        p.rows_cta = fit;
    if (p.rows_cta > N)
        p.rows_cta = N;
    while (p.rows_cta > 1 && static_cast<long long>(B) * ((N + p.rows_cta - 1) / p.rows_cta) < 304)
        --p.rows_cta;
    p.head_cta = p.heads;
    const long long ctas = static_cast<long long>(B) * ((N + p.rows_cta - 1) / p.rows_cta);
    if (ctas < 152) {
        const long long split = (row_items * p.rows_cta + kRotThreads - 1) / kRotThreads;
        const long long parts = split < 152 / ctas ? split : 152 / ctas;
        if (parts > 1)
            p.head_cta = static_cast<int>((p.heads + parts - 1) / parts);
    }
    const long long gx = static_cast<long long>(B) * ((N + p.rows_cta - 1) / p.rows_cta);
    const int gy = (p.heads + p.head_cta - 1) / p.head_cta;
    if (gx >= (1ll << 31))
        return PA_ERR_BAD_DIMS;
    const RotFn fn = o.dtype == PA_F32 ? pick_rotary<float>(mode) : o.dtype == PA_F16 ? pick_rotary<__half>(mode) : pick_rotary<__nv_bfloat16>(mode);
    const size_t smem = static_cast<size_t>(p.rows_cta) * (rot / 2) * sizeof(float2);
    fn<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), kRotThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    if (cudaGetLastError() != cudaSuccess)
        return PA_ERR_CUDA;
    count_launches(1);
    return PA_OK;
}
