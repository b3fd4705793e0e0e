// pa_q8_decode.cu -- attention over a cache in 8 bits, whole or over selected
// blocks (include/pa_q8.h).
//
// Work: segments (sequence, KV head, group of 8 NT query rows), each a run of
// 16-token tiles, laid end to end in units of 8 tiles; every CTA takes an equal
// range of units.  A segment cut between CTAs leaves partial states (maximum,
// sum, values) in the workspace, and the last CTA to finish one joins them.
//
// Tiles: a warp streams its own tiles through a ring of shared memory with
// 8- and 16-byte asynchronous copies.  Each lane copies exactly the bytes that it
// will use as matrix fragments and reads back only its own, so that the ring
// needs no barrier and no bank is hit twice:
//   S^T = K Q^T:   lane (g, t) has rows g and g + 8 of K, D / 4 channels in runs
//                  of 16; the channels' order is the same in Q's fragments;
//   O^T += V^T P^T: lane (g, t) has tokens 2t, 2t + 1, 2t + 8, 2t + 9 of V,
//                  channels D / 8 g ...: two tokens' codes interleaved are V^T's
//                  fragment.
// Codes become fp16 exactly (byte u = code + 128 under the exponent of 1024 is
// 1024 + u; less 1152).  A query row is scaled by a power of two into fp16's
// range, which loses nothing of a 16-bit row; float32 rows are two fp16 parts.
//
// Scales: the key scale multiplies the score.  The value scale joins the
// exponent, t = s + log2(v_scale), so that weights times value scale come out of
// the exponential; the softmax's sum takes them back through 1 / v_scale.  The
// maximum subtracted is t's: fp16 weights are as exact as their share in the
// output.  It is raised only when a score passes it by 2^8 (a vote instead of a
// reduction per tile; weights stay below 2^14).
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kDecodeThreads = kWarps * 32;
constexpr int kTile = 16;                 // tokens of a tile
constexpr int kUnit = kWarps;             // tiles of a unit
constexpr int kMaxEntries = 8192;         // prefix sums in shared memory
constexpr int kMaxCtas = 304;             // two per SM
constexpr int kMeta = 32;                 // bytes of a tile's scales and places
constexpr float kLift = 6.f, kSlack = 8.f;  // weights are 2^(t - m + 6), t - m <= 8

struct DecodeParams {
    const void* q;
    const int8_t* k;
    const int8_t* v;
    const float* ks;
    const float* vs;
    const int32_t* table;
    const int32_t* lens;
    void* out;
    const int32_t* selected;
    const int32_t* counts;
    int* counters;     // [segments] pieces done
    float2* part_ml;   // [CTA][2][8 NT] maximum, sum
    float* part_o;     // [CTA][2][8 NT][D]
    int* status;
    float scale;       // scale * log2(e)
    int B, H, KV, R, NQ, groups, shift, maxb, num_blocks, cap, budget, causal, dtype, entries, stages;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy8(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds8(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
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

__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) { mma_16816<false>(d, a, b0, b1); }

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// log2 and exp2 in float32 of the hardware (2 units in the last place or so).
__device__ __forceinline__ float fast_log2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// QP: fp16 parts of a query row and of a weight (2: float32).
template <int D, int NT, int QP>
__global__ void __launch_bounds__(kDecodeThreads, NT == 1 && QP == 1 ? 2 : 1) pa_q8_decode_kernel(const __grid_constant__ DecodeParams p)
{
    constexpr int kRows = 8 * NT, kSteps = D / 16, kTileBytes = 2 * kTile * D, kStage = kTileBytes + kMeta;
    constexpr int kChunks = D / 64;  // 16-byte runs of a key row per lane
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    __shared__ int sm_last;
    grid_dependents_launch();
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

    // prefix sums of the units of the entries (sequences, or sequences and KV
    // heads where each has its own blocks); `copies` segments share an entry's length
    int* prefix = reinterpret_cast<int*>(smem);
    const uint32_t ring0 = smem_u32(smem) + static_cast<uint32_t>((p.entries + 1) * 4 + 15) / 16 * 16;
    float* merge = reinterpret_cast<float*>(smem + ((p.entries + 1) * 4 + 15) / 16 * 16);
    const int copies = p.selected ? p.groups : p.KV * p.groups;
    {
        int* sums = reinterpret_cast<int*>(&sm_m[0][0]);
        const int per = (p.entries + kDecodeThreads - 1) / kDecodeThreads;
        const int e0 = min(tid * per, p.entries), e1 = min(e0 + per, p.entries);
        int sum = 0;
        for (int e = e0; e < e1; ++e) {
            int tokens;
            if (p.selected) {
                const int c = __ldg(p.counts + e);
                if ((c < 0 || c > p.budget) && blockIdx.x == 0)
                    q8_report(p.status, PA_STATUS_BAD_LENGTH);
                tokens = min(max(c, 0), p.budget) << p.shift;
            } else {
                const int n = __ldg(p.lens + e);
                if ((n < 0 || n > p.cap) && blockIdx.x == 0)
                    q8_report(p.status, PA_STATUS_BAD_LENGTH);
                tokens = min(max(n, 0), p.cap);
            }
            const int u = max(1, (tokens + kTile * kUnit - 1) / (kTile * kUnit));
            prefix[e] = u;
            sum += u;
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFullWarp, incl, o);
            if (lane >= o)
                incl += y;
        }
        if (lane == 31)
            sums[warp] = incl;
        __syncthreads();
        int at = incl - sum;
        for (int w = 0; w < warp; ++w)
            at += sums[w];
        for (int e = e0; e < e1; ++e) {
            const int u = prefix[e];
            prefix[e] = at;
            at += u;
        }
        if (tid == kDecodeThreads - 1)
            prefix[p.entries] = at;
        __syncthreads();
    }
    const int64_t U = static_cast<int64_t>(prefix[p.entries]) * copies;
    const int G = static_cast<int>(min(static_cast<int64_t>(gridDim.x), U));
    if (static_cast<int>(blockIdx.x) >= G)
        return;
    const int64_t u_end = (static_cast<int64_t>(blockIdx.x) + 1) * U / G;
    const int64_t u_begin = static_cast<int64_t>(blockIdx.x) * U / G;
    const uint32_t ring = ring0 + static_cast<uint32_t>(warp * p.stages * kStage);

    for (int64_t u = u_begin; u < u_end;) {
        // the segment of unit u: entry e, copy c of it
        int e = 0;
        {
            int hi = p.entries;
            while (hi - e > 1) {
                const int mid = (e + hi) >> 1;
                if (static_cast<int64_t>(prefix[mid]) * copies <= u)
                    e = mid;
                else
                    hi = mid;
            }
        }
        const int units = prefix[e + 1] - prefix[e];
        const int c = static_cast<int>((u - static_cast<int64_t>(prefix[e]) * copies) / units);
        const int64_t s_begin = static_cast<int64_t>(prefix[e]) * copies + static_cast<int64_t>(c) * units, s_end = s_begin + units;
        const int64_t stop = min(s_end, u_end);
        const int b = p.selected ? e / p.KV : e;
        const int kh = p.selected ? e % p.KV : c / p.groups;
        const int grp = p.selected ? c : c % p.groups;
        const int64_t segment = (static_cast<int64_t>(b) * p.KV + kh) * p.groups + grp;
        const int n = min(max(__ldg(p.lens + b), 0), p.cap);
        const int32_t* sel = p.selected ? p.selected + static_cast<int64_t>(e) * p.budget : nullptr;
        const int nsel = p.selected ? min(max(__ldg(p.counts + e), 0), p.budget) : 0;
        const int tokens = p.selected ? nsel << p.shift : n;  // places in the list of blocks
        const int nb = (n + (1 << p.shift) - 1) >> p.shift;
        const int32_t* table = p.table + static_cast<int64_t>(b) * p.maxb;
        // this warp's tiles: first, first + 8, ... below last
        const int first = static_cast<int>(u - s_begin) * kUnit + warp;
        const int last = min(static_cast<int>(stop - s_begin) * kUnit, (tokens + kTile - 1) / kTile);
        const int row_base = grp * kRows;

        // ---- query rows: fragments of B, scaled by a power of two
        uint32_t qf[QP][NT][kSteps][2];
        float rowf[NT][2];   // of this lane's two score columns: scale * log2(e) / the power of two
        int lim[NT][2];      // keys that the column's row sees
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = row_base + nt * 8 + g;
            float x[kSteps * 4];
            float a = 0.f;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                float y[16];
                if (row < p.R) {
                    const int64_t at = (static_cast<int64_t>(b) * p.KV + kh) * p.R * D + static_cast<int64_t>(row) * D + ch * 64 + t * 16;
                    if (p.dtype == PA_F32)
                        q8_load16(y, static_cast<const float*>(p.q) + at);
                    else if (p.dtype == PA_F16)
                        q8_load16(y, static_cast<const __half*>(p.q) + at);
                    else
                        q8_load16(y, static_cast<const __nv_bfloat16*>(p.q) + at);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        y[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[ch * 16 + i] = y[i];
                    a = q8_amax(a, y[i]);
                }
            }
            a = fmaxf(a, __shfl_xor_sync(kFullWarp, a, 1));
            a = fmaxf(a, __shfl_xor_sync(kFullWarp, a, 2));
            // 2^up brings the largest magnitude into [2^11, 2^12)
            const int ex = max(static_cast<int>(__float_as_uint(a) >> 23) - 127, -100), up = 11 - ex;
            const float f1 = __uint_as_float(static_cast<uint32_t>(127 + up / 2) << 23);
            const float f2 = __uint_as_float(static_cast<uint32_t>(127 + up - up / 2) << 23);
            const float d1 = __uint_as_float(static_cast<uint32_t>(127 - up / 2) << 23);
            const float d2 = __uint_as_float(static_cast<uint32_t>(127 - (up - up / 2)) << 23);
            const float factor = p.scale * d1 * d2;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                float z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    z[i] = x[4 * s + i] * f1 * f2;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half2 hi = __floats2half2_rn(z[2 * i], z[2 * i + 1]);
                    qf[0][nt][s][i] = half2_bits(hi);
                    if constexpr (QP == 2) {
                        const float2 back = __half22float2(hi);
                        qf[1][nt][s][i] = half2_bits(__floats2half2_rn(z[2 * i] - back.x, z[2 * i + 1] - back.y));
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                rowf[nt][i] = __shfl_sync(kFullWarp, factor, (2 * t + i) * 4);
                const int r = row_base + nt * 8 + 2 * t + i;
                lim[nt][i] = r >= p.R ? 0 : p.causal ? min(n, n - p.NQ + r % p.NQ + 1) : n;
            }
        }
        const int all_see = p.causal ? n - p.NQ + 1 : n;  // every row sees the keys below

        float o[kSteps][NT][4];
        float mx[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[nt][i] = -INFINITY;
                l[nt][i] = 0.f;
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[s][nt][i] = 0.f;
        }

        // ---- copies: block numbers are looked up one tile ahead, selected ones two
        int blk[2], blk_next[2], phys[2];
        auto look_selected = [&](int tile) {  // logical blocks of a tile's halves (-1: none)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int place = tile * kTile + 8 * x;
                int j = -1;
                if (tile < last && place < tokens) {
                    j = place >> p.shift;
                    if (sel)
                        j = __ldg(sel + j);
                }
                blk_next[x] = j;
            }
        };
        auto look_table = [&]() {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                blk[x] = blk_next[x];
                if (sel && (blk[x] < 0 || blk[x] >= nb)) {
                    if (blk[x] != -1)
                        q8_report(p.status, PA_STATUS_BAD_BLOCK);
                    blk[x] = -1;
                }
                phys[x] = blk[x] >= 0 ? __ldg(table + blk[x]) : -1;
            }
        };
        auto issue = [&](int tile, int stage) {
            if (tile < last) {
                const uint32_t st = ring + static_cast<uint32_t>(stage * kStage);
                const int in_block = (tile * kTile) & ((1 << p.shift) - 1);
                int64_t at[2];
                int place[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (phys[x] >= p.num_blocks || (blk[x] >= 0 && phys[x] < 0)) {
                        q8_report(p.status, PA_STATUS_BAD_BLOCK);
                        phys[x] = -1;
                    }
                    const int r = p.shift == 3 ? 0 : in_block + 8 * x;
                    place[x] = phys[x] >= 0 ? (blk[x] << p.shift) + r : INT_MAX - 64;
                    const int ph = max(phys[x], 0);
                    at[x] = (((static_cast<int64_t>(ph) << p.shift) + r) * p.KV + kh) * D;
                    if (lane < 2 && phys[x] >= 0) {
                        const float* src = (lane ? p.vs : p.ks) + static_cast<int64_t>(ph) * p.KV + kh;
                        copy4(st + kTileBytes + x * 8 + lane * 4, src);
                    }
                }
                if (lane == 2) {
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(st + kTileBytes + 16), "r"(place[0]), "r"(place[1]) : "memory");
                }
                const int64_t step = static_cast<int64_t>(p.KV) * D;
                // (a half without a block repeats row 0 of the pool: in bounds, weighed with zero)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int ch = 0; ch < kChunks; ++ch)
                        copy16(st + ((x * kChunks + ch) * 32 + lane) * 16, p.k + at[x] + g * step + ch * 64 + t * 16);
                const uint32_t sv = st + kTile * D;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int8_t* src = p.v + at[x] + (2 * t + i) * step + g * (D / 8);
                        if constexpr (D == 128)
                            copy16(sv + ((x * 2 + i) * 32 + lane) * 16, src);
                        else
                            copy8(sv + ((x * 2 + i) * 32 + lane) * 8, src);
                    }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        const int S = p.stages;
        look_selected(first);
        look_table();
        look_selected(first + kUnit);
        for (int i = 0; i < S - 1; ++i) {
            issue(first + i * kUnit, i);
            look_table();
            look_selected(first + (i + 2) * kUnit);
        }
        int stage = 0, fill = S - 1;
        for (int tile = first; tile < last; tile += kUnit) {
            // the oldest group is this tile's (S is 3, 4, 6 or 8)
            if (S == 3)
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            else if (S == 4)
                asm volatile("cp.async.wait_group 2;" ::: "memory");
            else if (S == 6)
                asm volatile("cp.async.wait_group 4;" ::: "memory");
            else
                asm volatile("cp.async.wait_group 6;" ::: "memory");
            __syncwarp();  // scales and places come from other lanes; the stage filled next has been read
            {
                const int ahead = tile + (S - 1) * kUnit;
                issue(ahead, fill);
                look_table();
                look_selected(ahead + 2 * kUnit);
            }
            const uint32_t st = ring + static_cast<uint32_t>(stage * kStage);
            const uint4 sc = lds16(st + kTileBytes);
            const uint2 pl = lds8(st + kTileBytes + 16);
            const int place[2] = {static_cast<int>(pl.x), static_cast<int>(pl.y)};
            const float ks[2] = {__uint_as_float(sc.x), __uint_as_float(sc.z)};
            float lv[2], iv[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float vs = fmaxf(__uint_as_float(x ? sc.w : sc.y), kMinScale);
                lv[x] = fast_log2(vs);
                iv[x] = __frcp_rn(vs);
            }
            // ---- S^T = K Q^T
            float sacc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sacc[nt][i] = 0.f;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                const uint4 ka = lds16(st + (ch * 32 + lane) * 16), kb = lds16(st + ((kChunks + ch) * 32 + lane) * 16);
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t ua = wa[i] ^ 0x80808080u, ub = wb[i] ^ 0x80808080u;
                    const uint32_t a[4] = {codes2(ua, 0x4140), codes2(ub, 0x4140), codes2(ua, 0x4342), codes2(ub, 0x4342)};
#pragma unroll
                    for (int q = 0; q < QP; ++q)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma(sacc[nt], a, qf[q][nt][ch * 4 + i][0], qf[q][nt][ch * 4 + i][1]);
                }
            }
            // ---- scores in base 2 plus log2 of the value scale; hidden ones -inf
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sacc[nt][i] = fmaf(sacc[nt][i], rowf[nt][i & 1] * ks[i >> 1], lv[i >> 1]);
            if (max(place[0], place[1]) + 8 > all_see || row_base + kRows > p.R) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (place[i >> 1] + g >= lim[nt][i & 1])
                            sacc[nt][i] = -INFINITY;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    raise |= sacc[nt][i] > mx[nt][i & 1] + kSlack;
            if (__any_sync(kFullWarp, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float m = fmaxf(sacc[nt][i], sacc[nt][i + 2]);
                        m = fmaxf(m, __shfl_xor_sync(kFullWarp, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(kFullWarp, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(kFullWarp, m, 16));
                        m = fmaxf(m, mx[nt][i]);
                        const float down = m == -INFINITY ? 1.f : fast_exp2(mx[nt][i] - m);
                        mx[nt][i] = m;
                        l[nt][i] *= down;
#pragma unroll
                        for (int s = 0; s < kSteps; ++s) {
                            o[s][nt][i] *= down;
                            o[s][nt][i + 2] *= down;
                        }
                    }
            }
            // ---- weights, and as fragments of P^T
            uint32_t pf[QP][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float base = mx[nt][i & 1] == -INFINITY ? 0.f : mx[nt][i & 1] - kLift;
                    w[i] = fast_exp2(sacc[nt][i] - base);
                    l[nt][i & 1] = sacc[nt][i] == -INFINITY ? l[nt][i & 1] : fmaf(w[i], iv[i >> 1], l[nt][i & 1]);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const __half2 hi = __floats2half2_rn(w[2 * x], w[2 * x + 1]);
                    pf[0][nt][x] = movm_trans(half2_bits(hi));
                    if constexpr (QP == 2) {
                        const float2 back = __half22float2(hi);
                        pf[1][nt][x] = movm_trans(half2_bits(__floats2half2_rn(w[2 * x] - back.x, w[2 * x + 1] - back.y)));
                    }
                }
            }
            // ---- O^T += V^T P^T
            const uint32_t sv = st + kTile * D;
            uint32_t vw[4][D / 32];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == 128) {
                    const uint4 v = lds16(sv + (i * 32 + lane) * 16);
                    vw[i][0] = v.x, vw[i][1] = v.y, vw[i][2] = v.z, vw[i][3] = v.w;
                } else {
                    const uint2 v = lds8(sv + (i * 32 + lane) * 8);
                    vw[i][0] = v.x, vw[i][1] = v.y;
                }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                uint32_t mixed[2][2];  // [half of the tokens][channels 0 1 | 2 3]
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mixed[x][0] = __byte_perm(vw[2 * x][w], vw[2 * x + 1][w], 0x5140) ^ 0x80808080u;
                    mixed[x][1] = __byte_perm(vw[2 * x][w], vw[2 * x + 1][w], 0x7362) ^ 0x80808080u;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t a[4] = {codes2(mixed[0][i], 0x4140), codes2(mixed[0][i], 0x4342), codes2(mixed[1][i], 0x4140),
                                           codes2(mixed[1][i], 0x4342)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (QP == 1) {
                            mma(o[2 * w + i][nt], a, pf[0][nt][0], pf[0][nt][1]);
                        } else {
                            // a tile's products by themselves: added to the sums by rounded
                            // additions (the tensor core's own cut off what does not fit)
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            mma(d, a, pf[QP - 1][nt][0], pf[QP - 1][nt][1]);
                            mma(d, a, pf[0][nt][0], pf[0][nt][1]);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                o[2 * w + i][nt][j] += d[j];
                        }
                    }
                }
            }
            stage = stage + 1 == S ? 0 : stage + 1;
            fill = fill + 1 == S ? 0 : fill + 1;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the rings are free

        // ---- the warps' states together
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float s = l[nt][i];
                s += __shfl_xor_sync(kFullWarp, s, 4);
                s += __shfl_xor_sync(kFullWarp, s, 8);
                s += __shfl_xor_sync(kFullWarp, s, 16);
                if (g == 0) {
                    sm_m[warp][nt * 8 + 2 * t + i] = mx[nt][i];
                    sm_l[warp][nt * 8 + 2 * t + i] = s;
                }
#pragma unroll
                for (int s2 = 0; s2 < kSteps; ++s2) {
                    // step s2 = 2 w + x: channels D / 8 g + 4 w + 2 x, + 1
                    float2 two = make_float2(o[s2][nt][i], o[s2][nt][i + 2]);
                    *reinterpret_cast<float2*>(merge + (static_cast<size_t>(warp) * kRows + nt * 8 + 2 * t + i) * D + g * (D / 8) + 2 * s2) = two;
                }
            }
        __syncthreads();
        const bool whole = u == s_begin && stop == s_end;
        const int slot = u == u_begin && u != s_begin ? 0 : 1;  // a piece of a segment begun earlier, or one that goes on
        const int64_t record = static_cast<int64_t>(blockIdx.x) * 2 + slot;
        for (int x = tid; x < kRows * D; x += kDecodeThreads) {
            const int row = x / D, d = x % D;
            if (row_base + row >= p.R)
                break;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                m = fmaxf(m, sm_m[w][row]);
            float sum = 0.f, val = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = sm_m[w][row] == -INFINITY ? 0.f : fast_exp2(sm_m[w][row] - m);
                sum = fmaf(sm_l[w][row], f, sum);
                val = fmaf(merge[(static_cast<size_t>(w) * kRows + row) * D + d], f, val);
            }
            if (whole) {
                const float y = sum == 0.f ? 0.f : val / sum;
                const int64_t at = ((static_cast<int64_t>(b) * p.KV + kh) * p.R + row_base + row) * D + d;
                if (p.dtype == PA_F32)
                    static_cast<float*>(p.out)[at] = y;
                else if (p.dtype == PA_F16)
                    static_cast<__half*>(p.out)[at] = __float2half_rn(y);
                else
                    static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
            } else {
                p.part_o[(record * kRows + row) * D + d] = val;
                if (d == 0)
                    p.part_ml[record * kRows + row] = make_float2(m, sum);
            }
        }
        if (!whole) {
            // pieces of the segment: CTAs c0 .. c1
            const int c0 = static_cast<int>(((s_begin + 1) * G - 1) / U), c1 = static_cast<int>((s_end * G - 1) / U);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int before = atomicAdd(p.counters + segment, 1);
                sm_last = before == c1 - c0;
                if (before == c1 - c0)
                    p.counters[segment] = 0;
            }
            __syncthreads();
            if (sm_last) {
                __threadfence();
                for (int x = tid; x < kRows * D; x += kDecodeThreads) {
                    const int row = x / D, d = x % D;
                    if (row_base + row >= p.R)
                        break;
                    float m = -INFINITY, sum = 0.f, val = 0.f;
                    for (int i = c0; i <= c1; ++i) {
                        // the first CTA's range may begin with this segment or earlier
                        const int64_t begin = static_cast<int64_t>(i) * U / G;
                        const int64_t rec = static_cast<int64_t>(i) * 2 + (begin > s_begin ? 0 : 1);
                        const float2 ml = __ldcg(p.part_ml + rec * kRows + row);
                        const float v = __ldcg(p.part_o + (rec * kRows + row) * D + d);
                        const float now = fmaxf(m, ml.x);
                        const float fa = m == -INFINITY ? 0.f : fast_exp2(m - now), fb = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - now);
                        sum = sum * fa + ml.y * fb;
                        val = val * fa + v * fb;
                        m = now;
                    }
                    const float y = sum == 0.f ? 0.f : val / sum;
                    const int64_t at = ((static_cast<int64_t>(b) * p.KV + kh) * p.R + row_base + row) * D + d;
                    if (p.dtype == PA_F32)
                        static_cast<float*>(p.out)[at] = y;
                    else if (p.dtype == PA_F16)
                        static_cast<__half*>(p.out)[at] = __float2half_rn(y);
                    else
                        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
                }
            }
        }
        __syncthreads();  // the next segment's copies overwrite the merged states
        u = stop;
    }
}

struct Variant {
    const void* fn;
    int rows, ctas, stages;
    size_t tile;
};

template <int D>
Variant variant(int dtype, int R)
{
    Variant v;
    v.tile = static_cast<size_t>(2) * kTile * D + kMeta;
    if (dtype == PA_F32) {
        v.rows = R > 8 ? 16 : 8;
        v.fn = R > 8 ? reinterpret_cast<const void*>(pa_q8_decode_kernel<D, 2, 2>) : reinterpret_cast<const void*>(pa_q8_decode_kernel<D, 1, 2>);
    } else {
        v.rows = R > 16 ? 32 : R > 8 ? 16 : 8;
        v.fn = R > 16  ? reinterpret_cast<const void*>(pa_q8_decode_kernel<D, 4, 1>)
               : R > 8 ? reinterpret_cast<const void*>(pa_q8_decode_kernel<D, 2, 1>)
                       : reinterpret_cast<const void*>(pa_q8_decode_kernel<D, 1, 1>);
    }
    v.ctas = dtype != PA_F32 && R <= 8 ? 2 : 1;
    return v;
}

Variant variant_of(int D, int dtype, int R) { return D == 64 ? variant<64>(dtype, R) : variant<128>(dtype, R); }

// Sizes that pa_q8_decode refuses, apart from those of the cache.
int decode_sizes(int B, int H, int KV, int NQ)
{
    if (H < 1 || KV < 1 || H % KV != 0 || NQ < 1)
        return PA_ERR_BAD_DIMS;
    if (NQ > PA_MAX_NQ || static_cast<long long>(H / KV) * NQ > 1024 || B > kMaxBatch || KV > 1024)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

struct Workspace {
    size_t zero, ml, o, total;
};

Workspace workspace_of(int B, int H, int KV, int D, int NQ)
{
    const size_t R = static_cast<size_t>(H / KV) * NQ;
    const size_t groups = (R + 7) / 8;  // at most: passes of 8 rows
    Workspace w;
    w.zero = (static_cast<size_t>(B) * KV * groups * 4 + 255) / 256 * 256;
    w.ml = static_cast<size_t>(kMaxCtas) * 2 * 32 * 8;
    w.o = static_cast<size_t>(kMaxCtas) * 2 * 32 * D * 4;
    w.total = w.zero + w.ml + w.o;
    return w;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_q8_workspace_bytes(int B, int H, int KV, int D, int NQ)
{
    if (B < 1 || decode_sizes(B, H, KV, NQ) != PA_OK || (D != 64 && D != 128))
        return 0;
    return workspace_of(B, H, KV, D, NQ).total;
}

extern "C" size_t pa_q8_workspace_zero_bytes(int B, int H, int KV, int D, int NQ)
{
    if (B < 1 || decode_sizes(B, H, KV, NQ) != PA_OK || (D != 64 && D != 128))
        return 0;
    return workspace_of(B, H, KV, D, NQ).zero;
}

extern "C" int pa_q8_decode(const void* q, const int8_t* k_cache, const int8_t* v_cache, const float* k_scale, const float* v_scale,
                            const int32_t* block_table, const int32_t* seq_lens, void* out, float scale, int B, int H, int KV,
                            int D, int NQ, int BLOCK, const pa_q8_opts* opts, void* stream)
{
    if (!opts)
        return PA_ERR_NULL_POINTER;
    const pa_q8_opts& o = *opts;
    int rc = q8_sizes(B, KV, D, BLOCK, o.max_blocks, o.num_blocks, o.dtype);
    if (rc == PA_OK)
        rc = decode_sizes(B, H, KV, NQ);
    if (rc != PA_OK)
        return rc;
    if ((o.selected != nullptr) != (o.counts != nullptr))
        return PA_ERR_NULL_POINTER;
    if (o.selected && (o.budget < 1 || static_cast<long long>(o.budget) * BLOCK >= (1ll << 30)))
        return PA_ERR_BAD_DIMS;
    if (o.selected && static_cast<long long>(B) * KV > kMaxEntries)
        return PA_ERR_UNSUPPORTED;
    if (B == 0)
        return PA_OK;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out)
        return PA_ERR_NULL_POINTER;
    if (!q8_a16(q) || !q8_a16(out) || !q8_a16(k_cache) || !q8_a16(v_cache) || !q8_a4(k_scale) || !q8_a4(v_scale) ||
        !q8_a4(block_table) || !q8_a4(seq_lens) || !q8_a4(o.selected) || !q8_a4(o.counts) || !q8_a4(o.status))
        return PA_ERR_ALIGNMENT;
    const int R = H / KV * NQ;
    const Workspace ws = workspace_of(B, H, KV, D, NQ);
    if (!o.workspace || o.workspace_bytes < ws.total || (reinterpret_cast<uintptr_t>(o.workspace) & 255))
        return PA_ERR_WORKSPACE;
    const size_t blocks = static_cast<size_t>(o.num_blocks) * KV, pool = blocks * BLOCK * D, b4 = static_cast<size_t>(B) * 4;
    const size_t rows = static_cast<size_t>(B) * H * NQ * D * (o.dtype == PA_F32 ? 4 : 2);
    const Q8Range r[] = {{out, rows, true},
                         {o.workspace, ws.total, true},
                         {o.status, 4, true},
                         {q, rows, false},
                         {k_cache, pool, false},
                         {v_cache, pool, false},
                         {k_scale, blocks * 4, false},
                         {v_scale, blocks * 4, false},
                         {block_table, b4 * o.max_blocks, false},
                         {seq_lens, b4, false},
                         {o.selected, b4 * KV * o.budget, false},
                         {o.counts, b4 * KV, false}};
    if (q8_overlap(r, 12))
        return PA_ERR_BAD_DIMS;
    const Variant v = variant_of(D, o.dtype, R);
    DecodeParams p{};
    p.groups = (R + v.rows - 1) / v.rows;
    p.entries = o.selected ? B * KV : B;
    const long long copies = o.selected ? p.groups : static_cast<long long>(KV) * p.groups;
    const long long most = o.selected ? static_cast<long long>(o.budget) * BLOCK : static_cast<long long>(o.max_blocks) * BLOCK;
    if (p.entries * ((most + kTile * kUnit - 1) / (kTile * kUnit)) * copies >= (1ll << 50) ||
        p.entries * ((most + kTile * kUnit - 1) / (kTile * kUnit)) >= (1ll << 31))
        return PA_ERR_BAD_DIMS;
    p.q = q;
    p.k = k_cache;
    p.v = v_cache;
    p.ks = k_scale;
    p.vs = v_scale;
    p.table = block_table;
    p.lens = seq_lens;
    p.out = out;
    p.selected = o.selected;
    p.counts = o.counts;
    unsigned char* w = static_cast<unsigned char*>(o.workspace);
    p.counters = reinterpret_cast<int*>(w);
    p.part_ml = reinterpret_cast<float2*>(w + ws.zero);
    p.part_o = reinterpret_cast<float*>(w + ws.zero + ws.ml);
    p.status = o.status;
    p.scale = scale * kLog2e;
    p.B = B;
    p.H = H;
    p.KV = KV;
    p.R = R;
    p.NQ = NQ;
    p.shift = BLOCK == 8 ? 3 : BLOCK == 16 ? 4 : BLOCK == 32 ? 5 : 6;
    p.maxb = o.max_blocks;
    p.num_blocks = o.num_blocks;
    p.cap = o.max_blocks * BLOCK;
    p.budget = o.budget;
    p.causal = o.causal ? 1 : 0;
    p.dtype = o.dtype;
    // ring depth: what fits beside the prefix sums, and the states merged in the same memory
    const size_t head = ((static_cast<size_t>(p.entries) + 1) * 4 + 15) / 16 * 16;
    const size_t room = static_cast<size_t>(v.ctas == 2 ? 108 : 220) * 1024 - head;
    const int fit = static_cast<int>(room / (kWarps * v.tile));
    p.stages = fit >= 8 ? 8 : fit >= 6 ? 6 : fit >= 4 ? 4 : 3;
    size_t body = kWarps * v.tile * p.stages;
    const size_t merge = static_cast<size_t>(kWarps) * v.rows * D * 4;
    if (body < merge)
        body = merge;
    int sms = 0, dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PA_ERR_CUDA;
    int grid = sms * v.ctas;
    grid = grid > kMaxCtas ? kMaxCtas : grid;
    void* args[] = {&p};
    return q8_launch(v.fn, dim3(grid), kDecodeThreads, head + body, static_cast<cudaStream_t>(stream), args);
}
