// pa_q8_select.cu -- blocks of a cache in 8 bits that a step's queries look at
// most (include/pa_q8.h).
//
// One kernel, a CTA or a cluster of them per sequence and KV head.  The query
// rows become whole numbers in shared memory, positive and negative parts apart,
// so that sum_d max(c min, c max) = c+ . max + c- . min is a product of whole
// numbers (dp4a): exact, in any order.  Four lanes share a block, a quarter of
// the channels each; four rows are summed over those lanes together.  Table
// entries are read before the length is known, and the next blocks' bounds
// while this step's are used.
//
// The scores go to the first CTA of the cluster, which finds the score of the
// last block taken by counting them in 256 bins over their range, then over the
// bin that it falls into, until that bin is taken whole: mostly two rounds.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kSelectRows = 128;        // query rows in shared memory at once
constexpr int kSelectBlocks = 32768;    // blocks of a table row at most
constexpr int kBins = 256;

struct SelectParams {
    const void* q;
    const int8_t* bounds;
    const float* k_scale;
    const int32_t* table;
    const int32_t* lens;
    int32_t* selected;
    int32_t* counts;
    int* status;
    int KV, R, maxb, num_blocks, budget, first, last, shift, cap, dtype;
};

// Unsigned integers in the order of the scores: NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t score_order(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float q8_element(const void* q, int dtype, int64_t i)
{
    if (dtype == PA_F32)
        return static_cast<const float*>(q)[i];
    if (dtype == PA_F16)
        return __half2float(static_cast<const __half*>(q)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(q)[i]);
}

// grid (C, B * KV), clusters of C along x; T threads.
template <int D, int C, int T>
__global__ void __launch_bounds__(T, 768 / T) pa_q8_select_kernel(const __grid_constant__ SelectParams p)
{
    constexpr int kWarps = T / 32, kStep = kWarps * C * 8;  // blocks that the cluster takes together
    constexpr int kWords = D / 16;                 // words of a lane's quarter of a row
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t* keys = smem;                         // [maxb] scores in order (the first CTA's)
    const int most = (p.maxb + kStep - 1) / kStep * kWarps * 8;  // blocks of a CTA
    float* own = reinterpret_cast<float*>(smem + ((p.maxb + 3) & ~3));  // [most] this CTA's scores
    uint32_t* codes = smem + ((p.maxb + 3) & ~3) + most;  // [rows][4 quarters][positive words | negative words]
    constexpr int kQuarter = D / 8 + 4, kRow = 4 * kQuarter;  // words; the four quarters in banks of their own
    __shared__ float steps[kSelectRows];
    __shared__ __align__(16) uint32_t hist[2][kBins];
    __shared__ uint32_t wide[kWarps][2];
    __shared__ int cnt[kWarps][2];
    grid_dependents_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int seg = blockIdx.y, b = seg / p.KV, h = seg - b * p.KV;
    const int rank = C == 1 ? 0 : static_cast<int>(blockIdx.x);
    if (C > 1)  // the first CTA's shared memory may be written once it runs
        asm volatile("barrier.cluster.arrive;" ::: "memory");
    grid_dependency_wait();
    int n = __ldg(p.lens + b);
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.maxb;
    // the cluster's warps take eight blocks each in turn
    const int j0 = (warp * C + rank) * 8 + g;
    int phys = j0 < p.maxb ? __ldg(table + j0) : -1;
    int phys1 = j0 + kStep < p.maxb ? __ldg(table + j0 + kStep) : -1;
    const int64_t q0 = static_cast<int64_t>(seg) * p.R * D;
    if (n < 0 || n > p.cap) {
        if (h == 0 && rank == 0 && tid == 0)
            q8_report(p.status, PA_STATUS_BAD_LENGTH);
        n = n < 0 ? 0 : p.cap;
    }
    const int nb = (n + (1 << p.shift) - 1) >> p.shift;
    const int m = min(nb, p.budget);
    int32_t* sel = p.selected + static_cast<int64_t>(seg) * p.budget;
    const int lo = p.first, hi = nb - p.last;
    const int need = p.budget - p.first - p.last;
    if (rank == 0) {
        for (int i = m + tid; i < p.budget; i += T)
            sel[i] = -1;
        if (tid == 0)
            p.counts[seg] = m;
        if (nb <= p.budget) {
            for (int i = tid; i < nb; i += T)
                sel[i] = i;
        } else {
            for (int i = tid; i < p.first; i += T)
                sel[i] = i;
            for (int i = tid; i < p.last; i += T)
                sel[p.first + need + i] = hi + i;
        }
    }
    if (nb <= p.budget || need == 0) {  // the same in every CTA of the cluster
        if (C > 1)
            asm volatile("barrier.cluster.wait;" ::: "memory");
        return;
    }

    // scores
    struct Bounds {
        uint32_t mn[kWords], mx[kWords];
        float ks;
        bool there;
    };
    auto fetch = [&](Bounds& x, int j, int ph) {
        x.there = j < nb && static_cast<uint32_t>(ph) < static_cast<uint32_t>(p.num_blocks);
        if (!x.there && j < nb)
            q8_report(p.status, PA_STATUS_BAD_BLOCK);
        const int64_t at = static_cast<int64_t>(x.there ? ph : 0) * p.KV + h;
        const uint4* src = reinterpret_cast<const uint4*>(p.bounds + at * 2 * D + t * (D / 4));
        if (x.there) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = __ldg(src + i), w = __ldg(src + i + D / 16);
                x.mn[4 * i] = v.x, x.mn[4 * i + 1] = v.y, x.mn[4 * i + 2] = v.z, x.mn[4 * i + 3] = v.w;
                x.mx[4 * i] = w.x, x.mx[4 * i + 1] = w.y, x.mx[4 * i + 2] = w.z, x.mx[4 * i + 3] = w.w;
            }
            x.ks = __ldg(p.k_scale + at);
        }
    };
    for (int r0 = 0; r0 < p.R; r0 += kSelectRows) {
        const int rows = min(kSelectRows, p.R - r0), rows4 = (rows + 3) & ~3;
        // two steps of blocks are on their way, the entries of the third
        Bounds x, next;
        if (r0 > 0) {
            phys = j0 < nb ? __ldg(table + j0) : -1;
            phys1 = j0 + kStep < nb ? __ldg(table + j0 + kStep) : -1;
            __syncthreads();
        }
        fetch(x, j0, phys);
        fetch(next, j0 + kStep, phys1);
        int phys2 = j0 + 2 * kStep < nb ? __ldg(table + j0 + 2 * kStep) : -1;
        for (int r = warp; r < rows4; r += kWarps) {
            float v[D / 32];
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                v[i] = r < rows ? q8_element(p.q, p.dtype, q0 + static_cast<int64_t>(r0 + r) * D + lane * (D / 32) + i) : 0.f;
                a = q8_amax(a, v[i]);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
                a = fmaxf(a, __shfl_xor_sync(kFullWarp, a, o));
            const float scale = q8_scale_of(a), inv = 1.f / scale;
            if (lane == 0)
                steps[r] = scale;
            int8_t* row = reinterpret_cast<int8_t*>(codes + r * kRow);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int d = lane * (D / 32) + i, c = q8_code(v[i], scale, inv);
                int8_t* at = row + (d / (D / 4)) * (kQuarter * 4) + d % (D / 4);
                at[0] = static_cast<int8_t>(max(c, 0));
                at[D / 4] = static_cast<int8_t>(min(c, 0));
            }
        }
        __syncthreads();
        int slot = warp * 8 + g;
        for (int base = j0 - g; base < nb; base += kStep, slot += kWarps * 8) {
            const int j = base + g;
            float best = -INFINITY;
            bool any = false;
            for (int r = 0; r < rows; r += 4) {
                int sum[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4* c = reinterpret_cast<const uint4*>(codes + (r + k) * kRow + t * kQuarter);
                    int s = 0;
#pragma unroll
                    for (int i = 0; i < kWords / 4; ++i) {
                        const uint4 up = c[i], dn = c[i + D / 64];
                        s = __dp4a(static_cast<int>(up.x), static_cast<int>(x.mx[4 * i]), s);
                        s = __dp4a(static_cast<int>(up.y), static_cast<int>(x.mx[4 * i + 1]), s);
                        s = __dp4a(static_cast<int>(up.z), static_cast<int>(x.mx[4 * i + 2]), s);
                        s = __dp4a(static_cast<int>(up.w), static_cast<int>(x.mx[4 * i + 3]), s);
                        s = __dp4a(static_cast<int>(dn.x), static_cast<int>(x.mn[4 * i]), s);
                        s = __dp4a(static_cast<int>(dn.y), static_cast<int>(x.mn[4 * i + 1]), s);
                        s = __dp4a(static_cast<int>(dn.z), static_cast<int>(x.mn[4 * i + 2]), s);
                        s = __dp4a(static_cast<int>(dn.w), static_cast<int>(x.mn[4 * i + 3]), s);
                    }
                    sum[k] = s;
                }
                // lane t of the four ends with the total of row r + t
                const int o0 = __shfl_xor_sync(kFullWarp, t & 1 ? sum[0] : sum[1], 1);
                const int o1 = __shfl_xor_sync(kFullWarp, t & 1 ? sum[2] : sum[3], 1);
                const int a0 = (t & 1 ? sum[1] : sum[0]) + o0, a1 = (t & 1 ? sum[3] : sum[2]) + o1;
                const int o2 = __shfl_xor_sync(kFullWarp, t & 2 ? a0 : a1, 2);
                const int total = (t & 2 ? a1 : a0) + o2;
                if (r + t < rows) {
                    const float score = __fmul_rn(__fmul_rn(steps[r + t], x.ks), static_cast<float>(total));
                    any |= score == score;
                    best = fmaxf(best, score);  // (a NaN leaves the other)
                }
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                best = fmaxf(best, __shfl_xor_sync(kFullWarp, best, o));
                any |= __shfl_xor_sync(kFullWarp, static_cast<int>(any), o) != 0;
            }
            if (j < nb && t == 0) {
                float s = x.there && any ? best : __int_as_float(0x7fc00000);
                if (r0 > 0) {
                    const float before = own[slot];
                    s = before != before ? s : s != s ? before : fmaxf(s, before);
                }
                own[slot] = s;
            }
            x = next;
            if (base + kStep < nb) {
                fetch(next, j + 2 * kStep, phys2);
                phys2 = j + 3 * kStep < nb ? __ldg(table + j + 3 * kStep) : -1;
            }
        }
    }
    // to the first CTA; a warp moves its own
    __syncwarp();
    uint32_t to = smem_u32(keys);
    if (C > 1) {
        asm volatile("barrier.cluster.wait;" ::: "memory");
        asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_u32(keys)));
    }
    for (int base = (warp * C + rank) * 8 + lane % 8 + lane / 8 * kStep, slot = warp * 8 + lane % 8 + lane / 8 * kWarps * 8; base < nb;
         base += 4 * kStep, slot += 4 * kWarps * 8)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + static_cast<uint32_t>(base) * 4), "r"(score_order(own[slot])) : "memory");
    if (C > 1) {
        asm volatile("barrier.cluster.arrive;" ::: "memory");
        if (rank != 0)
            return;  // (the first CTA alone waits: only its shared memory was written)
        asm volatile("barrier.cluster.wait;" ::: "memory");
    } else {
        __syncthreads();
    }

    // the range of the candidates' scores
    uint32_t least = 0xffffffffu, largest = 0;
    for (int i = tid; i < 2 * kBins; i += T)
        hist[0][i] = 0;
    for (int j = lo + tid; j < hi; j += T) {
        least = min(least, keys[j]);
        largest = max(largest, keys[j]);
    }
    least = __reduce_min_sync(kFullWarp, least);
    largest = __reduce_max_sync(kFullWarp, largest);
    if (lane == 0) {
        wide[warp][0] = least;
        wide[warp][1] = largest;
    }
    __syncthreads();
    least = __reduce_min_sync(kFullWarp, lane < kWarps ? wide[lane][0] : 0xffffffffu);
    largest = __reduce_max_sync(kFullWarp, lane < kWarps ? wide[lane][1] : 0u);
    // taken: scores >= t_ge, and of those equal to t_eq the first n_eq
    uint32_t t_ge = 0, t_eq = 0, from = least, width = largest - least;  // candidates in [from, from + width]
    int n_eq = 0, want = need;
    for (int round = 0;; ++round) {
        const int shift = max(0, 32 - __clz(width) - 8);  // 256 bins over the range
        uint32_t* bins = hist[round & 1];
        for (int j = lo + tid; j < hi; j += T) {
            const uint32_t key = keys[j], d = key - from;
            if (key >= from && d <= width)
                atomicAdd(&bins[d >> shift], 1u);
        }
        __syncthreads();
        // every warp for itself: eight bins a lane, from the top
        constexpr int kOwn = kBins / 32;
        const uint4 v0 = *reinterpret_cast<const uint4*>(bins + kBins - kOwn * (lane + 1)), v1 = *reinterpret_cast<const uint4*>(bins + kBins - kOwn * (lane + 1) + 4);
        const uint32_t v[kOwn] = {v1.w, v1.z, v1.y, v1.x, v0.w, v0.z, v0.y, v0.x};
        uint32_t sum = 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            sum += v[i];
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kFullWarp, incl, o);
            if (lane >= o)
                incl += y;
        }
        const int at_lane = __ffs(__ballot_sync(kFullWarp, incl >= static_cast<uint32_t>(want))) - 1;
        uint32_t at = incl - sum, bin = 0, left = 0, count = 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            if (at < static_cast<uint32_t>(want)) {
                bin = static_cast<uint32_t>(kBins - 1 - lane * kOwn - i);
                left = static_cast<uint32_t>(want) - at;
                count = v[i];
            }
            at += v[i];
        }
        bin = __shfl_sync(kFullWarp, bin, at_lane);
        left = __shfl_sync(kFullWarp, left, at_lane);
        count = __shfl_sync(kFullWarp, count, at_lane);
        from += bin << shift;
        want = static_cast<int>(left);
        if (left == count) {  // the bin is taken whole
            t_ge = from;
            break;
        }
        if (shift == 0) {  // its scores are equal: the first of them
            t_eq = from;
            t_ge = from + 1;
            n_eq = want;
            break;
        }
        width = (1u << shift) - 1;
        if (round > 0) {  // (the bins of the round before this one: all have read them)
            for (int i = tid; i < kBins; i += T)
                hist[(round + 1) & 1][i] = 0;
            __syncthreads();
        }
    }
    // counts of the warps' ranges, then the places
    const int chunk = ((hi - lo + kWarps - 1) / kWarps + 31) & ~31;
    const int w0 = min(lo + warp * chunk, hi), w1 = min(w0 + chunk, hi);
    int ge = 0, eq = 0;
    for (int j = w0 + lane; j < w1; j += 32) {
        ge += keys[j] >= t_ge;
        eq += n_eq > 0 && keys[j] == t_eq;
    }
    ge = __reduce_add_sync(kFullWarp, ge);
    eq = __reduce_add_sync(kFullWarp, eq);
    if (lane == 0) {
        cnt[warp][0] = ge;
        cnt[warp][1] = eq;
    }
    __syncthreads();
    int bge = __reduce_add_sync(kFullWarp, lane < warp ? cnt[lane][0] : 0), beq = __reduce_add_sync(kFullWarp, lane < warp ? cnt[lane][1] : 0);
    const uint32_t below = (1u << lane) - 1;
    for (int base = w0; base < w1; base += 32) {
        const int j = base + lane;
        const uint32_t key = j < w1 ? keys[j] : 0;
        const bool is_ge = j < w1 && key >= t_ge, is_eq = j < w1 && n_eq > 0 && key == t_eq;
        const uint32_t mg = __ballot_sync(kFullWarp, is_ge), me = __ballot_sync(kFullWarp, is_eq);
        const int a = bge + __popc(mg & below), e = beq + __popc(me & below);
        if (is_ge || (is_eq && e < n_eq))
            sel[p.first + a + min(e, n_eq)] = j;
        bge += __popc(mg);
        beq += __popc(me);
    }
}

template <int D>
const void* select_kernel(int C)
{
    return C == 1   ? reinterpret_cast<const void*>(pa_q8_select_kernel<D, 1, 256>)
           : C == 2 ? reinterpret_cast<const void*>(pa_q8_select_kernel<D, 2, 256>)
           : C == 4 ? reinterpret_cast<const void*>(pa_q8_select_kernel<D, 4, 256>)
           : C == 8 ? reinterpret_cast<const void*>(pa_q8_select_kernel<D, 8, 256>)
                    : reinterpret_cast<const void*>(pa_q8_select_kernel<D, 16, 256>);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_q8_select(const void* q, const int8_t* bounds, const float* k_scale, const int32_t* block_table,
                            const int32_t* seq_lens, int32_t* selected, int32_t* counts, int B, int H, int KV, int D, int NQ,
                            int BLOCK, const pa_q8_select_opts* opts, void* stream)
{
    if (!opts)
        return PA_ERR_NULL_POINTER;
    const pa_q8_select_opts& o = *opts;
    const int rc = q8_sizes(B, KV, D, BLOCK, o.max_blocks, o.num_blocks, o.dtype);
    if (rc != PA_OK)
        return rc;
    if (H < 1 || H % KV != 0 || NQ < 1 || o.budget < 1 || o.budget >= (1 << 30) || o.keep_first < 0 || o.keep_last < 0 ||
        static_cast<long long>(o.keep_first) + o.keep_last > o.budget)
        return PA_ERR_BAD_DIMS;
    if (NQ > PA_MAX_NQ || static_cast<long long>(H / KV) * NQ > 1024 || o.max_blocks > kSelectBlocks ||
        static_cast<long long>(B) * KV > 32768)
        return PA_ERR_UNSUPPORTED;
    if (B == 0)
        return PA_OK;
    if (!q || !bounds || !k_scale || !block_table || !seq_lens || !selected || !counts)
        return PA_ERR_NULL_POINTER;
    if (!q8_a16(q) || !q8_a16(bounds) || !q8_a4(k_scale) || !q8_a4(block_table) || !q8_a4(seq_lens) || !q8_a4(selected) ||
        !q8_a4(counts) || !q8_a4(o.status))
        return PA_ERR_ALIGNMENT;
    const size_t blocks = static_cast<size_t>(o.num_blocks) * KV, b4 = static_cast<size_t>(B) * 4;
    const Q8Range r[] = {{selected, b4 * KV * o.budget, true},
                         {counts, b4 * KV, true},
                         {o.status, 4, true},
                         {q, static_cast<size_t>(B) * H * NQ * D * (o.dtype == PA_F32 ? 4 : 2), false},
                         {bounds, blocks * 2 * D, false},
                         {k_scale, blocks * 4, false},
                         {block_table, b4 * o.max_blocks, false},
                         {seq_lens, b4, false}};
    if (q8_overlap(r, 8))
        return PA_ERR_BAD_DIMS;
    SelectParams p{};
    p.q = q;
    p.bounds = bounds;
    p.k_scale = k_scale;
    p.table = block_table;
    p.lens = seq_lens;
    p.selected = selected;
    p.counts = counts;
    p.status = o.status;
    p.KV = KV;
    p.R = H / KV * NQ;
    p.maxb = o.max_blocks;
    p.num_blocks = o.num_blocks;
    p.budget = o.budget;
    p.first = o.keep_first;
    p.last = o.keep_last;
    p.shift = BLOCK == 8 ? 3 : BLOCK == 16 ? 4 : BLOCK == 32 ? 5 : 6;
    p.cap = o.max_blocks * BLOCK;
    p.dtype = o.dtype;
    // CTAs per segment: as many as have a step of blocks each, up to a cluster of 16,
    // while the SMs hold them all at once (one each, or three in clusters up to 8)
    int C = 16;
    while (C > 1 && (static_cast<long long>(B) * KV * C > (C == 16 ? 152 : 456) || 64 * (C / 2) >= o.max_blocks))
        C /= 2;
    const int T = 256;
    const int most = (o.max_blocks + T / 4 * C - 1) / (T / 4 * C) * (T / 4);
    const int rows = p.R < kSelectRows ? (p.R + 3) & ~3 : kSelectRows;
    const size_t smem = 4 * (static_cast<size_t>((o.max_blocks + 3) & ~3) + most + static_cast<size_t>(rows) * (D / 2 + 16));
    void* args[] = {&p};
    return q8_launch(D == 64 ? select_kernel<64>(C) : select_kernel<128>(C), dim3(C, B * KV), T, smem,
                     static_cast<cudaStream_t>(stream), args, C);
}
