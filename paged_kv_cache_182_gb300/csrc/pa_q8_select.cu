// pa_q8_select.cu -- blocks of a cache in 8 bits that a step's queries look at
// most (include/pa_q8.h).
//
// One kernel, a CTA or a cluster of them per sequence and KV head.  The query
// rows become whole numbers in shared memory, positive and negative parts apart,
// so that sum_d max(c min, c max) = c+ . max + c- . min is a product of whole
// numbers (dp4a): exact, in any order.  Four lanes share a block, a quarter of
// the channels each; four rows are summed over those lanes together.  The scores
// go to the first CTA of the cluster, which finds the score of the last block
// taken two bits at a time and writes the indices in order.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectRows = 128;        // query rows in shared memory at once
constexpr int kSelectBlocks = 32768;    // blocks of a table row at most
constexpr int kStepBlocks = kSelectWarps * 8;

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

// grid (C, B * KV), clusters of C along x.
template <int D, int C>
__global__ void __launch_bounds__(kSelectThreads) pa_q8_select_kernel(const __grid_constant__ SelectParams p)
{
    constexpr int kWords = D / 16;                 // words of a lane's quarter of a row
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t* keys = smem;                         // [maxb] scores in order (the first CTA's)
    const int per = ((p.maxb + C - 1) / C + 7) & ~7;
    float* own = reinterpret_cast<float*>(C == 1 ? smem : smem + ((p.maxb + 3) & ~3));  // [per] this CTA's scores
    uint32_t* codes = smem + ((p.maxb + 3) & ~3) + (C == 1 ? 0 : per);  // [rows][4 quarters][positive words | negative words]
    __shared__ float steps[kSelectRows];
    __shared__ int2 sums[2][kSelectWarps];
    __shared__ int cnt[kSelectWarps][2];
    grid_dependents_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = blockIdx.y, b = seg / p.KV, h = seg % p.KV;
    const int rank = C == 1 ? 0 : static_cast<int>(blockIdx.x);
    if (C > 1)  // the first CTA's shared memory may be written once it runs
        asm volatile("barrier.cluster.arrive;" ::: "memory");
    grid_dependency_wait();
    int n = __ldg(p.lens + b);
    if (n < 0 || n > p.cap) {
        if (h == 0 && rank == 0 && tid == 0)
            q8_report(p.status, PA_STATUS_BAD_LENGTH);
        n = n < 0 ? 0 : p.cap;
    }
    const int nb = (n + (1 << p.shift) - 1) >> p.shift;
    const int m = min(nb, p.budget);
    int32_t* sel = p.selected + static_cast<int64_t>(seg) * p.budget;
    if (rank == 0) {
        for (int i = m + tid; i < p.budget; i += kSelectThreads)
            sel[i] = -1;
        if (tid == 0)
            p.counts[seg] = m;
    }
    if (nb <= p.budget) {  // the same in every CTA of the cluster
        if (rank == 0)
            for (int i = tid; i < nb; i += kSelectThreads)
                sel[i] = i;
        if (C > 1)
            asm volatile("barrier.cluster.wait;" ::: "memory");
        return;
    }
    const int lo = p.first, hi = nb - p.last;
    const int need = p.budget - p.first - p.last;
    if (rank == 0) {
        for (int i = tid; i < p.first; i += kSelectThreads)
            sel[i] = i;
        for (int i = tid; i < p.last; i += kSelectThreads)
            sel[p.first + need + i] = hi + i;
    }
    if (need == 0) {
        if (C > 1)
            asm volatile("barrier.cluster.wait;" ::: "memory");
        return;
    }

    // scores of this CTA's blocks [j0, j1)
    const int j0 = min(rank * per, nb), j1 = min(j0 + per, nb);
    const int g = lane >> 2, t = lane & 3;
    const int64_t q0 = static_cast<int64_t>(seg) * p.R * D;
    for (int r0 = 0; r0 < p.R; r0 += kSelectRows) {
        const int rows = min(kSelectRows, p.R - r0), rows4 = (rows + 3) & ~3;
        if (r0 > 0)
            __syncthreads();
        for (int r = warp; r < rows4; r += kSelectWarps) {
            float x[D / 32];
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                x[i] = r < rows ? q8_element(p.q, p.dtype, q0 + static_cast<int64_t>(r0 + r) * D + lane * (D / 32) + i) : 0.f;
                a = q8_amax(a, x[i]);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
                a = fmaxf(a, __shfl_xor_sync(kFullWarp, a, o));
            const float scale = q8_scale_of(a), inv = 1.f / scale;
            // (rows behind the last repeat step 0: they give 0, replaced below)
            if (lane == 0)
                steps[r] = scale;
            int8_t* row = reinterpret_cast<int8_t*>(codes + r * (D / 2));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int d = lane * (D / 32) + i, c = q8_code(x[i], scale, inv);
                int8_t* at = row + (d / (D / 4)) * (D / 2) + d % (D / 4);
                at[0] = static_cast<int8_t>(max(c, 0));
                at[D / 4] = static_cast<int8_t>(min(c, 0));
            }
        }
        __syncthreads();
        for (int base = j0 + warp * 8; base < j1; base += kStepBlocks) {
            const int j = base + g;
            int phys = -1;
            if (j < j1) {
                phys = __ldg(p.table + static_cast<int64_t>(b) * p.maxb + j);
                if (phys < 0 || phys >= p.num_blocks) {
                    phys = -1;
                    q8_report(p.status, PA_STATUS_BAD_BLOCK);
                }
            }
            uint32_t mn[kWords], mx[kWords];
            float ks = 0.f;
            if (phys >= 0) {
                const int64_t at = static_cast<int64_t>(phys) * p.KV + h;
                const uint4* src = reinterpret_cast<const uint4*>(p.bounds + at * 2 * D + t * (D / 4));
#pragma unroll
                for (int i = 0; i < kWords / 4; ++i) {
                    const uint4 v = __ldg(src + i), w = __ldg(src + i + D / 16);
                    mn[4 * i] = v.x, mn[4 * i + 1] = v.y, mn[4 * i + 2] = v.z, mn[4 * i + 3] = v.w;
                    mx[4 * i] = w.x, mx[4 * i + 1] = w.y, mx[4 * i + 2] = w.z, mx[4 * i + 3] = w.w;
                }
                ks = __ldg(p.k_scale + at);
            } else {
#pragma unroll
                for (int i = 0; i < kWords; ++i)
                    mn[i] = mx[i] = 0;
            }
            float best = -INFINITY;
            bool any = false;
            for (int r = 0; r < rows; r += 4) {
                int sum[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4* c = reinterpret_cast<const uint4*>(codes + (r + k) * (D / 2) + t * (D / 8));
                    int s = 0;
#pragma unroll
                    for (int i = 0; i < kWords / 4; ++i) {
                        const uint4 up = c[i], dn = c[i + D / 64];
                        s = __dp4a(static_cast<int>(up.x), static_cast<int>(mx[4 * i]), s);
                        s = __dp4a(static_cast<int>(up.y), static_cast<int>(mx[4 * i + 1]), s);
                        s = __dp4a(static_cast<int>(up.z), static_cast<int>(mx[4 * i + 2]), s);
                        s = __dp4a(static_cast<int>(up.w), static_cast<int>(mx[4 * i + 3]), s);
                        s = __dp4a(static_cast<int>(dn.x), static_cast<int>(mn[4 * i]), s);
                        s = __dp4a(static_cast<int>(dn.y), static_cast<int>(mn[4 * i + 1]), s);
                        s = __dp4a(static_cast<int>(dn.z), static_cast<int>(mn[4 * i + 2]), s);
                        s = __dp4a(static_cast<int>(dn.w), static_cast<int>(mn[4 * i + 3]), s);
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
                    const float score = __fmul_rn(__fmul_rn(steps[r + t], ks), static_cast<float>(total));
                    any |= score == score;
                    best = fmaxf(best, score);  // (a NaN leaves the other)
                }
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                best = fmaxf(best, __shfl_xor_sync(kFullWarp, best, o));
                any |= __shfl_xor_sync(kFullWarp, static_cast<int>(any), o) != 0;
            }
            if (j < j1 && t == 0) {
                float s = phys >= 0 && any ? best : __int_as_float(0x7fc00000);
                if (r0 > 0) {
                    const float before = own[j - j0];
                    s = before != before ? s : s != s ? before : fmaxf(s, before);
                }
                own[j - j0] = s;
            }
        }
    }
    __syncthreads();
    // to the first CTA
    if (C == 1) {
        for (int j = tid; j < nb; j += kSelectThreads)
            keys[j] = score_order(own[j]);
        __syncthreads();
    } else {
        asm volatile("barrier.cluster.wait;" ::: "memory");
        uint32_t to;
        asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_u32(keys)));
        for (int j = j0 + tid; j < j1; j += kSelectThreads)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + static_cast<uint32_t>(j) * 4),
                         "r"(score_order(own[j - j0]))
                         : "memory");
        asm volatile("barrier.cluster.arrive;" ::: "memory");
        asm volatile("barrier.cluster.wait;" ::: "memory");
        if (rank != 0)
            return;
    }

    // the score of the last block taken: the largest T that `need` candidates reach
    uint32_t T = 0, t_ge = 0, t_eq = 0;
    int n_eq = 0;
    bool whole = false;
    for (int s = 30; s >= 0 && !whole; s -= 2) {
        const uint32_t c1 = T | 1u << s, c2 = T | 2u << s, c3 = T | 3u << s;
        int x = 0, y = 0;
        for (int j = lo + tid; j < hi; j += kSelectThreads) {
            const uint32_t k = keys[j];
            x += (k >= c1 ? 1 : 0) + (k >= c2 ? 1 << 16 : 0);
            y += k >= c3 ? 1 : 0;
        }
        x = static_cast<int>(__reduce_add_sync(kFullWarp, static_cast<uint32_t>(x)));
        y = __reduce_add_sync(kFullWarp, y);
        int2* sum = sums[(s >> 1) & 1];
        if (lane == 0)
            sum[warp] = make_int2(x, y);
        __syncthreads();
        const int2 v = lane < kSelectWarps ? sum[lane] : make_int2(0, 0);
        const uint32_t xx = __reduce_add_sync(kFullWarp, static_cast<uint32_t>(v.x));
        const int n1 = static_cast<int>(xx & 0xffffu), n2 = static_cast<int>(xx >> 16), n3 = __reduce_add_sync(kFullWarp, v.y);
        int got = 0;
        if (n3 >= need) {
            T = c3;
            got = n3;
        } else if (n2 >= need) {
            T = c2;
            got = n2;
        } else if (n1 >= need) {
            T = c1;
            got = n1;
        }
        whole = got == need;  // all that reach T are taken
    }
    if (whole) {
        t_ge = T;
    } else {  // more than are wanted have the score T: the first of them
        t_eq = T;
        t_ge = T + 1;
    }
    // counts of the warps' ranges, then the places
    const int chunk = ((hi - lo + kSelectWarps - 1) / kSelectWarps + 31) & ~31;
    const int w0 = min(lo + warp * chunk, hi), w1 = min(w0 + chunk, hi);
    int ge = 0, eq = 0;
    for (int j = w0 + lane; j < w1; j += 32) {
        ge += keys[j] >= t_ge;
        eq += !whole && keys[j] == t_eq;
    }
    ge = __reduce_add_sync(kFullWarp, ge);
    eq = __reduce_add_sync(kFullWarp, eq);
    if (lane == 0) {
        cnt[warp][0] = ge;
        cnt[warp][1] = eq;
    }
    __syncthreads();
    const int cg = lane < kSelectWarps ? cnt[lane][0] : 0, ce = lane < kSelectWarps ? cnt[lane][1] : 0;
    n_eq = whole ? 0 : need - __reduce_add_sync(kFullWarp, cg);
    int bge = __reduce_add_sync(kFullWarp, lane < warp ? cg : 0), beq = __reduce_add_sync(kFullWarp, lane < warp ? ce : 0);
    const uint32_t below = (1u << lane) - 1;
    for (int base = w0; base < w1; base += 32) {
        const int j = base + lane;
        const uint32_t key = j < w1 ? keys[j] : 0;
        const bool is_ge = j < w1 && key >= t_ge, is_eq = j < w1 && !whole && key == t_eq;
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
    return C == 1   ? reinterpret_cast<const void*>(pa_q8_select_kernel<D, 1>)
           : C == 2 ? reinterpret_cast<const void*>(pa_q8_select_kernel<D, 2>)
           : C == 4 ? reinterpret_cast<const void*>(pa_q8_select_kernel<D, 4>)
                    : reinterpret_cast<const void*>(pa_q8_select_kernel<D, 8>);
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
    // CTAs per segment: as many as the SMs hold at once, with a step of blocks each
    int C = 8;
    while (C > 1 && (static_cast<long long>(B) * KV * C > 304 || kStepBlocks * (C / 2) >= o.max_blocks))
        C /= 2;
    const int per = ((o.max_blocks + C - 1) / C + 7) & ~7;
    const int rows = p.R < kSelectRows ? (p.R + 3) & ~3 : kSelectRows;
    const size_t smem = 4 * (static_cast<size_t>((o.max_blocks + 3) & ~3) + (C == 1 ? 0 : per) + static_cast<size_t>(rows) * (D / 2));
    void* args[] = {&p};
    return q8_launch(D == 64 ? select_kernel<64>(C) : select_kernel<128>(C), dim3(C, B * KV), kSelectThreads, smem,
                     static_cast<cudaStream_t>(stream), args, C);
}
