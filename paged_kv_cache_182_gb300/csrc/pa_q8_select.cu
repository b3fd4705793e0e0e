// pa_q8_select.cu -- blocks of a cache in 8 bits that a step's queries look at
// most (include/pa_q8.h).
//
// One kernel, a CTA or a cluster of them per sequence and KV head.  The query
// rows become whole numbers, positive and negative parts apart, so that
// sum_d max(c min, c max) = c- . min + c+ . max is a product of whole numbers of
// length 2 D.  The tensor cores take it in fp16 with float32 sums: a bound + 128 is
// a subnormal fp16 number as it stands (the row's 128 sum c is taken off
// beforehand), a code is exact, and all sums are below 2^24 of the unit 2^-24:
// nothing is rounded, in any order.  (Integer products, dp4a, run at a tenth of
// the rate here: 42 us for 8 x 8 x 4096 blocks and 4 rows, now 25; 40 for 4 x 8 x 2048
// and 32 rows, now 20.)  A warp has 16 blocks in hand and 16 on their way (three
// steps, CTAs of 128 threads, or three CTAs per SM at 80 registers: 35 to 49 us for
// the first); table entries are read before the length is known.
//
// The scores go to the first CTA of the cluster, which finds the score of the
// last block taken by counting them in 256 bins over their range, then over the
// bin that it falls into, until that bin is taken whole: mostly two rounds.
//
// What bounds it: latency.  8 heads of 2048 blocks (one sequence, clusters of 16)
// take 9.3 us, 24 x 8 x 750 blocks (one CTA each) 17.1 us, 2.2 TB/s, 24 uneven sequences
// of 63 to 750 14.5 us, 1.1 TB/s: the chain from length to table, bounds, scores, cluster
// barrier, rounds of bins and places.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kSelectRows = 128;        // query rows in shared memory at once
constexpr int kSelectBlocks = 32768;    // blocks of a table row at most
constexpr int kBins = 256;
constexpr int kRing = 2;                // steps of a warp's blocks in shared memory
__host__ __device__ constexpr int kStepBytes(int D) { return 16 * 2 * D + 64; }  // bounds of 16 blocks, their scales

struct SelectParams {
    const void* q;
    const int8_t* bounds;
    const float* k_scale;
    const int32_t* table;
    const int32_t* lens;
    int32_t* selected;
    int32_t* counts;
    int* status;
    int KV, R, chunk, maxb, num_blocks, budget, first, last, shift, cap, dtype;
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
__global__ void __launch_bounds__(T, 512 / T) pa_q8_select_kernel(const __grid_constant__ SelectParams p)
{
    constexpr int kWarps = T / 32, kStep = kWarps * C * 16;  // blocks that the cluster takes together
    constexpr int kChunks = D / 32, kSteps = D / 8;          // 64 bytes of a block's bounds; MMA steps
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t* keys = smem;                         // [maxb] scores in order (the first CTA's)
    // [most] this CTA's scores, one CTA's in the keys' place; the warps' rings;
    // fragments of the rows [8 rows][step][lane]
    const int most = C == 1 ? 0 : (p.maxb + kStep - 1) / kStep * kWarps * 16;
    uint32_t* const behind = smem + (p.maxb + 15) / 16 * 16;
    float* own = reinterpret_cast<float*>(C == 1 ? smem : behind);
    unsigned char* rings = reinterpret_cast<unsigned char*>(behind + most);
    unsigned char* ring = rings + (threadIdx.x >> 5) * kRing * kStepBytes(D);
    uint2* codes = reinterpret_cast<uint2*>(rings + kWarps * kRing * kStepBytes(D));
    __shared__ float offs[kSelectRows];            // what a row's sums begin with
    __shared__ float steps[kSelectRows];
    __shared__ __align__(16) uint32_t hist[2][kBins];
    __shared__ uint32_t wide[kWarps][2];
    __shared__ int cnt[kWarps][2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int seg = blockIdx.y, b = seg / p.KV, h = seg - b * p.KV;
    const int rank = C == 1 ? 0 : static_cast<int>(blockIdx.x);
    if (C > 1)  // the first CTA's shared memory may be written once it runs
        asm volatile("barrier.cluster.arrive;" ::: "memory");
    grid_begin();
    int n = __ldg(p.lens + b);
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.maxb;
    // the cluster's warps take 16 blocks each in turn, a lane those of rows g and g + 8
    const int j0 = (warp * C + rank) * 16 + g;
    auto entry = [&](int j, int end) { return j < end ? __ldg(table + j) : -1; };
    int phys[kRing][2];
#pragma unroll
    for (int s = 0; s < kRing; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            phys[s][i] = entry(j0 + s * kStep + 8 * i, p.maxb);
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

    // scores.  A lane copies the bytes that it will use itself (and one scale of two).
    const uint32_t ring0 = smem_u32(ring);
    uint32_t there = 0;  // of the steps on their way, two bits each: the lane's blocks are in the pool
    auto issue = [&](int j, const int* ph, int stage) {
        const uint32_t to = ring0 + stage * kStepBytes(D);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool ok = j + 8 * i < nb && static_cast<uint32_t>(ph[i]) < static_cast<uint32_t>(p.num_blocks);
            if (!ok && j + 8 * i < nb)
                q8_report(p.status, PA_STATUS_BAD_BLOCK);
            there = there << 1 | (ok ? 1u : 0u);
            if (ok) {
                const int64_t at = static_cast<int64_t>(ph[i]) * p.KV + h;
                const int8_t* src = p.bounds + at * 2 * D + t * 16;
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    q8_copy16(to + ((i * kChunks + c) * 32 + lane) * 16, src + c * 64);
                if (t == i)
                    q8_copy4(to + 32 * D + (g + 8 * i) * 4, p.k_scale + at);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int r0 = 0; r0 < p.R; r0 += p.chunk) {
        const int rows = min(p.chunk, p.R - r0), rows8 = (rows + 7) & ~7;
        // kRing - 1 steps are on their way, the entries of the next
        if (r0 > 0) {
#pragma unroll
            for (int s = 0; s < kRing; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    phys[s][i] = entry(j0 + s * kStep + 8 * i, nb);
            __syncthreads();
        }
#pragma unroll
        for (int s = 0; s < kRing - 1; ++s)
            issue(j0 + s * kStep, phys[s], s);
        int ahead[2] = {phys[kRing - 1][0], phys[kRing - 1][1]};
        for (int r = warp; r < rows8; r += kWarps) {
            constexpr int kOwn = D / 32;  // channels of a lane
            float v[kOwn];
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                v[i] = r < rows ? q8_element(p.q, p.dtype, q0 + static_cast<int64_t>(r0 + r) * D + lane * kOwn + i) : 0.f;
                a = q8_amax(a, v[i]);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
                a = fmaxf(a, __shfl_xor_sync(kFullWarp, a, o));
            const float scale = q8_scale_of(a), inv = 1.f / scale;
            int sum = 0;
            uint32_t up[kOwn / 2], down[kOwn / 2];
#pragma unroll
            for (int i = 0; i < kOwn; i += 2) {
                const int c0 = q8_code(v[i], scale, inv), c1 = q8_code(v[i + 1], scale, inv);
                sum += c0 + c1;
                const __half2 u = __floats2half2_rn(static_cast<float>(max(c0, 0)), static_cast<float>(max(c1, 0)));
                const __half2 d = __floats2half2_rn(static_cast<float>(min(c0, 0)), static_cast<float>(min(c1, 0)));
                up[i / 2] = *reinterpret_cast<const uint32_t*>(&u);
                down[i / 2] = *reinterpret_cast<const uint32_t*>(&d);
            }
            sum = __reduce_add_sync(kFullWarp, sum);
            if (lane == 0) {
                steps[r] = scale;
                offs[r] = static_cast<float>(sum) * (-128.f / 16777216.f);
            }
            // channel d: chunk d / 64, lane's part (d % 64) / 16, step (d % 16) / 4 of the chunk
            const int d = lane * kOwn;
            uint2* to = codes + ((r >> 3) * kSteps + (d / 64) * 4 + d % 16 / 4) * 32 + (r & 7) * 4 + d % 64 / 16;
            if constexpr (D == 128) {
                to[0] = make_uint2(down[0], down[1]);
                to[kSteps / 2 * 32] = make_uint2(up[0], up[1]);
            } else {
                reinterpret_cast<uint32_t*>(to)[d % 4 / 2] = down[0];
                reinterpret_cast<uint32_t*>(to + kSteps / 2 * 32)[d % 4 / 2] = up[0];
            }
        }
        __syncthreads();
        int slot = warp * 16 + g, stage = 0;
        for (int base = j0 - g; base < nb; base += kStep, slot += kWarps * 16) {
            const int j = base + g;
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
            __syncwarp();  // the scales of the other lanes; the stage filled next has been read
            issue(j + (kRing - 1) * kStep, ahead, stage == 0 ? kRing - 1 : stage - 1);
            ahead[0] = entry(j + kRing * kStep, nb);
            ahead[1] = entry(j + kRing * kStep + 8, nb);
            const unsigned char* now = ring + stage * kStepBytes(D);
            const bool ok[2] = {(there >> (2 * kRing - 1) & 1u) != 0, (there >> (2 * kRing - 2) & 1u) != 0};
            const float ks[2] = {*reinterpret_cast<const float*>(now + 32 * D + g * 4), *reinterpret_cast<const float*>(now + 32 * D + g * 4 + 32)};
            stage = stage + 1 == kRing ? 0 : stage + 1;
            float best[2] = {-INFINITY, -INFINITY};
            bool any[2] = {false, false};
            for (int r = 0; r < rows; r += 8) {
                float acc[4];
                acc[0] = acc[2] = offs[r + 2 * t];
                acc[1] = acc[3] = offs[r + 2 * t + 1];
                const uint2* q = codes + (r >> 3) * kSteps * 32 + lane;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const uint4 va = *reinterpret_cast<const uint4*>(now + (c * 32 + lane) * 16);
                    const uint4 vb = *reinterpret_cast<const uint4*>(now + ((kChunks + c) * 32 + lane) * 16);
                    const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t ua = wa[i] ^ 0x80808080u, ub = wb[i] ^ 0x80808080u;
                        const uint32_t a[4] = {__byte_perm(ua, 0, 0x4140), __byte_perm(ub, 0, 0x4140), __byte_perm(ua, 0, 0x4342),
                                               __byte_perm(ub, 0, 0x4342)};
                        const uint2 f = q[(c * 4 + i) * 32];
                        mma_16816<false>(acc, a, f.x, f.y);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r + 2 * t + (i & 1) < rows) {
                        const float score = __fmul_rn(__fmul_rn(steps[r + 2 * t + (i & 1)], ks[i >> 1]), acc[i] * 16777216.f);
                        any[i >> 1] |= score == score;
                        best[i >> 1] = fmaxf(best[i >> 1], score);  // (a NaN leaves the other)
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    best[i] = fmaxf(best[i], __shfl_xor_sync(kFullWarp, best[i], o));
                    any[i] |= __shfl_xor_sync(kFullWarp, static_cast<int>(any[i]), o) != 0;
                }
                if (j + 8 * i < nb && t == 0) {
                    float s = ok[i] && any[i] ? best[i] : __int_as_float(0x7fc00000);
                    if (r0 > 0) {
                        const float before = own[slot + 8 * i];
                        s = before != before ? s : s != s ? before : fmaxf(s, before);
                    }
                    own[slot + 8 * i] = s;
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    // to the first CTA; a warp moves its own
    __syncwarp();
    uint32_t to = smem_u32(keys);
    if (C > 1) {
        asm volatile("barrier.cluster.wait;" ::: "memory");
        asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_u32(keys)));
    }
    for (int base = (warp * C + rank) * 16 + lane % 16 + lane / 16 * kStep, slot = warp * 16 + lane % 16 + lane / 16 * kWarps * 16;
         base < nb; base += 2 * kStep, slot += 2 * kWarps * 16)
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
const void* select_kernel(int C, int T)
{
    return T == 128 ? reinterpret_cast<const void*>(pa_q8_select_kernel<D, 1, 128>)
           : C == 1 ? reinterpret_cast<const void*>(pa_q8_select_kernel<D, 1, 256>)
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
    // Smaller CTAs, four per SM, where two per SM do not hold all segments and a table
    // leaves them the room: 100 x 8 segments of 64 / 256 / 512 blocks 13.5 / 24.4 / 37.2 us
    // (CTAs of 256 threads: 16.9 / 26.5 / 37.7), 40 x 8 of 64 / 512 7.9 / 21.6 (10.6 / 22.5);
    // 80 x 8 of 1024 alone are slower, 56.5 (52.6).
    const int T = static_cast<long long>(B) * KV > 304 && o.max_blocks <= 4096 ? 128 : 256;
    // CTAs per segment: as many as have a step of blocks each, up to a cluster of 16,
    // while the SMs hold them all at once (one each, or two in clusters up to 8).  One
    // CTA / clusters: 8 x 2048 blocks 25 / 9.5 us, 64 x 4096 47 / 25, 128 x 1024 12.9 / 11.8
    constexpr size_t kRoom = 223 * 1024;  // (227 KB with the kernel's own arrays)
    int C = 16;
    while (C > 1 && (static_cast<long long>(B) * KV * C > (C == 16 ? 152 : 304) || T / 2 * (C / 2) >= o.max_blocks))
        C /= 2;
    const size_t keys = static_cast<size_t>(o.max_blocks + 15) / 16 * 64, ring = T / 32 * kRing * kStepBytes(D);
    const auto scores = [&](int c) { return c == 1 ? size_t{0} : static_cast<size_t>((o.max_blocks + T / 2 * c - 1) / (T / 2 * c)) * (T / 2) * 4; };
    const size_t row8 = static_cast<size_t>(8) * 4 * D;  // fragments of eight rows
    if (keys + scores(C) + ring + row8 > kRoom)
        C = 1;  // (a very long table: the scores stay where the keys are)
    // rows together: all, or what there is room for
    size_t room = (kRoom - keys - scores(C) - ring) / row8 * 8;
    p.chunk = static_cast<int>(room < kSelectRows ? room : kSelectRows);
    const size_t rows = p.R < p.chunk ? static_cast<size_t>(p.R + 7) & ~static_cast<size_t>(7) : p.chunk;
    const size_t smem = keys + scores(C) + ring + rows * 4 * D;
    void* args[] = {&p};
    return q8_launch(D == 64 ? select_kernel<64>(C, T) : select_kernel<128>(C, T), dim3(C, B * KV), T, smem,
                     static_cast<cudaStream_t>(stream), args, C);
}
