// pa_evict.cu -- cache eviction by accumulated attention weight
// (include/pa_evict.h).
//
// Two kernels:
//
// pa_evict_select -- a CTA or a cluster of CTAs per sequence finds the weight
//   of the last token that is kept: a radix select over the weights' ordered
//   bit patterns, histograms of 11, 11 and 10 bits summed over the cluster
//   through distributed shared memory.  It ends early once the chosen bin is
//   taken whole (two passes for distinct weights).  The weights stay in
//   registers, 8 a thread, loaded before the length is known (the ranges are
//   those of the table's capacity).  Then it writes the kept indices and
//   weights in token order: each warp owns a contiguous range of tokens, the
//   ranges' counts are summed over warps and CTAs, and ballots place the
//   tokens inside a range.  Bound by latency: 12 us for 64 sequences of up to
//   16384 tokens, 10.5 for one of 32768, of which a third are cluster barriers
//   and remote histogram reads.
//
// The rows then move by one of two kernels, which set up while the selection
// runs (programmatic launch):
//
// pa_evict_shift (in place) -- kept[r] >= r, so a destination slot is either
//   unmoved or the source of a lower or equal rank.  A CTA owns a slice of the
//   columns of one sequence's K or V and walks the ranks in order, several
//   runs of rows in flight: a run is written when it and all runs before it
//   have been read, which is all that the overlap asks for, and no CTA waits
//   for another.  (Runs of whole rows dealt to all CTAs, each waiting for the
//   flags of the runs that it overwrites, took 34 us where this takes 22.)
//   Bound by memory: 25 of 64 sequences over a budget of 2048, 100 MB read and
//   written at 6.9 TB/s once the pipeline is full, 5 us to fill it.
//
// pa_evict_gather (into other blocks) -- nothing overlaps: one CTA per run of
//   whole rows, 16 KB.  8192 rows of 2 KB of K and of V: 13 us, 5.2 TB/s.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_evict.h"
#include "pa_ptx.cuh"
#include "pa_vjp.cuh"

namespace pa {
namespace {

constexpr int kBins = 2048;
constexpr int kKeys = 8;            // weights in flight per thread of the selection
constexpr int kMoveThreads = 256;
constexpr int kRunBytes = 16384;    // in place: a run of rows' slices
constexpr int kRuns = 6;            // in flight
constexpr int kMoveBytes = 16384;   // other blocks: rows of one item, at most (one row when longer)
constexpr int kMoveRows = 256;
constexpr int kMaxRowBytes = 65536;
constexpr unsigned kAll32 = 0xffffffffu;

struct EvictParams {
    unsigned char* pool[2];  // K, V
    const int32_t* table;
    const int32_t* dst;      // destination table (block_table when in place)
    const int32_t* lens;
    const float* weights;
    int32_t* new_lens;
    int32_t* kept;
    float* weights_out;
    int* status;
    int B, BLOCK, maxb, dst_maxb, num_blocks, budget, first, last, in_place;
    int cap;                 // max_blocks * BLOCK
    int row_bytes;           // KV * D * element bytes
    int rows_item;           // other blocks: rows per item
    int slices;              // in place: column slices of a row
    int shift;               // log2 of BLOCK, or -1
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The two 32-bit words at the same shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ uint2 cluster_load2(const uint32_t* p, uint32_t rank)
{
    uint2 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %2, %3;\n\t"
        "ld.shared::cluster.v2.u32 {%0, %1}, [a];\n\t}"
        : "=r"(v.x), "=r"(v.y)
        : "r"(smem_u32(p)), "r"(rank)
        : "memory");
    return v;
}

// One of them.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* p, uint32_t rank)
{
    uint32_t v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %1, %2;\n\t"
        "ld.shared::cluster.u32 %0, [a];\n\t}"
        : "=r"(v)
        : "r"(smem_u32(p)), "r"(rank)
        : "memory");
    return v;
}

// Exclusive sum of v[0 .. n-1] below `warp` (n at most 32, the same in every lane).
__device__ __forceinline__ uint32_t sum_below(const uint32_t* v, int stride, int n, int warp)
{
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(kAll32, lane < n && lane < warp ? v[lane * stride] : 0u);
}

// Unsigned integers in the order of the weights: NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t order_of(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int clamped_len(const EvictParams& p, int b, bool report)
{
    const int n = __ldg(p.lens + b);
    if (n >= 0 && n <= p.cap)
        return n;
    if (report && p.status)
        atomicOr(p.status, PA_STATUS_BAD_LENGTH);
    return n < 0 ? 0 : p.cap;
}

// T threads a CTA, C CTAs a cluster.
template <int T, int C>
__global__ void __launch_bounds__(T) pa_evict_select(const __grid_constant__ EvictParams p)
{
    constexpr int kSelThreads = T, kSelWarps = T / 32, kOwn = kBins / T;
    __shared__ __align__(8) uint32_t hist[2][kBins];
    __shared__ uint32_t wsum[kSelWarps];
    __shared__ uint32_t pick[3];               // chosen digit, still needed in it, its count
    __shared__ uint32_t cnt[kSelWarps][2];     // tokens taken outright / at the threshold, by warp
    __shared__ uint32_t tot[2];                // the same of the CTA
    grid_dependents_launch();  // the move waits for this grid before it reads the kept list
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = C == 1 ? 0 : static_cast<int>(cluster_rank());
    const int b = blockIdx.x / C;
    const int step = C * kSelThreads, me = rank * kSelThreads + tid;
    const float* w = p.weights + static_cast<int64_t>(b) * p.cap;
    // This CTA's and warp's tokens: contiguous ranges of the table's capacity, in
    // token order, so that the weights are on their way before the length is
    // known.  A warp's batch is kKeys * 32 weights, loaded together; ranges of one
    // batch stay in registers, longer ones are read again in every pass.
    const int per = (p.cap + C - 1) / C;
    const int sub = ((per + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int64_t first_j = static_cast<int64_t>(rank) * per + static_cast<int64_t>(warp) * sub;
    int w0 = static_cast<int>(min(first_j, static_cast<int64_t>(p.cap)));
    int w1 = min(w0 + min(sub, max(0, per - warp * sub)), p.cap);
    float x[kKeys];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const int j = base + u * 32 + lane;
            x[u] = j < w1 ? __ldg(w + j) : 0.f;
        }
    };
    const bool resident = sub <= kKeys * 32;
    if (resident)
        load(w0);
    const int n = clamped_len(p, b, me == 0);
    float* wo = p.weights_out + static_cast<int64_t>(b) * p.cap;
    int32_t* kept = p.kept + static_cast<int64_t>(b) * p.budget;

    const int m = min(n, p.budget);
    if (me == 0)
        p.new_lens[b] = m;
    for (int j = m + me; j < p.cap; j += step)
        wo[j] = 0.f;
    if (n <= p.budget) {  // the same for every CTA of the cluster
        for (int j = me; j < p.budget; j += step)
            kept[j] = j < n ? j : -1;
        for (int j = me; j < n; j += step)
            wo[j] = __ldg(w + j);
        return;
    }
    const int lo = p.first, hi = n - p.last;
    int need = p.budget - p.first - p.last;
    for (int j = me; j < p.first; j += step) {
        kept[j] = j;
        wo[j] = __ldg(w + j);
    }
    for (int i = me; i < p.last; i += step) {
        kept[p.first + need + i] = hi + i;
        wo[p.first + need + i] = __ldg(w + hi + i);
    }
    if (need == 0)
        return;
    // of them, the tokens to choose from: [lo, hi)
    const int batch0 = w0;
    w1 = min(w1, hi);
    const int j_lo = max(w0, lo);

    // taken: order >= t_ge, and of those with order == t_eq the first n_eq
    uint32_t prefix = 0, mask = 0, t_ge = 0, t_eq = 0, n_eq = 0;
    for (int i = tid; i < 2 * kBins; i += kSelThreads)
        (&hist[0][0])[i] = 0;
    __syncthreads();
    uint32_t k = static_cast<uint32_t>(need);
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
        uint32_t* h = hist[pass & 1];
        for (int base = batch0; base < w1; base += kKeys * 32) {
            if (!resident)
                load(base);
#pragma unroll
            for (int u = 0; u < kKeys; ++u) {
                const int j = base + u * 32 + lane;
                const uint32_t key = order_of(x[u]);
                const bool in = j >= j_lo && j < w1 && (key & mask) == prefix;
                // weights crowd into few digits, but counting up by one is
                // combined within the warp by the hardware: aggregating equal
                // digits by hand (match, then one add) took twice as long
                if (in)
                    atomicAdd(&h[(key >> shift) & digits], 1u);
            }
        }
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
        // kOwn bins a thread, from the top
        uint32_t v[kOwn], sum = 0;
        const int top = kBins - 1 - kOwn * tid;
#pragma unroll
        for (int i = 0; i < kOwn; i += 2) {
            uint2 two = C == 1 ? *reinterpret_cast<const uint2*>(&h[top - i - 1]) : make_uint2(0, 0);
            if (C > 1) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint2 r = cluster_load2(&h[top - i - 1], c);
                    two.x += r.x;
                    two.y += r.y;
                }
            }
            v[i] = two.y;
            v[i + 1] = two.x;
            sum += two.x + two.y;
        }
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kAll32, incl, o);
            if (lane >= o)
                incl += y;
        }
        if (lane == 31)
            wsum[warp] = incl;
        __syncthreads();
        const uint32_t before = incl - sum + sum_below(wsum, 1, kSelWarps, warp);
        if (before < k && k <= before + sum) {
            uint32_t at = before;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                if (at < k && k <= at + v[i]) {
                    pick[0] = static_cast<uint32_t>(top - i);
                    pick[1] = k - at;
                    pick[2] = v[i];
                }
                at += v[i];
            }
        }
        __syncthreads();
        prefix |= pick[0] << shift;
        mask |= digits << shift;
        k = pick[1];
        if (k == pick[2]) {  // the whole bin is taken
            t_ge = prefix;
            break;
        }
        if (pass == 2) {
            t_eq = prefix;
            t_ge = prefix + 1;
            n_eq = k;
        } else if (pass == 1) {
            // pass 2 counts in hist[0] again: every CTA has read it (they have
            // all passed this pass's cluster barrier)
            for (int i = tid; i < kBins; i += kSelThreads)
                hist[0][i] = 0;
            __syncthreads();
        }
    }

    // counts of the ranges, then the places
    uint32_t ge = 0, eq = 0;
    for (int base = batch0; base < w1; base += kKeys * 32) {
        if (!resident)
            load(base);
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const int j = base + u * 32 + lane;
            const bool in = j >= j_lo && j < w1;
            const uint32_t key = order_of(x[u]);
            ge += in && key >= t_ge;
            eq += in && n_eq > 0 && key == t_eq;
        }
    }
    ge = __reduce_add_sync(kAll32, ge);
    eq = __reduce_add_sync(kAll32, eq);
    if (lane == 0) {
        cnt[warp][0] = ge;
        cnt[warp][1] = eq;
    }
    __syncthreads();
    uint32_t bge = sum_below(&cnt[0][0], 2, kSelWarps, warp), beq = sum_below(&cnt[0][1], 2, kSelWarps, warp);
    if (C > 1) {
        if (tid == kSelThreads - 1) {
            tot[0] = bge + ge;  // the last warp's: all of the CTA's
            tot[1] = beq + eq;
        }
        cluster_sync();
        for (int c = 0; c < rank; ++c) {
            bge += cluster_load(&tot[0], c);
            beq += cluster_load(&tot[1], c);
        }
    }
    const uint32_t below = (1u << lane) - 1;
    for (int base = batch0; base < w1; base += kKeys * 32) {
        if (!resident)
            load(base);
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const int j = base + u * 32 + lane;
            const uint32_t key = order_of(x[u]);
            const bool in = j >= j_lo && j < w1;
            const bool is_ge = in && key >= t_ge, is_eq = in && n_eq > 0 && key == t_eq;
            const uint32_t mg = __ballot_sync(kAll32, is_ge), me_ = __ballot_sync(kAll32, is_eq);
            const uint32_t g = bge + __popc(mg & below), e = beq + __popc(me_ & below);
            if (is_ge || (is_eq && e < n_eq)) {
                const int r = p.first + static_cast<int>(g + min(e, n_eq));
                kept[r] = j;
                wo[r] = x[u];
            }
            bge += __popc(mg);
            beq += __popc(me_);
        }
    }
    if (C > 1)
        cluster_sync();  // the others have read this CTA's shared memory
}

// A token's block.  (The move looks up four a row, on its way to every copy: with
// shifts in place of divisions a call of 19569 rows takes 55 us instead of 70.)
__device__ __forceinline__ int block_of(const EvictParams& p, int j) { return p.shift >= 0 ? j >> p.shift : j / p.BLOCK; }

// Slot of token j by a table row, or -1 (reported) when its block is outside the pool.
__device__ __forceinline__ int slot_of(const EvictParams& p, int phys, int j, bool report)
{
    if (phys >= 0 && phys < p.num_blocks)
        return phys * p.BLOCK + (j - block_of(p, j) * p.BLOCK);
    if (report && p.status)
        atomicOr(p.status, PA_STATUS_BAD_BLOCK);
    return -1;
}

// grid (slices * 2, B): a slice of VS 16-byte vectors of K or V of a sequence, S
// runs in flight.  Each thread looks up LOOK rows of a run, three steps ahead of
// their copy: kept index, then table entries, then slots.
template <int VS, int S>
__global__ void __launch_bounds__(kMoveThreads) pa_evict_shift(const __grid_constant__ EvictParams p)
{
    constexpr int RUN = kRunBytes / (16 * VS), LOOK = (RUN + kMoveThreads - 1) / kMoveThreads;
    static_assert(RUN % kMoveThreads == 0 || RUN < kMoveThreads, "rows looked up by the threads");
    extern __shared__ __align__(16) unsigned char ring[];  // [S runs][RUN rows][VS vectors]
    __shared__ int src[2][RUN], dst[S + 1][RUN];
    const int tid = threadIdx.x;
    const int kv = blockIdx.x & 1, slice = blockIdx.x >> 1, b = blockIdx.y;
    const int n = clamped_len(p, b, false);
    grid_dependency_wait();  // the kept list
    if (n <= p.budget)
        return;
    const int runs = (p.budget + RUN - 1) / RUN;
    const int32_t* kept = p.kept + static_cast<int64_t>(b) * p.budget;
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.maxb;
    const bool report = blockIdx.x == 0;
    const int v0 = slice * VS, nv = min(VS, (p.row_bytes >> 4) - v0);  // vectors of this slice
    unsigned char* pool = p.pool[kv] + v0 * 16;
    const int v = tid % VS, rr = tid / VS;
    constexpr int kStep = kMoveThreads / VS;  // rows the CTA copies at once

    int j1[LOOK], j2[LOOK], ps[LOOK], pd[LOOK];  // the run three and two ahead: kept; its entries
    auto fetch_kept = [&](int run) {
#pragma unroll
        for (int k = 0; k < LOOK; ++k) {
            const int at = tid + k * kMoveThreads, r = run * RUN + at;
            j1[k] = at < RUN && r < p.budget ? kept[r] : -1;
        }
    };
    auto fetch_entries = [&](int run) {
#pragma unroll
        for (int k = 0; k < LOOK; ++k) {
            j2[k] = j1[k];
            if (j2[k] >= 0) {
                ps[k] = __ldg(table + block_of(p, j2[k]));
                pd[k] = __ldg(table + block_of(p, run * RUN + tid + k * kMoveThreads));
            }
        }
    };
    auto put_slots = [&](int run) {
#pragma unroll
        for (int k = 0; k < LOOK; ++k) {
            const int at = tid + k * kMoveThreads;
            if (at < RUN) {
                const int r = run * RUN + at;
                int f = -1, t = -1;
                if (j2[k] >= 0 && j2[k] != r) {
                    f = slot_of(p, ps[k], j2[k], report);
                    t = slot_of(p, pd[k], r, report);
                }
                src[run & 1][at] = t < 0 ? -1 : f;
                dst[run % (S + 1)][at] = f < 0 ? -1 : t;
            }
        }
    };
    auto issue = [&](int run) {  // reads of a run
        if (v < nv) {
#pragma unroll
            for (int k = 0; k < RUN / kStep; ++k) {
                const int row = rr + k * kStep;
                const int f = src[run & 1][row];
                if (f >= 0)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     smem_u32(ring + (((run % S) * RUN + row) * VS + v) * 16)),
                                 "l"(pool + static_cast<int64_t>(f) * p.row_bytes + v * 16)
                                 : "memory");
            }
        }
    };
    fetch_kept(0);
    fetch_entries(0);
    fetch_kept(1);
    for (int run = 0; run < runs + S - 1; ++run) {
        // reads of `run`; writes of run - (S - 1)
        if (run < runs) {
            put_slots(run);
            fetch_entries(run + 1);
            fetch_kept(run + 2);
        }
        __syncthreads();  // the slots are there; the ring's run - S has been written out
        if (run < runs)
            issue(run);
        asm volatile("cp.async.commit_group;" ::: "memory");
        const int done = run - (S - 1);
        if (done >= 0) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
            __syncthreads();  // run `done` has been read by every thread, and all before it
            if (v < nv) {
#pragma unroll
                for (int k = 0; k < RUN / kStep; ++k) {
                    const int row = rr + k * kStep;
                    const int t = dst[done % (S + 1)][row];
                    if (t >= 0)
                        *reinterpret_cast<uint4*>(pool + static_cast<int64_t>(t) * p.row_bytes + v * 16) =
                            *reinterpret_cast<const uint4*>(ring + (((done % S) * RUN + row) * VS + v) * 16);
                }
            }
        }
    }
}

// grid (items of a sequence's rows * 2, B): whole rows of K or V.
__global__ void __launch_bounds__(kMoveThreads) pa_evict_gather(const __grid_constant__ EvictParams p)
{
    extern __shared__ __align__(16) unsigned char rows[];
    __shared__ int src[kMoveRows], dst[kMoveRows];
    const int tid = threadIdx.x;
    const int kv = blockIdx.x & 1, b = blockIdx.y;
    const int r0 = (blockIdx.x >> 1) * p.rows_item;
    const int m = min(clamped_len(p, b, false), p.budget);
    const int nr = min(p.rows_item, m - r0);
    grid_dependency_wait();  // the kept list
    if (nr <= 0)
        return;
    const int32_t* kept = p.kept + static_cast<int64_t>(b) * p.budget;
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.maxb;
    const int32_t* to = p.dst + static_cast<int64_t>(b) * p.dst_maxb;
    for (int i = tid; i < nr; i += kMoveThreads) {
        const int r = r0 + i;
        const int pd = __ldg(to + block_of(p, r)), j = kept[r];
        const int s = slot_of(p, __ldg(table + block_of(p, j)), j, kv == 0), d = slot_of(p, pd, r, kv == 0);
        src[i] = d < 0 ? -1 : s;
        dst[i] = s < 0 ? -1 : d;
    }
    __syncthreads();
    const int vpr = p.row_bytes >> 4;
    unsigned char* pool = p.pool[kv];
    const int total = nr * vpr;
    for (int i = tid; i < total; i += kMoveThreads) {
        const int r = i / vpr, v = i - r * vpr;
        if (src[r] >= 0)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(rows + static_cast<size_t>(i) * 16)),
                         "l"(pool + static_cast<int64_t>(src[r]) * p.row_bytes + v * 16)
                         : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // every thread writes what it has read itself
    for (int i = tid; i < total; i += kMoveThreads) {
        const int r = i / vpr, v = i - r * vpr;
        if (dst[r] >= 0)
            *reinterpret_cast<uint4*>(pool + static_cast<int64_t>(dst[r]) * p.row_bytes + v * 16) =
                *reinterpret_cast<const uint4*>(rows + static_cast<size_t>(i) * 16);
    }
}

int rows_per_item(int row_bytes)
{
    int r = kMoveBytes / row_bytes;
    return r < 1 ? 1 : r > kMoveRows ? kMoveRows : r;
}

bool a4(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 3) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Sizes that both entry points refuse; row bytes and capacity on success.
int evict_sizes(int B, int KV, int D, int max_blocks, int BLOCK, int budget, int dtype, int* row_bytes, int* cap)
{
    if (B < 0 || KV < 1 || D < 1 || max_blocks < 1 || BLOCK < 1 || budget < 1 || budget >= (1 << 30) ||
        static_cast<long long>(max_blocks) * BLOCK >= (1ll << 30))
        return PA_ERR_BAD_DIMS;
    if ((dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16) || B > kMaxBatch)
        return PA_ERR_UNSUPPORTED;
    const long long rb = static_cast<long long>(KV) * D * (dtype == PA_F32 ? 4 : 2);
    if (rb % 16 != 0 || rb > kMaxRowBytes)
        return PA_ERR_UNSUPPORTED;
    *row_bytes = static_cast<int>(rb);
    *cap = max_blocks * BLOCK;
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_cache_evict(void* k_cache, void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                              const float* weights, int32_t* new_lens, int32_t* kept, float* weights_out, int B, int KV,
                              int D, int BLOCK, const pa_evict_opts* opts, void* stream)
{
    if (!opts)
        return PA_ERR_NULL_POINTER;
    const pa_evict_opts& o = *opts;
    int rb = 0, cap = 0;
    const int rc = evict_sizes(B, KV, D, o.max_blocks, BLOCK, o.budget, o.dtype, &rb, &cap);
    if (rc != PA_OK)
        return rc;
    const int m = o.budget < cap ? o.budget : cap;
    if (o.num_blocks < 1 || static_cast<long long>(o.num_blocks) * BLOCK >= (1ll << 31) || o.keep_first < 0 ||
        o.keep_last < 0 || static_cast<long long>(o.keep_first) + o.keep_last > o.budget ||
        (o.dst_table && (o.dst_table == block_table || o.dst_max_blocks < 1 || static_cast<long long>(o.dst_max_blocks) * BLOCK < m)))
        return PA_ERR_BAD_DIMS;
    if (B == 0)
        return PA_OK;
    if (!k_cache || !v_cache || !block_table || !seq_lens || !weights || !new_lens || !kept || !weights_out)
        return PA_ERR_NULL_POINTER;
    if ((reinterpret_cast<uintptr_t>(k_cache) & 15) || (reinterpret_cast<uintptr_t>(v_cache) & 15) || !a4(block_table) ||
        !a4(seq_lens) || !a4(weights) || !a4(new_lens) || !a4(kept) || !a4(weights_out) || !a4(o.dst_table))
        return PA_ERR_ALIGNMENT;
    const size_t pool = static_cast<size_t>(o.num_blocks) * BLOCK * rb;
    const struct {
        const void* x;
        size_t bytes;
        bool written;
    } all[] = {{k_cache, pool, true},
               {v_cache, pool, true},
               {new_lens, static_cast<size_t>(B) * 4, true},
               {kept, static_cast<size_t>(B) * o.budget * 4, true},
               {weights_out, static_cast<size_t>(B) * cap * 4, true},
               {block_table, static_cast<size_t>(B) * o.max_blocks * 4, false},
               {seq_lens, static_cast<size_t>(B) * 4, false},
               {weights, static_cast<size_t>(B) * cap * 4, false},
               {o.dst_table, o.dst_table ? static_cast<size_t>(B) * o.dst_max_blocks * 4 : 0, false}};
    for (int i = 0; i < 9; ++i)
        for (int j = 0; j < i; ++j)
            if ((all[i].written || all[j].written) && overlap(all[i].x, all[i].bytes, all[j].x, all[j].bytes))
                return PA_ERR_BAD_DIMS;

    EvictParams p{};
    p.pool[0] = static_cast<unsigned char*>(k_cache);
    p.pool[1] = static_cast<unsigned char*>(v_cache);
    p.table = block_table;
    p.dst = o.dst_table ? o.dst_table : block_table;
    p.lens = seq_lens;
    p.weights = weights;
    p.new_lens = new_lens;
    p.kept = kept;
    p.weights_out = weights_out;
    p.status = o.status;
    p.B = B;
    p.BLOCK = BLOCK;
    p.maxb = o.max_blocks;
    p.dst_maxb = o.dst_table ? o.dst_max_blocks : o.max_blocks;
    p.num_blocks = o.num_blocks;
    p.budget = o.budget;
    p.first = o.keep_first;
    p.last = o.keep_last;
    p.in_place = o.dst_table ? 0 : 1;
    p.cap = cap;
    p.row_bytes = rb;
    p.rows_item = rows_per_item(rb);
    p.shift = -1;
    for (int e = 0; e < 30; ++e)
        if (1 << e == BLOCK)
            p.shift = e;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // short sequences: a CTA of 256 threads holds 2048 weights in registers;
    // else 1024 threads and 8192, and a cluster of up to 8 of them (16 weights a
    // thread and half the CTAs: 28.9 against 26.6 us for a call of 32768 tokens,
    // 37.2 against 36.0 for 64 of up to 16384; twice the CTAs: 28.7 and 39.1)
    const bool small = cap <= 2048;
    const int C = cap <= 8192 ? 1 : cap <= 16384 ? 2 : cap <= 32768 ? 4 : 8;
    const void* sel = small    ? reinterpret_cast<const void*>(pa_evict_select<256, 1>)
                      : C == 1 ? reinterpret_cast<const void*>(pa_evict_select<1024, 1>)
                      : C == 2 ? reinterpret_cast<const void*>(pa_evict_select<1024, 2>)
                      : C == 4 ? reinterpret_cast<const void*>(pa_evict_select<1024, 4>)
                               : reinterpret_cast<const void*>(pa_evict_select<1024, 8>);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(B) * C);
    cfg.blockDim = dim3(small ? 256 : 1024);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 1 : 0;
    void* args[1] = {&p};
    // In place, six runs of 16 KB in flight per CTA; slices of 128 bytes, or of 64
    // or 32 (with two or four times the rows in a run) where wider ones would leave
    // SMs idle.  Calls with 128-, 64- and 32-byte slices: one sequence, 8192 rows
    // of 2 KB 63.5 / 41.0 / 34.8 us; one, 19569 of 512 bytes 129.0 / 72.0 / 57.4;
    // four, 4096 of 2 KB 43.8 / 38.4 / 56.1; sixteen, 2048 of 2 KB 57.7 / 62.9 /
    // 97.4; 64 ragged ones 36.9 / 39.3 / 58.2.
    const void* move;
    size_t smem;
    dim3 grid;
    if (p.in_place) {
        int vs = 8;
        while (vs > 2 && 2ll * B * ((rb + 16 * vs - 1) / (16 * vs)) < 152)
            vs /= 2;
        p.slices = (rb + 16 * vs - 1) / (16 * vs);
        grid = dim3(2u * p.slices, static_cast<unsigned>(B));
        move = vs == 8   ? reinterpret_cast<const void*>(pa_evict_shift<8, kRuns>)
               : vs == 4 ? reinterpret_cast<const void*>(pa_evict_shift<4, kRuns>)
                         : reinterpret_cast<const void*>(pa_evict_shift<2, kRuns>);
        smem = kRuns * kRunBytes;
    } else {
        grid = dim3(2u * ((m + p.rows_item - 1) / p.rows_item), static_cast<unsigned>(B));
        move = reinterpret_cast<const void*>(pa_evict_gather);
        smem = static_cast<size_t>(p.rows_item) * rb;
    }
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(move, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return PA_ERR_CUDA;
    if (cudaLaunchKernelExC(&cfg, sel, args) != cudaSuccess)
        return PA_ERR_CUDA;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelExC(&cfg, move, args) != cudaSuccess)
        return PA_ERR_CUDA;
    count_launches(2);
    return PA_OK;
}
