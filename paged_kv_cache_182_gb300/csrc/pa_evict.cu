// pa_evict.cu -- cache eviction by accumulated attention weight
// (include/pa_evict.h).
//
// Two kernels:
//
// pa_evict_select -- one cluster of CTAs per sequence finds the weight of the
//   last token that is kept (a radix select: histograms of 11, 11 and 10 bits
//   of the weights' ordered bit patterns, summed over the cluster through
//   distributed shared memory; it ends early once the chosen bin is taken
//   whole), then writes the kept indices and weights in token order: each
//   warp owns a contiguous range of tokens, the ranges' counts are summed
//   over warps and CTAs, and ballots place the tokens inside a range.
//
// pa_evict_move -- the rows.  kept[r] >= r, so a destination slot is either
//   unmoved or the source of a lower or equal rank: an item (sequence, run of
//   ranks, K or V) reads all of its rows into shared memory, raises its flag,
//   and writes them once the items whose sources it overwrites have raised
//   theirs.  Those items have lower ranks, items are dealt in rank order by a
//   ticket, and reading never waits, so every wait ends.  Into fresh blocks
//   there is nothing to wait for.
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

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 32768;   // rows of one item, at most (one row when longer)
constexpr int kMoveRows = 256;      // rows of one item, at most
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
    int* ticket;             // workspace: ticket, then the items' flags
    int* flags;
    int* status;
    unsigned long long wait_ns;
    int B, BLOCK, maxb, dst_maxb, num_blocks, budget, first, last, in_place;
    int cap;                 // max_blocks * BLOCK
    int row_bytes;           // KV * D * element bytes
    int rows_item, chunks;   // ranks per item, items per sequence and pool
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

// The 32-bit word at the same shared-memory place in CTA `rank` of the cluster.
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

template <int C>
__global__ void __launch_bounds__(kSelThreads) pa_evict_select(const __grid_constant__ EvictParams p)
{
    __shared__ uint32_t hist[2][kBins];
    __shared__ uint32_t wsum[kSelWarps];
    __shared__ uint32_t pick[3];               // chosen digit, still needed in it, its count
    __shared__ uint32_t cnt[kSelWarps][2];     // tokens taken outright / at the threshold, by warp
    __shared__ uint32_t tot[2];                // the same of the CTA
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = C == 1 ? 0 : static_cast<int>(cluster_rank());
    const int b = blockIdx.x / C;
    const int step = C * kSelThreads, me = rank * kSelThreads + tid;
    const int n = clamped_len(p, b, me == 0);
    const float* w = p.weights + static_cast<int64_t>(b) * p.cap;
    float* wo = p.weights_out + static_cast<int64_t>(b) * p.cap;
    int32_t* kept = p.kept + static_cast<int64_t>(b) * p.budget;

    if (p.in_place) {
        // the move's flags and ticket start at zero
        for (int i = me; i < 2 * p.chunks; i += step)
            p.flags[static_cast<int64_t>(b) * 2 * p.chunks + i] = 0;
        if (b == 0 && me == 0)
            *p.ticket = 0;
    }
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
    // this CTA's and warp's tokens: contiguous ranges in token order
    const int per = (hi - lo + C - 1) / C;
    const int c0 = min(lo + rank * per, hi), c1 = min(c0 + per, hi);
    const int sub = ((c1 - c0 + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int w0 = min(c0 + warp * sub, c1), w1 = min(w0 + sub, c1);

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
        for (int j0 = w0; j0 < w1; j0 += 32) {
            const int j = j0 + lane;
            const uint32_t key = j < w1 ? order_of(__ldg(w + j)) : 0u;
            const bool in = j < w1 && (key & mask) == prefix;
            // one addition per distinct digit of the warp: accumulated weights
            // crowd into few digits
            const uint32_t d = in ? (key >> shift) & digits : 0xffffffffu;
            const uint32_t same = __match_any_sync(kAll32, d);
            if (in && (same & ((1u << lane) - 1)) == 0)
                atomicAdd(&h[d], static_cast<uint32_t>(__popc(same)));
        }
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
        // four bins a thread, from the top
        uint32_t v[4], sum = 0;
        const int top = kBins - 1 - 4 * tid;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = 0;
            if (C == 1) {
                v[i] = h[top - i];
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    v[i] += cluster_load(&h[top - i], c);
            }
            sum += v[i];
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
        uint32_t before = incl - sum;
        for (int i = 0; i < warp; ++i)
            before += wsum[i];
        if (before < k && k <= before + sum) {
            uint32_t at = before;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
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
    for (int j = w0 + lane; j < w1; j += 32) {
        const uint32_t key = order_of(__ldg(w + j));
        ge += key >= t_ge;
        eq += n_eq > 0 && key == t_eq;
    }
    ge = __reduce_add_sync(kAll32, ge);
    eq = __reduce_add_sync(kAll32, eq);
    if (lane == 0) {
        cnt[warp][0] = ge;
        cnt[warp][1] = eq;
    }
    __syncthreads();
    if (tid < 2) {
        uint32_t s = 0;
        for (int i = 0; i < kSelWarps; ++i)
            s += cnt[i][tid];
        tot[tid] = s;
    }
    if (C > 1)
        cluster_sync();
    uint32_t bge = 0, beq = 0;
    for (int c = 0; c < rank; ++c) {
        bge += cluster_load(&tot[0], c);
        beq += cluster_load(&tot[1], c);
    }
    for (int i = 0; i < warp; ++i) {
        bge += cnt[i][0];
        beq += cnt[i][1];
    }
    const uint32_t below = (1u << lane) - 1;
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int j = j0 + lane;
        const float x = j < w1 ? __ldg(w + j) : 0.f;
        const uint32_t key = order_of(x);
        const bool is_ge = j < w1 && key >= t_ge, is_eq = j < w1 && n_eq > 0 && key == t_eq;
        const uint32_t mg = __ballot_sync(kAll32, is_ge), me_ = __ballot_sync(kAll32, is_eq);
        const uint32_t g = bge + __popc(mg & below), e = beq + __popc(me_ & below);
        if (is_ge || (is_eq && e < n_eq)) {
            const int r = p.first + static_cast<int>(g + min(e, n_eq));
            kept[r] = j;
            wo[r] = x;
        }
        bge += __popc(mg);
        beq += __popc(me_);
    }
    if (C > 1)
        cluster_sync();  // the others have read this CTA's shared memory
}

__device__ __forceinline__ int load_acquire(const int* p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void store_release(int* p, int v)
{
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kMoveThreads) pa_evict_move(const __grid_constant__ EvictParams p)
{
    extern __shared__ __align__(16) unsigned char rows[];
    __shared__ int s_item;
    __shared__ int src[kMoveRows], dst[kMoveRows];
    const int tid = threadIdx.x;
    int item = blockIdx.x;
    if (p.in_place) {
        if (tid == 0)
            s_item = atomicAdd(p.ticket, 1);
        __syncthreads();
        item = s_item;
    }
    // ranks slowest: an item's predecessors were dealt long before it
    const int kv = item & 1;
    const int c = (item >> 1) / p.B, b = (item >> 1) - c * p.B;
    const int n = clamped_len(p, b, false);
    const int m = min(n, p.budget);
    const int r0 = c * p.rows_item;
    if (r0 >= m || (p.in_place && n <= p.budget))
        return;  // nothing moves (and nothing is waited for: no source lies here)
    const int nr = min(p.rows_item, m - r0);
    const int32_t* kept = p.kept + static_cast<int64_t>(b) * p.budget;
    int* flag = p.flags + static_cast<int64_t>(b) * 2 * p.chunks + kv;
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.maxb;
    const int32_t* to = p.dst + static_cast<int64_t>(b) * p.dst_maxb;
    for (int i = tid; i < nr; i += kMoveThreads) {
        const int r = r0 + i, j = kept[r];
        int s = -1, d = -1;
        if (!p.in_place || j != r) {
            const int ps = table[j / p.BLOCK], pd = to[r / p.BLOCK];
            if (ps < 0 || ps >= p.num_blocks || pd < 0 || pd >= p.num_blocks) {
                if (p.status)
                    atomicOr(p.status, PA_STATUS_BAD_BLOCK);
            } else {
                s = ps * p.BLOCK + j % p.BLOCK;
                d = pd * p.BLOCK + r % p.BLOCK;
            }
        }
        src[i] = s;
        dst[i] = d;
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
    __syncthreads();
    if (p.in_place) {
        if (tid == 0) {
            __threadfence();
            store_release(flag + 2 * c, 1);
            // ranks whose sources are this item's destinations r0 .. r0 + nr - 1:
            // kept ascends and kept[r] >= r, so they lie in [lo, r0 + nr)
            int lo = 0, up = r0;  // first rank with kept >= r0
            while (lo < up) {
                const int mid = (lo + up) >> 1;
                if (kept[mid] >= r0)
                    up = mid;
                else
                    lo = mid + 1;
            }
            bool ok = true;
            const uint64_t start = global_timer_ns();
            for (int k = lo / p.rows_item; k < c && ok; ++k)
                while (load_acquire(flag + 2 * k) == 0)
                    if (global_timer_ns() - start > p.wait_ns) {
                        ok = false;
                        break;
                    }
            if (!ok && p.status)
                atomicOr(p.status, PA_STATUS_TIMEOUT);
            s_item = ok;
        }
        __syncthreads();
        if (!s_item)
            return;
    }
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

// ticket (256 bytes) | flags [B][chunks][2]
size_t evict_workspace(int B, int row_bytes, int cap, int budget)
{
    const int m = budget < cap ? budget : cap;
    const int chunks = (m + rows_per_item(row_bytes) - 1) / rows_per_item(row_bytes);
    return 256 + static_cast<size_t>(B) * 2 * chunks * sizeof(int);
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

extern "C" size_t pa_cache_evict_workspace_bytes(int B, int KV, int D, int max_blocks, int BLOCK, int budget, int dtype)
{
    int rb, cap;
    if (evict_sizes(B, KV, D, max_blocks, BLOCK, budget, dtype, &rb, &cap) != PA_OK || B == 0)
        return 0;
    return evict_workspace(B, rb, cap, budget);
}

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
        (o.dst_table && (o.dst_max_blocks < 1 || static_cast<long long>(o.dst_max_blocks) * BLOCK < m)))
        return PA_ERR_BAD_DIMS;
    if (B == 0)
        return PA_OK;
    if (!k_cache || !v_cache || !block_table || !seq_lens || !weights || !new_lens || !kept || !weights_out)
        return PA_ERR_NULL_POINTER;
    if ((reinterpret_cast<uintptr_t>(k_cache) & 15) || (reinterpret_cast<uintptr_t>(v_cache) & 15) || !a4(block_table) ||
        !a4(seq_lens) || !a4(weights) || !a4(new_lens) || !a4(kept) || !a4(weights_out) || !a4(o.dst_table))
        return PA_ERR_ALIGNMENT;
    const size_t need = evict_workspace(B, rb, cap, o.budget);
    if (!o.workspace || o.workspace_bytes < need)
        return PA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(o.workspace) & 255)
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
               {o.workspace, need, true},
               {block_table, static_cast<size_t>(B) * o.max_blocks * 4, false},
               {seq_lens, static_cast<size_t>(B) * 4, false},
               {weights, static_cast<size_t>(B) * cap * 4, false},
               {o.dst_table, o.dst_table ? static_cast<size_t>(B) * o.dst_max_blocks * 4 : 0, false}};
    for (int i = 0; i < 10; ++i)
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
    p.ticket = static_cast<int*>(o.workspace);
    p.flags = p.ticket + 64;
    p.status = o.status;
    p.wait_ns = o.wait_limit_ns ? o.wait_limit_ns : kWaitLimitNs;
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
    p.chunks = (m + p.rows_item - 1) / p.rows_item;
    const long long items = 2ll * p.chunks * B;
    if (items >= (1ll << 31))
        return PA_ERR_BAD_DIMS;
    const size_t smem = static_cast<size_t>(p.rows_item) * rb;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // one CTA of a cluster per 4096 tokens of capacity, at most 8
    const int C = cap <= 4096 ? 1 : cap <= 16384 ? 4 : 8;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(B) * C);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[1] = {&p};
    const void* sel = C == 1   ? reinterpret_cast<const void*>(pa_evict_select<1>)
                      : C == 4 ? reinterpret_cast<const void*>(pa_evict_select<4>)
                               : reinterpret_cast<const void*>(pa_evict_select<8>);
    const void* move = reinterpret_cast<const void*>(pa_evict_move);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(move, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return PA_ERR_CUDA;
    if (cudaLaunchKernelExC(&cfg, sel, args) != cudaSuccess)
        return PA_ERR_CUDA;
    pa_evict_move<<<static_cast<unsigned>(items), kMoveThreads, smem, st>>>(p);
    if (cudaGetLastError() != cudaSuccess)
        return PA_ERR_CUDA;
    count_launches(2);
    return PA_OK;
}
