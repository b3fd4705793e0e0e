// pa_blocks.cu -- block tables and slots of a serving step (include/pa_blocks.h).
//
// One kernel, no CTA waits for another: every CTA sums up what all sequences
// give back and take (two prefix sums over at most 4096 sequences), so that each
// of them knows which block any place of any table gets: the i-th block taken is
// entry free_count + returned - 1 - i of the stack with the returned blocks on
// top, a free block below free_count or a table entry that its sequence gives
// back above.  Nothing that a CTA reads is written in the call: a sequence gives
// back or takes, never both, and blocks are either taken off the old stack or
// added to it.  The work (entries taken, entries put back, slots) is dealt to
// the CTAs in equal ranges.
//
// What bounds it: latency.  64 sequences of a token each take 4.4 us: a launch,
// lengths, two sums, the stack's top, the table.  500 sequences of up to 2000 rows
// (8 MB of slots and positions, a floor of 1.3 us) take 9.4: every CTA's own sums,
// then four slots a thread and turn (one at a time: 12).  The grid is sized by the
// slots alone: 39,000 blocks given back in a step of 431 rows take one CTA 52 us.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_blocks.h"
#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_ptx.cuh"
#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;

struct PlanParams {
    int32_t* table;
    const int32_t* lens;
    int32_t* stack;
    const int32_t* count;
    int32_t* new_lens;
    int32_t* new_count;
    int32_t* slots;
    int32_t* positions;
    int32_t* kept;
    int32_t* granted;
    const int32_t* add;
    const int32_t* keep;
    const int32_t* starts;
    int* status;
    int B, N, BLOCK, maxb, num_blocks, cap, shift;
    int vectors;  // rows of slots and positions are whole 16-byte vectors
};

struct Sequence {
    int n, keep, add, have, need;
};

__device__ __forceinline__ int div_block(const PlanParams& p, int x) { return p.shift >= 0 ? x >> p.shift : x / p.BLOCK; }

// Blocks of x tokens (x + BLOCK may pass 2^31, not 2^32).
__device__ __forceinline__ int blocks_of(const PlanParams& p, int x)
{
    const uint32_t up = static_cast<uint32_t>(x) + static_cast<uint32_t>(p.BLOCK) - 1u;
    return static_cast<int>(p.shift >= 0 ? up >> p.shift : up / static_cast<uint32_t>(p.BLOCK));
}

__device__ __forceinline__ Sequence sequence(const PlanParams& p, int b, int& bad)
{
    Sequence s;
    const int n = __ldg(p.lens + b), k = p.keep ? __ldg(p.keep + b) : INT_MAX, a = p.add ? __ldg(p.add + b) : p.N;
    s.n = min(max(n, 0), p.cap);
    s.keep = p.keep ? min(max(k, 0), s.n) : s.n;
    s.add = min(max(a, 0), p.N);
    if (s.n != n || (p.keep && s.keep != k) || s.add != a)
        bad |= PA_STATUS_BAD_LENGTH;
    s.have = blocks_of(p, s.n);
    s.need = blocks_of(p, s.keep + s.add);
    return s;
}

// Exclusive sums of x and y over the CTA's threads; the totals in tx, ty.
__device__ __forceinline__ void exclusive_sums(int& x, int& y, int& tx, int& ty, int2* part)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int ux = __shfl_up_sync(kFullWarp, ix, o), uy = __shfl_up_sync(kFullWarp, iy, o);
        if (lane >= o) {
            ix += ux;
            iy += uy;
        }
    }
    if (lane == 31)
        part[warp] = make_int2(ix, iy);
    __syncthreads();
    const int2 w = lane < kPlanWarps ? part[lane] : make_int2(0, 0);
    tx = __reduce_add_sync(kFullWarp, w.x);
    ty = __reduce_add_sync(kFullWarp, w.y);
    const int bx = __reduce_add_sync(kFullWarp, lane < warp ? w.x : 0), by = __reduce_add_sync(kFullWarp, lane < warp ? w.y : 0);
    x = bx + ix - x;
    y = by + iy - y;
    __syncthreads();
}

// Last b with at[b] <= i (at is not decreasing, at[0] = 0).
__device__ __forceinline__ int owner(const int* at, int B, int i)
{
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) pa_plan_kernel(const __grid_constant__ PlanParams p)
{
    extern __shared__ __align__(8) int smem[];
    int* taken = smem;             // [B] blocks taken by the sequences before
    int* given = smem + p.B;       // [B] blocks given back by the sequences before
    int2* span = reinterpret_cast<int2*>(smem + 2 * p.B);  // [B] (first new token, rows; -1 refused)
    int* held = reinterpret_cast<int*>(span + p.B);        // [B] blocks it had
    __shared__ int2 part[kPlanWarps];
    grid_begin();
    const int tid = threadIdx.x, B = p.B;
    const bool lead = blockIdx.x == 0;
    const int per = (B + kPlanThreads - 1) / kPlanThreads;  // consecutive sequences per thread
    const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
    int bad = 0, back = 0, more = 0;
    for (int b = b0; b < b1; ++b) {
        const Sequence s = sequence(p, b, bad);
        back += max(s.have - s.need, 0);
        more += s.need <= p.maxb ? max(s.need - s.have, 0) : 0;
    }
    int given_all, wanted_all;
    exclusive_sums(back, more, given_all, wanted_all, part);
    int count = __ldg(p.count);
    if (count < 0 || count > p.num_blocks) {
        bad |= PA_STATUS_BAD_LENGTH;
        count = min(max(count, 0), p.num_blocks);
    }
    // (a stack that overflows is the caller's mistake: what does not fit is dropped)
    const int room = p.num_blocks - count;
    const int put = min(given_all, room);
    if (put < given_all)
        bad |= PA_STATUS_BAD_LENGTH;
    const int there = count + put;
    int granted_more = 0;
    for (int b = b0; b < b1; ++b) {
        int ignore = 0;
        const Sequence s = sequence(p, b, ignore);
        const int m = s.need <= p.maxb ? max(s.need - s.have, 0) : 0;
        const bool fits = s.need <= p.maxb, ok = fits && (m == 0 || more <= there - m);
        given[b] = back;
        taken[b] = min(more, there);
        span[b] = make_int2(s.keep, ok ? s.add : -1);
        held[b] = s.have;
        back += max(s.have - s.need, 0);
        more += m;
        if (ok && m > 0)
            granted_more = more;
        if (!ok)
            bad |= fits ? PA_STATUS_NO_BLOCKS : PA_STATUS_BAD_LENGTH;
        if (lead) {
            p.new_lens[b] = ok ? s.keep + s.add : s.n;
            if (p.kept)
                p.kept[b] = ok ? s.keep : s.n;
            if (p.granted)
                p.granted[b] = ok ? s.add : 0;
        }
    }
    // blocks taken in all: the largest sum that was granted
    granted_more = __reduce_max_sync(kFullWarp, granted_more);
    if ((tid & 31) == 0)
        part[tid >> 5].x = granted_more;
    __syncthreads();
    const int taken_all = __reduce_max_sync(kFullWarp, (tid & 31) < kPlanWarps ? part[tid & 31].x : 0);
    const int left = there - taken_all;
    if (lead && tid == 0)
        *p.new_count = left;
    if (lead && bad)
        q8_report(p.status, bad);

    // block i from the bottom of the stack with the returned ones on top
    auto entry = [&](int at) -> int {
        if (at < count)
            return p.stack[at];
        const int i = at - count, b = owner(given, B, i);
        const int need = blocks_of(p, span[b].x + max(span[b].y, 0));
        return p.table[static_cast<int64_t>(b) * p.maxb + need + i - given[b]];
    };
    const int step = gridDim.x * kPlanThreads, me = blockIdx.x * kPlanThreads + tid;
    for (int i = me; i < taken_all; i += step) {
        const int b = owner(taken, B, i);
        const int phys = entry(there - 1 - i);
        if (phys < 0 || phys >= p.num_blocks)
            q8_report(p.status, PA_STATUS_BAD_BLOCK);
        p.table[static_cast<int64_t>(b) * p.maxb + held[b] + i - taken[b]] = phys;
    }
    for (int at = count + me; at < left; at += step)
        p.stack[at] = entry(at);
    // slots, four rows of a sequence at a time
    const uint32_t quads = (static_cast<uint32_t>(p.N) + 3) / 4, total = static_cast<uint32_t>(B) * quads;
    for (uint32_t x = me; x < total; x += step) {
        const uint32_t b = x / quads;
        const int j0 = static_cast<int>(x - b * quads) * 4;
        const int2 s = span[b];
        int slot[4] = {-1, -1, -1, -1}, pos[4] = {-1, -1, -1, -1};
        if (j0 < s.y) {
            const int had = held[b], start = p.starts ? __ldg(p.starts + b) : s.x;
            int blk = -1, base = -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = s.x + j0 + k;
                if (j0 + k >= s.y)
                    break;
                if (div_block(p, t) != blk) {
                    blk = div_block(p, t);
                    const int phys = blk < had ? p.table[static_cast<int64_t>(b) * p.maxb + blk] : entry(there - 1 - (taken[b] + blk - had));
                    base = phys < 0 || phys >= p.num_blocks ? INT_MIN : (phys - blk) * p.BLOCK;
                }
                slot[k] = base == INT_MIN ? -1 : base + t;
                pos[k] = start + j0 + k;
            }
        }
        const int64_t at = static_cast<int64_t>(b) * p.N + j0;
        if (p.vectors) {
            *reinterpret_cast<int4*>(p.slots + at) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            if (p.positions)
                *reinterpret_cast<int4*>(p.positions + at) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j0 + k < p.N) {
                    p.slots[at + k] = slot[k];
                    if (p.positions)
                        p.positions[at + k] = pos[k];
                }
        }
    }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_plan_blocks(int32_t* block_table, const int32_t* seq_lens, int32_t* free_blocks, const int32_t* free_count,
                              int32_t* new_lens, int32_t* new_free_count, int32_t* slots, int B, int N, int BLOCK,
                              const pa_blocks_opts* opts, void* stream)
{
    if (!opts)
        return PA_ERR_NULL_POINTER;
    const pa_blocks_opts& o = *opts;
    if (B < 0 || N < 0 || BLOCK < 1 || o.max_blocks < 1 || o.num_blocks < 1 ||
        static_cast<long long>(o.max_blocks) * BLOCK >= (1ll << 30) || static_cast<long long>(o.num_blocks) * BLOCK >= (1ll << 31) ||
        static_cast<long long>(B) * o.max_blocks >= (1ll << 31) || static_cast<long long>(B) * N >= (1ll << 31))
        return PA_ERR_BAD_DIMS;
    if (B > kMaxBatch || N > PA_MAX_PREFILL)
        return PA_ERR_UNSUPPORTED;
    if (!free_blocks || !free_count || !new_free_count ||
        (B > 0 && (!block_table || !seq_lens || !new_lens || (N > 0 && !slots))))
        return PA_ERR_NULL_POINTER;
    const void* all4[] = {block_table, seq_lens, free_blocks, free_count, new_lens, new_free_count, slots,
                          o.add,       o.keep,   o.starts,    o.positions, o.status, o.kept,         o.granted};
    for (const void* x : all4)
        if (!q8_a4(x))
            return PA_ERR_ALIGNMENT;
    const size_t b4 = static_cast<size_t>(B) * 4;
    const Q8Range r[] = {{block_table, b4 * o.max_blocks, true}, {free_blocks, static_cast<size_t>(o.num_blocks) * 4, true},
                         {new_lens, b4, true},                   {new_free_count, 4, true},
                         {slots, b4 * N, true},                  {o.positions, b4 * N, true},
                         {seq_lens, b4, false},                  {free_count, 4, false},
                         {o.add, b4, false},                     {o.keep, b4, false},
                         {o.starts, b4, false},                  {o.status, 4, true},
                         {o.kept, b4, true},                     {o.granted, b4, true}};
    if (q8_overlap(r, 14))
        return PA_ERR_BAD_DIMS;
    PlanParams p{};
    p.table = block_table;
    p.lens = seq_lens;
    p.stack = free_blocks;
    p.count = free_count;
    p.new_lens = new_lens;
    p.new_count = new_free_count;
    p.slots = slots;
    p.positions = N > 0 ? o.positions : nullptr;
    p.kept = o.kept;
    p.granted = o.granted;
    p.add = o.add;
    p.keep = o.keep;
    p.starts = o.starts;
    p.status = o.status;
    p.B = B;
    p.N = N;
    p.BLOCK = BLOCK;
    p.maxb = o.max_blocks;
    p.num_blocks = o.num_blocks;
    p.cap = o.max_blocks * BLOCK;
    p.shift = -1;
    for (int e = 0; e < 30; ++e)
        if (1 << e == BLOCK)
            p.shift = e;
    p.vectors = N % 4 == 0 && q8_a16(slots) && q8_a16(p.positions) ? 1 : 0;
    // a CTA for about 512 groups of four rows, and two per SM at most
    long long grid = (static_cast<long long>(B) * ((N + 3) / 4) + 511) / 512;
    grid = grid < 1 ? 1 : grid > 304 ? 304 : grid;
    const size_t smem = static_cast<size_t>(B) * 20;
    void* args[] = {&p};
    return q8_launch(reinterpret_cast<const void*>(pa_plan_kernel), dim3(static_cast<unsigned>(grid)), kPlanThreads, smem,
                     static_cast<cudaStream_t>(stream), args);
}
