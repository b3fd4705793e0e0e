// pa_q8_decode.cu -- attention over a cache in 8 bits, whole or over selected
// blocks (include/pa_q8.h).
//
// Work: segments (sequence, KV head, group of 8 NT query rows), each a run of
// tiles of 32 tokens.  Teams of up to four CTAs take neighbouring heads of the
// same tokens, whose cache lines lie together (24 to 64 uneven sequences, 89 MB: 29.6 us,
// one CTA a team 32.8).  A team takes a segment whole, an equal piece of one, or,
// where there are more segments than teams, a range of all segments' tiles laid end
// to end, in which every piece costs a charge besides its tiles (without charges
// 42 us for the uneven batch at the time, 25 instead of 20 for one long sequence; ranges
// alone, without whole segments and equal pieces, 24.9 instead of 20.1 for 64 MB of 24
// even sequences).  Of many short
// segments a warp takes whole ones by itself, and no states are joined.  The states of a
// segment cut between CTAs (maximum, sum, values) go to the workspace, and the last
// CTA to finish one joins them: about 4 us, which whole segments save (64 MB of 24
// even sequences 20 us, of 16, which are cut, 22).  A CTA starts the copies of its
// next piece before it joins its warps' states of the last.
//
// What bounds it: memory, at 6.3 TB/s while it streams (one sequence of 268 MB in
// 54 us, of 537 MB in 97); a call besides costs about 5.7 us before the first tiles are
// there (lengths, ranges, table, then copies that all begin at once) and 3 to 5 behind
// the last (67 MB of one sequence 20.6 us).  With 32 query rows a head it is the
// instructions: 1.3 a cycle on two warps a scheduler, tensor cores active 28 %
// (fp16, 31.7 us for 16 x 2048 tokens).
//
// Tiles: a warp streams its own tiles through a ring of shared memory with
// 16-byte asynchronous copies, whole lines of 128 bytes together (copies in the
// order of the fragments, four lines of 32 bytes at once, kept the L1's tags busy:
// 512 MB of one sequence 124 us instead of 101 at the time), swizzled so that the
// reads meet no bank twice:
//   S^T = K Q^T:   lane (g, t) has rows g and g + 8 of K, D / 4 channels in runs
//                  of 16; the channels' order is the same in Q's fragments;
//   O^T += V^T P^T: lane (g, t) has tokens 2t, 2t + 1, 2t + 8, 2t + 9 of V,
//                  channels D / 8 g ...: two tokens' codes interleaved are V^T's
//                  fragment.
// More than eight rows of 16 bits take the products' 16-row side instead, S = Q K^T
// and O += P V (16 x 2048 tokens, 32 rows a head: 27.8 -> 25.5 us, weights of one part).
// Codes become fp16 exactly (byte u = code + 128 under the exponent of 1024 is
// 1024 + u; less 1152).  Keys of 16-bit rows skip the subtraction: u by itself is a
// subnormal number, and 128 times the row's sum is taken off beforehand.  A query
// row is scaled by a power of two, its largest element to 2^11: a 16-bit row keeps its
// digits but for those below 2^-35 of its largest element (fp16's last subnormal);
// float32 rows are two fp16 parts.
//
// Scales: the key scale multiplies the score.  The value scale joins the
// exponent, t = s + log2(v_scale), so that weights times value scale come out of
// the exponential; the softmax's sum takes them back through 1 / v_scale.  The
// maximum subtracted is t's: fp16 weights are as exact as their share in the
// output.  A weight is two fp16 parts, 22 bits, so that fp16 and float32 outputs are
// off by their own rounding alone (one part: fp16 outputs 2.5e-4 to 2.8e-4 instead of
// 2.1e-4, and 3 to 5 % less time at eight rows, where memory bounds the call).  Only
// bfloat16 rows beyond eight a head take one part, 11 bits: their own rounding of 2^-8
// hides it (1.7e-3 either way), and the second part's products cost 26.4 -> 31.7 us at
// 32 rows.  Where value scales lie far from one, 2^(t - m) may be 0 in float32 for a
// key whose share in the sum, 2^(s - m), is not small beside the others': from the
// first scale beyond 2^+-32 on, a warp sums the latter by themselves (a second
// exponential per weight), and sums are scaled in two steps where 2^d alone is 0
// (scaled_sum).  Up to 2^96 no weight above 2^-36 of the row's largest is lost.  It is raised only when a score passes it by 2^8 (a vote instead of a
// reduction per tile; weights stay below 2^14).
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kTile = 32;                 // tokens of a tile: two MMA groups of 16
constexpr int kMaxEntries = 4096;         // prefix sums in shared memory
constexpr int kRecordRows = 304 * 32;     // query rows of all CTAs, at most
constexpr int kMaxCtas = kRecordRows / 8; // CTAs, at most (passes have 8 query rows or more)
constexpr int kChargeBytes = 32 << 13;    // a piece's start and end count for so many bytes of tiles on an SM
constexpr int kJoinBytes = 22 << 13;      // joining the pieces of a segment, besides (of 4, 11, 16 and 30 none is better)
constexpr int kMeta = 64;                 // bytes of a tile's scales and places
constexpr float kLift = 6.f, kSlack = 8.f;  // weights are 2^(t - m + 6), t - m <= 8
constexpr float kNear = 32.f;             // log2 of value scales that share a weight's exponential with the sum
constexpr int kNowhere = INT_MAX - 64;    // place of a part of a tile that has no block

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
    int* counters;     // [CTA] pieces done of the cut segment whose first piece the CTA has
    float2* part_ml;   // [CTA][2][8 NT] maximum, sum
    float* part_o;     // [CTA][2][8 NT][D]
    int* status;
    float scale;       // scale * log2(e)
    int B, H, KV, R, NQ, groups, shift, maxb, num_blocks, cap, budget, causal, dtype, entries, copies, lg_team;
};

__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds4(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds8(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) { mma_16816<false>(d, a, b0, b1); }

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// log2 of the hardware.
__device__ __forceinline__ float fast_log2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// l 2^d (d <= 0), also where 2^d by itself would be 0.
__device__ __forceinline__ float scaled_sum(float l, float d)
{
    float y = l * fast_exp2(fmaxf(d, -120.f));
    if (d < -120.f)
        y = (l > 3.402823466e38f ? 3.402823466e38f : l) * fast_exp2(-120.f) * fast_exp2(d + 120.f);
    return y;
}

// QP: fp16 parts of a query row (2: float32).  PW: fp16 parts of a weight.  HB: blocks
// a tile may touch (2; 4 where BLOCK is 8).  Query fragments stay in registers, or in
// shared memory where the accumulators of four groups of rows leave no room.
template <int D, int NT, int QP, int C, int PW>
struct Shape {
    static constexpr int kRows = 8 * NT, kSteps = D / 16;
    // more than eight rows of 16 bits: rows on the 16-row side of the products
    static constexpr bool kWide = NT >= 2 && QP == 1;
    static constexpr int kWarps = NT == 1 && QP == 1 ? 12 / C : 8, kThreads = kWarps * 32;
    static constexpr int kJoint = NT * QP == 4 && QP == 2 ? 1 : 2;  // MMA groups of a tile taken together
    static constexpr int kTileBytes = 2 * kTile * D, kStage = kTileBytes + kMeta;
    static constexpr int kStages = 2 * (D == 128 ? 1 : 2);
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kCharge = kChargeBytes / C / kTileBytes, kJoin = kJoinBytes / C / kTileBytes;  // in tiles
    // CTAs that stream at the memory's rate: one of 12 warps takes 64 GB/s, of 6 warps 34.5, of 4 23
    static constexpr int kFull = C == 1 ? 98 : C == 2 ? 182 : 274;
    // A warp's state in shared memory: steps of 16 + 4 floats, rows 4 (mod 32) floats
    // apart (wide: rows of D + 4, four floats together in an order of their own), so
    // that neither its writes nor its reads meet a bank twice
    static constexpr int kStateStep = 20, kStateRow = kWide ? D + 4 : kSteps * kStateStep + 4, kState = kRows * kStateRow * 4;
    static constexpr int kGroup = C == 3 ? 1 : 2;  // warps' states joined at once beside a ring in use
    static constexpr int kLastGroup = kRing >= kWarps * kState ? kWarps : kWarps / 2;  // ... and in the place of the ring
    static_assert(kRing >= kLastGroup * kState, "states fit");
    static constexpr int kQueryBytes = QP * kSteps * NT * 32 * 8;
};

template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v)
{
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = v;
    } else if constexpr (std::is_same_v<T, __half>) {
        *reinterpret_cast<uint2*>(p) = make_uint2(half2_bits(__floats2half2_rn(v.x, v.y)), half2_bits(__floats2half2_rn(v.z, v.w)));
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}

__device__ __forceinline__ void store_out(const DecodeParams& p, int64_t at, float4 v)
{
    if (p.dtype == PA_F32)
        store4(static_cast<float*>(p.out) + at, v);
    else if (p.dtype == PA_F16)
        store4(static_cast<__half*>(p.out) + at, v);
    else
        store4(static_cast<__nv_bfloat16*>(p.out) + at, v);
}

__device__ __forceinline__ void fma4(float4& a, float f, float4 v)
{
    a.x = fmaf(f, v.x, a.x);
    a.y = fmaf(f, v.y, a.y);
    a.z = fmaf(f, v.z, a.z);
    a.w = fmaf(f, v.w, a.w);
}

// A segment of which this CTA has left a record: its first team, its pieces (0:
// another CTA joins them), where its rows go.
struct OpenPiece {
    int first, pieces;
    int* counter;
    int64_t out;
    int rows;
};

// kMany: more segments than CTAs, so that a warp may take whole ones by itself.
template <int D, int NT, int QP, int HB, int C, int PW, bool kMany>
__global__ void __launch_bounds__(Shape<D, NT, QP, C, PW>::kThreads, C) pa_q8_decode_kernel(const __grid_constant__ DecodeParams p)
{
    using Sh = Shape<D, NT, QP, C, PW>;
    constexpr int kRows = Sh::kRows, kSteps = Sh::kSteps, kTileBytes = Sh::kTileBytes, kStage = Sh::kStage, S = Sh::kStages;
    constexpr int kWarps = Sh::kWarps, kThreads = Sh::kThreads;
    constexpr int kChunks = D / 64;  // 16-byte runs of a key row per lane
    constexpr bool kWide = Sh::kWide;
    // float16 has a code + 128 as a subnormal number, with no arithmetic: the sum of
    // the row's 128 is taken off the score beforehand.  (Keys only: the values'
    // weights have one sign, and their sum would swamp the output.)
    constexpr bool kSmall = QP == 1;
    constexpr float kUnit = kSmall ? 8192.f : 1.f;  // 2^13 of the 2^24 by the key scale, 2^11 by the row's factor: neither overflows
    constexpr int J = Sh::kJoint, kCharge = Sh::kCharge;
    extern __shared__ __align__(16) unsigned char smem[];  // ring | query fragments | states | prefix sums
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    // (by warp where each has a segment of its own)
    constexpr int kSets = kMany ? kWarps : 1;
    static_assert(!kMany || NT == 1);
    __shared__ float sm_f[kSets * kRows];  // of a row's scores: scale * log2(e) / the power of two
    __shared__ float sm_off[kSets * kRows];  // what a row's scores begin with (kSmall)
    __shared__ int sm_lim[kSets * kRows];  // keys that the row sees
    __shared__ OpenPiece sm_open[2];
    grid_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * S * kStage);
    // a copy takes kRowsCopy rows of D bytes, 16 bytes a lane, whole lines together;
    // the places of the 16-byte runs (and, at D = 64, the order of V's rows) are such
    // that the reads below meet no bank twice
    constexpr int kRuns = D / 16, kRowsCopy = 32 / kRuns;
    const int copy_run = lane % kRuns;
    const int copy_row = D == 128 ? lane / kRuns : (lane >> 2 & 3) * 2 + (lane >> 4);
    auto turn_of = [](int x) { return D == 128 ? 2 * x : (x >> 1) * 2; };  // order of a wide state's quads
    uint32_t copy_k, copy_v, read_k, read_v;
    if constexpr (D == 128) {
        copy_k = copy_row * 128 + (copy_run ^ (copy_row & 1) << 2) * 16;
        copy_v = copy_row * 128 + (copy_run ^ (copy_row >> 1 & 1) << 1) * 16;  // (rows 4 to 7 of 8: ^ 64)
        read_k = g * 128 + (t ^ (g & 1) << 2) * 16;
        read_v = 2 * t * 128 + (g ^ t << 1) * 16;
    } else {
        copy_k = copy_row * 64 + copy_run * 16;
        copy_v = (lane >> 2) * 64 + (copy_run ^ (lane >> 3 & 1) << 1) * 16;
        read_k = g * 64 + t * 16;
        read_v = t * 64 + (g ^ (t >> 1) << 2) * 8;
    }
    uint2* sm_q = reinterpret_cast<uint2*>(smem + Sh::kRing);  // [QP][step][group of rows][lane]
    int* prefix = reinterpret_cast<int*>(smem + Sh::kRing + Sh::kQueryBytes + Sh::kGroup * Sh::kState);

    // prefix sums of the tiles of the entries (sequences, or sequences and KV
    // heads where each has its own blocks), each with the charge of a piece
    int longest = 0;
    auto tiles_of = [&](int e) -> int {
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
        const int u = max(1, (tokens + kTile - 1) / kTile);
        longest = max(longest, u);
        return kCharge + u;
    };
    {
        int* sums = reinterpret_cast<int*>(&sm_m[0][0]);
        const int per = (p.entries + kThreads - 1) / kThreads;
        const int e0 = min(tid * per, p.entries), e1 = min(e0 + per, p.entries);
        int sum = 0;
        for (int e = e0; e < e1; ++e) {
            const int v = tiles_of(e);
            prefix[e] = v;
            sum += v;
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFullWarp, incl, o);
            if (lane >= o)
                incl += y;
        }
        const int most = __reduce_max_sync(kFullWarp, longest);
        if (lane == 31) {
            sums[warp] = incl;
            sums[kWarps + warp] = most;
        }
        __syncthreads();
        int at = incl - sum;
        for (int w = 0; w < kWarps; ++w) {
            at += w < warp ? sums[w] : 0;
            longest = max(longest, sums[kWarps + w]);
        }
        for (int e = e0; e < e1; ++e) {
            const int v = prefix[e];
            prefix[e] = at;
            at += v;
        }
        if (tid == kThreads - 1)
            prefix[p.entries] = at;
        __syncthreads();
    }
    // Teams of CTAs walk the same tokens of neighbouring KV heads (or of groups of
    // rows of one head); `copies` segments of a team share an entry's length.
    const int copies = p.copies, team = blockIdx.x >> p.lg_team, member = blockIdx.x & ((1 << p.lg_team) - 1);
    const int teams = gridDim.x >> p.lg_team, segments = p.entries * copies;
    const int U = prefix[p.entries] * copies;  // (below 2^31: the host has seen to it)
    const int G = min(teams, (U + kCharge + 3) / (kCharge + 4));
    // U = G share + extra: the first `extra` teams take one tile more
    const int share = U / G, extra = U - G * share;
    auto owner_of = [&](int x) { return x < extra * (share + 1) ? x / (share + 1) : extra + (x - extra * (share + 1)) / share; };
    // Segments whole, or in equal pieces of at most `piece` tiles, one a team, or the
    // shares.  Estimates in tiles of one CTA: the longest run of tiles, but no less
    // than what the memory's rate allows for them all, and what a join costs; of the
    // shares also that a team starts a second segment.
    int piece = 0;
    if (segments <= teams) {
        const int tiles = U - segments * kCharge, least = (tiles << p.lg_team) / Sh::kFull;
        const int whole = max(longest, least);
        piece = whole <= max(share, least) + Sh::kJoin ? longest : 0;
        if (segments < teams) {
            // tiles / (teams - segments) always does; pieces end on average half a piece early,
            // so that two smaller sizes are tried where it counts (0.3 us; nine sequences of
            // 64 MB 24.2 -> 21.3 us): with few segments they are nearly the same, with nearly as
            // many as teams there is no room to cut
            int cut = static_cast<int>(static_cast<float>(tiles) * fast_rcp(static_cast<float>(teams - segments)));
            cut = max(4, cut + (cut >> 20) + 1);  // (not below the quotient)
            if (segments * 4 > teams && segments * 4 < 3 * teams && longest < 1 << 18 && (segments * 2 < teams || 0.9f * longest * segments > tiles)) {
                constexpr int kTries = 2;
                int size[kTries], sum[kTries];
                float inv[kTries];
#pragma unroll
                for (int i = 0; i < kTries; ++i) {
                    inv[i] = fast_rcp(static_cast<float>(teams) - static_cast<float>(segments) * (0.45f + 0.25f * i));
                    size[i] = max(4, static_cast<int>(static_cast<float>(tiles) * inv[i]) + 1);
                    inv[i] = fast_rcp(static_cast<float>(size[i]));
                    sum[i] = 0;
                }
                // ceil(x / size): x - 1/2 is too far from a multiple for the rounding to matter
                for (int e = lane; e < p.entries; e += 32) {
                    const float x = static_cast<float>(prefix[e + 1] - prefix[e] - kCharge) - 0.5f;
#pragma unroll
                    for (int i = 0; i < kTries; ++i)
                        sum[i] += static_cast<int>(x * inv[i]) + 1;
                }
#pragma unroll
                for (int i = kTries - 1; i >= 0; --i)
                    if (__reduce_add_sync(kFullWarp, sum[i]) * copies <= teams)
                        cut = min(cut, size[i]);
            }
            if (cut < longest && max(cut, least) + Sh::kJoin < whole && cut <= share + (segments - 1) * 5 / 4)
                piece = cut;
        }
    }
    // Short ones: a warp takes a segment by itself, the next at a distance of all warps of
    // the grid.  A tile of a warp's own costs about 7 / C of a share's (1.0 us), its start
    // and end one more; a share its starts (charged) and a join.  8 heads of 128 channels,
    // by itself / shares: 100 sequences of 64 tokens 8.0 / 19.6 us, of 256 17.4 / 27.2,
    // of 1024 50 / 54.5, 60 of 512 22.7 / 29.0; 800 of 64 tokens 33 / 226.
    const int solo_step = gridDim.x * kWarps, solo_end = segments << p.lg_team;
    bool solo = false;
    if (kMany && piece == 0) {
        const int rounds = (solo_end + solo_step - 1) / solo_step;
        solo = 7.f * rounds * (longest + 1) <= static_cast<float>(C) * share + 36.f;
    }
    const int stride = solo ? 1 : kWarps, rows_at = solo ? warp * kRows : 0;
    int u_begin, u_end, first_team = 0, own_pieces = 1;
    if (solo) {
        u_begin = warp * gridDim.x + blockIdx.x;
        u_end = solo_end;
    } else if (piece > 0) {
        int e = copies == 1 ? team : team / copies;
        first_team = e * copies;
        if (piece < longest) {
            // every warp for itself: the entry whose pieces hold this team
            int before = 0;
            bool found = false;
            for (int e0 = 0; e0 < p.entries && !found; e0 += 32) {
                const int v = e0 + lane < p.entries ? (prefix[e0 + lane + 1] - prefix[e0 + lane] - kCharge + piece - 1) / piece : 0;
                int incl = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(kFullWarp, incl, o);
                    if (lane >= o)
                        incl += y;
                }
                const uint32_t here = __ballot_sync(kFullWarp, (before + incl) * copies > team);
                if (here != 0) {
                    const int at = __ffs(here) - 1;
                    e = e0 + at;
                    own_pieces = __shfl_sync(kFullWarp, v, at);
                    first_team = (before + __shfl_sync(kFullWarp, incl, at) - own_pieces) * copies;
                    found = true;
                }
                before += __shfl_sync(kFullWarp, incl, 31);
            }
            if (!found)
                return;
        } else if (team >= segments) {
            return;
        }
        const int length = prefix[e + 1] - prefix[e];
        const int cc = copies == 1 ? 0 : (team - first_team) / own_pieces, i = team - first_team - cc * own_pieces;
        first_team += cc * own_pieces;
        const int tiles = length - kCharge, each = tiles / own_pieces, over = tiles - each * own_pieces;
        const int base = prefix[e] * copies + cc * length + kCharge;
        u_begin = i == 0 ? base - kCharge : base + i * each + min(i, over);
        u_end = base + (i + 1) * each + min(i + 1, over);
    } else {
        if (team >= G)
            return;
        u_begin = team * share + min(team, extra);
        u_end = u_begin + share + (team < extra ? 1 : 0);
    }

    // ---- a piece: tiles from .. stop - 1 of a segment (tiles s_begin .. s_end - 1)
    int u = u_begin, s_begin = 0, s_end = 0, from = 0, stop = 0;
    int b = 0, kh = 0, grp = 0, row_base = 0, n = 0, tokens = 0, nb = 0, first = 0, last = 0;
    const int32_t* sel;
    const int32_t* table;
    uint4 raw[kChunks][QP * 2];  // query rows: one warp a group of eight; 16 elements a chunk

    // ---- copies.  The lanes look up the blocks of the warp's next kWindow tiles together.
    constexpr int kWindow = 32 / HB, kPart = kTile / HB;  // tokens of a block within a tile, at most
    const uint32_t step = static_cast<uint32_t>(p.KV) * D;
    const uint32_t copy_at = copy_row * step + copy_run * 16;
    const int own = lane >> 1 & (HB - 1);     // the part whose scale and place this lane stores
    uint32_t w_row = 0;                       // of this lane's part of the window: its first row of the pool
    int w_place = 0, blk_next = -1, phys_next = -1;
    auto look_up = [&](int window) {
        const int tile = first + (window * kWindow + lane / HB) * stride;
        const int place = tile * kTile + kPart * (lane % HB);
        int j = -1;
        if (tile < last && place < tokens) {
            j = place >> p.shift;
            if (sel) {
                j = __ldg(sel + j);
                if (j < 0 || j >= nb) {
                    if (j != -1)
                        q8_report(p.status, PA_STATUS_BAD_BLOCK);
                    j = -1;
                }
            }
        }
        blk_next = j;
        phys_next = j >= 0 ? __ldg(table + j) : -1;
    };
    auto take_up = [&](int window) {
        const int tile = first + (window * kWindow + lane / HB) * stride;
        const int in_block = (tile * kTile + kPart * (lane % HB)) & ((1 << p.shift) - 1);
        const bool there = static_cast<uint32_t>(phys_next) < static_cast<uint32_t>(p.num_blocks);
        if (!there && blk_next >= 0)
            q8_report(p.status, PA_STATUS_BAD_BLOCK);
        // (without a block: the first rows of the pool are read in its place, and hidden)
        w_row = there ? (static_cast<uint32_t>(phys_next) << p.shift) + in_block : 0u;
        w_place = there ? (blk_next << p.shift) + in_block : kNowhere;
    };
    auto issue = [&](int k, uint32_t st) {  // the warp's k-th tile
        if (first + k * stride < last) {
            const int at_window = k & (kWindow - 1);
            if (at_window == 0 && k > 0)
                take_up(k / kWindow);
            if (at_window == kWindow / 2)
                look_up(k / kWindow + 1);
            const uint32_t own_row = __shfl_sync(kFullWarp, w_row, at_window * HB + own);
            const int own_place = __shfl_sync(kFullWarp, w_place, at_window * HB + own);
            if (lane < 2 * HB) {
                q8_copy4(st + kTileBytes + lane * 4, (lane & 1 ? p.vs : p.ks) + static_cast<uint64_t>(own_row >> p.shift) * p.KV + kh);
                if ((lane & 1) == 0)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + kTileBytes + 32 + 2 * lane), "r"(own_place) : "memory");
            }
#pragma unroll
            for (int x = 0; x < HB; ++x) {
                const uint64_t at = static_cast<uint64_t>(__shfl_sync(kFullWarp, w_row, at_window * HB + x)) * step + (kh * D + copy_at);
                const int8_t* k0 = p.k + at;
                const int8_t* v0 = p.v + at;
#pragma unroll
                for (int i = 0; i < kPart / kRowsCopy; ++i) {
                    const uint32_t to = st + (x * (kPart / kRowsCopy) + i) * 512;
                    q8_copy16(to + copy_k, k0 + i * kRowsCopy * step);
                    q8_copy16(to + kTile * D + (D == 128 && i & 1 ? copy_v ^ 64 : copy_v), v0 + i * kRowsCopy * step);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Takes up the piece at tile u and starts its first copies; false when only a
    // charge is left of this CTA's range (the next one has the tiles).
    auto begin = [&]() -> bool {
        int e = 0, c;
        if (solo) {
            const int all = copies << p.lg_team;
            e = u / all;
            c = u - e * all;
            s_begin = from = 0;
            s_end = stop = prefix[e + 1] - prefix[e] - kCharge;
        } else {
            int hi = p.entries;
            while (hi - e > 1) {
                const int mid = (e + hi) >> 1;
                if (prefix[mid] * copies <= u)
                    e = mid;
                else
                    hi = mid;
            }
            const int length = prefix[e + 1] - prefix[e];
            const int cc = copies == 1 ? 0 : (u - prefix[e] * copies) / length;
            s_end = prefix[e] * copies + (cc + 1) * length;
            s_begin = s_end - length + kCharge;  // its first tile, behind the charge
            from = max(u, s_begin);
            stop = min(s_end, u_end);
            if (stop <= s_begin)
                return false;
            c = (cc << p.lg_team) + member;
        }
        b = p.selected ? e / p.KV : e;
        kh = p.selected ? e - b * p.KV : p.groups == 1 ? c : c / p.groups;
        grp = p.selected ? c : p.groups == 1 ? 0 : c - kh * p.groups;
        row_base = grp * kRows;
        const int length = __ldg(p.lens + b);
        n = min(max(length, 0), p.cap);
        if (p.selected && length != n)  // (without lists the prefix sums have told)
            q8_report(p.status, PA_STATUS_BAD_LENGTH);
        sel = p.selected ? p.selected + static_cast<int64_t>(e) * p.budget : nullptr;
        tokens = p.selected ? min(max(__ldg(p.counts + e), 0), p.budget) << p.shift : n;  // places in the list of blocks
        nb = (n + (1 << p.shift) - 1) >> p.shift;
        table = p.table + static_cast<int64_t>(b) * p.maxb;
        // this warp's tiles: first, first + kWarps, ... below last
        first = from - s_begin + (solo ? 0 : warp);
        last = min(stop - s_begin, (tokens + kTile - 1) / kTile);
        look_up(0);
        if (warp < NT || solo) {
            const int row = row_base + (solo ? 0 : warp * 8) + g;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                const int64_t at = ((static_cast<int64_t>(b) * p.KV + kh) * p.R + row) * D + ch * 64 + t * 16;
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.q) + at * (QP * 2));
#pragma unroll
                for (int i = 0; i < QP * 2; ++i)
                    raw[ch][i] = row < p.R ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        __syncwarp();  // the ring's last tiles have been read
        take_up(0);
#pragma unroll
        for (int i = 0; i < S - 1; ++i)
            issue(i, ring + i * kStage);
        return true;
    };
    // values, maxima and sums: by steps of channels and groups of eight rows, two rows
    // a lane (wide: by 16 rows and eight channels, rows g and g + 8)
    constexpr int kStats = kWide ? NT : 2 * NT, kOct = D / 8;
    float o[kSteps * NT][4];
    float mx[kStats], l[kStats];
    int open = 0;  // pieces of this CTA that leave a record: at most the first and the last
    bool have = false;
    for (;;) {
        // ---- what the end of the piece in hand needs, and the start of the next
        const bool whole = from == s_begin && stop == s_end;
        // a piece of a segment begun by an earlier CTA, or one that goes on
        const int slot = u_begin > s_begin ? 0 : 1;
        const int64_t out0 = ((static_cast<int64_t>(b) * p.KV + kh) * p.R + row_base) * D;
        const int rows_left = p.R - row_base;
        if (have && !whole && tid == 0) {
            const int c0 = piece > 0 ? first_team : owner_of(s_begin), count = piece > 0 ? own_pieces : owner_of(s_end - 1) - c0 + 1;
            // (of the segments that begin in a CTA, one at most goes on in the next)
            sm_open[open] = {c0, count, p.counters + (c0 << p.lg_team) + member, out0, rows_left};
        }
        if (have)
            u = solo ? u + solo_step : stop;
        const bool more = u < u_end && begin();
        if (have && solo) {
            // ---- the warp's own state is all there is
            if constexpr (kMany) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float sum = l[k];
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        sum += __shfl_xor_sync(kFullWarp, sum, x);
                    const float r = sum == 0.f ? 0.f : 1.f / sum;
                    if (2 * t + k < rows_left) {
                        const int64_t to = out0 + (2 * t + k) * D + D / 8 * g;
#pragma unroll
                        for (int s2 = 0; s2 < kSteps; s2 += 2)
                            store_out(p, to + 2 * s2, make_float4(o[s2][k] * r, o[s2][k + 2] * r, o[s2 + 1][k] * r, o[s2 + 1][k + 2] * r));
                    }
                }
            }
        } else if (have) {
            // ---- the warps' states together
            auto row_of = [&](int k) { return kWide ? (k >> 1) * 16 + (k & 1) * 8 + g : (k >> 1) * 8 + 2 * t + (k & 1); };
#pragma unroll
            for (int k = 0; k < kStats; ++k) {
                float s = l[k];
#pragma unroll
                for (int x = kWide ? 1 : 4; x < (kWide ? 4 : 32); x <<= 1)
                    s += __shfl_xor_sync(kFullWarp, s, x);
                if (kWide ? t == 0 : g == 0) {
                    sm_m[warp][row_of(k)] = mx[k];
                    sm_l[warp][row_of(k)] = s;
                }
            }
            __syncthreads();  // (without a next piece, the rings of all warps are free then)
            constexpr int kQuads = D / 4, kItems = kRows * kQuads;  // four channels each
            constexpr int kPer = (kItems + kThreads - 1) / kThreads;
            float4 val[kPer];
#pragma unroll
            for (int x = 0; x < kPer; ++x)
                val[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            float* state = reinterpret_cast<float*>(more ? smem + Sh::kRing + Sh::kQueryBytes : smem);  // [warp][row] in steps
            const int group = more ? Sh::kGroup : Sh::kLastGroup;
            for (int w0 = 0; w0 < kWarps; w0 += group) {
                if (w0 > 0)
                    __syncthreads();
                if (warp >= w0 && warp < w0 + group) {
#pragma unroll
                    for (int k = 0; k < kStats; ++k) {
                        const int row = row_of(k);
                        float m = -INFINITY;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w)
                            m = fmaxf(m, sm_m[w][row]);
                        const float f = mx[k] == -INFINITY ? 0.f : fast_exp2(mx[k] - m);
                        float* to = state + ((warp - w0) * kRows + row) * Sh::kStateRow;
                        if constexpr (kWide) {  // channels D / 4 t ...: two of eight octets' columns
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int j = 0; j < kOct; j += 4) {
                                    const int at = (k >> 1) * kOct + j, i = (k & 1) * 2 + e, quad = t * (D / 16) + ((e * kOct + j) / 4 ^ turn_of(t));
                                    *reinterpret_cast<float4*>(to + quad * 4) = make_float4(o[at][i] * f, o[at + 1][i] * f, o[at + 2][i] * f, o[at + 3][i] * f);
                                }
                        } else {
#pragma unroll
                            for (int s2 = 0; s2 < kSteps; ++s2)  // channels D / 8 g + 2 s2, + 1
                                *reinterpret_cast<float2*>(to + 2 * g + s2 * Sh::kStateStep) =
                                    make_float2(o[s2 * NT + (k >> 1)][k & 1] * f, o[s2 * NT + (k >> 1)][(k & 1) + 2] * f);
                        }
                    }
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    const int x = tid + k * kThreads, row = x / kQuads, quad = x % kQuads;
                    if (x < kItems) {
                        const float* at = state + row * Sh::kStateRow;
                        if constexpr (kWide) {
                            const int lane_t = quad / (D / 16);
                            at += (lane_t * (D / 16) + (quad % (D / 16) ^ turn_of(lane_t))) * 4;
                            for (int w = 0; w < group; ++w) {
                                const float4 v = *reinterpret_cast<const float4*>(at + w * kRows * Sh::kStateRow);
                                val[k].x += v.x, val[k].y += v.y, val[k].z += v.z, val[k].w += v.w;
                            }
                        } else {
                            at += quad / (D / 32) * 2 + quad % (D / 32) * 2 * Sh::kStateStep;
                            for (int w = 0; w < group; ++w) {
                                const float2 v0 = *reinterpret_cast<const float2*>(at + w * kRows * Sh::kStateRow);
                                const float2 v1 = *reinterpret_cast<const float2*>(at + w * kRows * Sh::kStateRow + Sh::kStateStep);
                                val[k].x += v0.x, val[k].y += v0.y, val[k].z += v1.x, val[k].w += v1.y;
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int x = tid + k * kThreads, row = x / kQuads, quad = x % kQuads;
                if (x >= kItems || row >= rows_left)
                    break;
                float m = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    m = fmaxf(m, sm_m[w][row]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    sum += scaled_sum(sm_l[w][row], sm_m[w][row] - m);
                if (whole) {
                    const float r = sum == 0.f ? 0.f : 1.f / sum;
                    store_out(p, out0 + static_cast<int64_t>(x) * 4, make_float4(val[k].x * r, val[k].y * r, val[k].z * r, val[k].w * r));
                } else {
                    *reinterpret_cast<float4*>(p.part_o + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * kRows * D + x * 4) = val[k];
                    if (quad == 0)
                        p.part_ml[(static_cast<int64_t>(blockIdx.x) * 2 + slot) * kRows + row] = make_float2(m, sum);
                }
            }
            open += whole ? 0 : 1;
        }
        if (!more)
            break;
        have = true;

        // ---- query rows as fragments of B, scaled by a power of two
        uint32_t qf[kWide ? 1 : QP][kWide ? 1 : NT][kWide ? 1 : kSteps][2];
        if (warp < NT || solo) {
            float x[kSteps * 4], a = 0.f;
#pragma unroll
            for (int i = 0; i < kSteps * 4; i += QP == 2 ? 1 : 2) {
                const uint4 v = raw[i / 16][i % 16 / (QP == 2 ? 4 : 8)];
                const int word = QP == 2 ? i % 4 : i % 8 / 2;
                const uint32_t w = word == 0 ? v.x : word == 1 ? v.y : word == 2 ? v.z : v.w;
                if constexpr (QP == 2) {
                    x[i] = __uint_as_float(w);
                } else {
                    const float2 two = p.dtype == PA_F16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
                                                         : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
                    x[i] = two.x;
                    x[i + 1] = two.y;
                }
            }
#pragma unroll
            for (int i = 0; i < kSteps * 4; ++i)
                a = fmaxf(a, fabsf(x[i]));
            a = fmaxf(a, __shfl_xor_sync(kFullWarp, a, 1));
            a = fmaxf(a, __shfl_xor_sync(kFullWarp, a, 2));
            // 2^up brings the largest magnitude into [2^11, 2^12)
            const int up = 11 - max(static_cast<int>(__float_as_uint(a) >> 23) - 127, -100);
            const float lift = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            float total = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                uint32_t w[QP][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float z0 = x[4 * s + 2 * i] * lift, z1 = x[4 * s + 2 * i + 1] * lift;
                    const __half2 hi = __floats2half2_rn(z0, z1);
                    const float2 back = __half22float2(hi);
                    w[0][i] = half2_bits(hi);
                    if constexpr (QP == 2)
                        w[QP - 1][i] = half2_bits(__floats2half2_rn(z0 - back.x, z1 - back.y));
                    total += back.x + back.y;
                }
#pragma unroll
                for (int q = 0; q < QP; ++q) {
                    if constexpr (kWide) {  // fragments of 16 rows: rows g, g + 8, and again 8 channels on
                        uint32_t* to = reinterpret_cast<uint32_t*>(sm_q) + ((s * (NT / 2) + warp / 2) * 32 + lane) * 4 + warp % 2;
                        to[0] = w[q][0];
                        to[2] = w[q][1];
                    } else if (solo) {
                        qf[q][0][s][0] = w[q][0];
                        qf[q][0][s][1] = w[q][1];
                    } else {
                        sm_q[((q * kSteps + s) * NT + warp) * 32 + lane] = make_uint2(w[q][0], w[q][1]);
                    }
                }
            }
            total += __shfl_xor_sync(kFullWarp, total, 1);
            total += __shfl_xor_sync(kFullWarp, total, 2);
            if (t == 0) {
                const int in = solo ? 0 : warp * 8, r = row_base + in + g, at = rows_at + in + g;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
                sm_f[at] = p.scale * down * (kSmall ? 2048.f : 1.f);
                sm_off[at] = kSmall ? total * (-128.f / 16777216.f) : 0.f;
                sm_lim[at] = r >= p.R ? 0 : p.causal ? min(n, n - p.NQ + r % p.NQ + 1) : n;
            }
        }
        if (solo)
            __syncwarp();
        else
            __syncthreads();
        if (!kWide && !solo) {
#pragma unroll
            for (int q = 0; q < QP; ++q)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const uint2 w = sm_q[((q * kSteps + s) * NT + nt) * 32 + lane];
                        qf[q][nt][s][0] = w.x;
                        qf[q][nt][s][1] = w.y;
                    }
        }
        float rowf[kStats], off[kStats];  // of this lane's rows (wide: read when they are needed)
        if constexpr (!kWide) {
#pragma unroll
            for (int k = 0; k < kStats; ++k) {
                rowf[k] = sm_f[rows_at + (k >> 1) * 8 + 2 * t + (k & 1)];
                off[k] = sm_off[rows_at + (k >> 1) * 8 + 2 * t + (k & 1)];
            }
        }
        // parts that begin here or before are seen by every row
        const int all_see = row_base + kRows > p.R ? INT_MIN : (p.causal ? n - p.NQ + 1 : n) - kPart;

#pragma unroll
        for (int k = 0; k < kStats; ++k) {
            mx[k] = -INFINITY;
            l[k] = 0.f;
        }
#pragma unroll
        for (int s = 0; s < kSteps * NT; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[s][i] = 0.f;

        uint32_t st = ring, fill = ring + (S - 1) * kStage;
        int ahead = S - 1;
        bool apart = false;  // a value scale far from one has been met
        for (int tile = first; tile < last; tile += stride) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");  // this tile's
            __syncwarp();  // the copies of the other lanes; the stage filled next has been read
            issue(ahead++, fill);
            if constexpr (kWide) {
                constexpr int M = NT / 2;  // groups of 16 rows
                float ks[HB], lv[HB], iv[HB];
                int place[HB];
#pragma unroll
                for (int x = 0; x < HB; ++x) {
                    const uint2 sc = lds8(st + kTileBytes + x * 8);
                    ks[x] = fmaxf(__uint_as_float(sc.x), kMinScale) * kUnit;
                    const float vs = fmaxf(__uint_as_float(sc.y), kMinScale);
                    lv[x] = fast_log2(vs);
                    iv[x] = fast_rcp(vs);
                    place[x] = static_cast<int>(lds4(st + kTileBytes + 32 + x * 4));
                    apart |= fabsf(lv[x]) > kNear && place[x] < kNowhere;
                }
                if (apart) {
#pragma unroll
                    for (int x = 0; x < HB; ++x)
                        iv[x] = 0.f;
                }
                // ---- S = Q K^T, eight tokens at a time
                float s[M][4][4];
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[m][e][i] = sm_off[m * 16 + (i >> 1) * 8 + g];
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch) {
                    uint32_t w[4][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 v = lds16(st + e * 8 * D + (read_k ^ ch * 64));
                        w[e][0] = v.x, w[e][1] = v.y, w[e][2] = v.z, w[e][3] = v.w;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a[M][4];
#pragma unroll
                        for (int m = 0; m < M; ++m) {
                            const uint4 v = reinterpret_cast<const uint4*>(sm_q)[((ch * 4 + i) * M + m) * 32 + lane];
                            a[m][0] = v.x, a[m][1] = v.y, a[m][2] = v.z, a[m][3] = v.w;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t u = w[e][i] ^ 0x80808080u, b0 = __byte_perm(u, 0, 0x4140), b1 = __byte_perm(u, 0, 0x4342);
#pragma unroll
                            for (int m = 0; m < M; ++m)
                                mma(s[m][e], a[m], b0, b1);
                        }
                    }
                }
                // ---- scores in base 2 plus log2 of the value scale, less the maximum; hidden ones -inf
                bool hide = false, raise = false;
#pragma unroll
                for (int x = 0; x < HB; ++x)
                    hide |= place[x] > all_see;
                float top[2 * M];
#pragma unroll
                for (int k = 0; k < 2 * M; ++k) {
                    const int m = k >> 1, i0 = (k & 1) * 2;
                    const float base = mx[k] == -INFINITY ? 0.f : mx[k] - kLift;
                    top[k] = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int x = HB == 4 ? e : e >> 1;
                        const float f = sm_f[m * 16 + (k & 1) * 8 + g] * ks[x], add = lv[x] - base;
                        s[m][e][i0] = fmaf(s[m][e][i0], f, add);
                        s[m][e][i0 + 1] = fmaf(s[m][e][i0 + 1], f, add);
                    }
                    if (hide) {
                        const int lim = sm_lim[m * 16 + (k & 1) * 8 + g];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if ((HB == 4 ? place[e & (HB - 1)] : place[e >> 1] + (e & 1) * 8) + 2 * t + i >= lim)
                                    s[m][e][i0 + i] = -INFINITY;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top[k] = fmaxf(top[k], fmaxf(s[m][e][i0], s[m][e][i0 + 1]));
                    raise |= top[k] > (mx[k] == -INFINITY ? -INFINITY : kLift + kSlack);
                }
                if (__any_sync(kFullWarp, raise)) {
#pragma unroll
                    for (int k = 0; k < 2 * M; ++k) {
                        const int m = k >> 1, i0 = (k & 1) * 2;
                        const float base = mx[k] == -INFINITY ? 0.f : mx[k] - kLift;
                        float high = top[k];
                        high = fmaxf(high, __shfl_xor_sync(kFullWarp, high, 1));
                        high = fmaxf(high, __shfl_xor_sync(kFullWarp, high, 2));
                        high = fmaxf(high + base, mx[k]);
                        const float down = high == -INFINITY ? 1.f : fast_exp2(mx[k] - high);
                        const float less = high == -INFINITY ? 0.f : base - (high - kLift);
                        l[k] = scaled_sum(l[k], mx[k] - high);
                        mx[k] = high;
#pragma unroll
                        for (int j = 0; j < kOct; ++j) {
                            o[m * kOct + j][i0] *= down;
                            o[m * kOct + j][i0 + 1] *= down;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[m][e][i0] += less;
                            s[m][e][i0 + 1] += less;
                        }
                    }
                }
                if (apart) {
#pragma unroll
                    for (int m = 0; m < M; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                l[m * 2 + (i >> 1)] += fast_exp2(s[m][e][i] - lv[HB == 4 ? e : e >> 1]);
                }
                // ---- weights, as they are the fragments of P
                uint32_t pf[2][PW][M][4];
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = fast_exp2(s[m][e][i]);
                        const float inv = iv[HB == 4 ? e : e >> 1];
                        l[m * 2] = fmaf(w[0] + w[1], inv, l[m * 2]);
                        l[m * 2 + 1] = fmaf(w[2] + w[3], inv, l[m * 2 + 1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const __half2 hi = __floats2half2_rn(w[2 * i], w[2 * i + 1]);
                            pf[e >> 1][0][m][(e & 1) * 2 + i] = half2_bits(hi);
                            if constexpr (PW == 2) {
                                const float2 back = __half22float2(hi);
                                pf[e >> 1][PW - 1][m][(e & 1) * 2 + i] = half2_bits(__floats2half2_rn(w[2 * i] - back.x, w[2 * i + 1] - back.y));
                            }
                        }
                    }
                // ---- O += P V, eight channels at a time
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t sv = st + kTile * D + j * 16 * D;
                    uint32_t vw[4][D / 32];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (D == 128) {
                            const uint4 v = lds16(sv + (i >> 1) * 8 * D + (i & 1) * 128 + read_v);
                            vw[i][0] = v.x, vw[i][1] = v.y, vw[i][2] = v.z, vw[i][3] = v.w;
                        } else {
                            const uint2 v = lds8(sv + (i >> 1) * 8 * D + (i & 1) * 256 + read_v);
                            vw[i][0] = v.x, vw[i][1] = v.y;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < D / 32; ++w)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t pick = half ? 0x7362 : 0x5140;
                            const uint32_t lo = __byte_perm(vw[0][w], vw[1][w], pick) ^ 0x80808080u;
                            const uint32_t hi = __byte_perm(vw[2][w], vw[3][w], pick) ^ 0x80808080u;
                            uint32_t vb[2][2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                vb[i][0] = codes2(lo, i ? 0x4342 : 0x4140);
                                vb[i][1] = codes2(hi, i ? 0x4342 : 0x4140);
                            }
#pragma unroll
                            for (int x = PW - 1; x >= 0; --x)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
#pragma unroll
                                    for (int m = 0; m < M; ++m)
                                        mma(o[m * kOct + w * 4 + half * 2 + i], pf[j][x][m], vb[i][0], vb[i][1]);
                        }
                }
            } else {
#pragma unroll 1
            for (int j0 = 0; j0 < 2; j0 += J) {
                constexpr int B2 = HB / 2;  // blocks of a group of 16
                float ks[J][B2], lv[J][B2], iv[J][B2];
                int place[J][2];
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int x = 0; x < B2; ++x) {
                        const int part = (j0 + j) * B2 + x;
                        const uint2 sc = lds8(st + kTileBytes + part * 8);
                        ks[j][x] = fmaxf(__uint_as_float(sc.x), kMinScale) * kUnit;
                        const float vs = fmaxf(__uint_as_float(sc.y), kMinScale);
                        lv[j][x] = fast_log2(vs);
                        iv[j][x] = fast_rcp(vs);
                        place[j][x] = static_cast<int>(lds4(st + kTileBytes + 32 + part * 4));
                        apart |= fabsf(lv[j][x]) > kNear && place[j][x] < kNowhere;
                        if constexpr (B2 == 1)
                            place[j][1] = place[j][0] + 8;
                    }
                if (__builtin_expect(apart, 0)) {  // (out of the way: float32, 16 rows 28.9 -> 27.4 us; the other form is no faster so)
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int x = 0; x < B2; ++x)
                            iv[j][x] = 0.f;
                }
                // ---- S^T = K Q^T
                float sacc[J][NT][4];
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sacc[j][nt][i] = off[nt * 2 + (i & 1)];
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch) {
                    uint32_t wa[J][4], wb[J][4];
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const uint32_t at = st + (j0 + j) * 16 * D + (read_k ^ ch * 64);
                        const uint4 ka = lds16(at), kb = lds16(at + 8 * D);
                        wa[j][0] = ka.x, wa[j][1] = ka.y, wa[j][2] = ka.z, wa[j][3] = ka.w;
                        wb[j][0] = kb.x, wb[j][1] = kb.y, wb[j][2] = kb.z, wb[j][3] = kb.w;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            const uint32_t ua = wa[j][i] ^ 0x80808080u, ub = wb[j][i] ^ 0x80808080u;
                            const uint32_t a[4] = {kSmall ? __byte_perm(ua, 0, 0x4140) : codes2(ua, 0x4140),
                                                   kSmall ? __byte_perm(ub, 0, 0x4140) : codes2(ub, 0x4140),
                                                   kSmall ? __byte_perm(ua, 0, 0x4342) : codes2(ua, 0x4342),
                                                   kSmall ? __byte_perm(ub, 0, 0x4342) : codes2(ub, 0x4342)};
#pragma unroll
                            for (int q = 0; q < QP; ++q)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma(sacc[j][nt], a, qf[q][nt][ch * 4 + i][0], qf[q][nt][ch * 4 + i][1]);
                                }
                        }
                    }
                }
                // ---- scores in base 2 plus log2 of the value scale; hidden ones -inf
                bool hide = false, raise = false;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    hide |= (B2 == 1 ? place[j][0] : max(place[j][0], place[j][1])) > all_see;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sacc[j][nt][i] = fmaf(sacc[j][nt][i], rowf[nt * 2 + (i & 1)] * ks[j][i >> 1 & (B2 - 1)], lv[j][i >> 1 & (B2 - 1)]);
                }
                if (hide) {
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (place[j][i >> 1] + g >= sm_lim[rows_at + nt * 8 + 2 * t + (i & 1)])
                                    sacc[j][nt][i] = -INFINITY;
                }
                float top[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top[nt][i] = fmaxf(sacc[0][nt][i], sacc[0][nt][i + 2]);
                        if constexpr (J == 2)
                            top[nt][i] = fmaxf(top[nt][i], fmaxf(sacc[J - 1][nt][i], sacc[J - 1][nt][i + 2]));
                        raise |= top[nt][i] > mx[nt * 2 + i] + kSlack;
                    }
                if (__any_sync(kFullWarp, raise)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float m = top[nt][i];
                            m = fmaxf(m, __shfl_xor_sync(kFullWarp, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(kFullWarp, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(kFullWarp, m, 16));
                            m = fmaxf(m, mx[nt * 2 + i]);
                            const float down = m == -INFINITY ? 1.f : fast_exp2(mx[nt * 2 + i] - m);
                            l[nt * 2 + i] = scaled_sum(l[nt * 2 + i], mx[nt * 2 + i] - m);
                            mx[nt * 2 + i] = m;
#pragma unroll
                            for (int s = 0; s < kSteps; ++s) {
                                o[s * NT + nt][i] *= down;
                                o[s * NT + nt][i + 2] *= down;
                            }
                        }
                }
                // ---- weights, and as fragments of P^T
                static_assert(PW == 2);
                uint32_t pf[J][PW][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    // (a row that has seen nothing: its scores are -inf, and so is what is left of them)
                    const float base[2] = {fmaxf(mx[nt * 2], -3.402823466e38f) - kLift, fmaxf(mx[nt * 2 + 1], -3.402823466e38f) - kLift};
                    if (__builtin_expect(apart, 0)) {
#pragma unroll
                        for (int j = 0; j < J; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                l[nt * 2 + (i & 1)] += fast_exp2(sacc[j][nt][i] - base[i & 1] - lv[j][i >> 1 & (B2 - 1)]);
                    }
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        float w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = fast_exp2(sacc[j][nt][i] - base[i & 1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if constexpr (B2 == 1)
                                l[nt * 2 + i] = fmaf(w[i] + w[i + 2], iv[j][0], l[nt * 2 + i]);
                            else
                                l[nt * 2 + i] = fmaf(w[i], iv[j][0], fmaf(w[i + 2], iv[j][B2 - 1], l[nt * 2 + i]));
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const __half2 hi = __floats2half2_rn(w[2 * x], w[2 * x + 1]);
                            pf[j][0][nt][x] = movm_trans(half2_bits(hi));
                            const float2 back = __half22float2(hi);
                            pf[j][1][nt][x] = movm_trans(half2_bits(__floats2half2_rn(w[2 * x] - back.x, w[2 * x + 1] - back.y)));
                        }
                    }
                }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const uint32_t sv = st + kTile * D + (j0 + j) * 16 * D;
                    uint32_t vw[4][D / 32];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (D == 128) {
                            const uint4 v = lds16(sv + (i >> 1) * 8 * D + (i & 1) * 128 + read_v);
                            vw[i][0] = v.x, vw[i][1] = v.y, vw[i][2] = v.z, vw[i][3] = v.w;
                        } else {
                            const uint2 v = lds8(sv + (i >> 1) * 8 * D + (i & 1) * 256 + read_v);
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
                        uint32_t a[2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            a[i][0] = codes2(mixed[0][i], 0x4140), a[i][1] = codes2(mixed[0][i], 0x4342);
                            a[i][2] = codes2(mixed[1][i], 0x4140), a[i][3] = codes2(mixed[1][i], 0x4342);
                        }
                        if constexpr (QP == 1) {
#pragma unroll
                            for (int x = PW - 1; x >= 0; --x)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    mma(o[2 * w + i], a[i], pf[j][x][0][0], pf[j][x][0][1]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    // a group's products by themselves: added to the sums by rounded
                                    // additions (the tensor core's own cut off what does not fit)
                                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma(d, a[i], pf[j][1][nt][0], pf[j][1][nt][1]);
                                    mma(d, a[i], pf[j][0][nt][0], pf[j][0][nt][1]);
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        o[(2 * w + i) * NT + nt][y] += d[y];
                                }
                        }
                    }
                }
            }
            }
            st = st + kStage == ring + S * kStage ? ring : st + kStage;
            fill = fill + kStage == ring + S * kStage ? ring : fill + kStage;
        }
    }

    // ---- the pieces that left a record: the last CTA to finish one of a segment joins them all
    if (open > 0) {
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            for (int i = 0; i < open; ++i) {
                const int before = atomicAdd(sm_open[i].counter, 1);
                if (before == sm_open[i].pieces - 1)
                    *sm_open[i].counter = 0;
                else
                    sm_open[i].pieces = 0;
            }
            __threadfence();
        }
        __syncthreads();
    }
    constexpr int kQuads = D / 4, kItems = kRows * kQuads;
    constexpr int kBatch = 20;  // pieces loaded together
    for (int which = 0; which < open; ++which) {
        // a row to each set of D / 4 lanes; their lanes hold the pieces' factors
        const int c0 = sm_open[which].first, pieces = sm_open[which].pieces, rows_left = sm_open[which].rows;
        const int64_t out0 = sm_open[which].out;
        if (pieces == 0)
            continue;
        // (the first team's range begins with the segment or earlier, the others' inside it)
        auto record_of = [&](int i) { return ((static_cast<int64_t>(c0 + i) << p.lg_team) + member) * 2 + (i > 0 ? 0 : 1); };
        for (int x0 = warp * 32; x0 < kItems; x0 += kThreads) {
            const int x = x0 + lane, row = x / kQuads, in_row = lane % kQuads;
            const bool live = row < rows_left;
            float m = -INFINITY, sum = 0.f;
            float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < pieces; i0 += kQuads) {  // (one turn, mostly)
                const int many = min(kQuads, pieces - i0);
                const float* src = p.part_o + x * 4;
                float4 v[kBatch];
                auto load = [&](int i) {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        v[k] = live && i + k < many ? __ldcg(reinterpret_cast<const float4*>(src + record_of(i0 + i + k) * kRows * D))
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                };
                load(0);
                float2 ml = make_float2(-INFINITY, 0.f);
                if (live && in_row < many)
                    ml = __ldcg(p.part_ml + record_of(i0 + in_row) * kRows + row);
                float top = ml.x;
#pragma unroll
                for (int k = 1; k < kQuads; k <<= 1)
                    top = fmaxf(top, __shfl_xor_sync(kFullWarp, top, k));
                top = fmaxf(top, m);
                const float f = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - top), old = m == -INFINITY ? 0.f : fast_exp2(m - top);
                float part = scaled_sum(ml.y, ml.x - top);
#pragma unroll
                for (int k = 1; k < kQuads; k <<= 1)
                    part += __shfl_xor_sync(kFullWarp, part, k);
                sum = scaled_sum(sum, m - top) + part;
                all.x *= old, all.y *= old, all.z *= old, all.w *= old;
                m = top;
                for (int i = 0; i < many; i += kBatch) {
                    if (i > 0)
                        load(i);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        fma4(all, __shfl_sync(kFullWarp, f, (lane & ~(kQuads - 1)) + ((i + k) & (kQuads - 1))), v[k]);
                }
            }
            const float r = sum == 0.f ? 0.f : 1.f / sum;
            if (live)
                store_out(p, out0 + static_cast<int64_t>(x) * 4, make_float4(all.x * r, all.y * r, all.z * r, all.w * r));
        }
    }
}

struct Variant {
    const void* fn;
    int rows, threads, ctas, charge;
    size_t body;  // shared memory apart from the prefix sums
    const void* many;  // for more segments than CTAs
};

template <int D, int NT, int QP, int C, int PW = 2>
Variant variant(int BLOCK)
{
    using Sh = Shape<D, NT, QP, C, PW>;
    static_assert(C > 1 || Sh::kRing + Sh::kQueryBytes + Sh::kGroup * Sh::kState + (kMaxEntries + 1) * 4 + 4096 <= 227 * 1024, "with the arrays of its own");
    constexpr bool kMany = NT == 1;
    return {BLOCK == 8 ? reinterpret_cast<const void*>(pa_q8_decode_kernel<D, NT, QP, 4, C, PW, false>)
                       : reinterpret_cast<const void*>(pa_q8_decode_kernel<D, NT, QP, 2, C, PW, false>),
            Sh::kRows, Sh::kThreads, C, Sh::kCharge, static_cast<size_t>(Sh::kRing) + Sh::kQueryBytes + Sh::kGroup * Sh::kState,
            BLOCK == 8 ? reinterpret_cast<const void*>(pa_q8_decode_kernel<D, NT, QP, 4, C, PW, kMany>)
                       : reinterpret_cast<const void*>(pa_q8_decode_kernel<D, NT, QP, 2, C, PW, kMany>)};
}

// `segments`: of 8 query rows.  One CTA of 12 warps per SM streams a segment twice as
// fast as one of two with 6 each and keeps up to a segment per SM whole; two fill
// in for each other's starts and ends, which counts where CTAs take several pieces.
// 64 MB, one / two: one sequence of 8 heads 20.7 / 24.4 us, 13 even ones 19.7 / 23.0,
// 40 even ones 31.9 / 26.9, 192 selected lists 26.7 / 18.0; 12 to 19 uneven
// sequences (26 to 51 MB) 20 to 25 / 16 to 21.  Lists that were selected are mostly
// of one length, sequences seldom.  Three of 4 warps are for as many segments as
// they still keep whole: 40 sequences of 512 / 1024 tokens 14.9 / 22.3 us (two: 24.0 /
// 30.0), 40 uneven ones of 43 MB 21.5 (24.6); with fewer segments they are slower (24
// even sequences 21.7, two: 20.0), with more no better (60 of 512 tokens 27.4, 22.8).
template <int D>
Variant variant(int BLOCK, int dtype, int R, long long segments, int sms, int entries, bool even)
{
    if (dtype == PA_F32)
        return R > 8 ? variant<D, 2, 2, 1>(BLOCK) : variant<D, 1, 2, 1>(BLOCK);
    if (R > 8 && dtype == PA_BF16)  // (weights of one part: see above)
        return R > 16 ? variant<D, 4, 1, 1, 1>(BLOCK) : variant<D, 2, 1, 1, 1>(BLOCK);
    if (R > 8)
        return R > 16 ? variant<D, 4, 1, 1>(BLOCK) : variant<D, 2, 1, 1>(BLOCK);
    const size_t sums = 4 * static_cast<size_t>(entries);
    const Variant two = variant<D, 1, 1, 2>(BLOCK), three = variant<D, 1, 1, 3>(BLOCK);
    if (segments > 2 * sms && segments <= 3 * sms && three.body + sums <= 75000)
        return three;
    return segments > (even ? sms : sms / 2) && two.body + sums <= 114000 ? two : variant<D, 1, 1, 1>(BLOCK);
}

// Sizes that pa_q8_decode refuses, apart from those of the cache.
int decode_sizes(int B, int H, int KV, int NQ)
{
    if (H < 1 || KV < 1 || H % KV != 0 || NQ < 1)
        return PA_ERR_BAD_DIMS;
    if (NQ > PA_MAX_NQ || static_cast<long long>(H / KV) * NQ > 1024 || B > kMaxBatch || KV > 1024)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// The counters lie at the same place whatever the sizes, the records behind them: a
// workspace may serve calls of unlike sizes in turn, and no record of one is where
// another has its counters.
constexpr size_t kZeroBytes = (kMaxCtas * sizeof(int) + 255) / 256 * 256;
constexpr size_t kMlBytes = static_cast<size_t>(kRecordRows) * 2 * sizeof(float2);

size_t workspace_bytes(int D) { return kZeroBytes + kMlBytes + static_cast<size_t>(kRecordRows) * 2 * D * sizeof(float); }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_q8_workspace_bytes(int B, int H, int KV, int D, int NQ)
{
    if (B < 1 || decode_sizes(B, H, KV, NQ) != PA_OK || (D != 64 && D != 128))
        return 0;
    return workspace_bytes(D);
}

extern "C" size_t pa_q8_workspace_zero_bytes(int B, int H, int KV, int D, int NQ)
{
    if (B < 1 || decode_sizes(B, H, KV, NQ) != PA_OK || (D != 64 && D != 128))
        return 0;
    return kZeroBytes;
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
    const size_t need = workspace_bytes(D);
    if (!o.workspace || o.workspace_bytes < need || (reinterpret_cast<uintptr_t>(o.workspace) & 255))
        return PA_ERR_WORKSPACE;
    const size_t blocks = static_cast<size_t>(o.num_blocks) * KV, pool = blocks * BLOCK * D, b4 = static_cast<size_t>(B) * 4;
    const size_t rows = static_cast<size_t>(B) * H * NQ * D * (o.dtype == PA_F32 ? 4 : 2);
    const Q8Range r[] = {{out, rows, true},
                         {o.workspace, need, true},
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
    int sms = 0, dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PA_ERR_CUDA;
    const long long segments = static_cast<long long>(B) * KV;
    const int entries = o.selected ? B * KV : B;
    const Variant v = D == 64 ? variant<64>(BLOCK, o.dtype, R, segments, sms, entries, o.selected) : variant<128>(BLOCK, o.dtype, R, segments, sms, entries, o.selected);
    DecodeParams p{};
    p.groups = (R + v.rows - 1) / v.rows;
    p.entries = entries;
    const long long copies = o.selected ? p.groups : static_cast<long long>(KV) * p.groups;
    const long long most = o.selected ? static_cast<long long>(o.budget) * BLOCK : static_cast<long long>(o.max_blocks) * BLOCK;
    const long long tiles = (most + kTile - 1) / kTile + v.charge;
    if (p.entries * tiles * copies >= (1ll << 31))
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
    p.part_ml = reinterpret_cast<float2*>(w + kZeroBytes);
    p.part_o = reinterpret_cast<float*>(w + kZeroBytes + kMlBytes);
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
    const int grid = sms * v.ctas > kRecordRows / v.rows ? kRecordRows / v.rows : sms * v.ctas;
    // Teams: the copies of one length that run side by side (rows of the same or of
    // neighbouring heads, whose cache lines lie together)
    p.lg_team = copies % 4 == 0 ? 2 : copies % 2 == 0 ? 1 : 0;
    if (grid % (1 << p.lg_team) != 0)
        p.lg_team = 0;
    p.copies = static_cast<int>(copies >> p.lg_team);
    void* args[] = {&p};
    return q8_launch(entries * copies > grid ? v.many : v.fn, dim3(grid), v.threads, v.body + (static_cast<size_t>(entries) + 1) * 4, static_cast<cudaStream_t>(stream), args);
}
