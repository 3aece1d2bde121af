// paged_plan.cu -- the work list of a prefill over the paged cache, from the lengths on the
// device: one thread block, about 3 us for up to 32 sequences and 5 us for more (latencies one
// after the other), so that neither the host nor each of the prefill's thread blocks has to look
// for its rows.
//
// A sequence's tiles are cut into pieces of at most Q tiles where that pays.  Q is chosen for
// the whole call: each warp takes one share of the tiles that an SM gets on average (0.15 to 3
// of them, or no cut at all) and estimates when the last SM is done as the largest of
//   - all tiles and entries, shared out evenly;
//   - ceil(n(a) / SMs) (a + an entry's cost) for the n(a) entries of a tiles or more, for eight
//     lengths a: entries of that length have to be taken in that many rounds;
// plus the merge of the pieces.  Longest entries come first.  Against the best of twenty Qs in a
// simulation of that order over 120 random batches the choice costs 0.5 % on average and 10 % at
// worst.  Where an SM's share is twice the longest entry cutting gained nothing (in none of 37
// such batches), and the search is left out.  (Qs that fill one, two or three whole rounds, as
// the rule was before, cost 10 % on average and up to 5 x: a long sequence among many short ones
// was not cut.  12 mixed sequences 67.5 -> 62.5 us, one of 64000 keys among 256 of 110 690 -> 196.)
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace yoco {

constexpr int kPlanThreads = 512;
constexpr int kPlanRanked = 256;  // sequences that are ordered by length
constexpr int kPlanTries = 16;    // Qs, one to a warp
__constant__ const float kPlanShare[kPlanTries] = {0.f,  3.f,  2.f,   1.5f, 1.2f, 1.f,  .85f, .7f,  // (0: no cut)
                                                   .6f, .5f, .42f, .35f, .3f,  .25f, .2f,  .15f};
constexpr int kPlanNoCut = 1 << 30;

struct PlanSeq {
    int first, n, pos, blocks, tiles;  // tiles: of the row block that sees most, give or take one
};

__device__ __forceinline__ PlanSeq plan_seq(const PagedView &pv, const int32_t *cu, int rows, int T_R, int b, int *err) {
    PlanSeq s{0, 0, 0, 0, 0};
    const int len = paged_len(pv, b, err);  // (asked for before the rows are known: one latency, not two)
    s.n = paged_rows(cu, rows, b, s.first, err);
    if (s.n == 0) return s;
    s.blocks = (s.n + T_R - 1) / T_R;
    s.pos = len - s.n;
    const int last = s.pos + (s.blocks - 1) * T_R;
    s.tiles = paged_range(pv, last, s.pos + s.n - 1).ntiles;
    // with a window a last row block of few rows sees less than the one before it
    if (pv.window > 0 && s.blocks > 1) s.tiles = max(s.tiles, paged_range(pv, last - T_R, last - 1).ntiles);
    return s;
}

__device__ __forceinline__ int plan_pieces(int tiles, int Q) { return max(1, (tiles + Q - 1) / Q); }

template <typename T> __device__ __forceinline__ T plan_sum(T x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

struct PlanArgs {
    const int32_t *cu;
    int rows, T_R, slots, max_split, min_piece;
    float entry_cost, split_cost;
    int cap;
    PagedPlan *plan;
    PagedEntry *entries, *cuts;
    int *err;
};

// sizes are tried where something may be gained by them, and where the list has room for cuts
// (rows counted twice by overlapping cu_rows may pass its end: then nothing is cut)
__device__ __forceinline__ bool plan_tries(const PlanArgs &a, int Hkv, float W, long long nblocks, int longest) {
    return a.max_split > 0 && nblocks <= a.cap - a.max_split / Hkv &&
           2.f * ((float)longest + a.entry_cost) > (W + (float)(nblocks * Hkv) * a.entry_cost) / (float)a.slots;
}

// A warp's try: its Q, and what the call is estimated to take with it, in tiles of an SM; seq(b)
// is {row blocks, tiles} of sequence b
template <typename Seq>
__device__ __forceinline__ float plan_cost(const PlanArgs &a, int B, int Hkv, int warp, float W, Seq seq, int &q) {
    const int lane = threadIdx.x & 31;
    q = warp == 0 ? kPlanNoCut : max(a.min_piece, (int)ceilf(min(W / (float)a.slots * kPlanShare[warp], 1e9f)));
    int n = 0, split = 0, most = 0;
#pragma unroll 1
    for (int b = lane; b < B; b += 32) {
        const int2 s = seq(b);
        if (s.x == 0) continue;
        const int pc = plan_pieces(s.y, q);
        n += s.x * pc;
        split += pc > 1 ? s.x * pc : 0;
        most = max(most, (s.y + pc - 1) / pc);
    }
    n = __reduce_add_sync(0xffffffffu, n) * Hkv;
    split = __reduce_add_sync(0xffffffffu, split) * Hkv;
    most = __reduce_max_sync(0xffffffffu, most);
    float cost = (W + (float)n * a.entry_cost) / (float)a.slots;
    int over[8] = {0, 0, 0, 0, 0, 0, 0, 0};  // entries of at least that part of the longest
    constexpr float part[8] = {1.f, .85f, .7f, .6f, .5f, .42f, .34f, .25f};
#pragma unroll 1
    for (int b = lane; b < B; b += 32) {
        const int2 s = seq(b);
        if (s.x == 0) continue;
        const int pc = plan_pieces(s.y, q), len = (s.y + pc - 1) / pc;
#pragma unroll
        for (int k = 0; k < 8; ++k) over[k] += (float)len >= part[k] * (float)most ? s.x * pc : 0;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int rounds = (__reduce_add_sync(0xffffffffu, over[k]) * Hkv + a.slots - 1) / a.slots;
        cost = max(cost, (float)rounds * (part[k] * (float)most + a.entry_cost));
    }
    cost += split > 0 ? .75f * a.entry_cost + (float)split * a.split_cost : 0.f;
    return split <= a.max_split ? cost : 3e38f;
}

// entry e: number idx of sequence b's, whose partial results and cut row blocks start at slot0, cut0
__device__ __forceinline__ void plan_entry(const PlanArgs &a, const PagedView &pv, const PlanSeq &s, int b, int pc, int idx,
                                           int e, int slot0, int cut0) {
    const int per = (s.tiles + pc - 1) / pc;
    // the row blocks that see most come first; a cut sequence's row blocks of one piece are
    // neighbours (they read the same keys)
    const int piece = idx / s.blocks, j = s.blocks - 1 - (idx - piece * s.blocks);
    PagedEntry o;
    o.b = b;
    o.row0 = s.first + j * a.T_R;
    o.nrow = min(a.T_R, s.n - j * a.T_R);
    o.pos0 = s.pos + j * a.T_R;
    o.range = paged_range(pv, o.pos0, o.pos0 + o.nrow - 1);
    // one may see a tile more than `tiles`, or many fewer: the last piece takes what is left
    o.pieces = min(pc, max(1, per > 0 ? (o.range.ntiles + per - 1) / per : 1));
    o.i0 = min(piece * per, o.range.ntiles);
    o.i1 = piece == pc - 1 ? o.range.ntiles : min(o.i0 + per, o.range.ntiles);
    if (piece >= o.pieces) o.nrow = 0;
    o.slot = slot0 + idx;
    o.stride = s.blocks;
    o.pad = 0;
    const int4 *from = reinterpret_cast<const int4 *>(&o);
#pragma unroll
    for (int x = 0; x < 4; ++x) reinterpret_cast<int4 *>(a.entries + e)[x] = from[x];
    if (pc > 1 && piece == 0) {  // for the merge
#pragma unroll
        for (int x = 0; x < 4; ++x) reinterpret_cast<int4 *>(a.cuts + cut0 + idx)[x] = from[x];
    }
}

// Up to 32 sequences: lane b of every warp has sequence b in registers, one barrier (for the tries).
__global__ void __launch_bounds__(kPlanThreads)
paged_plan_small_kernel(const PagedView pv, const PlanArgs a) {
    __shared__ float c_cost[kPlanTries];
    __shared__ int c_q[kPlanTries];
    static_assert(kPlanTries <= kPlanThreads / 32 && kPlanTries <= 32, "a warp for each try, a lane for each cost");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, B = pv.B;
    constexpr int kWarps = kPlanThreads / 32;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    PlanSeq s{0, 0, 0, 0, 0};
    if (lane < B) s = plan_seq(pv, a.cu, a.rows, a.T_R, lane, warp == 0 ? a.err : nullptr);
    const float W = plan_sum((float)s.blocks * (float)s.tiles) * (float)pv.Hkv;
    const long long nblocks = plan_sum((long long)s.blocks);
    const int longest = __reduce_max_sync(0xffffffffu, s.tiles);
    int Q = kPlanNoCut;
    if (plan_tries(a, pv.Hkv, W, nblocks, longest)) {
        if (warp < kPlanTries) {
            int q;
            const float cost = plan_cost(a, B, pv.Hkv, warp, W, [&](int) { return make_int2(s.blocks, s.tiles); }, q);
            if (lane == 0) {
                c_cost[warp] = cost;
                c_q[warp] = q;
            }
        }
        __syncthreads();
        // (costs are positive: their bits are in their order)
        const unsigned mine = lane < kPlanTries ? __float_as_uint(c_cost[lane]) : 0xffffffffu;
        const unsigned least = __reduce_min_sync(0xffffffffu, mine);
        Q = c_q[__ffs(__ballot_sync(0xffffffffu, mine == least)) - 1];
    }
    // longest entries first: where this lane's sequence starts is what all before it take
    const int pc = plan_pieces(s.tiles, Q), len = s.blocks > 0 ? (s.tiles + pc - 1) / pc : -1;
    long long start = 0, slot0 = 0, cut0 = 0, all = 0, all_cut = 0;
#pragma unroll 4
    for (int o = 0; o < B; ++o) {
        const int o_len = __shfl_sync(0xffffffffu, len, o), o_blocks = __shfl_sync(0xffffffffu, s.blocks, o);
        const int o_pc = __shfl_sync(0xffffffffu, pc, o);
        const long long n = (long long)o_blocks * o_pc;
        all += n;
        all_cut += o_pc > 1 ? o_blocks : 0;
        if (o_len > len || (o_len == len && o < lane)) {
            start += n;
            slot0 += o_pc > 1 ? n : 0;
            cut0 += o_pc > 1 ? o_blocks : 0;
        }
    }
    if (threadIdx.x == 0) {
        a.plan->entries = (int)min(all, (long long)a.cap);
        a.plan->cut = (int)min(all_cut, (long long)a.cap);
        a.plan->next = 0;
    }
    // sequences to warps, or several warps to each of a few
    const int share = max(1, kWarps / (B > 1 ? 1 << (32 - __clz(B - 1)) : 1));
    const int first = (int)min(start, (long long)a.cap), slot = (int)min(slot0, (long long)a.cap);
    const int cut = (int)min(cut0, (long long)a.cap);
    for (int k = warp / share; k < B; k += kWarps / share) {
        PlanSeq t;
        t.first = __shfl_sync(0xffffffffu, s.first, k);
        t.n = __shfl_sync(0xffffffffu, s.n, k);
        t.pos = __shfl_sync(0xffffffffu, s.pos, k);
        t.blocks = __shfl_sync(0xffffffffu, s.blocks, k);
        t.tiles = __shfl_sync(0xffffffffu, s.tiles, k);
        const int t_pc = __shfl_sync(0xffffffffu, pc, k), t_first = __shfl_sync(0xffffffffu, first, k);
        const int t_slot = __shfl_sync(0xffffffffu, slot, k), t_cut = __shfl_sync(0xffffffffu, cut, k);
        const int n = (int)min((long long)t.blocks * t_pc, (long long)(a.cap - t_first));
        for (int idx = (warp % share) * 32 + lane; idx < n; idx += 32 * share)
            plan_entry(a, pv, t, k, t_pc, idx, t_first + idx, t_slot, t_cut);
    }
}

__global__ void __launch_bounds__(kPlanThreads)
paged_plan_kernel(const PagedView pv, const PlanArgs a) {
    extern __shared__ int sh[];
    int *tiles = sh, *blocks = tiles + pv.B, *order = blocks + pv.B;
    int *start = order + pv.B, *slot0 = start + pv.B + 1, *cut0 = slot0 + pv.B + 1;
    __shared__ float r_W[kPlanThreads / 32], c_cost[kPlanTries];
    __shared__ long long r_sum[3][kPlanThreads / 32];
    __shared__ int r_longest[kPlanThreads / 32], c_q[kPlanTries];
    static_assert(kPlanTries <= kPlanThreads / 32, "a warp for each");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = pv.B;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");

    float W = 0.f;
    long long nblocks = 0;
    int longest = 0;
#pragma unroll 1
    for (int b = tid; b < B; b += kPlanThreads) {
        const PlanSeq s = plan_seq(pv, a.cu, a.rows, a.T_R, b, a.err);
        tiles[b] = s.tiles;
        blocks[b] = s.blocks;
        W += (float)s.blocks * (float)s.tiles;
        nblocks += s.blocks;
        longest = max(longest, s.tiles);
    }
    W = plan_sum(W);
    nblocks = plan_sum(nblocks);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
        r_longest[warp] = longest;
        r_W[warp] = W;
        r_sum[0][warp] = nblocks;
    }
    __syncthreads();
    W = 0.f;
    nblocks = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        W += r_W[w];
        nblocks += r_sum[0][w];
        longest = max(longest, r_longest[w]);
    }
    W *= (float)pv.Hkv;  // tiles of all heads
    int Q = kPlanNoCut;
    if (plan_tries(a, pv.Hkv, W, nblocks, longest)) {
        if (warp < kPlanTries) {
            int q;
            const float cost = plan_cost(a, B, pv.Hkv, warp, W, [&](int b) { return make_int2(blocks[b], tiles[b]); }, q);
            if (lane == 0) {
                c_cost[warp] = cost;
                c_q[warp] = q;
            }
        }
        __syncthreads();
        int best = 0;
        for (int k = 1; k < kPlanTries; ++k)
            if (c_cost[k] < c_cost[best]) best = k;
        Q = c_q[best];
    }
    // longest entries first: ranked, or, of many sequences, by 32nds of the longest (in a class
    // the order is any: it decides who runs when, not what comes out)
    int *length = slot0;  // (its own use comes later)
    __shared__ int at_class[32];
    if (tid < 32) at_class[tid] = 0;
    __syncthreads();
    const int cut_longest = max(1, min(longest, Q));
#pragma unroll 1
    for (int b = tid; b < B; b += kPlanThreads) {
        const int pc = plan_pieces(tiles[b], Q);
        length[b] = (tiles[b] + pc - 1) / pc;
        if (B > kPlanRanked) {
            length[b] = 31 - (int)(31ll * length[b] / cut_longest);
            atomicAdd(&at_class[length[b]], 1);
        }
    }
    __syncthreads();
    if (B > kPlanRanked) {
        if (warp == 0) {
            const int n = at_class[lane];
            int inc = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += v;
            }
            at_class[lane] = inc - n;
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int b = tid; b < B; b += kPlanThreads) {
        int at = 0;
        if (B <= kPlanRanked) {
            const int mine = length[b];
            for (int o = 0; o < B; ++o) at += length[o] > mine || (length[o] == mine && o < b);
        } else {
            at = atomicAdd(&at_class[length[b]], 1);
        }
        order[at] = b;
    }
    __syncthreads();
    // where each sequence's entries, partial results and cut row blocks start
    const int each = (B + kPlanThreads - 1) / kPlanThreads;
    const int p0 = min(B, tid * each), p1 = min(B, p0 + each);
    long long sum[3] = {0, 0, 0}, inc[3];
    for (int p = p0; p < p1; ++p) {
        const int b = order[p], pc = plan_pieces(tiles[b], Q);
        const long long n = (long long)blocks[b] * pc;
        sum[0] += n;
        sum[1] += pc > 1 ? n : 0;
        sum[2] += pc > 1 ? blocks[b] : 0;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        inc[k] = sum[k];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc[k], off);
            if (lane >= off) inc[k] += v;
        }
        if (lane == 31) r_sum[k][warp] = inc[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        long long run = inc[k] - sum[k];
        for (int w = 0; w < warp; ++w) run += r_sum[k][w];
        sum[k] = run;
    }
    const long long top = 0x7fffffff;
    for (int p = p0; p <= p1; ++p) {
        if (p == p1 && p1 != B) break;  // the next thread's
        start[p] = (int)min(sum[0], top);
        slot0[p] = (int)min(sum[1], top);
        cut0[p] = (int)min(sum[2], top);
        if (p == p1) break;
        const int b = order[p], pc = plan_pieces(tiles[b], Q);
        const long long n = (long long)blocks[b] * pc;
        sum[0] += n;
        sum[1] += pc > 1 ? n : 0;
        sum[2] += pc > 1 ? blocks[b] : 0;
    }
    __syncthreads();
    const int total = min(start[B], a.cap);
    if (tid == 0) {
        a.plan->entries = total;
        a.plan->cut = cut0[B];
        a.plan->next = 0;
    }
    for (int e = tid; e < total; e += kPlanThreads) {
        int lo = 0, hi = B;  // the sequence: start[lo] <= e < start[lo + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= e) lo = mid;
            else hi = mid;
        }
        const int b = order[lo], idx = e - start[lo];
        const PlanSeq s = plan_seq(pv, a.cu, a.rows, a.T_R, b, a.err);
        plan_entry(a, pv, s, b, plan_pieces(s.tiles, Q), idx, e, slot0[lo], cut0[lo]);
    }
}

}  // namespace yoco

namespace yoco_host {
using namespace yoco;

cudaError_t paged_plan(const PagedArgs &a, const PagedGrid &g, cudaStream_t st) {
    const bool small = a.cache->B <= 32;
    cudaError_t e = small ? cudaSuccess
                          : cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)((6 * (size_t)kPagedMaxB + 3) * sizeof(int)));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = small ? 0 : (6 * (size_t)a.cache->B + 3) * sizeof(int);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    const PlanArgs p{a.cu, a.rows, g.rows, g.slots, g.max_split, g.min_piece, g.entry_cost, g.split_cost, g.cap,
                     (PagedPlan *)g.plan, (PagedEntry *)g.entries, (PagedEntry *)g.cuts, a.err};
    return cudaLaunchKernelEx(&cfg, small ? paged_plan_small_kernel : paged_plan_kernel, paged_view(a), p);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_plan)
