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

// (documents shorten row blocks one by one: plan_range)
template <bool MOD>
__device__ __forceinline__ PlanSeq plan_seq(const PagedView &pv, const PagedMod &mod, const int32_t *cu, int rows, int T_R, int b,
                                            int *err) {
    PlanSeq s{0, 0, 0, 0, 0};
    int prefix = 0;
    if constexpr (MOD) prefix = mod.prefix ? mod.prefix[b] : 0;
    const int len = paged_len(pv, b, err);  // (asked for before the rows are known: one latency, not two)
    s.n = paged_rows(cu, rows, b, s.first, err);
    if (s.n == 0) return s;
    s.blocks = (s.n + T_R - 1) / T_R;
    s.pos = len - s.n;
    const int last = s.pos + (s.blocks - 1) * T_R;
    auto tiles = [&](int p0, int p1) {
        if constexpr (MOD) return paged_range_mod(pv, p0, p1, len, prefix, 0).ntiles;
        else return paged_range(pv, p0, p1).ntiles;
    };
    s.tiles = tiles(last, s.pos + s.n - 1);
    // with a window a last row block of few rows sees less than the one before it
    if (pv.window > 0 && s.blocks > 1) s.tiles = max(s.tiles, tiles(last - T_R, last - 1));
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
    void *entries, *cuts;  // PagedKind<MOD>::Entry
    int *doc_lo;           // a scored call's
    int units;             // with documents: row blocks that are planned one by one; 0: more than there is room for
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
    // (a lane to each, and the loops above not unrolled: one block that runs each line once or twice takes as
    // long as its code takes to come.  8192 rows of documents 96.9 us; loops unrolled by two 98.0, four 99.4)
    int n_over = 0;
    float its_part = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int sum = __reduce_add_sync(0xffffffffu, over[k]);
        n_over = lane == k ? sum : n_over;
        its_part = lane == k ? part[k] : its_part;
    }
    const int rounds = (n_over * Hkv + a.slots - 1) / a.slots;
    cost = max(cost, (float)rounds * (its_part * (float)most + a.entry_cost));
    cost = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(cost)));  // (positive: in their bits' order)
    cost += split > 0 ? .75f * a.entry_cost + (float)split * a.split_cost : 0.f;
    return split <= a.max_split ? cost : 3e38f;
}

// the Q of the least cost, the first of several (costs are positive: their bits are in their order)
__device__ __forceinline__ int plan_best(const float *cost, const int *q) {
    const int lane = threadIdx.x & 31;
    const unsigned mine = lane < kPlanTries ? __float_as_uint(cost[lane]) : 0xffffffffu;
    const unsigned least = __reduce_min_sync(0xffffffffu, mine);
    return q[__ffs(__ballot_sync(0xffffffffu, mine == least)) - 1];
}

// what row block j of sequence b sees, number g of the call's (row bounds that overlap may pass the
// list's end: such a block is taken to see everything)
__device__ __forceinline__ PagedRangeMod plan_range(const PlanArgs &a, const PagedView &pv, const PagedMod &mod,
                                                    const PlanSeq &s, int b, int j, int g) {
    const int pos0 = s.pos + j * a.T_R, n = min(a.T_R, s.n - j * a.T_R);
    return paged_range_mod(pv, pos0, pos0 + n - 1, s.pos + s.n, mod.prefix ? mod.prefix[b] : 0,
                           mod.doc && g < a.cap ? a.doc_lo[g] : 0);
}

// entry e: piece `piece` of row block j of sequence b, one of pc of at most `per` tiles; its partial
// result is `slot`, the next piece's slot + stride; cut: where the merge finds its row block
template <bool MOD>
__device__ __forceinline__ void plan_entry(const PlanArgs &a, const PagedView &pv, const PagedMod &mod, const PlanSeq &s, int b,
                                           int j, int g, int piece, int pc, int e, int slot, int stride, int cut) {
    typedef typename PagedKind<MOD>::Entry Entry;
    const int per = (s.tiles + pc - 1) / pc;
    Entry o;
    o.b = b;
    o.row0 = s.first + j * a.T_R;
    o.nrow = min(a.T_R, s.n - j * a.T_R);
    o.pos0 = s.pos + j * a.T_R;
    if constexpr (MOD) o.range = plan_range(a, pv, mod, s, b, j, g);
    else o.range = paged_range(pv, o.pos0, o.pos0 + o.nrow - 1);
    // one may see a tile more than `tiles`, or many fewer: the last piece takes what is left
    o.pieces = min(pc, max(1, per > 0 ? (o.range.ntiles + per - 1) / per : 1));
    o.i0 = min(piece * per, o.range.ntiles);
    o.i1 = piece == pc - 1 ? o.range.ntiles : min(o.i0 + per, o.range.ntiles);
    if (piece >= o.pieces) o.nrow = 0;
    o.slot = slot;
    o.stride = stride;
    o.pad = 0;
    const int4 *from = reinterpret_cast<const int4 *>(&o);
    constexpr int kQuads = sizeof(Entry) / 16;
#pragma unroll
    for (int x = 0; x < kQuads; ++x) reinterpret_cast<int4 *>((Entry *)a.entries + e)[x] = from[x];
    if (pc > 1 && piece == 0) {  // for the merge
#pragma unroll
        for (int x = 0; x < kQuads; ++x) reinterpret_cast<int4 *>((Entry *)a.cuts + cut)[x] = from[x];
    }
}

// The same for number idx of sequence b's entries: the row blocks that see most come first; a cut
// sequence's row blocks of one piece are neighbours (they read the same keys).  block0: the number
// of its first row block.
template <bool MOD>
__device__ __forceinline__ void plan_seq_entry(const PlanArgs &a, const PagedView &pv, const PagedMod &mod, const PlanSeq &s,
                                               int b, int pc, int idx, int e, int slot0, int cut0, int block0) {
    const int piece = idx / s.blocks, j = s.blocks - 1 - (idx - piece * s.blocks);
    plan_entry<MOD>(a, pv, mod, s, b, j, block0 + j, piece, pc, e, slot0 + idx, s.blocks, cut0 + idx);
}

// Up to 32 sequences: lane b of every warp has sequence b in registers, one barrier (for the tries).
template <bool MOD>
__global__ void __launch_bounds__(kPlanThreads)
paged_plan_small_kernel(const PagedView pv, const PagedMod mod, const PlanArgs a) {
    __shared__ float c_cost[kPlanTries];
    __shared__ int c_q[kPlanTries];
    static_assert(kPlanTries <= kPlanThreads / 32 && kPlanTries <= 32, "a warp for each try, a lane for each cost");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, B = pv.B;
    constexpr int kWarps = kPlanThreads / 32;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    PlanSeq s{0, 0, 0, 0, 0};
    if (lane < B) s = plan_seq<MOD>(pv, mod, a.cu, a.rows, a.T_R, lane, warp == 0 ? a.err : nullptr);
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
        Q = plan_best(c_cost, c_q);
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
            plan_seq_entry<MOD>(a, pv, mod, t, k, t_pc, idx, t_first + idx, t_slot, t_cut, 0);
    }
}

// With documents each row block is looked at (four lanes read its rows' document starts) and, where
// there is room for them, planned by itself as if it were a sequence: what they see may differ by
// much.  (As one sequence with the longest block's tiles 8192 rows of documents of 700 with a
// question of 100 rows that sees all of them were not cut: 157 us.)
template <bool MOD>
__global__ void __launch_bounds__(kPlanThreads)
paged_plan_kernel(const PagedView pv, const PagedMod mod, const PlanArgs a) {
    extern __shared__ int sh[];
    const int room = max(pv.B, MOD ? a.units : 0);
    int *tiles = sh, *blocks = tiles + room, *order = blocks + room;
    int *start = order + room, *slot0 = start + room + 1, *cut0 = slot0 + room + 1;
    [[maybe_unused]] int *block0 = cut0 + room + 1;  // [B + 1] row blocks before the sequence's
    __shared__ float r_W[kPlanThreads / 32], c_cost[kPlanTries];
    __shared__ long long r_sum[3][kPlanThreads / 32];
    __shared__ int r_longest[kPlanThreads / 32], c_q[kPlanTries];
    static_assert(kPlanTries <= kPlanThreads / 32, "a warp for each");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int B = pv.B;  // sequences, or row blocks that are planned one by one
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");

    float W = 0.f;
    long long nblocks = 0;
    int longest = 0;
    const bool docs = MOD && mod.doc;
    bool single = false;  // row blocks are planned one by one
#pragma unroll 1
    for (int b = tid; b < B; b += kPlanThreads) {
        const PlanSeq s = plan_seq<MOD>(pv, mod, a.cu, a.rows, a.T_R, b, a.err);
        tiles[b] = docs ? 0 : s.tiles;
        blocks[b] = s.blocks;
        nblocks += s.blocks;
        if (!docs) {
            W += (float)s.blocks * (float)s.tiles;
            longest = max(longest, s.tiles);
        }
    }
    if (docs) {
        __syncthreads();
        const int each = (B + kPlanThreads - 1) / kPlanThreads;
        const int p0 = min(B, tid * each), p1 = min(B, p0 + each);
        long long mine = 0, sum;
        for (int b = p0; b < p1; ++b) mine += blocks[b];
        sum = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += v;
        }
        if (lane == 31) r_sum[1][warp] = sum;
        __syncthreads();
        long long run = sum - mine;
        for (int w = 0; w < warp; ++w) run += r_sum[1][w];
        for (int b = p0; b < p1; ++b) {
            block0[b] = (int)min(run, 0x7fffffffll);
            run += blocks[b];
        }
        if (p0 < B && p1 == B) block0[B] = (int)min(run, 0x7fffffffll);
        __syncthreads();
        // (row bounds that overlap may pass what there is room for)
        single = block0[B] <= a.units;
        const int all = min(block0[B], a.cap);
        for (int g0 = tid / 4; g0 - (tid & 31) / 4 < all; g0 += kPlanThreads / 4) {
            const int g = min(g0, all - 1);
            int lo = 0, hi = B;  // the sequence: block0[lo] <= g < block0[lo + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (block0[mid] <= g) lo = mid;
                else hi = mid;
            }
            const PlanSeq s = plan_seq<MOD>(pv, mod, a.cu, a.rows, a.T_R, lo, nullptr);
            const int j = g - block0[lo], r1 = min(s.n, (j + 1) * a.T_R);
            int least = 0x7fffffff;
            for (int r = j * a.T_R + (lane & 3); r < r1; r += 48) {  // (twelve loads on their way at a time)
#pragma unroll
                for (int k = 0; k < 12; ++k) least = min(least, mod.doc[s.first + min(r + 4 * k, r1 - 1)]);
            }
#pragma unroll
            for (int off = 2; off > 0; off >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, off));
            if ((lane & 3) == 0 && g0 < all) {
                a.doc_lo[g] = least;
                const int n = plan_range(a, pv, mod, s, lo, j, g).ntiles;
                if (single) {
                    tiles[g] = n;
                    blocks[g] = 1;
                } else {
                    atomicMax(&tiles[lo], n);
                }
                W += (float)n;
                longest = max(longest, n);
            }
            __syncwarp();
        }
        __syncthreads();  // (r_sum is written again)
        if (single) B = all;
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
        Q = plan_best(c_cost, c_q);
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
        const int b = order[lo], idx = e - start[lo], pc = plan_pieces(tiles[b], Q);
        if (single) {
            int seq = 0, end = pv.B;  // row block b's sequence
            while (end - seq > 1) {
                const int mid = (seq + end) >> 1;
                if (block0[mid] <= b) seq = mid;
                else end = mid;
            }
            PlanSeq s = plan_seq<MOD>(pv, mod, a.cu, a.rows, a.T_R, seq, nullptr);
            s.tiles = tiles[b];
            plan_entry<MOD>(a, pv, mod, s, seq, b - block0[seq], b, idx, pc, e, slot0[lo] + idx, 1, cut0[lo]);
        } else {
            PlanSeq s = plan_seq<MOD>(pv, mod, a.cu, a.rows, a.T_R, b, nullptr);
            s.tiles = tiles[b];
            plan_seq_entry<MOD>(a, pv, mod, s, b, pc, idx, e, slot0[lo], cut0[lo], docs ? block0[b] : 0);
        }
    }
}

}  // namespace yoco

namespace yoco_host {
using namespace yoco;

template <bool MOD> static cudaError_t plan_launch(const PagedArgs &a, const PagedGrid &g, cudaStream_t st) {
    const bool docs = a.scores && a.scores->doc_first, small = a.cache->B <= 32 && !docs;
    // row blocks of any bounds that do not overlap: as many as the list has entries for them
    const int64_t most = (int64_t)a.rows / g.rows + std::min(a.cache->B, a.rows);
    const int units = docs && most <= kPagedMaxB ? (int)most : 0;
    const size_t n = (size_t)std::max(a.cache->B, units);
    cudaError_t e = cudaSuccess;
    if (!small)
        e = cudaFuncSetAttribute(paged_plan_kernel<MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)((7 * (size_t)kPagedMaxB + 4) * sizeof(int)));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = small ? 0 : (6 * n + 3 + (docs ? (size_t)a.cache->B + 1 : 0)) * sizeof(int);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    const PlanArgs p{a.cu, a.rows, g.rows, g.slots, g.max_split, g.min_piece, g.entry_cost, g.split_cost, g.cap,
                     (PagedPlan *)g.plan, g.entries, g.cuts, g.doc_lo, units, a.err};
    return cudaLaunchKernelEx(&cfg, small ? paged_plan_small_kernel<MOD> : paged_plan_kernel<MOD>, paged_view(a), paged_mod(a), p);
}

cudaError_t paged_plan(const PagedArgs &a, const PagedGrid &g, cudaStream_t st) {
    return a.scores ? plan_launch<true>(a, g, st) : plan_launch<false>(a, g, st);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_plan)
