// paged.cuh -- what the kernels over the paged cache share: the cache's device view,
// the lengths it may hold, and which 128-key tiles the rows of a block see.
//
// Sequence b of length L keeps slot p at row p % page of page table[b][p / page] of
// k, v [num_pages, Hkv, page, d].  The row at position p sees slot m when m <= p and,
// with a window W > 0, p - W < m or m < sinks.  Rows at negative positions (more new
// rows than the sequence holds) see nothing and come out as zeros.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"

namespace yoco {

struct PagedView {
    const int32_t *table;  // [B, max_pages]
    const int32_t *lens;   // [B]
    int32_t B, Hkv, max_pages, num_pages;
    int32_t shift;         // log2 of the page size
    int32_t window, sinks; // 0: no window
};

constexpr int kPagedTile = 128;  // keys per tile

// workspace status codes of bad metadata (kErrMagic | code); the call goes on without
// touching what they name
constexpr int kErrPagedLen = 0x60;   // a length below zero or past the table
constexpr int kErrPagedPage = 0x61;  // a page number outside the pool
constexpr int kErrPagedRows = 0x62;  // cu_rows decreases or leaves [0, rows]

__device__ __forceinline__ void paged_report(int *err, int code) {
    if (err) atomicExch(err, (int)(kErrMagic | (uint32_t)code));
}

// length of sequence b; one that no table row can hold counts as empty
__device__ __forceinline__ int paged_len(const PagedView &pv, int b, int *err) {
    const int L = pv.lens[b];
    if (L < 0 || L > (int)((uint32_t)pv.max_pages << pv.shift)) {
        paged_report(err, kErrPagedLen);
        return 0;
    }
    return L;
}

// first row and number of rows of sequence b among the call's rows (cu == nullptr: row b)
__device__ __forceinline__ int paged_rows(const int32_t *cu, int rows, int b, int &first, int *err) {
    if (!cu) {
        first = b;
        return 1;
    }
    const int c0 = cu[b], c1 = cu[b + 1];
    if (c0 < 0 || c1 < c0 || c1 > rows) {
        paged_report(err, kErrPagedRows);
        first = 0;
        return 0;
    }
    first = c0;
    return c1 - c0;
}

// page that holds slots [e << shift, ...) of sequence b, or -1 where the table names none
__device__ __forceinline__ int paged_page(const PagedView &pv, int b, int e, int *err) {
    if (e >= pv.max_pages) return -1;
    const int p = pv.table[(size_t)b * pv.max_pages + e];
    if ((unsigned)p >= (unsigned)pv.num_pages) {
        paged_report(err, kErrPagedPage);
        return -1;
    }
    return p;
}

// The slots seen by rows at positions p_lo .. p_hi, in order: whole chunks of up to a page
// (at most 128 slots) of the sinks that lie before the window's first chunk, then from that
// chunk on.  Place v of this list is slot slot(v); tile i is places 128 i .. 128 i + 127.
// Slot m of them is seen by some row when m < hi and (m >= lo or m < sinks).  Cutting the
// list by chunks, not by 128 slots, lets a few sinks and the window's start share a tile.
struct PagedRange {
    int lo, hi, base, sink_slots, places, ntiles;
    __device__ __forceinline__ int slot(int v) const { return v < sink_slots ? v : v - sink_slots + base; }
    // some place of tile i is no row's
    __device__ __forceinline__ bool edge(int i, int sinks) const {
        const int v = i * kPagedTile;
        return v + kPagedTile > places || !(v >= sink_slots + lo - base || v + kPagedTile <= min(sinks, sink_slots));
    }
    __device__ __forceinline__ bool seen(int m, int sinks) const { return m < hi && (m >= lo || m < sinks); }
};

__device__ __forceinline__ PagedRange paged_range(const PagedView &pv, int p_lo, int p_hi) {
    PagedRange r;
    const int cs = min(pv.shift, 7);
    r.hi = max(p_hi + 1, 0);
    r.lo = pv.window > 0 ? max(0, p_lo - pv.window + 1) : 0;
    r.base = (r.lo >> cs) << cs;
    r.sink_slots = min(((pv.sinks + (1 << cs) - 1) >> cs) << cs, r.base);
    r.places = r.hi > 0 ? r.sink_slots + r.hi - r.base : 0;
    r.ntiles = (r.places + kPagedTile - 1) / kPagedTile;
    return r;
}

// ---------------------------------------------- chunks of rows (prefill)
//
// Rows of a sequence go to blocks of T_R; where that leaves SMs idle or one sequence much
// longer than the rest, a sequence's tiles are cut into pieces of at most Q tiles, each
// (piece, kv head, block) a thread block of its own.  Q is chosen on the device from the
// lengths as they are (nothing on the host needs to know them) by every thread block alike.

// one sequence's part of a call: its rows, its row blocks and the tiles of its last block
struct PagedSeq {
    int first, n, pos, blocks, tiles;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedView &pv, const int32_t *cu, int rows, int T_R, int b, int *err) {
    PagedSeq s{0, 0, 0, 0, 0};
    if (b < 0 || b >= pv.B) return s;
    s.n = paged_rows(cu, rows, b, s.first, err);
    if (s.n == 0) return s;
    s.blocks = (s.n + T_R - 1) / T_R;
    s.pos = paged_len(pv, b, err) - s.n;
    s.tiles = paged_range(pv, s.pos + (s.blocks - 1) * T_R, s.pos + s.n - 1).ntiles;
    return s;
}

__device__ __forceinline__ int paged_pieces(const PagedSeq &s, int Q) { return max(1, (s.tiles + Q - 1) / Q); }

constexpr int kPagedNoSplit = 1 << 30;
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Q for the call; one whole warp, `s` its lanes' sequences B - 1 - lane.  `slots` blocks are
// resident at a time, at most max_split may be pieces of something; a piece has min_piece
// tiles or more, and a block costs block_cost tiles beside its own.  Nothing is cut where
// the row blocks keep the slots busy for two rounds and none is longer than a slot's share.
// Else the smallest Q with which all blocks fit one, two or three rounds of `slots` is
// compared with no cut: by the tiles and blocks to a slot, the last round's idle part, and
// never less than the longest block.
__device__ __forceinline__ int paged_plan(const PagedView &pv, const int32_t *cu, int rows, int T_R, int slots,
                                          int max_split, int min_piece, float block_cost, const PagedSeq &s,
                                          int *err) {
    if (max_split == 0) return kPagedNoSplit;
    const int lane = threadIdx.x & 31;
    int units = s.blocks * pv.Hkv, longest = s.tiles;
    float W = (float)units * (float)s.tiles;
    for (int b = pv.B - 33 - lane; b + lane >= 0; b -= 32) {
        const PagedSeq o = paged_seq(pv, cu, rows, T_R, b, err);
        units += o.blocks * pv.Hkv;
        longest = max(longest, o.tiles);
        W += (float)(o.blocks * pv.Hkv) * (float)o.tiles;
    }
    W = warp_sum(W);
    units = __reduce_add_sync(0xffffffffu, units);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (units >= 2 * slots && (float)longest * (float)slots <= W) return kPagedNoSplit;
    if (pv.B > 32)  // many sequences: pieces of 1 / 1.5 of a slot's share (at most max_split of them)
        return max(min_piece, (int)ceilf(min(1e9f, 2.f * W / (float)max_split)) + 1);
    auto cost = [&](int items, int most) {
        const float x = (float)items / (float)slots, one = (float)most + block_cost;
        return max(one, (W + (float)items * block_cost) / (float)slots + (ceilf(x) - x) * one);
    };
    int best_q = kPagedNoSplit;
    float best = cost(units, longest);
    for (int k = 1; k <= 3; ++k) {
        int Q = max(min_piece, (int)ceilf(W / (float)(slots * k)));
        for (int it = 0; it < 6; ++it) {
            const int pc = paged_pieces(s, Q), mine = s.blocks * pv.Hkv * pc;
            const int items = __reduce_add_sync(0xffffffffu, mine);
            const int split = __reduce_add_sync(0xffffffffu, pc > 1 ? mine : 0);
            if (items <= slots * k && split <= max_split) {
                const float c = cost(items, __reduce_max_sync(0xffffffffu, (s.tiles + pc - 1) / pc)) + block_cost;
                if (c < best) {
                    best = c;
                    best_q = Q;
                }
                break;
            }
            Q = max(Q + 1, (int)min(1e9f, (float)Q * (float)items / (float)(slots * k)));
        }
    }
    return best_q;
}

// What one thread block of the prefill kernels works on: rows [row0, row0 + nrow) of the
// call, at positions pos0 .., all query heads of kv head hk, and tiles [i0, i1) of what they
// see.  `pieces` blocks share the rows (1: nothing to join); this one's partial result goes
// to `slot`, piece p's to slot + (p - piece) stride.
struct PagedBlock {
    int b, hk, row0, nrow, pos0, i0, i1, pieces, slot, stride;
    PagedRange range;
};

// Block `item` of the call, or with SPLIT the item-th (row block, kv head) of the sequences
// that are cut, as its first piece.  From the last sequence to the first; within a
// sequence that is cut all row blocks of one (piece, kv head) are neighbours (they read the
// same keys), within one that is not the row blocks that see most come first.  One whole
// warp, `s` its lanes' sequences B - 1 - lane; nrow = 0 when there is no such block.
template <bool SPLIT>
__device__ __forceinline__ void paged_block(const PagedView &pv, const int32_t *cu, int rows, int T_R, int Q, int item,
                                            PagedSeq s, PagedBlock &o, int *err) {
    const int lane = threadIdx.x & 31;
    o.nrow = 0;
    o.pieces = 1;
    int before = 0, slots = 0;
    for (int hi = pv.B; hi > 0; hi -= 32) {
        if (hi < pv.B) s = paged_seq(pv, cu, rows, T_R, hi - 1 - lane, err);
        const int pc = paged_pieces(s, Q), units = s.blocks * pv.Hkv;
        const int mine = SPLIT ? (pc > 1 ? units : 0) : units * pc, cut = pc > 1 ? units * pc : 0;
        int inc = mine, inc_s = cut;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off), u = __shfl_up_sync(0xffffffffu, inc_s, off);
            if (lane >= off) {
                inc += v;
                inc_s += u;
            }
        }
        const int total = __shfl_sync(0xffffffffu, inc, 31);
        if (item < before + total) {
            const int src = __ffs(__ballot_sync(0xffffffffu, before + inc > item)) - 1;
            const int first = __shfl_sync(0xffffffffu, s.first, src), n = __shfl_sync(0xffffffffu, s.n, src);
            const int pos = __shfl_sync(0xffffffffu, s.pos, src), nb = __shfl_sync(0xffffffffu, s.blocks, src);
            const int tiles = __shfl_sync(0xffffffffu, s.tiles, src), p = __shfl_sync(0xffffffffu, pc, src);
            const int idx = item - before - __shfl_sync(0xffffffffu, inc - mine, src);
            slots += __shfl_sync(0xffffffffu, inc_s - cut, src);
            int piece = 0, j;
            if (p > 1) {
                j = nb - 1 - idx % nb;
                o.hk = idx / nb % pv.Hkv;
                piece = idx / nb / pv.Hkv;
            } else {
                o.hk = idx % pv.Hkv;
                j = nb - 1 - idx / pv.Hkv;
            }
            const int per = (tiles + p - 1) / p;
            o.b = hi - 1 - src;
            o.row0 = first + j * T_R;
            o.pos0 = pos + j * T_R;
            o.stride = pv.Hkv * nb;
            o.slot = slots + idx;
            const int nr = min(T_R, n - j * T_R);
            o.range = paged_range(pv, o.pos0, o.pos0 + nr - 1);
            // a block may see a tile more or less than the last one: the last piece takes what is left
            o.pieces = min(p, max(1, per > 0 ? (o.range.ntiles + per - 1) / per : 1));
            o.i0 = min(piece * per, o.range.ntiles);
            o.i1 = piece == p - 1 ? o.range.ntiles : min(o.i0 + per, o.range.ntiles);
            if (piece < o.pieces) o.nrow = nr;
            return;
        }
        before += total;
        slots += __shfl_sync(0xffffffffu, inc_s, 31);
    }
}

// ------------------------------------------------ one row per sequence (decode)
//
// The tiles of every (sequence, kv head), one after the other, are cut into equal runs,
// one run per thread block: the blocks finish together however the lengths differ, and
// nothing on the host needs to know them.  A (sequence, kv head) that a cut runs through
// is left as partial results (at most two per block: its run's first and last), merged
// by paged_merge_kernel.

constexpr int kPagedMaxB = 4096;

// what block c tells the merge about the first unit of its run
struct PagedCut {
    int unit;             // b * Hkv + kv head when block c is the second of the blocks that share it, else -1
    int c_first, c_last;  // the blocks that share it
    int slot_first;       // which of c_first's two partials is its
};

// tiles of all sequences before b into pre[b] (shared memory, B + 1 entries); all
// THREADS threads; `sums` one int per warp
template <int THREADS>
__device__ __forceinline__ void paged_prefix(const PagedView &pv, int *pre, int *sums, int *err) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (pv.B + THREADS - 1) / THREADS;
    const int b0 = min(pv.B, tid * each), b1 = min(pv.B, b0 + each);
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int L = paged_len(pv, b, err);
        const int n = paged_range(pv, L - 1, L - 1).ntiles;
        pre[b] = n;
        mine += n;
    }
    int inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += v;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int run = inc - mine;
    for (int w = 0; w < warp; ++w) run += sums[w];
    for (int b = b0; b < b1; ++b) {
        const int n = pre[b];
        pre[b] = run;
        run += n;
    }
    if (b0 < pv.B && b1 == pv.B) pre[pv.B] = run;
    __syncthreads();
}

// Walks a run of tiles, unit by unit.
struct PagedWalk {
    int g, g1;             // tiles left: [g, g1)
    int b, hk, n;          // unit
    int t0, t1;            // its tiles in this run
    __device__ __forceinline__ bool start(const PagedView &pv, const int *pre, int from, int to) {
        g = from;
        g1 = to;
        if (g >= g1) return false;
        int lo = 0, hi = pv.B;  // the b with pre[b] Hkv <= g < pre[b + 1] Hkv
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] * pv.Hkv <= g) lo = mid;
            else hi = mid;
        }
        b = lo;
        n = pre[b + 1] - pre[b];
        const int local = g - pre[b] * pv.Hkv;
        hk = local / n;
        t0 = local - hk * n;
        t1 = min(n, t0 + (g1 - g));
        return true;
    }
    __device__ __forceinline__ bool next(const PagedView &pv, const int *pre) {
        g += t1 - t0;
        if (g >= g1) return false;
        if (++hk == pv.Hkv) {
            hk = 0;
            do ++b; while (pre[b + 1] == pre[b]);
            n = pre[b + 1] - pre[b];
        }
        t0 = 0;
        t1 = min(n, g1 - g);
        return true;
    }
    // the whole unit lies in this run
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n; }
};

// block c's note for the merge; one thread.  `each` tiles to a run
__device__ __forceinline__ PagedCut paged_cut(const PagedView &pv, const int *pre, const PagedWalk &w, int c, int each) {
    PagedCut cut{-1, 0, 0, 0};
    const int u0 = pre[w.b] * pv.Hkv + w.hk * w.n;
    cut.c_first = u0 / each;
    cut.c_last = (u0 + w.n - 1) / each;
    cut.slot_first = u0 % each ? 1 : 0;
    if (cut.c_first + 1 == c) cut.unit = w.b * pv.Hkv + w.hk;
    return cut;
}

}  // namespace yoco

namespace yoco_host {
struct PagedArgs;
yoco::PagedView paged_view(const PagedArgs &a);
// bf16, 128-byte swizzle, what lies outside reads as zeros
bool paged_map(CUtensorMap *m, const void *ptr, int rank, const uint64_t *dims, const uint64_t *strides,
               const uint32_t *box);
// a pool's k or v as {d, slot of the page, kv head, page}, boxes of 64 channels x up to a tile's slots
bool paged_kv_map(CUtensorMap *m, const void *ptr, const yoco_paged_kv *c);
}  // namespace yoco_host
