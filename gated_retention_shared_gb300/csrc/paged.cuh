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

// The tiles seen by rows at positions p_lo .. p_hi: `nsink` tiles from slot 0 on, then
// those from tile lo_tile on.  A slot m of them is seen by some row when
// m < hi and (m >= lo or m < sinks).
struct PagedRange {
    int lo, hi, lo_tile, nsink, ntiles;
    __device__ __forceinline__ int key0(int i) const { return (i < nsink ? i : lo_tile + i - nsink) * kPagedTile; }
};

__device__ __forceinline__ PagedRange paged_range(const PagedView &pv, int p_lo, int p_hi) {
    PagedRange r;
    r.hi = max(p_hi + 1, 0);
    r.lo = pv.window > 0 ? max(0, p_lo - pv.window + 1) : 0;
    r.lo_tile = r.lo / kPagedTile;
    r.nsink = min((pv.sinks + kPagedTile - 1) / kPagedTile, r.lo_tile);
    r.ntiles = r.hi > 0 ? r.nsink + (r.hi + kPagedTile - 1) / kPagedTile - r.lo_tile : 0;
    return r;
}

// Row block j of all sequences (T_R rows to a block), counted from the last block of the
// last sequence: within a sequence the blocks that see most keys come first.  One whole
// warp; false when there are not so many.
__device__ __forceinline__ bool paged_find_block(const int32_t *cu, int rows, int B, int T_R, int j, int &b, int &blk,
                                                 int *err) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int hi = B; hi > 0; hi -= 32) {
        const int s = hi - 1 - lane;
        int first, n = 0;
        if (s >= 0) n = (paged_rows(cu, rows, s, first, err) + T_R - 1) / T_R;
        int inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        const int total = __shfl_sync(0xffffffffu, inc, 31);
        if (j < before + total) {
            const int src = __ffs(__ballot_sync(0xffffffffu, before + inc > j)) - 1;
            b = hi - 1 - src;
            const int nn = __shfl_sync(0xffffffffu, n, src);
            blk = nn - 1 - (j - before - (__shfl_sync(0xffffffffu, inc, src) - nn));
            return true;
        }
        before += total;
    }
    return false;
}

// What one thread block of the prefill kernels works on: rows [row0, row0 + nrow) of the
// call, at positions pos0 .., all query heads of kv head hk, and tiles [i0, i1) of the
// keys they see.  `pieces` blocks share the rows (1: no merge).
struct PagedBlock {
    int b, hk, row0, nrow, pos0, i0, i1, pieces;
    PagedRange range;
};

constexpr int kPagedMinTiles = 4;  // a split of the keys is at least this long (but for the last)

// split `sp` of `splits` of row block j; one whole warp; nrow = 0 when there is no such block
__device__ __forceinline__ void paged_block(const PagedView &pv, const int32_t *cu, int rows, int T_R, int j, int hk,
                                            int sp, int splits, PagedBlock &o, int *err) {
    int blk = 0;
    o.nrow = 0;
    o.hk = hk;
    if (!paged_find_block(cu, rows, pv.B, T_R, j, o.b, blk, err)) return;
    int first;
    const int n = paged_rows(cu, rows, o.b, first, err);
    o.row0 = first + blk * T_R;
    o.nrow = min(T_R, n - blk * T_R);
    o.pos0 = paged_len(pv, o.b, err) - n + blk * T_R;
    o.range = paged_range(pv, o.pos0, o.pos0 + o.nrow - 1);
    const int per = max((o.range.ntiles + splits - 1) / splits, kPagedMinTiles);
    o.pieces = max(1, (o.range.ntiles + per - 1) / per);
    o.i0 = min(sp * per, o.range.ntiles);
    o.i1 = min(o.i0 + per, o.range.ntiles);
    if (sp >= o.pieces) o.nrow = 0;
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
