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

// These kernels are started while the one before them in the stream may still run, and wait for
// its end (griddepcontrol.wait).  What that one may write -- a call's plan, notes and partial
// results, and as well a caller's Q, K and V: the O of one call can be the Q of the next -- is not
// read-only while they run, so it is not loaded through the read-only path, whose loads the
// compiler may also move ahead of the wait.
__device__ __forceinline__ int paged_ld(const int *p) {
    int v;
    asm volatile("ld.global.b32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// 16 bytes of a tensor (no clobber: nothing here writes what it reads, and it keeps its place
// behind the wait, which is volatile too)
__device__ __forceinline__ uint4 paged_ld16(const void *p) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

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
// longer than the rest, a sequence's tiles are cut into pieces.  paged_plan_kernel writes
// the list of (row block, piece) from the lengths as they are on the device; the prefill
// kernels take its entries, once for every kv head.
struct alignas(16) PagedEntry {
    int b, row0, nrow, pos0;   // rows [row0, row0 + nrow) of the call, at positions pos0 ..
    int i0, i1;                // tiles of what they see
    int pieces, slot, stride;  // pieces > 1: this one's partial result is `slot`, piece 0's
                               // neighbour slot + stride (each times Hkv, plus the kv head)
    PagedRange range;
    int pad;
};
static_assert(sizeof(PagedEntry) == 64, "entries are read by 16 lanes");

struct PagedPlan {
    int entries;  // in the list
    int next;     // entry x kv head that a block takes next, counted from the grid's size
    int cut;      // row blocks in more than one piece: cuts[0 .. cut) are their first entries
};

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
