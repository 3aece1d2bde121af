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
constexpr int kErrPagedRefs = 0x63;  // more table entries name a page than refs says
constexpr int kErrPagedSeq = 0x64;   // a sequence that cannot be forked from or to
constexpr int kErrPagedRoom = 0x65;  // not enough free pages: no sequence grew

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

// ---------------------------------------------- scores and masks of the scored calls
//
// The row at position p >= 0 of a sequence of length L sees slot m < L when
//     m >= doc[row]  and  ( m < prefix[b]  or  m <= p and (W == 0 or p - W < m or m < sinks) ).
// Kernels are templates on MOD: false is the plain calls' code.
struct PagedMod {
    const float *slopes;        // [Hq], or nullptr
    const int32_t *prefix;      // [B], or nullptr
    const int32_t *doc;         // [rows], or nullptr
    float cap2;                 // cap log2(e); 0: no cap
    float qk;                   // what q.k is multiplied by: scale / cap with a cap, else scale log2(e)
    // with a cap, for |q.k| <= quick: cap2 tanh(qk s) = s (a[0] + a[1] s^2 + .. + a[degree] s^(2 degree)),
    // the others 0
    float a[6], quick;
    int degree;
    float hidden;  // a product whose weight comes out as 0 that way
};

// As PagedRange: the slots that some row of a block sees lie in `dlo <= m < hi` and (m >= lo or
// m < see), dlo the least of its rows' document starts, `see` the end of the prefix or the sinks.
// Whole chunks of the slots up to `see`, from slot `first` on, come before the window's.
struct PagedRangeMod {
    int lo, hi, base, sink_slots, places, ntiles;
    int first, dlo, see, pre;  // pre: end of the prefix
    __device__ __forceinline__ int slot(int v) const { return v < sink_slots ? v + first : v - sink_slots + base; }
    __device__ __forceinline__ bool edge(int i, int) const {
        const int v = i * kPagedTile;
        if (v + kPagedTile > places) return true;
        if (v >= sink_slots) return v - sink_slots + base < max(lo, dlo);
        return v + kPagedTile > sink_slots || v + first < dlo || v + first + kPagedTile > see;
    }
    __device__ __forceinline__ bool seen(int m, int) const { return m < hi && m >= dlo && (m >= lo || m < see); }
};

__device__ __forceinline__ PagedRangeMod paged_range_mod(const PagedView &pv, int p_lo, int p_hi, int L, int prefix, int dlo) {
    PagedRangeMod r;
    const int cs = min(pv.shift, 7);
    r.pre = p_hi < 0 ? 0 : max(0, min(prefix, L));
    r.dlo = max(dlo, 0);
    r.see = max(min(pv.sinks, max(p_hi + 1, 0)), r.pre);
    r.hi = max(max(p_hi + 1, 0), r.pre);
    r.lo = pv.window > 0 ? max(0, p_lo - pv.window + 1) : 0;
    r.base = (max(r.lo, min(r.dlo, r.hi)) >> cs) << cs;
    r.first = (min(r.dlo, r.see) >> cs) << cs;
    r.sink_slots = r.dlo < r.see ? max(0, min(((r.see + (1 << cs) - 1) >> cs) << cs, r.base) - r.first) : 0;
    r.places = r.dlo < r.hi ? r.sink_slots + r.hi - r.base : 0;
    r.ntiles = (r.places + kPagedTile - 1) / kPagedTile;
    return r;
}

// the row sees nothing at all
__device__ __forceinline__ bool paged_blind(int pos, int doc, int pre) {
    return pos < 0 || (doc > pos && max(doc, 0) >= pre);
}

// C tanh(u): in [-0.8, 0.8] (paged_cap_near) u times the minimax polynomial of tanh(u) / u in u^2 (own fit
// by reweighted least squares, relative error 6e-8), outside C - 2 C / (1 + e^2u), where nothing cancels.
// The error stays relative to the result, so a cap far above the scores costs no precision.
constexpr float kCapNear = 0.8f;
__device__ __forceinline__ float paged_cap_near(float u, float C) {
    const float x = u * u;
    float q = fmaf(x, -0.00435529966f, 0.019093302f);
    q = fmaf(x, q, -0.0531143173f);
    q = fmaf(x, q, 0.133210484f);
    q = fmaf(x, q, -0.333326749f);
    q = fmaf(x, q, 0.999999942f);
    return C * (u * q);
}
__device__ __forceinline__ float paged_cap(float u, float C) {
    const float near = paged_cap_near(u, C);
    float e, i;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(u * 2.8853900817779268f));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(i) : "f"(1.f + e));
    return fabsf(u) < kCapNear ? near : fmaf(-2.f * C, i, C);
}

// what a tensor-core kernel's rows do to their scores before the softmax, beyond the plain calls'
constexpr int kModMask = 1, kModCap = 2, kModBias = 4, kModWide = 8, kModShort = 16;

constexpr float kPagedLog2E = 1.4426950408889634f;
// the tensor-core prefill's quick way (paged_prefill_tc.cu): the polynomial of degree 3 reaches to half the
// cap, caps below kWideCap get one of degree 5 for all of the cap, those from kShortCap on one of degree 2
// for 0.26 of it (4096 rows, scores of deviation 2, us with 2, 3 and 5: cap 50 110 114 129, cap 40 116 114 128,
// cap 30 242 114 129, cap 20 273 126 128, cap 15 267 129 with 3 and 5, cap 10 279 140, cap 8 278 258)
constexpr float kWideCap = 20.f, kShortCap = 45.f;
__host__ __device__ constexpr int paged_cap_degree(int mode) { return mode & kModWide ? 5 : mode & kModShort ? 2 : 3; }
// and how large scores and slopes may be, times log2(e)
constexpr float kQuickScore = 22.f, kQuickSlope = 22.f / 15.f;

// ---------------------------------------------- chunks of rows (prefill)
//
// Rows of a sequence go to blocks of T_R; where that leaves SMs idle or one sequence much
// longer than the rest, a sequence's tiles are cut into pieces.  paged_plan_kernel writes
// the list of (row block, piece) from the lengths as they are on the device; the prefill
// kernels take its entries, once for every kv head.
template <typename Range> struct alignas(16) PagedEntryOf {
    int b, row0, nrow, pos0;   // rows [row0, row0 + nrow) of the call, at positions pos0 ..
    int i0, i1;                // tiles of what they see
    int pieces, slot, stride;  // pieces > 1: this one's partial result is `slot`, piece 0's
                               // neighbour slot + stride (each times Hkv, plus the kv head)
    Range range;
    int pad;
};
typedef PagedEntryOf<PagedRange> PagedEntry;
typedef PagedEntryOf<PagedRangeMod> PagedEntryMod;
static_assert(sizeof(PagedEntry) == 64 && sizeof(PagedEntryMod) == 80, "entries are read by as many lanes as they have words");

template <bool MOD> struct PagedKind {
    typedef PagedRange Range;
    typedef PagedEntry Entry;
};
template <> struct PagedKind<true> {
    typedef PagedRangeMod Range;
    typedef PagedEntryMod Entry;
};

// what the newest row of sequence b, of length L, sees (the decode's rows)
template <bool MOD>
__device__ __forceinline__ typename PagedKind<MOD>::Range paged_newest(const PagedView &pv, const PagedMod &mod, int b, int L) {
    if constexpr (MOD) return paged_range_mod(pv, L - 1, L - 1, L, mod.prefix ? mod.prefix[b] : 0, mod.doc ? mod.doc[b] : 0);
    else return paged_range(pv, L - 1, L - 1);
}

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
template <int THREADS, bool MOD>
__device__ __forceinline__ void paged_prefix(const PagedView &pv, const PagedMod &mod, int *pre, int *sums, int *err) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (pv.B + THREADS - 1) / THREADS;
    const int b0 = min(pv.B, tid * each), b1 = min(pv.B, b0 + each);
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int L = paged_len(pv, b, err);
        const int n = paged_newest<MOD>(pv, mod, b, L).ntiles;
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
yoco::PagedMod paged_mod(const PagedArgs &a);
// bf16, 128-byte swizzle, what lies outside reads as zeros
bool paged_map(CUtensorMap *m, const void *ptr, int rank, const uint64_t *dims, const uint64_t *strides,
               const uint32_t *box);
// a pool's k or v as {d, slot of the page, kv head, page}, boxes of 64 channels x up to a tile's slots
bool paged_kv_map(CUtensorMap *m, const void *ptr, const yoco_paged_kv *c);
}  // namespace yoco_host
