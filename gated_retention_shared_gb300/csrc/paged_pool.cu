// paged_pool.cu -- handing out the pages of a paged cache: sequences that grow, shrink, end and
// fork, and moving the used pages together (yoco_paged_resize, _fork, _compact, _copy).
//
// refs[p] is how many table entries name page p; the free pages are those with 0.  Which pages a
// call hands out goes by their numbers alone (the lowest free ones, in the order of the sequences
// and slots), so nothing depends on the order of threads: the warps of a cluster count the free
// (or used) pages of runs of kPoolRun, taken in turn (the lowest pages, which are handed out, are
// then every warp's work), and a page's rank is what lies in the runs before plus its rank in the
// run; number r of those that are wanted is found in the prefix sums of what the sequences need.
//
// A resize and a compact are one cluster of eight blocks, its phases divided by cluster barriers,
// and one grid that copies: these calls are latencies one after the other, and a launch for each
// phase cost more than what eight SMs lack in bandwidth (a search round of 8 x 4 sequences, two
// resizes and a fork, 38 -> 21 us; a serving round of two resizes of 1024 sequences over 200000
// pages 44 -> 26).  A compact's grid copies at 6.9 TB/s (1.16 GB
// moved: 168 us), the copy rate.
//
// A resize: 1. sequences that shrink give pages back; 2. one block decides, per growing sequence,
// whether the page it writes next has to be copied, and sums up what is needed, while the others
// count free pages; 3. pages are handed out; 4. the second grid copies.  Of the sequences that
// share a page and all grow the first keeps it: a table in shared memory, keyed by the page, has
// how many they are and which is first.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace yoco {

constexpr int kPoolThreads = 256;
constexpr int kClusterBlocks = 8, kClusterThreads = 1024;
constexpr int kClusterWarps = kClusterBlocks * kClusterThreads / 32;
constexpr int kShareEach = kPagedMaxB / kClusterThreads;
constexpr int kPoolLoads = 16;  // of refs, of a lane at a time
constexpr int kPoolRun = 32 * kPoolLoads, kPoolRuns = 8192;  // pages to a run, or more where the runs would not be enough
constexpr int kPoolUnroll = 4, kPoolStep = kPoolUnroll * kClusterBlocks * kClusterThreads;  // table entries of a thread at a time
constexpr int kShareSlots = 2 * kPagedMaxB;  // of the table of shared pages

struct PoolView {
    int32_t *table, *lens, *refs;
    int32_t B, max_pages, num_pages, shift;
    int4 *moves;
    // scratch
    // pages needed by the sequences before b are start[b], the first of its own goes to table entry
    // first[b] (both in every block's shared memory)
    int *old;     // [B] page that it copies, or -1
    int *fill;    // [B] slots of it in use
    int *copies;  // [B + 1] copies made by the sequences before b
    int *rank;    // [num_pages] a compact's: of a page that moves, among those; a resize's: the pages
                  // that are handed out, in order
    int *err;
};

__device__ __forceinline__ int pool_pages(const PoolView &v, int len) { return (len + (1 << v.shift) - 1) >> v.shift; }

// a length that the table can hold
__device__ __forceinline__ bool pool_len_ok(const PoolView &v, int len) {
    return len >= 0 && len <= (int)((uint32_t)v.max_pages << v.shift);
}

// sequence b's length now and after the call; one that is left alone has both the same
__device__ __forceinline__ void pool_lens(const PoolView &v, const int32_t *new_lens, int b, int &L, int &N, bool report) {
    L = v.lens[b];
    N = new_lens[b];
    if (!pool_len_ok(v, L) || (N >= 0 && !pool_len_ok(v, N))) {
        if (report) paged_report(v.err, kErrPagedLen);
        L = N = 0;
    } else if (N < 0) {
        N = L;
    }
}

// whether a table entry names a page; below 0 it says that there is none (a window has left it)
__device__ __forceinline__ bool pool_names(const PoolView &v, int p) {
    if (p >= v.num_pages) paged_report(v.err, kErrPagedPage);
    return (unsigned)p < (unsigned)v.num_pages;
}

// exclusive prefix sums of x over the block's threads; `sums` one per warp; total: of all.  (Every
// warp scans the warps' sums by itself: a loop over them in every thread took 3000 cycles.)
template <typename N> __device__ __forceinline__ N pool_scan_warp(N x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const N y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    return x;
}
template <int THREADS, typename N> __device__ __forceinline__ N pool_scan(N x, N *sums, N &total) {
    static_assert(THREADS == 1024, "a lane for each warp's sum");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const N inc = pool_scan_warp(x);
    __syncthreads();  // `sums` may still be read
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    const N mine = sums[lane], all = pool_scan_warp(mine);
    total = __shfl_sync(0xffffffffu, all, 31);
    return inc - x + __shfl_sync(0xffffffffu, all - mine, warp);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// the same place in block `rank`'s shared memory
__device__ __forceinline__ uint32_t cluster_at(const int *at, int rank) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(to) : "r"((uint32_t)__cvta_generic_to_shared(at)), "r"(rank));
    return to;
}
__device__ __forceinline__ void cluster_put(int *at, int rank, int x) {
    asm volatile("st.shared::cluster.s32 [%0], %1;\n" ::"r"(cluster_at(at, rank)), "r"(x) : "memory");
}
__device__ __forceinline__ int cluster_get(const int *at, int rank) {
    int x;
    asm volatile("ld.shared::cluster.s32 %0, [%1];\n" : "=r"(x) : "r"(cluster_at(at, rank)) : "memory");
    return x;
}

struct PoolSmem {
    long long sums[kClusterThreads / 32];
    long long before[kPagedMaxB];  // entries that go back of the sequences before b
    int from[kPagedMaxB];        // first of them in the table
    int count[kPoolRuns];        // free (used) pages of each run, then of those before it
    int start[kPagedMaxB + 1];   // as in PoolView
    int first[kPagedMaxB];
};
struct PoolShared {  // the deciding block's table of shared pages
    int page[kShareSlots], grow[kShareSlots], first[kShareSlots];
};
constexpr size_t kResizeSmem = sizeof(PoolSmem) + sizeof(PoolShared);

// the place of `page` in the table, taken if it is not there yet (at most half of the table is)
__device__ __forceinline__ int pool_slot(PoolShared &t, int page) {
    int at = (int)((unsigned)page * 2654435761u >> 19) & (kShareSlots - 1);
    for (;;) {
        const int was = atomicCAS(&t.page[at], -1, page);
        if (was == -1 || was == page) return at;
        at = (at + 1) & (kShareSlots - 1);
    }
}

// b with before[b] <= i < before[b + 1]
template <typename N> __device__ __forceinline__ int pool_owner(const N *before, int B, N i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// pages to a run
__device__ __forceinline__ int pool_per(const PoolView &v) {
    const int least = (int)(((long long)v.num_pages + kPoolRuns - 1) / kPoolRuns);
    return max(kPoolRun, (least + 31) / 32 * 32);
}

// how many pages of [p0, p1) are used (or free), kPoolLoads loads of a lane in flight
template <bool USED> __device__ __forceinline__ int pool_count(const PoolView &v, int p0, int p1) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int p = p0 + lane; p < p1; p += 32 * kPoolLoads) {
        int r[kPoolLoads];
#pragma unroll
        for (int k = 0; k < kPoolLoads; ++k) r[k] = p + 32 * k < p1 ? __ldcg(v.refs + p + 32 * k) : (USED ? 0 : 1);
#pragma unroll
        for (int k = 0; k < kPoolLoads; ++k) n += (r[k] > 0) == USED;
    }
    return __reduce_add_sync(0xffffffffu, n);
}

// counts the runs of warp w of `warps` and tells every block
template <bool USED> __device__ __forceinline__ void pool_tell(const PoolView &v, PoolSmem &sm, int w, int warps, int per) {
    const int lane = threadIdx.x & 31;
    for (int run = w; (long long)run * per < v.num_pages; run += warps) {
        const int p0 = run * per, n = pool_count<USED>(v, p0, min(p0 + per, v.num_pages));
        if (lane < kClusterBlocks) cluster_put(&sm.count[run], lane, n);
    }
}

// the counts become those of the runs before each; their sum; all threads of the block
__device__ __forceinline__ int pool_before(const PoolView &v, PoolSmem &sm, int per) {
    const int runs = (v.num_pages + per - 1) / per, each = (runs + kClusterThreads - 1) / kClusterThreads;
    const int r0 = min(runs, (int)threadIdx.x * each), r1 = min(runs, r0 + each);
    int mine = 0, total;
    for (int k = r0; k < r1; ++k) mine += sm.count[k];
    int before = pool_scan<kClusterThreads>(mine, reinterpret_cast<int *>(sm.sums), total);
    for (int k = r0; k < r1; ++k) {
        const int n = sm.count[k];
        sm.count[k] = before;
        before += n;
    }
    __syncthreads();
    return total;
}

// Of the sequences that grow: what they need and which pages have to be copied, into v's scratch and
// the block's start and first; one block.  page[k]: the page that holds the last slot of its
// sequence b0 + k, where that is not full.  Sequences whose page is counted 0, or grows in more of
// them than it is counted, stay as they are (N becomes L) and its count is left alone: taken down for
// their copies it would reach 0, and the page be handed out or not by when the other blocks look.
__device__ __forceinline__ void pool_share(const PoolView &v, const int (&L)[kShareEach], int (&N)[kShareEach],
                                           const int (&page)[kShareEach], int each, PoolSmem &sm, PoolShared &t) {
    const int b0 = threadIdx.x * each;
    int refs[kShareEach], slot[kShareEach];
    bool any = false;
#pragma unroll
    for (int k = 0; k < kShareEach; ++k) {
        refs[k] = page[k] >= 0 ? __ldcg(v.refs + page[k]) : 0;
        slot[k] = -1;
        any |= refs[k] > 1;
    }
    if (__syncthreads_or(any)) {
        for (int i = threadIdx.x; i < kShareSlots; i += kClusterThreads) {
            t.page[i] = -1;
            t.grow[i] = 0;
            t.first[i] = kPagedMaxB;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kShareEach; ++k) {
            if (refs[k] <= 1) continue;
            slot[k] = pool_slot(t, page[k]);
            atomicAdd(&t.grow[slot[k]], 1);
            atomicMin(&t.first[slot[k]], b0 + k);
        }
        __syncthreads();
    }
    // what is needed and, in the low 13 bits, how many copies that makes (all that sequences ask for may
    // pass 32 bits: 4096 times 2^26 pages)
    static_assert(kPagedMaxB < 1 << 13, "the copies of all sequences are counted in 13 bits");
    long long sum = 0, all;
    int need[kShareEach];
    bool copy[kShareEach];
#pragma unroll
    for (int k = 0; k < kShareEach; ++k) {
        copy[k] = slot[k] >= 0;
        if (page[k] >= 0 && (refs[k] <= 0 || (copy[k] && t.grow[slot[k]] > refs[k]))) {
            paged_report(v.err, kErrPagedRefs);
            copy[k] = false;
            N[k] = L[k];
        }
        if (copy[k] && t.grow[slot[k]] >= refs[k] && t.first[slot[k]] == b0 + k) copy[k] = false;
        if (copy[k]) atomicSub(v.refs + page[k], 1);
        need[k] = N[k] > L[k] ? pool_pages(v, N[k]) - pool_pages(v, L[k]) + copy[k] : 0;
        sum += ((long long)need[k] << 13) + copy[k];
    }
    long long before = pool_scan<kClusterThreads>(sum, sm.sums, all);
    const long long top = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kShareEach; ++k) {
        const int b = b0 + k;
        if (k >= each || b >= v.B) break;
        sm.start[b] = (int)min(before >> 13, top);
        sm.first[b] = pool_pages(v, L[k]) - copy[k];
        v.old[b] = copy[k] ? page[k] : -1;
        v.fill[b] = L[k] & ((1 << v.shift) - 1);
        v.copies[b] = (int)(before & 8191);
        before += ((long long)need[k] << 13) + copy[k];
    }
    if (threadIdx.x < kClusterBlocks) cluster_put(&sm.start[v.B], threadIdx.x, (int)min(all >> 13, top));
    if (threadIdx.x == 0) v.copies[v.B] = (int)(all & 8191);
}

__global__ void __cluster_dims__(kClusterBlocks, 1, 1) __launch_bounds__(kClusterThreads)
pool_resize_kernel(const PoolView v, const int32_t *new_lens) {
    extern __shared__ long long smem8[];
    PoolSmem &sm = *reinterpret_cast<PoolSmem *>(smem8);
    PoolShared &shared = *reinterpret_cast<PoolShared *>(&sm + 1);
    const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.x;
    cluster_arrive();  // (waited for before another block's memory is written)
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    // 1. entries behind the ends of shorter sequences, numbered over all of them
    const int each = (v.B + kClusterThreads - 1) / kClusterThreads, b0 = tid * each;
    int L[kShareEach], N[kShareEach], page[kShareEach];
    long long mine = 0, drops;
#pragma unroll
    for (int k = 0; k < kShareEach; ++k) {
        L[k] = N[k] = 0;
        page[k] = -1;
        if (k < each && b0 + k < v.B) pool_lens(v, new_lens, b0 + k, L[k], N[k], rank == 0);
    }
#pragma unroll
    for (int k = 0; k < kShareEach; ++k) {
        if (k >= each || b0 + k >= v.B) break;
        sm.from[b0 + k] = pool_pages(v, N[k]);
        sm.before[b0 + k] = max(0, pool_pages(v, L[k]) - pool_pages(v, N[k]));
        mine += sm.before[b0 + k];
        if (rank == 0 && N[k] > L[k] && (L[k] & ((1 << v.shift) - 1))) {
            const int p = v.table[(size_t)(b0 + k) * v.max_pages + pool_pages(v, L[k]) - 1];
            if ((unsigned)p < (unsigned)v.num_pages) page[k] = p;
            else paged_report(v.err, kErrPagedPage);  // (the page that is written next has to be there)
        }
    }
    long long run = pool_scan<kClusterThreads>(mine, sm.sums, drops);
    cluster_wait();
    if (drops > 0) {  // (the same for every block)
#pragma unroll
        for (int k = 0; k < kShareEach; ++k) {
            if (k >= each || b0 + k >= v.B) break;
            const long long n = sm.before[b0 + k];
            sm.before[b0 + k] = run;
            run += n;
        }
        __syncthreads();
        for (long long i0 = rank * kClusterThreads + tid; i0 < drops; i0 += kPoolStep) {
            int32_t *at[kPoolUnroll];
            int p[kPoolUnroll], was[kPoolUnroll];
#pragma unroll
            for (int u = 0; u < kPoolUnroll; ++u) {
                const long long i = i0 + u * kClusterBlocks * kClusterThreads;
                at[u] = nullptr;
                if (i >= drops) continue;
                const int b = pool_owner(sm.before, v.B, i), e = sm.from[b] + (int)(i - sm.before[b]);
                if (YOCO_DCHECK(e < v.max_pages, 0x6B)) at[u] = v.table + (size_t)b * v.max_pages + e;
            }
#pragma unroll
            for (int u = 0; u < kPoolUnroll; ++u) p[u] = at[u] ? *at[u] : -1;
#pragma unroll
            for (int u = 0; u < kPoolUnroll; ++u) {
                was[u] = 1;
                if (!at[u]) continue;
                *at[u] = -1;
                if (pool_names(v, p[u])) was[u] = atomicSub(v.refs + p[u], 1);
            }
#pragma unroll
            for (int u = 0; u < kPoolUnroll; ++u) {
                if (was[u] > 0) continue;  // (else more entries name it than it was counted)
                atomicAdd(v.refs + p[u], 1);
                paged_report(v.err, kErrPagedRefs);
            }
        }
        cluster_sync();
    }
    // 2. the first block decides, the others count
    const int warps = kClusterWarps - kClusterThreads / 32, w = (rank - 1) * (kClusterThreads / 32) + (tid >> 5), per = pool_per(v);
    if (rank == 0) pool_share(v, L, N, page, each, sm, shared);
    else pool_tell<false>(v, sm, w, warps, per);
    cluster_sync();
    // 3. the free pages that are taken, in order
    const int total = sm.start[v.B], all = pool_before(v, sm, per);
    const bool room = total <= all;
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < kShareEach; ++k) {
            const int b = b0 + k;
            if (k >= each || b >= v.B) break;
            if (N[k] < L[k] || (N[k] > L[k] && room)) v.lens[b] = N[k];
            if (!room && v.old[b] >= 0) atomicAdd(v.refs + v.old[b], 1);
        }
        if (tid == 0) {
            v.moves[0] = make_int4(room ? v.copies[v.B] : 0, room ? all - total : all, 0, 0);
            if (!room) paged_report(v.err, kErrPagedRoom);
        }
    }
    if (!room || total == 0) return;
    if (rank != 0) {
        for (int b = tid; b < v.B; b += kClusterThreads) {
            sm.start[b] = cluster_get(&sm.start[b], 0);
            sm.first[b] = cluster_get(&sm.first[b], 0);
        }
        for (int run = w; (long long)run * per < v.num_pages; run += warps) {
            int r = sm.count[run];
            if (r >= total) break;
            for (int q = run * per + lane, p1 = min(run * per + per, v.num_pages); q - lane < p1 && r < total; q += 32 * kPoolLoads) {
                int refs[kPoolLoads];
#pragma unroll
                for (int k = 0; k < kPoolLoads; ++k) refs[k] = q + 32 * k < p1 ? __ldcg(v.refs + q + 32 * k) : 1;
#pragma unroll
                for (int k = 0; k < kPoolLoads; ++k) {
                    const bool free = refs[k] <= 0;
                    const unsigned who = __ballot_sync(0xffffffffu, free);
                    const int i = r + __popc(who & ((1u << lane) - 1));
                    r += __popc(who);
                    if (free && i < total) {
                        v.rank[i] = q + 32 * k;
                        v.refs[q + 32 * k] = 1;
                    }
                }
            }
        }
    }
    cluster_sync();
    // 4. to whom they go, shared out anew (given out by the runs' own warps, a run of free pages is one
    // warp's search after search: 34 us for the round of 1024 sequences)
    for (int i0 = rank * kClusterThreads + tid; i0 < total; i0 += kPoolStep) {
        int p[kPoolUnroll];
#pragma unroll
        for (int u = 0; u < kPoolUnroll; ++u) {
            const int i = i0 + u * kClusterBlocks * kClusterThreads;
            if (i < total) p[u] = __ldcg(v.rank + i);
        }
#pragma unroll
        for (int u = 0; u < kPoolUnroll; ++u) {
            const int i = i0 + u * kClusterBlocks * kClusterThreads;
            if (i >= total) break;
            const int b = pool_owner(sm.start, v.B, i), idx = i - sm.start[b], e = sm.first[b] + idx;
            if (!YOCO_DCHECK(b < v.B && e < v.max_pages, 0x6B)) continue;
            v.table[(size_t)b * v.max_pages + e] = p[u];
            if (idx == 0) {
                const int old = __ldcg(v.old + b);
                if (old >= 0) v.moves[1 + __ldcg(v.copies + b)] = make_int4(old, p[u], __ldcg(v.fill + b), 0);
            }
        }
    }
}

__global__ void __launch_bounds__(kPoolThreads)
pool_fork_kernel(const PoolView v, const int32_t *src, const int32_t *dst, int n) {
    __shared__ int refused;
    const int i = blockIdx.x, a = src[i], b = dst[i];
    bool bad = (unsigned)a >= (unsigned)v.B || (unsigned)b >= (unsigned)v.B;
    if (threadIdx.x == 0) refused = 0;
    __syncthreads();
    for (int k = threadIdx.x; k < n && !bad; k += kPoolThreads) {
        const int to = dst[k];
        if (to == a || (to == b && k < i)) refused = 1;
    }
    __syncthreads();
    // (a sequence that is forked to by this pair alone: no other block writes its length)
    bad = bad || refused;
    int L = 0;
    if (!bad) {
        L = v.lens[a];
        bad = v.lens[b] != 0;
        if (!pool_len_ok(v, L)) {
            if (threadIdx.x == 0) paged_report(v.err, kErrPagedLen);
            return;
        }
    }
    if (bad) {
        if (threadIdx.x == 0) paged_report(v.err, kErrPagedSeq);
        return;
    }
    __syncthreads();
    for (int e = threadIdx.x, held = pool_pages(v, L); e < held; e += kPoolThreads) {
        const int p = v.table[(size_t)a * v.max_pages + e];
        v.table[(size_t)b * v.max_pages + e] = p;
        if (pool_names(v, p)) atomicAdd(v.refs + p, 1);
    }
    if (threadIdx.x == 0) v.lens[b] = L;
}

// who moves where
__global__ void __cluster_dims__(kClusterBlocks, 1, 1) __launch_bounds__(kClusterThreads) pool_moves_kernel(const PoolView v) {
    extern __shared__ long long smem8[];
    PoolSmem &sm = *reinterpret_cast<PoolSmem *>(smem8);
    const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.x;
    cluster_arrive();  // (waited for before another block's memory is written)
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int w = rank * (kClusterThreads / 32) + (tid >> 5), per = pool_per(v);
    cluster_wait();
    pool_tell<true>(v, sm, w, kClusterWarps, per);
    cluster_sync();
    const int live = pool_before(v, sm, per);
    // used pages below page `live`: those of the runs before its own, and a part of that one
    int in_front, part, n = 0;
    const int edge = live / per;
    for (int p = edge * per + tid; p < live; p += kClusterThreads) n += __ldcg(v.refs + p) > 0;
    (void)pool_scan<kClusterThreads>(n, reinterpret_cast<int *>(sm.sums), part);
    in_front = part + (edge * per < v.num_pages ? sm.count[edge] : live);
    if (tid == 0 && rank == 0) v.moves[0] = make_int4(live - in_front, live, 0, 0);
    if (live == in_front) return;
    int *moves = reinterpret_cast<int *>(v.moves + 1);
    // (a run before page `live` has holes, one behind it pages that move)
    for (int run = w; (long long)run * per < v.num_pages; run += kClusterWarps) {
        int at = sm.count[run];
        for (int q = run * per + lane, p1 = min(run * per + per, v.num_pages); q - lane < p1; q += 32 * kPoolLoads) {
            int refs[kPoolLoads];
#pragma unroll
            for (int k = 0; k < kPoolLoads; ++k) refs[k] = q + 32 * k < p1 ? __ldcg(v.refs + q + 32 * k) : 0;
#pragma unroll
            for (int k = 0; k < kPoolLoads; ++k) {
                const int p = q + 32 * k;
                const bool is = refs[k] > 0;
                const unsigned who = __ballot_sync(0xffffffffu, is);
                const int used = at + __popc(who & ((1u << lane) - 1));  // used pages before p
                at += __popc(who);
                if (p >= p1) continue;
                if (is && p >= live) {
                    const int r = used - in_front;
                    if (!YOCO_DCHECK(r >= 0 && r < v.num_pages / 2, 0x6C)) continue;
                    v.rank[p] = r;
                    moves[4 * r] = p;
                    moves[4 * r + 2] = 1 << v.shift;
                    moves[4 * r + 3] = 0;
                } else if (!is && p < live) {
                    moves[4 * (p - used) + 1] = p;
                }
            }
        }
    }
}

// tables and counts follow the moves; the blocks of the copying grid, before they copy
__device__ __forceinline__ void pool_follow(const PoolView &v) {
    const int4 head = __ldcg(v.moves);
    const int count = head.x, live = head.y;
    for (int i = blockIdx.x * kPoolThreads + threadIdx.x; i < count; i += gridDim.x * kPoolThreads) {
        const int4 m = __ldcg(v.moves + 1 + i);
        v.refs[m.y] = v.refs[m.x];
        v.refs[m.x] = 0;
    }
    for (int b = blockIdx.x; b < v.B; b += gridDim.x) {
        const int L = paged_ld(v.lens + b);
        if (!pool_len_ok(v, L)) {
            if (threadIdx.x == 0) paged_report(v.err, kErrPagedLen);
            continue;
        }
        for (int e = threadIdx.x, held = pool_pages(v, L); e < held; e += kPoolThreads) {
            int32_t *at = v.table + (size_t)b * v.max_pages + e;
            const int p = paged_ld(at);
            if (p < live || !pool_names(v, p)) continue;
            const int r = paged_ld(v.rank + p);  // (of a page that was not counted as used: anything)
            const int4 m = (unsigned)r < (unsigned)count ? __ldcg(v.moves + 1 + r) : make_int4(-1, 0, 0, 0);
            if (m.x == p) *at = m.y;
            else paged_report(v.err, kErrPagedRefs);
        }
    }
}

// The copies of a list: block by block a (move, k or v, kv head), whose slots lie side by side.
constexpr int kCopyUnroll = 4;

template <bool FOLLOW>
__global__ void __launch_bounds__(kPoolThreads)
pool_copy_kernel(uint4 *k, uint4 *v, const int4 *moves, int most, int Hkv, int num_pages, int shift, int row16,
                 const PoolView view) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // (the list, where the call made it)
    if constexpr (FOLLOW) pool_follow(view);
    const int64_t items = (int64_t)min(max(__ldcg(moves).x, 0), most) * 2 * Hkv;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int head = (int)(it % Hkv), which = (int)(it / Hkv) & 1;
        const int4 m = __ldcg(moves + 1 + it / (2 * Hkv));
        if ((unsigned)m.x >= (unsigned)num_pages || (unsigned)m.y >= (unsigned)num_pages || m.z < 0 || m.z > 1 << shift) continue;
        const int n = m.z * row16;
        const int64_t head16 = (int64_t)row16 << shift;
        uint4 *pool = which ? v : k;
        const uint4 *from = pool + ((int64_t)m.x * Hkv + head) * head16;
        uint4 *to = pool + ((int64_t)m.y * Hkv + head) * head16;
        for (int i0 = threadIdx.x; i0 < n; i0 += kPoolThreads * kCopyUnroll) {
            uint4 x[kCopyUnroll];
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u)
                if (i0 + u * kPoolThreads < n) x[u] = from[i0 + u * kPoolThreads];
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u)
                if (i0 + u * kPoolThreads < n) to[i0 + u * kPoolThreads] = x[u];
        }
    }
}

}  // namespace yoco

namespace yoco_host {
using namespace yoco;

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// the view of a call, its scratch in `ws`; the bytes that takes
static size_t pool_view(const yoco_paged_kv *c, int32_t *refs, int32_t *moves, char *ws, PoolView &v) {
    v = {};
    // (the cache's members are const for the calls that only read them)
    v.table = const_cast<int32_t *>(c->page_table);
    v.lens = const_cast<int32_t *>(c->seq_lens);
    v.refs = refs;
    v.B = c->B;
    v.max_pages = c->max_pages;
    v.num_pages = c->num_pages;
    while ((1 << v.shift) < c->page_size) ++v.shift;
    v.err = (int *)ws;
    size_t at = 256;
    auto take = [&](size_t ints) {
        int *p = (int *)(ws + at);
        at += up256(ints * sizeof(int));
        return p;
    };
    v.old = take(c->B);
    v.fill = take(c->B);
    v.copies = take((size_t)c->B + 1);
    v.rank = take(c->num_pages);
    v.moves = (int4 *)take(4 * ((size_t)std::max(c->B, c->num_pages / 2) + 1));
    if (moves) v.moves = (int4 *)moves;
    return at;
}

size_t paged_pool_workspace(const yoco_paged_kv *c) {
    PoolView v;
    return pool_view(c, nullptr, nullptr, nullptr, v);
}

// `follow`: the call is a compact, its tables and counts are brought in line as well
static cudaError_t pool_copy(const yoco_paged_kv *c, const int4 *moves, int most, const PoolView *follow, bool early,
                             cudaStream_t st) {
    if (most <= 0) return cudaSuccess;
    int shift = 0;
    while ((1 << shift) < c->page_size) ++shift;
    const int64_t items = (int64_t)most * 2 * c->Hkv;
    const int row16 = c->d * (c->dtype == YOCO_BF16 ? 2 : 4) / 16;
    cudaLaunchConfig_t cfg = {};
    // a resize copies little or nothing: a grid that starts fast
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(items, (int64_t)device_sm_count() * (early && !follow ? 2 : 8)));
    cfg.blockDim = dim3(kPoolThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, follow ? pool_copy_kernel<true> : pool_copy_kernel<false>, (uint4 *)c->k, (uint4 *)c->v,
                              moves, most, c->Hkv, c->num_pages, shift, row16, follow ? *follow : PoolView{});
}

cudaError_t paged_resize(const yoco_paged_kv *c, int32_t *refs, const int32_t *new_lens, int32_t *moves, void *ws,
                         cudaStream_t st) {
    PoolView v;
    (void)pool_view(c, refs, moves, (char *)ws, v);
    // the shared-memory opt-in is set on every launch (it belongs to the current device)
    cudaError_t e = cudaFuncSetAttribute(pool_resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kResizeSmem);
    if (e != cudaSuccess) return e;
    count_launches(1);
    pool_resize_kernel<<<kClusterBlocks, kClusterThreads, kResizeSmem, st>>>(v, new_lens);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : pool_copy(c, v.moves, c->B, nullptr, true, st);
}

cudaError_t paged_fork(const yoco_paged_kv *c, int32_t *refs, const int32_t *src, const int32_t *dst, int n, void *ws,
                       cudaStream_t st) {
    PoolView v;
    (void)pool_view(c, refs, nullptr, (char *)ws, v);
    count_launches(1);
    pool_fork_kernel<<<n, kPoolThreads, 0, st>>>(v, src, dst, n);
    return cudaGetLastError();
}

cudaError_t paged_compact(const yoco_paged_kv *c, int32_t *refs, int32_t *moves, void *ws, cudaStream_t st) {
    PoolView v;
    (void)pool_view(c, refs, moves, (char *)ws, v);
    cudaError_t e = cudaFuncSetAttribute(pool_moves_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PoolSmem));
    if (e != cudaSuccess) return e;
    count_launches(1);
    pool_moves_kernel<<<kClusterBlocks, kClusterThreads, sizeof(PoolSmem), st>>>(v);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : pool_copy(c, v.moves, c->num_pages / 2, &v, true, st);
}

cudaError_t paged_copy(const yoco_paged_kv *c, const int32_t *moves, int most, cudaStream_t st) {
    return pool_copy(c, (const int4 *)moves, most, nullptr, false, st);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_pool)
