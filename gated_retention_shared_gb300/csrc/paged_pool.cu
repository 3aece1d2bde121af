// paged_pool.cu -- handing out the pages of a paged cache: sequences that grow, shrink, end and
// fork, and moving the used pages together (yoco_paged_resize, _fork, _compact, _copy).
//
// refs[p] is how many table entries name page p; the free pages are those with 0.  Which pages a
// call hands out goes by their numbers alone (the lowest free ones, in the order of the sequences
// and slots), so nothing depends on the order of threads.  With chunks of kPoolChunk pages counted
// first, a page's rank among the free (or used) ones is what lies in the chunks before its own
// plus its rank in the chunk; entry number r of those that are wanted is found in the prefix sums
// of what the sequences need.
//
// A resize: 1. sequences that shrink give pages back; 2. one block decides, per growing sequence,
// whether the page it writes next has to be copied, and sums up what is needed; 3. free pages are
// counted; 4. handed out; 5. copies are made.  Of the sequences that share a page and all grow the
// first keeps it: each takes its count off refs; where that leaves 0, all of them grow, and the
// least b - B, written to refs itself, says which is first.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace yoco {

constexpr int kPoolChunk = 4096;      // pages counted by a block
constexpr int kPoolThreads = 256;
constexpr int kPoolEach = kPoolChunk / kPoolThreads;
constexpr int kShareThreads = 1024;   // the deciding block
constexpr int kShareEach = kPagedMaxB / kShareThreads;

struct PoolView {
    int32_t *table, *lens, *refs;
    int32_t B, max_pages, num_pages, shift, chunks;
    int4 *moves;
    // scratch
    int *start;   // [B + 1] pages needed by the sequences before b
    int *first;   // [B] table entry that the first of them goes to
    int *old;     // [B] page that it copies, or -1
    int *fill;    // [B] slots of it in use
    int *copies;  // [B + 1] copies made by the sequences before b
    int *count;   // [chunks] free (used) pages
    int *rank;    // [num_pages] of a page that moves, among those
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

// page e of sequence b, or -1
__device__ __forceinline__ int pool_page(const PoolView &v, int b, int e) {
    const int p = v.table[(size_t)b * v.max_pages + e];
    if ((unsigned)p < (unsigned)v.num_pages) return p;
    paged_report(v.err, kErrPagedPage);
    return -1;
}

__global__ void __launch_bounds__(kPoolThreads) pool_release_kernel(const PoolView v, const int32_t *new_lens) {
    const int b = blockIdx.x;
    int L, N;
    pool_lens(v, new_lens, b, L, N, threadIdx.x == 0);
    for (int e = pool_pages(v, N) + threadIdx.x, e1 = pool_pages(v, L); e < e1; e += kPoolThreads) {
        const int p = pool_page(v, b, e);
        v.table[(size_t)b * v.max_pages + e] = -1;
        if (p >= 0 && atomicSub(v.refs + p, 1) <= 0) {  // more entries name it than it was counted
            atomicAdd(v.refs + p, 1);
            paged_report(v.err, kErrPagedRefs);
        }
    }
}

// exclusive prefix sums of x over the block's threads; `sums` one per warp; total: of all
template <int THREADS, typename N> __device__ __forceinline__ N pool_scan(N x, N *sums, N &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    N inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const N y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
    }
    __syncthreads();  // `sums` may still be read
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    N before = 0;
    total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        before += w < warp ? sums[w] : 0;
        total += sums[w];
    }
    return before + inc - x;
}

__global__ void __launch_bounds__(kShareThreads) pool_share_kernel(const PoolView v, const int32_t *new_lens) {
    __shared__ long long sums[kShareThreads / 32];  // (what all sequences ask for may pass 32 bits)
    const int each = (v.B + kShareThreads - 1) / kShareThreads, b0 = threadIdx.x * each;
    int page[kShareEach], need[kShareEach], at[kShareEach], fill[kShareEach];
    bool copy[kShareEach], last[kShareEach];  // last: all who have the page grow
#pragma unroll
    for (int k = 0; k < kShareEach; ++k) {
        page[k] = -1;
        need[k] = at[k] = fill[k] = 0;
        copy[k] = false;
        if (k >= each || b0 + k >= v.B) continue;
        int L, N;
        pool_lens(v, new_lens, b0 + k, L, N, false);
        if (N <= L) continue;
        at[k] = pool_pages(v, L);
        need[k] = pool_pages(v, N) - at[k];
        fill[k] = L & ((1 << v.shift) - 1);
        if (fill[k] == 0) continue;
        page[k] = pool_page(v, b0 + k, at[k] - 1);
        if (page[k] >= 0) copy[k] = __ldcg(v.refs + page[k]) > 1;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kShareEach; ++k)
        if (copy[k]) atomicSub(v.refs + page[k], 1);
    __threadfence();
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kShareEach; ++k) {
        const int left = copy[k] ? __ldcg(v.refs + page[k]) : 1;
        last[k] = left <= 0;
        if (left < 0) paged_report(v.err, kErrPagedRefs);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kShareEach; ++k)
        if (last[k]) atomicMin(v.refs + page[k], b0 + k - v.B);
    __threadfence();
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kShareEach; ++k)
        if (last[k] && __ldcg(v.refs + page[k]) == b0 + k - v.B) copy[k] = false;
    __syncthreads();
    long long sum = 0, made = 0;
#pragma unroll
    for (int k = 0; k < kShareEach; ++k) {
        if (last[k] && !copy[k]) v.refs[page[k]] = 1;
        if (copy[k]) {
            ++need[k];
            --at[k];
        }
        sum += need[k];
        made += copy[k];
    }
    long long all, all_made;
    long long before = pool_scan<kShareThreads>(sum, sums, all);
    long long made_before = pool_scan<kShareThreads>(made, sums, all_made);
    const long long top = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kShareEach; ++k) {
        const int b = b0 + k;
        if (k >= each || b >= v.B) break;
        v.start[b] = (int)min(before, top);
        v.first[b] = at[k];
        v.old[b] = copy[k] ? page[k] : -1;
        v.fill[b] = fill[k];
        v.copies[b] = (int)made_before;
        before += need[k];
        made_before += copy[k];
    }
    if (threadIdx.x == 0) {
        v.start[v.B] = (int)min(all, top);
        v.copies[v.B] = (int)all_made;
    }
}

// pages of the chunk that are free (or used)
template <bool USED> __global__ void __launch_bounds__(kPoolThreads) pool_count_kernel(const PoolView v) {
    __shared__ int sums[kPoolThreads / 32];
    int n = 0;
    for (int k = 0; k < kPoolEach; ++k) {
        const int p = blockIdx.x * kPoolChunk + k * kPoolThreads + threadIdx.x;
        if (p < v.num_pages) n += (v.refs[p] > 0) == USED;
    }
    int all;
    (void)pool_scan<kPoolThreads>(n, sums, all);
    if (threadIdx.x == 0) v.count[blockIdx.x] = all;
}

// of all chunks, and of those before this block's
__device__ __forceinline__ void pool_counts(const PoolView &v, int *sums, int chunk, int &before, int &all) {
    int n = 0, m = 0;
    for (int c = threadIdx.x; c < v.chunks; c += kPoolThreads) {
        const int x = v.count[c];
        n += x;
        m += c < chunk ? x : 0;
    }
    (void)pool_scan<kPoolThreads>(n, sums, all);
    (void)pool_scan<kPoolThreads>(m, sums, before);
}

__global__ void __launch_bounds__(kPoolThreads) pool_assign_kernel(const PoolView v, const int32_t *new_lens) {
    __shared__ int sums[kPoolThreads / 32];
    int before, all;
    pool_counts(v, sums, blockIdx.x, before, all);
    const int total = v.start[v.B];
    const bool room = total <= all;
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < v.B; b += kPoolThreads) {
            int L, N;
            pool_lens(v, new_lens, b, L, N, false);
            if (N < L || (N > L && room)) v.lens[b] = N;
            if (!room && v.old[b] >= 0) atomicAdd(v.refs + v.old[b], 1);
        }
        if (threadIdx.x == 0) {
            v.moves[0] = make_int4(room ? v.copies[v.B] : 0, room ? all - total : all, 0, 0);
            if (!room) paged_report(v.err, kErrPagedRoom);
        }
    }
    if (!room || before >= total) return;
    // each thread's pages side by side, so that ranks go by page number
    const int p0 = blockIdx.x * kPoolChunk + threadIdx.x * kPoolEach;
    unsigned free = 0;
    for (int k = 0; k < kPoolEach; ++k)
        if (p0 + k < v.num_pages && v.refs[p0 + k] <= 0) free |= 1u << k;
    int in_chunk;
    int r = before + pool_scan<kPoolThreads>(__popc(free), sums, in_chunk);
    for (; free && r < total; free &= free - 1, ++r) {
        const int p = p0 + __ffs(free) - 1;
        int lo = 0, hi = v.B;  // the sequence: start[lo] <= r < start[lo + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (v.start[mid] <= r) lo = mid;
            else hi = mid;
        }
        const int idx = r - v.start[lo], e = v.first[lo] + idx;
        if (!YOCO_DCHECK(lo < v.B && e < v.max_pages, 0x6B)) continue;
        v.table[(size_t)lo * v.max_pages + e] = p;
        v.refs[p] = 1;
        if (idx == 0 && v.old[lo] >= 0) v.moves[1 + v.copies[lo]] = make_int4(v.old[lo], p, v.fill[lo], 0);
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
        const int p = pool_page(v, a, e);
        v.table[(size_t)b * v.max_pages + e] = p;
        if (p >= 0) atomicAdd(v.refs + p, 1);
    }
    if (threadIdx.x == 0) v.lens[b] = L;
}

// who moves where
__global__ void __launch_bounds__(kPoolThreads) pool_moves_kernel(const PoolView v) {
    __shared__ int sums[kPoolThreads / 32];
    int before, live;
    pool_counts(v, sums, blockIdx.x, before, live);
    // used pages below page `live`: those of the chunks before its own, and a part of that one
    int in_front = 0, all;
    {
        const int edge = live / kPoolChunk;  // (past the last chunk where every page is used)
        int n = 0;
        for (int c = threadIdx.x; c < min(edge, v.chunks); c += kPoolThreads) n += v.count[c];
        for (int p = edge * kPoolChunk + threadIdx.x; p < live; p += kPoolThreads) n += v.refs[p] > 0;
        (void)pool_scan<kPoolThreads>(n, sums, in_front);
    }
    const int p0 = blockIdx.x * kPoolChunk + threadIdx.x * kPoolEach;
    unsigned used = 0;
    for (int k = 0; k < kPoolEach; ++k)
        if (p0 + k < v.num_pages && v.refs[p0 + k] > 0) used |= 1u << k;
    int at = before + pool_scan<kPoolThreads>(__popc(used), sums, all);  // used pages before p0
    int *moves = reinterpret_cast<int *>(v.moves + 1);
    for (int k = 0; k < kPoolEach && p0 + k < v.num_pages; ++k) {
        const int p = p0 + k;
        const bool is = used >> k & 1;
        if (is && p >= live) {
            const int r = at - in_front;
            if (!YOCO_DCHECK(r >= 0 && r < v.num_pages / 2, 0x6C)) continue;
            v.rank[p] = r;
            moves[4 * r] = p;
            moves[4 * r + 2] = 1 << v.shift;
            moves[4 * r + 3] = 0;
        } else if (!is && p < live) {
            moves[4 * (p - at) + 1] = p;
        }
        at += is;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) v.moves[0] = make_int4(live - in_front, live, 0, 0);
}

// tables and counts follow the moves
__global__ void __launch_bounds__(kPoolThreads) pool_follow_kernel(const PoolView v) {
    const int4 head = v.moves[0];
    const int count = head.x, live = head.y;
    for (int i = blockIdx.x * kPoolThreads + threadIdx.x; i < count; i += gridDim.x * kPoolThreads) {
        const int4 m = v.moves[1 + i];
        v.refs[m.y] = v.refs[m.x];
        v.refs[m.x] = 0;
    }
    for (int b = blockIdx.x; b < v.B; b += gridDim.x) {
        const int L = v.lens[b];
        if (!pool_len_ok(v, L)) {
            if (threadIdx.x == 0) paged_report(v.err, kErrPagedLen);
            continue;
        }
        for (int e = threadIdx.x, held = pool_pages(v, L); e < held; e += kPoolThreads) {
            int32_t *at = v.table + (size_t)b * v.max_pages + e;
            const int p = *at;
            if (p < live && p >= 0) continue;
            if ((unsigned)p >= (unsigned)v.num_pages) {
                paged_report(v.err, kErrPagedPage);
                continue;
            }
            const int r = v.rank[p];  // (of a page that was not counted as used: anything)
            if ((unsigned)r < (unsigned)count && v.moves[1 + r].x == p) *at = v.moves[1 + r].y;
            else paged_report(v.err, kErrPagedRefs);
        }
    }
}

// The copies of a list: block by block a (move, k or v, kv head), whose slots lie side by side.
constexpr int kCopyUnroll = 4;

__global__ void __launch_bounds__(kPoolThreads)
pool_copy_kernel(uint4 *k, uint4 *v, const int4 *moves, int most, int Hkv, int num_pages, int shift, int row16) {
    const int64_t items = (int64_t)min(max(moves[0].x, 0), most) * 2 * Hkv;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int head = (int)(it % Hkv), which = (int)(it / Hkv) & 1;
        const int4 m = moves[1 + it / (2 * Hkv)];
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
    v.chunks = (c->num_pages + kPoolChunk - 1) / kPoolChunk;
    v.err = (int *)ws;
    size_t at = 256;
    auto take = [&](size_t ints) {
        int *p = (int *)(ws + at);
        at += up256(ints * sizeof(int));
        return p;
    };
    v.start = take((size_t)c->B + 1);
    v.first = take(c->B);
    v.old = take(c->B);
    v.fill = take(c->B);
    v.copies = take((size_t)c->B + 1);
    v.count = take(v.chunks);
    v.rank = take(c->num_pages);
    v.moves = (int4 *)take(4 * ((size_t)std::max(c->B, c->num_pages / 2) + 1));
    if (moves) v.moves = (int4 *)moves;
    return at;
}

size_t paged_pool_workspace(const yoco_paged_kv *c) {
    PoolView v;
    return pool_view(c, nullptr, nullptr, nullptr, v);
}

static cudaError_t pool_copy(const yoco_paged_kv *c, const int4 *moves, int most, cudaStream_t st) {
    if (most <= 0) return cudaSuccess;
    int shift = 0;
    while ((1 << shift) < c->page_size) ++shift;
    const int64_t items = (int64_t)most * 2 * c->Hkv;
    const int blocks = (int)std::min<int64_t>(items, (int64_t)device_sm_count() * 8);
    const int row16 = c->d * (c->dtype == YOCO_BF16 ? 2 : 4) / 16;
    count_launches(1);
    pool_copy_kernel<<<blocks, kPoolThreads, 0, st>>>((uint4 *)c->k, (uint4 *)c->v, moves, most, c->Hkv, c->num_pages, shift,
                                                      row16);
    return cudaGetLastError();
}

cudaError_t paged_resize(const yoco_paged_kv *c, int32_t *refs, const int32_t *new_lens, int32_t *moves, void *ws,
                         cudaStream_t st) {
    PoolView v;
    (void)pool_view(c, refs, moves, (char *)ws, v);
    count_launches(4);
    pool_release_kernel<<<v.B, kPoolThreads, 0, st>>>(v, new_lens);
    pool_share_kernel<<<1, kShareThreads, 0, st>>>(v, new_lens);
    pool_count_kernel<false><<<v.chunks, kPoolThreads, 0, st>>>(v);
    pool_assign_kernel<<<v.chunks, kPoolThreads, 0, st>>>(v, new_lens);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : pool_copy(c, v.moves, c->B, st);
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
    count_launches(3);
    pool_count_kernel<true><<<v.chunks, kPoolThreads, 0, st>>>(v);
    pool_moves_kernel<<<v.chunks, kPoolThreads, 0, st>>>(v);
    pool_follow_kernel<<<std::max(v.B, 64), kPoolThreads, 0, st>>>(v);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : pool_copy(c, v.moves, c->num_pages / 2, st);
}

cudaError_t paged_copy(const yoco_paged_kv *c, const int32_t *moves, int most, cudaStream_t st) {
    return pool_copy(c, (const int4 *)moves, most, st);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_pool)
