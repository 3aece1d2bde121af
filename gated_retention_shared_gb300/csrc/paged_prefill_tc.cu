// paged_prefill_tc.cu -- attention of chunks of new rows over the paged cache on the tensor
// cores, bf16, head size 128 (with scores 64 too), up to 16 query heads to a kv head.
//
// A row of the MMA is one (token, query head of the kv head's group): 128 rows are
// TS = 128 / G tokens with their G heads, so the group reads each K and V tile once, and a
// block of 2 TS tokens meets the diagonal over 2 TS + 128 keys, not over 256 + 128.  A block
// has two such sets, A and B, each with a softmax warpgroup of its own, so that the tensor
// cores work on one set while the other's softmax runs.  Per 128-key tile i and set X:
//     S_X  = Q_X K_i^T                    (TMEM)
//     P_X  = 2^(c S_X - m)   masked       (bf16, shared memory)
//     O_X += P_X V_i                      (TMEM)
// with c = scale log2(e) and m a reference per row that moves only when a tile's maximum
// passes it by more than 8 / ln 2, O_X being rescaled then.  P is rounded to bf16 for the
// second product, its sum is kept in fp32 before that rounding.
//
// The sets take one P buffer in turn by 64-key halves (set B writes P(i) as P_A V(i) reads
// its halves, set A P(i + 1) as P_B V(i) does).  A block whose tokens fit set A (a short
// chunk, the end of a long one) leaves set B out and uses Q_B's place as a second P buffer, so
// that the softmax of tile i + 1 runs while P V(i) does.
//
// The kernel is a template: MODE 0 is the plain call's, the others are those of the scored calls
// (masks; a cap; a bias by distance; both), whose softmax is described at c_scores.  4096 fresh rows
// take 86 us plain, 90 with masks, 102 biased, 115 capped, 135 with both: in the tile loop the fp32 pipe
// (37 % with a cap) and the chain from S to P; the products are 54.
//
// Pages, rows out of sight and pages that are not there: as in paged_decode_tc.cu; set A's
// warps clear the V rows that no row of the block sees.  Where the plan (paged_plan.cu) cuts a
// row block's keys into pieces, the unnormalised sums are joined by paged_merge_rows_kernel;
// the partials lie column by column, so a warp's 32 rows store side by side.
//
// One block per SM; it takes entry after entry of the plan's list from a counter, longest first.
// The next entry is chosen three tiles before this one's end, gets barriers of its own (two
// groups in turn, set up anew while the other is in use) and its Q and first K tile while this one's
// last product runs and its rows are written; then all warps meet.
//
// Warps: 0 TMA producer, 1 issues S products, 2 issues P V products, 3 the next entry, 4-7 set
// A, 8-11 set B (thread = TMEM lane = row).  S and P V have issuers of their own so that
// S_X(i + 1) goes as soon as S_X(i) has been read, whatever P the other issuer waits for.
//
// What bounds it (512 rows over 131072 keys: 586-630 us with the card's power, 1.46 us a tile of
// 2 x 128 rows at the least; the products alone are 1.08): the softmax warps' own chain, about 2800 cycles a tile from S to P
// with no pipe above a third; and some 5 us an entry around its tiles (first S; last P V; rows out).  What counted, each timed as the kernel then was, on the long chunk if not said:
//   - no register spilled in the tile loop: shared memory leaves next to no L1, so each reload
//     is an L2 round trip (140 bytes of spills: 1.5 x the time).  Hence the 120 / 192 split;
//   - the exponentials in steps over 32 columns, not element by element (740 -> 690 us);
//   - one copy of the tile loop's code for both sets (a copy for each: 2 x the time, the
//     instruction cache);
//   - the waits of the other kernels: one whose first 16384 polls were a loop of nothing else that
//     fell through into what follows took 663 us against 586 (the cause was not shown);
//   - S and P V issuers apart (757 -> 740 us);
//   - little between a slot's release and its next copy (12 mixed sequences 63.4 -> 61.3 us);
//   - blocks that stay instead of one per entry: 600 short sequences 218 -> 172 us, 3 windows 129
//     -> 123, 16 prompts of 100 to 900 rows 67 -> 62; 12 mixed sequences, about one entry to a
//     block, 61.3 -> 62 (59 today).  The next kernel is let in when a block has found no further entry, not
//     at once (2 us);
//   - Q and K ahead, and so rows staged in V tiles: 600 sequences of 1 to 30 rows over 10 to 400 keys 203
//     -> 185 us, 8192 rows with a window of 500 82 -> 77, 16 prompts 47 -> 45, 8192 rows of documents
//     100.5 -> 98.6.  The first S ahead as well: the sequences 201, and capped tiles 3 % slower.
// Tried and slower: two warps to a row (half the columns each, 808 against 740 us), weights
// before the maximum is known (752); S read twice by halves made no difference, nor did both
// sets on one set's rows, tile by tile, where the rows fit one (its time is the reads').
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "tc.cuh"

namespace yoco {

using namespace tc;

constexpr int kCRows = 128;                    // rows of a set
constexpr int kCStages = 2;
constexpr int kCTile = kPagedTile * 128 * 2;   // 32 KB (at head size 64 Q, K and V use the first half of theirs)
constexpr int kCHalf = kCTile / 2;             // 64 channels (or keys) of 128 rows
constexpr int kCThreads = 384;
constexpr float kCGap = 8.f * kPagedLog2E;

struct PagedPreBars {
    uint64_t q_full;
    uint64_t kfull[kCStages], kempty[kCStages], vfull[kCStages], vempty[kCStages];
    uint64_t s_full[2], s_free[2];          // per set
    uint64_t p_ready[2][2], pv_done[2][2];  // per set (one set: per P buffer) and 64-key half
};

// what an entry needs; the next entry's is filled while this one's runs
template <bool MOD> struct PagedPreTask {
    PagedPreBars bar;
    typename PagedKind<MOD>::Entry blk;
    int hk;
    int more;  // there is such an entry
};

template <bool MOD> struct PagedPreSmem {
    PagedPreTask<MOD> task[2];
    uint64_t drain[2];
    int walive[2][4];
    uint32_t tmem_base;
    int abort_flag;
    int go[2];
};

constexpr size_t kCTileBytes = (size_t)3 * kCTile + (size_t)kCStages * 2 * kCTile;  // Q_A, Q_B, P, K/V rings
template <bool MOD> constexpr size_t kCSmem = kCTileBytes + sizeof(PagedPreSmem<MOD>) + 1024;
static_assert(kCSmem<true> <= 232448, "paged prefill tiles must fit shared memory");

__device__ __forceinline__ void cbar(int id) {  // the four warps of a set
    __syncwarp();
    asm volatile("bar.sync %0, 128;\n" ::"r"(id) : "memory");
}

__device__ __forceinline__ uint32_t c_chunk(int r, int c) {  // 16-byte chunk c (0..15) of row r, 128-byte swizzle
    return (uint32_t)(c >> 3) * kCHalf + (uint32_t)r * 128u + (uint32_t)(((c & 7) ^ (r & 7)) * 16);
}

__device__ __forceinline__ uint32_t c_pack(float lo, float hi) {
    const __nv_bfloat162 h2 = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h2);
}

__device__ __forceinline__ float c_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void c_bars_init(PagedPreBars &bar) {
    mbar_init(&bar.q_full, 1);
    for (int s = 0; s < kCStages; ++s) {
        mbar_init(&bar.kfull[s], 1);
        mbar_init(&bar.kempty[s], 1);
        mbar_init(&bar.vfull[s], 1);
        mbar_init(&bar.vempty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
        mbar_init(&bar.s_full[x], 1);
        mbar_init(&bar.s_free[x], 4);
        for (int hh = 0; hh < 2; ++hh) {
            mbar_init(&bar.p_ready[x][hh], 4);
            mbar_init(&bar.pv_done[x][hh], 1);
        }
    }
    fence_mbar_init();
}

// end of an entry for every warp; false when one of them has seen the abort flag
__device__ __forceinline__ bool c_end(volatile int *abort_flag) {
    uint32_t gone = *abort_flag != 0;
    __syncwarp();
    tc_fence_before();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %0, 0;\n\t"
        "bar.red.or.pred q, 9, 384, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
        : "+r"(gone)
        :
        : "memory");
    tc_fence_after();
    return gone == 0;
}
static_assert(kCThreads == 384, "c_end counts the block's threads");

__device__ __forceinline__ void c_regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 120;\n"); }

// 8 consecutive columns of lane (taddr.lane + t)
__device__ __forceinline__ void c_tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void c_tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// the low `n` of 32 bits (n clamped to [0, 32])
__device__ __forceinline__ uint32_t c_below(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// How a scored tile goes.  The reference of a row's exponentials need not be its maximum, only no
// less and not far above, so it is found from the raw products: with a cap (which is monotone) from
// their largest magnitude, with a bias from the largest of each 16 columns and the bias at their end.
// The cap and the bias are then part of the exponentials' argument,
//     2^(s Q(s^2) + (slope (m - p) - reference)),
// Q the polynomial of C tanh(k s) / s of degree 3 in s^2 (own minimax fit by reweighted least squares,
// relative error 5.4e-7 up to |k s| = 0.5, a 2000th of the rounding of the weights that follows), for
// caps below kWideCap of degree 5 (5.9e-7 up to 1; 4096 rows, cap 15: 267 -> 129 us, as most tiles went the
// exact way before; at cap 50, where none does, it is 114 -> 129), from kShortCap on of degree 2 (5.0e-7 up
// to 0.26; cap 50 114 -> 110 us, with a bias 135 -> 126).  The bracket is advanced by additions from every eighth column on: two
// scores to an instruction, degree + 2 more for two scores than without, and nothing more for the
// special-function unit.  That is where all products of the warp's rows are within the polynomial's range
// and scores within kQuickScore of 0, slopes
// below kQuickSlope and all that is seen lies behind the row: a reference is then at most 2 x 22 (cap) and
// 22 (bias) powers of two above the maximum, and what is 2^-60 of the largest weight still is a normal
// number (the smallest products as well took 122 us in place of 115 for 4096 rows).
// Other tiles take the exact way, score by score, in small steps over tensor memory: unrolled over the
// row's registers its code cost the quick tiles their place in the instruction cache (4096 rows, cap 30,
// 3 % of the tiles exact: 256 us).

// 16 places of the tile from place c0 on, in place: cap tanh(q.k scale / cap) - slope |p - m|, times
// log2(e), and -inf where `seen` has no bit.  Place c is slot v0 + first + c before the first run's end,
// v0 + delta + c from there on.
template <bool CAP, bool BIAS>
__device__ __forceinline__ void c_scores(uint32_t (&sv)[16], int c0, uint32_t seen, const PagedMod &mod, float c2, float slope,
                                         int pos, int v0, int sink_slots, int first, int delta) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        float y = __uint_as_float(sv[c]) * c2;
        if constexpr (CAP) y = paged_cap(y, mod.cap2);
        if constexpr (BIAS) {
            const int v = v0 + c0 + c, m = v + (v < sink_slots ? first : delta);
            y = fmaf(-slope, fabsf((float)(m - pos)), y);
        }
        sv[c] = seen & (1u << c) ? __float_as_uint(y) : 0xff800000u;
    }
}

__device__ __forceinline__ float c_max_nan(float a, float b) {  // NaN where one is NaN
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int MODE, int D>
__global__ void __launch_bounds__(kCThreads, 1)
paged_prefill_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, bf16_t *__restrict__ O, float *__restrict__ part,
                        PagedPlan *plan, const typename PagedKind<(MODE > 0)>::Entry *__restrict__ entries, int cap, int rows,
                        int Hq, const PagedView pv, const PagedMod mod, float c2, int *err) {
    constexpr bool MOD = MODE > 0, CAP = MODE & kModCap, BIAS = MODE & kModBias, SCORED = CAP || BIAS;
    constexpr int DEG = CAP ? paged_cap_degree(MODE) : 0;  // of the quick way's polynomial
    typedef typename PagedKind<MOD>::Entry Entry;
    typedef PagedPreTask<MOD> Task;
    constexpr int kWords = sizeof(Entry) / 4;
    constexpr int kHalves = D / 64, kChunks = D / 8;  // of a row: 64 channels, 16 bytes
    static_assert(D == 64 || D == 128, "halves of 64 channels");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    uint8_t *tiles = smem_raw + pad;
    uint8_t *sQ = tiles;                 // Q_A, Q_B
    uint8_t *sP = tiles + 2 * kCTile;
    uint8_t *ring = tiles + 3 * kCTile;  // stage s: K at ring + 2 s kCTile, V after it
    PagedPreSmem<MOD> &sm = *reinterpret_cast<PagedPreSmem<MOD> *>(tiles + kCTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = Hq / pv.Hkv, TS = kCRows / G;

    if (tid == 0) {
        c_bars_init(sm.task[0].bar);
        c_bars_init(sm.task[1].bar);
        for (int k = 0; k < 2; ++k) mbar_init(&sm.drain[k], 1);
        fence_mbar_init();
        sm.abort_flag = 0;
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    const int entry0 = (int)blockIdx.x / pv.Hkv;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    volatile int *abort_flag = &sm.abort_flag;
    auto fail = [&](int code) {
        *abort_flag = 1;
        paged_report(err, code);
    };
    // warp 3: the first entry with rows from `item` on, item by item of all blocks' common counter
    auto fetch = [&](int item, int entry, Task &task) {
        for (;;) {
            // (both loads at once: the list has room for `cap` entries)
            const int word = lane < kWords ? paged_ld(reinterpret_cast<const int *>(entries + min(entry, cap - 1)) + lane) : 0;
            const int count = paged_ld(&plan->entries);
            if (entry >= count) {
                if (lane == 0) task.more = 0;
                break;
            }
            if (lane < kWords) reinterpret_cast<int *>(&task.blk)[lane] = word;
            if (lane == 0) {
                task.hk = item - entry * pv.Hkv;
                task.more = 1;
            }
            if (__shfl_sync(0xffffffffu, word, 2) > 0) break;  // nrow
            if (lane == 0) item = (int)gridDim.x + atomicAdd(&plan->next, 1);
            item = __shfl_sync(0xffffffffu, item, 0);
            entry = item / pv.Hkv;
        }
        __syncwarp();
    };
    if (warp == 3) fetch(blockIdx.x, entry0, sm.task[0]);
    __syncthreads();
    if (!sm.task[0].more) return;
    // the TMA warp's lanes: a tile is `boxes` boxes of pages, 64 channels each
    const int psz = min(1 << pv.shift, kPagedTile), boxes = kHalves * (kPagedTile / psz);
    const int mine = lane / kHalves * psz;
    // what the table says of this lane's box of tile i (fetched ahead of use, so not yet looked
    // at); -1 past the last place
    // the entry's i-th tile.  A bias takes the nearest first: from the farthest on, each tile's scores
    // would pass the reference and the sums would be rescaled every time (4096 rows, slopes 2^(-i/3):
    // 135 us in place of 110, as the rest then was)
    auto tile_of = [&](const Entry &blk, int i) { return BIAS ? blk.i1 - 1 - i : blk.i0 + i; };
    auto look_up = [&](const Entry &blk, int i) -> int {
        const int v = tile_of(blk, i) * kPagedTile + mine, e = blk.range.slot(v) >> pv.shift;
        const bool there = lane < boxes && v < blk.range.places && e < pv.max_pages;
        return there ? pv.table[(size_t)blk.b * pv.max_pages + e] : -1;
    };
    // that page, or the one past the pool
    auto page_of = [&](const Entry &blk, int i, int entry_of_table) -> int {
        if ((unsigned)entry_of_table < (unsigned)pv.num_pages) return entry_of_table;
        if (lane < boxes && tile_of(blk, i) * kPagedTile + mine < blk.range.places) paged_report(err, kErrPagedPage);
        return pv.num_pages;
    };
    const int half = lane % kHalves;
    auto row_of = [&](const Entry &blk, int i) -> int {  // of tile i's box in its page
        return blk.range.slot(tile_of(blk, i) * kPagedTile + mine) & ((1 << pv.shift) - 1);
    };
    auto copy = [&](Task &task, int hk, int i, bool is_v, int page, int row) {  // K or V tile i into its (free) slot
        const int s = i % kCStages;
        uint8_t *st = ring + (size_t)s * 2 * kCTile + (is_v ? kCTile : 0);
        uint64_t *full = is_v ? &task.bar.vfull[s] : &task.bar.kfull[s];
        if (lane == 0) mbar_arrive_expect_tx(full, kHalves * kCHalf);
        __syncwarp();
        if (lane < boxes)
            tma_load_4d(st + half * kCHalf + mine * 128, is_v ? &tm_v : &tm_k, full, half * 64, row, hk, page);
    };
    auto copy_q = [&](Task &task) {
        if (lane == 0) {
            const int sets = task.blk.nrow > TS ? 2 : 1;
            mbar_arrive_expect_tx(&task.bar.q_full, (uint32_t)(sets * kHalves * TS * G * 128));
            for (int x = 0; x < sets; ++x)
                for (int hf = 0; hf < kHalves; ++hf)
                    tma_load_3d(sQ + x * kCTile + hf * kCHalf, &tm_q, &task.bar.q_full, hf * 64, task.hk * G,
                                task.blk.row0 + x * TS);
        }
        __syncwarp();
    };
    int pg0 = -1, pg1 = -1;
    // the entry's first pages and K tile
    auto first_k = [&](Task &task) {
        if (task.blk.i1 == task.blk.i0) return;
        pg0 = look_up(task.blk, 0);
        pg1 = task.blk.i1 - task.blk.i0 > 1 ? look_up(task.blk, 1) : -1;
        pg0 = page_of(task.blk, 0, pg0);
        copy(task, task.hk, 0, false, pg0, row_of(task.blk, 0));
    };
    if (warp == 0) {  // the first copies are on their way while tensor memory is taken
        if (sm.task[0].blk.i1 > sm.task[0].blk.i0) copy_q(sm.task[0]);
        first_k(sm.task[0]);
    } else if (warp == 3) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    // P buffer and barriers of set x at tile i, and how often they were used before
    auto p_slot = [](bool two, int x, int i) { return two ? x : (i & 1); };
    auto p_use = [](bool two, int i) { return two ? i : (i >> 1); };

    // where a wait gave up, products may still be running: none may be when tensor memory is given back
    auto drain = [&](int k) {
        if (lane == 0) {
            volatile int no_abort = 0;
            mma_commit(&sm.drain[k]);
            mbar_wait(&sm.drain[k], 0, &no_abort, 200000000ull);
        }
        __syncwarp();
    };

    if (warp == 0) {
        // -------------------------------------------------------------- TMA
        c_regs_dec();
        for (int n = 0;; ++n) {
            Task &task = sm.task[n & 1], &next = sm.task[(n + 1) & 1];
            const Entry &blk = task.blk;
            const int ntiles = blk.i1 - blk.i0;
            volatile int no_abort = 0;
            int nk = 0, nv = 0;  // tiles whose K / V copy was issued
            bool told = false;  // warp 3 takes the next entry late: who is done first takes the longest
            auto tell = [&]() {
                if (!told) asm volatile("bar.arrive 11, 64;\n" ::: "memory");
                told = true;
            };
            if (ntiles > 0) {
                nk = 1;
                const int c_i0 = BIAS ? blk.i1 - 1 : blk.i0, c_sink = blk.range.sink_slots, c_delta = blk.range.base - c_sink, c_hk = task.hk;
                bool ok = true;
                auto load = [&](int i, bool is_v, int page) {
                    const int s = i % kCStages, v = (BIAS ? c_i0 - i : c_i0 + i) * kPagedTile + mine;
                    int to = v < c_sink ? 0 : c_delta;
                    if constexpr (MOD) {
                        if (v < c_sink) to = blk.range.first;  // (from shared memory: a register more would spill)
                    }
                    const int row = (v + to) & ((1 << pv.shift) - 1);
                    if (i >= kCStages)
                        ok = mbar_wait(is_v ? &task.bar.vempty[s] : &task.bar.kempty[s], ((i / kCStages) + 1) & 1, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) return;
                    copy(task, c_hk, i, is_v, page, row);
                    ++(is_v ? nv : nk);
                };
                // K runs one tile ahead of V: its slot is free first
                for (int i = 0; i < ntiles && ok; ++i) {
                    const int pg2 = i + 2 < ntiles ? look_up(blk, i + 2) : -1;
                    if (i + 3 >= ntiles) tell();
                    if (i + 1 < ntiles) load(i + 1, false, pg1 = page_of(blk, i + 1, pg1));
                    if (ok) load(i, true, pg0);
                    pg0 = pg1;
                    pg1 = pg2;
                }
                tell();
                // leave no copy in flight (only the last two of each kind can be), no tile in use, nor a commit
                // on its way to a barrier that is set up anew: here Q and K, below V
                if (lane == 0) {
                    mbar_wait(&task.bar.q_full, 0, &no_abort, 200000000ull);
                    for (int k = max(0, nk - kCStages); k < nk; ++k)
                        mbar_wait(&task.bar.kfull[k % kCStages], (k / kCStages) & 1, &no_abort, 200000000ull);
                    for (int k = max(0, nk - kCStages); k < nk && ok; ++k)
                        ok = mbar_wait(&task.bar.kempty[k % kCStages], (k / kCStages) & 1, abort_flag);
                    if (!ok) fail(51);
                }
                __syncwarp();
            }
            tell();
            // the next entry's first K tile and Q come in while the last product runs and this one's rows
            // are written (Q after the last product where that reads P from Q_B's place)
            asm volatile("bar.sync 10, 64;\n" ::: "memory");
            const bool ahead = next.more && next.blk.i1 > next.blk.i0 && __all_sync(0xffffffffu, !*abort_flag);
            const bool early = blk.nrow > TS || ntiles == 0;
            if (ahead) first_k(next);
#pragma unroll 1
            for (int step = 0; step < 2; ++step) {
                if (step == (early ? 0 : 1)) {
                    if (ahead) copy_q(next);
                } else if (ntiles > 0) {
                    if (lane == 0) {
                        bool ok = true;
                        for (int k = max(0, nv - kCStages); k < nv; ++k)
                            mbar_wait(&task.bar.vfull[k % kCStages], (k / kCStages) & 1, &no_abort, 200000000ull);
                        for (int k = max(0, nv - kCStages); k < nv && ok; ++k)
                            ok = mbar_wait(&task.bar.vempty[k % kCStages], (k / kCStages) & 1, abort_flag);
                        if (!ok) fail(51);
                    }
                    __syncwarp();
                }
            }
            if (!c_end(abort_flag)) {
                if (ahead && lane == 0) {
                    mbar_wait(&next.bar.kfull[0], 0, &no_abort, 200000000ull);
                    mbar_wait(&next.bar.q_full, 0, &no_abort, 200000000ull);
                }
                break;
            }
            if (!next.more) break;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA: S = Q K^T
        c_regs_dec();
        for (int n = 0;; ++n) {
            PagedPreBars &bar = sm.task[n & 1].bar;
            const Entry &blk = sm.task[n & 1].blk;
            const int ntiles = blk.i1 - blk.i0;
            const bool two = blk.nrow > TS;
            if (lane == 0 && ntiles > 0) {
                const uint32_t id_s = idesc_bf16_f32(kCRows, kPagedTile, false, false);  // A = Q, B = K (K-major)
                bool ok = mbar_wait(&bar.q_full, 0, abort_flag);
                for (int i = 0; i < ntiles && ok; ++i) {
                    const int s = i % kCStages;
                    if (!(ok = mbar_wait(&bar.kfull[s], (i / kCStages) & 1, abort_flag))) break;
                    for (int x = 0; x < (two ? 2 : 1); ++x) {
                        // S_X(i) goes over S_X(i - 1) as soon as that has been read out
                        if (i > 0 && !(ok = mbar_wait(&bar.s_free[x], (i - 1) & 1, abort_flag))) break;
                        tc_fence_after();
                        const uint64_t dq = smem_desc_sw128(smem_u32(sQ + x * kCTile), 16, 1024);
                        const uint64_t dk = smem_desc_sw128(smem_u32(ring + (size_t)s * 2 * kCTile), 16, 1024);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t off = ((kk >> 2) * kCHalf + (kk & 3) * 32) >> 4;
                            mma_ss(tmem + 256 * x, dq + off, dk + off, id_s, kk > 0);
                        }
                        mma_commit(&bar.s_full[x]);
                    }
                    if (ok) mma_commit(&bar.kempty[s]);
                }
                if (!ok) fail(52);
            }
            if (!c_end(abort_flag)) {
                drain(0);
                break;
            }
            if (!sm.task[(n + 1) & 1].more) break;
        }
    } else if (warp == 2) {
        // ------------------------------------------------------ MMA: O += P V
        c_regs_dec();
        for (int n = 0;; ++n) {
            PagedPreBars &bar = sm.task[n & 1].bar;
            const Entry &blk = sm.task[n & 1].blk;
            const int ntiles = blk.i1 - blk.i0;
            const bool two = blk.nrow > TS;
            if (lane == 0) {
                const uint64_t dp0 = smem_desc_sw128(smem_u32(sP), 16, 1024), dv0 = smem_desc_sw128(smem_u32(ring + kCTile), kCHalf, 1024);
                const uint32_t id_o = idesc_bf16_f32(kCRows, D, false, true);  // A = P (K-major), B = V (N-major)
                bool ok = true;
                for (int i = 0; i < ntiles && ok; ++i) {
                    const int s = i % kCStages;
                    uint64_t dp = dp0 - (uint64_t)(!two && (i & 1) ? kCTile >> 4 : 0), dv = dv0 + (uint64_t)(s * (2 * kCTile >> 4));
                    asm volatile("" : "+l"(dp), "+l"(dv));
                    if (!(ok = mbar_wait(&bar.vfull[s], (i / kCStages) & 1, abort_flag))) break;
                    for (int x = 0; x < (two ? 2 : 1) && ok; ++x) {
                        const int b = p_slot(two, x, i);
                        for (int hh = 0; hh < 2; ++hh) {
                            if (!(ok = mbar_wait(&bar.p_ready[b][hh], p_use(two, i) & 1, abort_flag))) break;
                            tc_fence_after();
#pragma unroll
                            for (int k4 = 0; k4 < 4; ++k4) {
                                const int kk = 4 * hh + k4;
                                mma_ss(tmem + 256 * x + 128, dp + (uint64_t)((hh * kCHalf + k4 * 32) >> 4),
                                       dv + (uint64_t)((kk * 2048) >> 4), id_o, (i > 0 || kk > 0));
                            }
                            mma_commit(&bar.pv_done[b][hh]);
                        }
                    }
                    if (ok) mma_commit(&bar.vempty[s]);
                }
                if (!ok) fail(58);
            }
            if (!c_end(abort_flag)) {
                drain(1);
                break;
            }
            if (!sm.task[(n + 1) & 1].more) break;
        }
    } else if (warp == 3) {
        // -------------------------------------------- the next entry and its barriers
        c_regs_dec();
        for (int n = 0;; ++n) {
            Task &next = sm.task[(n + 1) & 1];
            asm volatile("bar.sync 11, 64;\n" ::: "memory");
            int item = 0;
            if (lane == 0) item = (int)gridDim.x + atomicAdd(&plan->next, 1);
            item = __shfl_sync(0xffffffffu, item, 0);
            fetch(item, item / pv.Hkv, next);
            // (let in before that the next kernel's blocks wait on SMs that other entries could use)
            if (!next.more) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
            if (n > 0 && lane == 0) {
                uint64_t *bars = reinterpret_cast<uint64_t *>(&next.bar);
                for (int k = 0; k < (int)(sizeof(PagedPreBars) / sizeof(uint64_t)); ++k) mbar_inval(bars + k);
                c_bars_init(next.bar);
            }
            __syncwarp();
            asm volatile("bar.sync 10, 64;\n" ::: "memory");
            if (!c_end(abort_flag) || !next.more) break;
        }
    } else {
        // ------------------------------------------ softmax, rescale, output
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;\n");
        const int x = (warp - 4) / 4;  // set
        const int q4 = warp & 3;       // TMEM lane quarter of this warp
        const int r = q4 * 32 + lane;  // row of the set = TMEM lane
        const int bar_id = 1 + x;
        const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
        const uint32_t colS = 256 * x, colO = 256 * x + 128;
        for (int n = 0;; ++n) {
        PagedPreBars &bar = sm.task[n & 1].bar;
        const Entry &blk = sm.task[n & 1].blk;
        const int hk = sm.task[n & 1].hk, ntiles = blk.i1 - blk.i0;
        const bool two = *(const volatile int *)&blk.nrow > TS;
        if (ntiles == 0) {  // nothing to see: zeros
            for (int e = tid - 128; e < blk.nrow * G * kChunks; e += 256)
                *reinterpret_cast<uint4 *>(O + ((size_t)(blk.row0 + e / (G * kChunks)) * Hq + hk * G) * D + (e % (G * kChunks)) * 8) =
                    make_uint4(0, 0, 0, 0);
        } else if (x == 0 || two) {
        const int toks = min(TS, blk.nrow - x * TS);       // tokens of the set
        const int set_lo = blk.pos0 + x * TS, set_hi = set_lo + toks - 1;
        const bool used = r < toks * G;
        const int pos = set_lo + r / G;
        const int sink_slots = blk.range.sink_slots, delta = blk.range.base - sink_slots;
        // tiles of which some place is no row's are those before e_lo and from e_hi on; set A clears
        // their V rows.  (A parity can only tell a phase from the one before: with two sets P(i - 1)
        // waited for P_B V(i - 2), so V(i - 2) has come; with one set every tile waits for V)
        int e_lo = 0, e_hi = 0x7fffffff;
        if (x == 0) {
            const auto &rg = blk.range;
            int lo = rg.lo;
            if constexpr (MOD) lo = max(lo, rg.dlo);
            const int from = rg.sink_slots + lo - rg.base;  // the first place that is seen for being in the window
            e_lo = (from + kPagedTile - 1) / kPagedTile - blk.i0;
            e_hi = rg.places / kPagedTile - blk.i0;
        }
        // a scored call's row sees the slots [lo, pos] and [doc, head): its window from its document's
        // start on, and of the document's slots the prefix and the sinks; all rows of the warp see
        // [all_lo, all_hi) and [all_doc, all_head)
        [[maybe_unused]] int lo = 0, doc = 0, head = 0, all_lo = 0, all_hi = 0, all_doc = 0, all_head = 0;
        [[maybe_unused]] float slope = 0.f;
        [[maybe_unused]] bool gentle = true, back = true;  // slopes for the quick way; no row sees past itself
        if constexpr (MOD) {
            if (used && mod.doc) doc = max(0, mod.doc[blk.row0 + x * TS + r / G]);
            lo = max(doc, pv.window > 0 ? pos + 1 - pv.window : 0);
            head = pos < 0 ? 0 : max(blk.range.pre, min(pv.sinks, pos + 1));
            all_lo = __reduce_max_sync(0xffffffffu, used ? lo : 0);
            all_hi = __reduce_min_sync(0xffffffffu, used ? pos + 1 : 0x7fffffff);
            all_doc = __reduce_max_sync(0xffffffffu, used ? doc : 0);
            all_head = __reduce_min_sync(0xffffffffu, used ? head : 0x7fffffff);
            if constexpr (BIAS) {
                if (used) slope = mod.slopes[hk * G + r % G] * kPagedLog2E;
                gentle = __all_sync(0xffffffffu, fabsf(slope) <= kQuickSlope);
                back = __all_sync(0xffffffffu, head <= pos + 1 || !used);
            }
        }
        float m_ref = -INFINITY, l = 0.f;  // base-2 units
        // One exit from the tile loop: a wait that gave up makes what follows garbage (the status word
        // says so), but every barrier is still served.  A warp gives up as one: tcgen05.ld and the
        // votes take whole warps.
        bool alive = true;
        for (int i = 0; i < ntiles && alive; ++i) {
            // place 0 of the tile, and what its slot is where it lies past the sinks' chunks
            const int v0 = tile_of(blk, i) * kPagedTile, key0 = v0 + delta;
            // every row of the set (a scored call: of the warp) sees every slot of the tile
            bool full;
            [[maybe_unused]] int first = 0, k0 = key0;  // of the first run's slots; of the tile's where it has one run
            [[maybe_unused]] bool run = true;
            if constexpr (MOD) {
                if (__builtin_expect(v0 < sink_slots, 0)) {
                    first = blk.range.first;
                    run = v0 + kPagedTile <= sink_slots;
                    k0 = v0 + first;
                }
                full = run && ((all_lo <= k0 && k0 + kPagedTile <= all_hi) || (all_doc <= k0 && k0 + kPagedTile <= all_head));
            }
            alive = mbar_wait_warp(&bar.s_full[x], i & 1, abort_flag);
            tc_fence_after();
            const uint32_t s_t = tmem + colS + lane_base;
            uint32_t sv[128];
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) tmem_ld32(s_t + cb * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * cb));
            tmem_wait_ld();
            if constexpr (!SCORED) {
                // S is in registers: the MMA may write S(i + 1) over it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.s_free[x]);
            }
            if constexpr (!MOD)
                full = v0 >= sink_slots && key0 + kPagedTile - 1 <= set_lo &&
                       (pv.window <= 0 || key0 > set_hi - pv.window || key0 + kPagedTile <= pv.sinks);
            [[maybe_unused]] uint32_t bits[4] = {~0u, ~0u, ~0u, ~0u};
            if (__builtin_expect(!full, 0)) {
                if constexpr (MOD) {
                    // [lo, pos] and [doc, head) of the second run's places, [doc, head) of the first run's
                    const int ch_c = sink_slots - v0, f_c = v0 + first;
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        bits[w] = (((c_below(pos + 1 - key0 - 32 * w) & ~c_below(lo - key0 - 32 * w)) |
                                    (c_below(head - key0 - 32 * w) & ~c_below(doc - key0 - 32 * w))) & ~c_below(ch_c - 32 * w)) |
                                  (c_below(head - f_c - 32 * w) & ~c_below(doc - f_c - 32 * w) & c_below(ch_c - 32 * w));
                } else {
                    // the places this row sees of the tile: sinks in the sinks' chunks, then a run up to its
                    // own position from the window's first slot on, and sinks that lie in those chunks
                    const int hi_c = pos + 1 - key0;
                    const int lo_c = pv.window > 0 ? pos + 1 - pv.window - key0 : -1;
                    const int sk_c = min(pv.sinks - key0, hi_c);
                    const int ch_c = sink_slots - v0, sc_c = min(ch_c, min(pv.sinks, pos + 1) - v0);
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        bits[w] = (((c_below(hi_c - 32 * w) & ~c_below(lo_c - 32 * w)) | c_below(sk_c - 32 * w)) &
                                   ~c_below(ch_c - 32 * w)) | c_below(sc_c - 32 * w);
                }
                if constexpr (!SCORED) {
#pragma unroll
                    for (int c = 0; c < kPagedTile; ++c)
                        sv[c] = (bits[c >> 5] & (1u << (c & 31))) ? sv[c] : 0xff800000u;  // -inf
                }
            }
            float mt;
            [[maybe_unused]] bool quick = true;
            if constexpr (SCORED) {
                // the largest products (with a cap in magnitude), with a bias of each 16 columns: of those
                // that the row sees
                constexpr int kGroups = BIAS ? 8 : 4;
                auto size = [](uint32_t w) { return CAP ? fabsf(__uint_as_float(w)) : __uint_as_float(w); };
                float top[kGroups];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) top[g] = -INFINITY;
                if (__builtin_expect(full, 1)) {
#pragma unroll
                    for (int j = 0; j < kPagedTile / 2; ++j) {  // (chain by chain in turn)
                        const int g = j % kGroups, c = kPagedTile / kGroups * g + 2 * (j / kGroups);
                        top[g] = fmax3(top[g], size(sv[c]), size(sv[c + 1]));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kPagedTile; ++c) {
                        const bool seen = bits[c >> 5] & (1u << (c & 31));
                        float &t = top[c / (kPagedTile / kGroups)];
                        t = fmaxf(t, seen ? size(sv[c]) : -INFINITY);
                        sv[c] = seen ? sv[c] : __float_as_uint(CAP ? mod.hidden : -INFINITY);  // (weight 0)
                    }
                }
                auto scored = [&](float s0) {  // cap tanh(s0 scale / cap), times log2(e)
                    if constexpr (!CAP) return s0 * c2;
                    const float x2 = s0 * s0;
                    float f = mod.a[DEG];
#pragma unroll
                    for (int k = DEG - 1; k >= 0; --k) f = fmaf(x2, f, mod.a[k]);
                    return s0 == -INFINITY ? s0 : s0 * f;
                };
                float most = 0.f;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) most = fmaxf(most, top[g]);
                if constexpr (CAP) quick = __all_sync(0xffffffffu, most <= mod.quick || !used);
                // (no slot past a row's position is one that it sees)
                if constexpr (BIAS) quick = quick && gentle && run && (back || k0 + kPagedTile <= all_hi);
                mt = -INFINITY;
                if constexpr (BIAS) {
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) mt = fmaxf(mt, fmaf(slope, 16.f * g, scored(top[g])));
                    mt += fmaf(slope, (float)(k0 - pos), fmaxf(15.f * slope, 0.f));
                } else {
                    mt = scored(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
                }
                if (__builtin_expect(!quick, 0)) {
                    mt = -INFINITY;
#pragma unroll 1
                    for (int c0 = 0; c0 < kPagedTile; c0 += 16) {
                        const uint32_t seen = (c0 < 64 ? (c0 < 32 ? bits[0] : bits[1]) : (c0 < 96 ? bits[2] : bits[3])) >> (c0 & 31);
                        uint32_t y[16];
                        tmem_ld16(s_t + c0, y);
                        tmem_wait_ld();
                        c_scores<CAP, BIAS>(y, c0, seen, mod, c2, slope, pos, v0, sink_slots, first, delta);
#pragma unroll
                        for (int c = 0; c < 16; ++c) mt = fmaxf(mt, __uint_as_float(y[c]));
                        tmem_st16(s_t + c0, y);
                    }
                    tmem_wait_st();
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) tmem_ld32(s_t + cb * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * cb));
                    tmem_wait_ld();
                }
                // S is in registers: the MMA may write S(i + 1) over it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.s_free[x]);
            } else {
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kPagedTile; c += 2)
                    mq[(c >> 1) & 3] = fmax3(mq[(c >> 1) & 3], __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
                mt = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * c2;
            }
            // rows past the set's tokens hold whatever shared memory held: they never move the
            // reference (no rescaling for their sake) and are never stored
            mt = used ? mt : -INFINITY;
            const bool move = (mt > m_ref + kCGap) || (m_ref == -INFINITY && mt > -INFINITY);
            const float m_old = m_ref;
            m_ref = move ? mt : m_ref;
            const float alpha = move ? (m_old == -INFINITY ? 0.f : c_ex2(m_old - mt)) : 1.f;
            const float mu = (m_ref == -INFINITY) ? 0.f : m_ref;
            const uint64_t c2x2 = f2_pack(c2, c2), nmu2 = f2_pack(-mu, -mu);
            // the argument's terms: (a[0] + a[1] s^2 + a[2] s^4 ..) s + b0 + step c; a tile that went the
            // exact way holds arguments already
            [[maybe_unused]] float a[DEG + 1], b0 = -mu, step = 0.f;
            if constexpr (SCORED) {
#pragma unroll
                for (int k = 0; k <= DEG; ++k) a[k] = CAP ? mod.a[k] : c2;
                if constexpr (BIAS) {
                    step = slope;
                    b0 = fmaf(slope, (float)(k0 - pos), -mu);
                }
                if (__builtin_expect(!quick, 0)) {
#pragma unroll
                    for (int k = 0; k <= DEG; ++k) a[k] = k == 0 ? 1.f : 0.f;
                    b0 = step = 0.f;
#pragma unroll
                    for (int c = 0; c < kPagedTile; ++c)  // (s^2 stays finite)
                        sv[c] = __float_as_uint(c_max_nan(__uint_as_float(sv[c]) - mu, -1e18f));
                }
            }
            uint64_t acc2[4] = {0, 0, 0, 0};  // packed zeros
            uint32_t pk[kPagedTile / 2];
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // 32 columns at a time, each step for all of them: element by element
                                           // they come out as chains of latencies
                if constexpr (SCORED) {
                    uint64_t ax2[DEG + 1];
#pragma unroll
                    for (int k = 0; k <= DEG; ++k) ax2[k] = f2_pack(a[k], a[k]);
                    const uint64_t b0x2 = f2_pack(b0, b0), step2 = f2_pack(2.f * step, 2.f * step);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {  // 16 columns at a time
                        uint64_t s2[8], f2[8], run[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int c = 32 * q + 16 * g + 2 * e;
                            s2[e] = f2_pack(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
                            run[e] = b0x2;
                            if constexpr (BIAS) {
                                const float at = fmaf(step, (float)c, b0);
                                run[e] = e & 3 ? f2_add(run[e - 1], step2) : f2_pack(at, at + step);
                            }
                            f2[e] = ax2[DEG];
                        }
                        if constexpr (CAP) {
                            uint64_t x2[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x2[e] = f2_mul(s2[e], s2[e]);
#pragma unroll
                            for (int k = DEG - 1; k >= 0; --k)
#pragma unroll
                                for (int e = 0; e < 8; ++e) f2[e] = f2_fma(x2[e], f2[e], ax2[k]);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int c = 32 * q + 16 * g + 2 * e;
                            float x0, x1;
                            f2_unpack(f2_fma(s2[e], f2[e], run[e]), x0, x1);
                            sv[c] = __float_as_uint(x0);
                            sv[c + 1] = __float_as_uint(x1);
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 16 * q; c < 16 * q + 16; ++c) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), c2x2, nmu2), x0, x1);
                        sv[2 * c] = __float_as_uint(x0);
                        sv[2 * c + 1] = __float_as_uint(x1);
                    }
                }
#pragma unroll
                for (int c = 32 * q; c < 32 * q + 32; ++c) sv[c] = __float_as_uint(c_ex2(__uint_as_float(sv[c])));
#pragma unroll
                for (int c = 16 * q; c < 16 * q + 16; ++c) {
                    const float e0 = __uint_as_float(sv[2 * c]), e1 = __uint_as_float(sv[2 * c + 1]);
                    acc2[c & 3] = f2_add(acc2[c & 3], f2_pack(e0, e1));
                    pk[c] = c_pack(e0, e1);
                }
            }
            float ls0, ls1;
            f2_unpack(f2_add(f2_add(acc2[0], acc2[1]), f2_add(acc2[2], acc2[3])), ls0, ls1);
            l = fmaf(l, alpha, ls0 + ls1);
            // O_X holds tiles < i; rows whose reference moved rescale it before P V(i)
            if (__builtin_expect(i > 0 && __any_sync(0xffffffffu, move), 0)) {
                alive &= mbar_wait_warp(&bar.pv_done[p_slot(two, x, i - 1)][1], p_use(two, i - 1) & 1, abort_flag);
                __syncwarp();
                tc_fence_after();
                const uint32_t o_t = tmem + colO + lane_base;
#pragma unroll 1
                for (int cb = 0; cb < D; cb += 8) {  // (in small steps: it is rare, and registers are not)
                    uint32_t ov[8];
                    c_tmem_ld8(o_t + cb, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                    c_tmem_st8(o_t + cb, ov);
                }
                tmem_wait_st();
            }
            // V rows that no row of the block sees: zero, once the tile has come
            const int at = BIAS ? ntiles - 1 - i : i;
            if (__builtin_expect(at < e_lo || at >= e_hi || !two, 0)) {
                alive &= mbar_wait_warp(&bar.vfull[i % kCStages], (i / kCStages) & 1, abort_flag);
                if (alive && !blk.range.seen(blk.range.slot(v0 + r), pv.sinks)) {
                    uint8_t *vr = ring + (size_t)(i % kCStages) * 2 * kCTile + kCTile + r * 128;
#pragma unroll 1
                    for (int ch = 0; ch < kChunks; ++ch)
                        *reinterpret_cast<uint4 *>(vr + (ch >> 3) * kCHalf + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
            }
            // the P buffer's halves are free once the product that read them last is done: with two
            // sets the other set's latest, with one the product two tiles back (before the first use of
            // a barrier the other parity counts as done)
            const int b = p_slot(two, x, i);
            uint64_t *done = bar.pv_done[two ? 1 - x : b];
            const uint32_t par = two ? (uint32_t)(x == 0 ? i + 1 : i) & 1u : (uint32_t)((i >> 1) + 1) & 1u;
            const uint32_t pb = smem_u32(sP) - (!two && (i & 1) ? (uint32_t)kCTile : 0u) + (uint32_t)r * 128u;  // (Q_B lies before P)
            uint32_t swz = (uint32_t)(r & 7) * 16u;
            asm volatile("" : "+r"(swz));  // (eight addresses kept over the loop would spill)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                alive &= mbar_wait_warp(done + hh, par, abort_flag);
#pragma unroll
                for (int c8 = 0; c8 < 8; ++c8) {
                    const int ch = hh * 8 + c8;
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(pb + hh * kCHalf + ((c8 * 16) ^ swz)),
                                 "r"(pk[4 * ch]), "r"(pk[4 * ch + 1]), "r"(pk[4 * ch + 2]), "r"(pk[4 * ch + 3])
                                 : "memory");
                }
                fence_proxy_async_smem();  // P as the tensor cores read it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_ready[b][hh]);
            }
        }
        if (!alive && lane == 0) fail(53);
        // the set agrees on going on
        if (lane == 0) sm.walive[x][q4] = alive ? 1 : 0;
        cbar(bar_id);
        alive = sm.walive[x][0] && sm.walive[x][1] && sm.walive[x][2] && sm.walive[x][3];
        if (alive) {
            if (r == 0) {
                const bool ok = mbar_wait(&bar.pv_done[p_slot(two, x, ntiles - 1)][1], p_use(two, ntiles - 1) & 1, abort_flag);
                if (!ok) fail(56);
                sm.go[x] = ok && !*abort_flag;
            }
            cbar(bar_id);
            if (sm.go[x]) {
                tc_fence_after();
                const uint32_t o_t = tmem + colO + lane_base;
                if (blk.pieces > 1) {
                    float *pp = part + (((size_t)blk.slot * pv.Hkv + hk) * 2 + x) * (D + 2) * kCRows + r;
#pragma unroll 1
                    for (int cb = 0; cb < D / 32; ++cb) {
                        uint32_t ov[32];
                        tmem_ld32(o_t + cb * 32, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) pp[(size_t)(cb * 32 + e) * kCRows] = __uint_as_float(ov[e]);
                    }
                    pp[(size_t)D * kCRows] = m_ref;
                    pp[(size_t)(D + 1) * kCRows] = l;
                } else {
                    // o = O / l as bf16, staged in a V tile that no product reads any more (set B's last
                    // comes after set A's: B takes the last tile's, A the other), then rows of 256 bytes side
                    // by side
                    uint8_t *stg = ring + (size_t)((ntiles + x) & 1) * 2 * kCTile + kCTile;
                    // (a row whose scores are all -inf: 0 / 0, NaN as softmax has it)
                    bool blind = pos < 0;  // sees nothing
                    if constexpr (MOD) blind = lo > pos && doc >= head;
                    const float inv = blind ? 0.f : 1.f / l;
#pragma unroll 1
                    for (int cb = 0; cb < D / 32; ++cb) {
                        uint32_t ov[32];
                        tmem_ld32(o_t + cb * 32, ov);
                        tmem_wait_ld();
                        if (__builtin_expect(blind, 0)) {  // sees nothing: zero, though 0 times a value may be NaN
#pragma unroll
                            for (int e = 0; e < 32; ++e) ov[e] = 0;
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = c_pack(__uint_as_float(ov[8 * q + 2 * e]) * inv,
                                              __uint_as_float(ov[8 * q + 2 * e + 1]) * inv);
                            *reinterpret_cast<uint4 *>(stg + c_chunk(r, cb * 4 + q)) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    cbar(bar_id);
                    const int ch = r % kChunks;
                    const uint32_t by_g = 0x10000u / (uint32_t)G + 1;  // row / G for rows below 128
#pragma unroll 8
                    for (int k = 0; k < kChunks; ++k) {
                        const int row = r / kChunks + kCRows / kChunks * k, t = (int)((uint32_t)row * by_g >> 16);
                        const int tok = blk.row0 + x * TS + t, h = hk * G + row - t * G;
                        if (row >= toks * G || !YOCO_DCHECK(tok < rows && h < Hq, 0x68)) continue;
                        *reinterpret_cast<uint4 *>(O + ((size_t)tok * Hq + h) * D + ch * 8) =
                            *reinterpret_cast<const uint4 *>(stg + c_chunk(row, ch));
                    }
                }
                tc_fence_before();
            }
        }
        }
        fence_proxy_async_smem();  // the next entry's copies go where this one's rows were staged
        if (!c_end(abort_flag) || !sm.task[(n + 1) & 1].more) break;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_dealloc(tmem, 512);
}

}  // namespace yoco

namespace yoco_host {
using namespace yoco;

template <int MODE, int D>
static cudaError_t launch(const PagedArgs &a, const PagedGrid &g, const CUtensorMap &mq, const CUtensorMap &mk,
                          const CUtensorMap &mv, cudaStream_t st) {
    // the shared-memory opt-in is set on every launch (it belongs to the current device)
    cudaError_t e = cudaFuncSetAttribute(paged_prefill_tc_kernel<MODE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kCSmem<(MODE > 0)>);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int64_t items = (int64_t)g.cap * a.cache->Hkv;
    if (items > 0x7fffffff) return cudaErrorInvalidValue;
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(items, g.slots));
    cfg.blockDim = dim3(kCThreads);
    cfg.dynamicSmemBytes = kCSmem<(MODE > 0)>;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    const PagedMod mod = paged_mod(a);
    return cudaLaunchKernelEx(&cfg, paged_prefill_tc_kernel<MODE, D>, mq, mk, mv, (bf16_t *)a.O, g.part, (PagedPlan *)g.plan,
                              (const typename PagedKind<(MODE > 0)>::Entry *)g.entries, g.cap, a.rows, a.Hq, paged_view(a), mod,
                              mod.qk, a.err);
}

template <int D>
static cudaError_t launch_scored(const PagedArgs &a, const PagedGrid &g, const CUtensorMap &mq, const CUtensorMap &mk,
                                 const CUtensorMap &mv, cudaStream_t st) {
    const bool cap = a.scores->softcap > 0.f, bias = a.scores->slopes != nullptr;
    if (cap) {
        constexpr int both = kModMask + kModCap;
        switch (paged_mod(a).degree) {
            case 2:
                if constexpr (D == 128)
                    return bias ? launch<both + kModShort + kModBias, D>(a, g, mq, mk, mv, st) : launch<both + kModShort, D>(a, g, mq, mk, mv, st);
                return cudaErrorInvalidValue;
            case 3: return bias ? launch<both + kModBias, D>(a, g, mq, mk, mv, st) : launch<both, D>(a, g, mq, mk, mv, st);
            default: return bias ? launch<both + kModWide + kModBias, D>(a, g, mq, mk, mv, st) : launch<both + kModWide, D>(a, g, mq, mk, mv, st);
        }
    }
    return bias ? launch<kModMask + kModBias, D>(a, g, mq, mk, mv, st) : launch<kModMask, D>(a, g, mq, mk, mv, st);
}

cudaError_t paged_prefill_tc(const PagedArgs &a, const PagedGrid &g, cudaStream_t st) {
    const int G = a.Hq / a.cache->Hkv, TS = kCRows / G, d = a.cache->d;
    CUtensorMap mq, mk, mv;
    // Q [rows, Hq, d] by boxes of TS tokens x G heads x 64 channels
    const uint64_t dims[3] = {(uint64_t)d, (uint64_t)a.Hq, (uint64_t)a.rows};
    const uint64_t strides[2] = {(uint64_t)d * 2, (uint64_t)a.Hq * d * 2};
    const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)TS};
    if (!paged_map(&mq, a.Q, 3, dims, strides, box) || !paged_kv_map(&mk, a.cache->k, a.cache) ||
        !paged_kv_map(&mv, a.cache->v, a.cache))
        return cudaErrorInvalidValue;
    if (d == 64) return a.scores ? launch_scored<64>(a, g, mq, mk, mv, st) : cudaErrorInvalidValue;
    return a.scores ? launch_scored<128>(a, g, mq, mk, mv, st) : launch<0, 128>(a, g, mq, mk, mv, st);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_prefill_tc)
