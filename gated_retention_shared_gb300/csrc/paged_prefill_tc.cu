// paged_prefill_tc.cu -- attention of chunks of new rows over the paged cache on the tensor
// cores, bf16, head size 128, up to 16 query heads to a kv head.
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
// Pages, rows out of sight and pages that are not there: as in paged_decode_tc.cu; set A's
// warps clear the V rows that no row of the block sees.  Where the plan (paged_plan.cu) cuts a
// row block's keys into pieces, the unnormalised sums are joined by paged_merge_rows_kernel;
// the partials lie column by column, so a warp's 32 rows store side by side.
//
// One block per SM; it takes entry after entry of the plan's list from a counter, longest first.
// The next entry is chosen three tiles before this one's end, gets barriers of its own (two
// groups in turn, set up anew while the other is in use) and its first K tile while this one's
// rows are written; then all warps meet.
//
// Warps: 0 TMA producer, 1 issues S products, 2 issues P V products, 3 the next entry, 4-7 set
// A, 8-11 set B (thread = TMEM lane = row).  S and P V have issuers of their own so that
// S_X(i + 1) goes as soon as S_X(i) has been read, whatever P the other issuer waits for.
//
// What bounds it (512 rows over 131072 keys: 586-630 us with the card's power, 1.46 us a tile of
// 2 x 128 rows at the least; the products alone are 1.08): the softmax warps' own chain, about 2800 cycles a tile from S to P
// with no pipe above a third; and some 6 us an entry around its tiles (first Q, K, S; last P V;
// rows out).  What counted, each timed as the kernel then was, on the long chunk if not said:
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
//     at once (2 us).
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

constexpr int kCD = 128;                       // head size
constexpr int kCRows = 128;                    // rows of a set
constexpr int kCStages = 2;
constexpr int kCTile = kPagedTile * kCD * 2;   // 32 KB
constexpr int kCHalf = kCTile / 2;             // 64 channels (or keys) of 128 rows
constexpr int kCThreads = 384;
constexpr float kCLog2e = 1.4426950408889634f;
constexpr float kCGap = 8.f * kCLog2e;

struct PagedPreBars {
    uint64_t q_full;
    uint64_t kfull[kCStages], kempty[kCStages], vfull[kCStages], vempty[kCStages];
    uint64_t s_full[2], s_free[2];          // per set
    uint64_t p_ready[2][2], pv_done[2][2];  // per set (one set: per P buffer) and 64-key half
};

// what an entry needs; the next entry's is filled while this one's runs
struct PagedPreTask {
    PagedPreBars bar;
    PagedEntry blk;
    int hk;
    int more;  // there is such an entry
};

struct PagedPreSmem {
    PagedPreTask task[2];
    uint64_t drain[2];
    int walive[2][4];
    uint32_t tmem_base;
    int abort_flag;
    int go[2];
};

constexpr size_t kCTileBytes = (size_t)3 * kCTile + (size_t)kCStages * 2 * kCTile;  // Q_A, Q_B, P, K/V rings
constexpr size_t kCSmem = kCTileBytes + sizeof(PagedPreSmem) + 1024;
static_assert(kCSmem <= 232448, "paged prefill tiles must fit shared memory");

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

__global__ void __launch_bounds__(kCThreads, 1)
paged_prefill_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, bf16_t *__restrict__ O, float *__restrict__ part,
                        PagedPlan *plan, const PagedEntry *__restrict__ entries, int cap, int rows, int Hq, const PagedView pv,
                        float c2, int *err) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    uint8_t *tiles = smem_raw + pad;
    uint8_t *sQ = tiles;                 // Q_A, Q_B
    uint8_t *sP = tiles + 2 * kCTile;
    uint8_t *ring = tiles + 3 * kCTile;  // stage s: K at ring + 2 s kCTile, V after it
    PagedPreSmem &sm = *reinterpret_cast<PagedPreSmem *>(tiles + kCTileBytes);
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
    auto fetch = [&](int item, int entry, PagedPreTask &task) {
        for (;;) {
            // (both loads at once: the list has room for `cap` entries)
            const int word = lane < 16 ? paged_ld(reinterpret_cast<const int *>(entries + min(entry, cap - 1)) + lane) : 0;
            const int count = paged_ld(&plan->entries);
            if (entry >= count) {
                if (lane == 0) task.more = 0;
                break;
            }
            if (lane < 16) reinterpret_cast<int *>(&task.blk)[lane] = word;
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
    const int psz = min(1 << pv.shift, kPagedTile), boxes = 2 * (kPagedTile / psz);
    const int mine = (lane >> 1) * psz;
    // what the table says of this lane's box of tile i (fetched ahead of use, so not yet looked
    // at); -1 past the last place
    auto look_up = [&](const PagedEntry &blk, int i) -> int {
        const int v = (blk.i0 + i) * kPagedTile + mine, e = blk.range.slot(v) >> pv.shift;
        const bool there = lane < boxes && v < blk.range.places && e < pv.max_pages;
        return there ? pv.table[(size_t)blk.b * pv.max_pages + e] : -1;
    };
    // that page, or the one past the pool
    auto page_of = [&](const PagedEntry &blk, int i, int entry_of_table) -> int {
        if ((unsigned)entry_of_table < (unsigned)pv.num_pages) return entry_of_table;
        if (lane < boxes && (blk.i0 + i) * kPagedTile + mine < blk.range.places) paged_report(err, kErrPagedPage);
        return pv.num_pages;
    };
    const int half = lane & 1;
    auto row_of = [&](const PagedEntry &blk, int i) -> int {  // of tile i's box in its page
        return blk.range.slot((blk.i0 + i) * kPagedTile + mine) & ((1 << pv.shift) - 1);
    };
    auto copy = [&](PagedPreTask &task, int hk, int i, bool is_v, int page, int row) {  // K or V tile i into its (free) slot
        const int s = i % kCStages;
        uint8_t *st = ring + (size_t)s * 2 * kCTile + (is_v ? kCTile : 0);
        uint64_t *full = is_v ? &task.bar.vfull[s] : &task.bar.kfull[s];
        if (lane == 0) mbar_arrive_expect_tx(full, kCTile);
        __syncwarp();
        if (lane < boxes)
            tma_load_4d(st + half * kCHalf + mine * 128, is_v ? &tm_v : &tm_k, full, half * 64, row, hk, page);
    };
    auto copy_q = [&](PagedPreTask &task) {
        if (lane == 0) {
            const int sets = task.blk.nrow > TS ? 2 : 1;
            mbar_arrive_expect_tx(&task.bar.q_full, (uint32_t)(sets * 2 * TS * G * 128));
            for (int x = 0; x < sets; ++x)
                for (int hf = 0; hf < 2; ++hf)
                    tma_load_3d(sQ + x * kCTile + hf * kCHalf, &tm_q, &task.bar.q_full, hf * 64, task.hk * G,
                                task.blk.row0 + x * TS);
        }
        __syncwarp();
    };
    int pg0 = -1, pg1 = -1;
    // the entry's first pages and K tile
    auto first_k = [&](PagedPreTask &task) {
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
            PagedPreTask &task = sm.task[n & 1], &next = sm.task[(n + 1) & 1];
            const PagedEntry &blk = task.blk;
            const int ntiles = blk.i1 - blk.i0;
            volatile int no_abort = 0;
            bool told = false;  // warp 3 takes the next entry late: who is done first takes the longest
            auto tell = [&]() {
                if (!told) asm volatile("bar.arrive 11, 64;\n" ::: "memory");
                told = true;
            };
            if (ntiles > 0) {
                if (n > 0) copy_q(task);
                int nk = 1, nv = 0;  // tiles whose K / V copy was issued
                const int c_i0 = blk.i0, c_sink = blk.range.sink_slots, c_delta = blk.range.base - c_sink, c_hk = task.hk;
                bool ok = true;
                auto load = [&](int i, bool is_v, int page) {
                    const int s = i % kCStages, v = (c_i0 + i) * kPagedTile + mine;
                    const int row = (v < c_sink ? v : v + c_delta) & ((1 << pv.shift) - 1);
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
                if (lane == 0) {
                    // leave no copy in flight (only the last two of each kind can be)
                    mbar_wait(&task.bar.q_full, 0, &no_abort, 200000000ull);
                    for (int k = max(0, nk - kCStages); k < nk; ++k)
                        mbar_wait(&task.bar.kfull[k % kCStages], (k / kCStages) & 1, &no_abort, 200000000ull);
                    for (int k = max(0, nv - kCStages); k < nv; ++k)
                        mbar_wait(&task.bar.vfull[k % kCStages], (k / kCStages) & 1, &no_abort, 200000000ull);
                    // nor a tile in use, nor a commit on its way to a barrier that is set up anew
                    for (int k = max(0, nk - kCStages); k < nk && ok; ++k)
                        ok = mbar_wait(&task.bar.kempty[k % kCStages], (k / kCStages) & 1, abort_flag);
                    for (int k = max(0, nv - kCStages); k < nv && ok; ++k)
                        ok = mbar_wait(&task.bar.vempty[k % kCStages], (k / kCStages) & 1, abort_flag);
                    if (!ok) fail(51);
                }
                __syncwarp();
            }
            tell();
            // the next entry's first K tile comes in while this one's rows are written
            asm volatile("bar.sync 10, 64;\n" ::: "memory");
            const bool ahead = next.more && next.blk.i1 > next.blk.i0 && __all_sync(0xffffffffu, !*abort_flag);
            if (ahead) first_k(next);
            if (!c_end(abort_flag)) {
                if (ahead && lane == 0) mbar_wait(&next.bar.kfull[0], 0, &no_abort, 200000000ull);
                break;
            }
            if (!next.more) break;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA: S = Q K^T
        c_regs_dec();
        for (int n = 0;; ++n) {
            PagedPreBars &bar = sm.task[n & 1].bar;
            const PagedEntry &blk = sm.task[n & 1].blk;
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
                        for (int kk = 0; kk < 8; ++kk) {
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
            const PagedEntry &blk = sm.task[n & 1].blk;
            const int ntiles = blk.i1 - blk.i0;
            const bool two = blk.nrow > TS;
            if (lane == 0) {
                const uint32_t id_o = idesc_bf16_f32(kCRows, kCD, false, true);  // A = P (K-major), B = V (N-major)
                bool ok = true;
                for (int i = 0; i < ntiles && ok; ++i) {
                    const int s = i % kCStages;
                    if (!(ok = mbar_wait(&bar.vfull[s], (i / kCStages) & 1, abort_flag))) break;
                    const uint64_t dp = smem_desc_sw128(smem_u32(!two && (i & 1) ? sQ + kCTile : sP), 16, 1024);
                    const uint64_t dv = smem_desc_sw128(smem_u32(ring + (size_t)s * 2 * kCTile + kCTile), kCHalf, 1024);
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
            PagedPreTask &next = sm.task[(n + 1) & 1];
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
        const PagedEntry &blk = sm.task[n & 1].blk;
        const int hk = sm.task[n & 1].hk, ntiles = blk.i1 - blk.i0;
        const bool two = *(const volatile int *)&blk.nrow > TS;
        if (ntiles == 0) {  // nothing to see: zeros
            for (int e = tid - 128; e < blk.nrow * G * (kCD / 8); e += 256)
                *reinterpret_cast<uint4 *>(O + ((size_t)(blk.row0 + e / (G * 16)) * Hq + hk * G) * kCD + (e % (G * 16)) * 8) =
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
            const PagedRange &rg = blk.range;
            const int from = rg.sink_slots + rg.lo - rg.base;  // the first place that is seen for being in the window
            e_lo = (from + kPagedTile - 1) / kPagedTile - blk.i0;
            e_hi = rg.places / kPagedTile - blk.i0;
        }
        float m_ref = -INFINITY, l = 0.f;  // base-2 units
        // One exit from the tile loop: a wait that gave up makes what follows garbage (the status word
        // says so), but every barrier is still served.  A warp gives up as one: tcgen05.ld and the
        // votes take whole warps.
        bool alive = true;
        for (int i = 0; i < ntiles && alive; ++i) {
            alive = mbar_wait_warp(&bar.s_full[x], i & 1, abort_flag);
            tc_fence_after();
            const uint32_t s_t = tmem + colS + lane_base;
            uint32_t sv[128];
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) tmem_ld32(s_t + cb * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * cb));
            tmem_wait_ld();
            // S is in registers: the MMA may write S(i + 1) over it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.s_free[x]);
            // place 0 of the tile, and what its slot is where it lies past the sinks' chunks
            const int v0 = (blk.i0 + i) * kPagedTile, key0 = v0 + delta;
            // every row of the set sees every slot of the tile
            const bool full = v0 >= sink_slots && key0 + kPagedTile - 1 <= set_lo &&
                              (pv.window <= 0 || key0 > set_hi - pv.window || key0 + kPagedTile <= pv.sinks);
            if (__builtin_expect(!full, 0)) {
                // the places this row sees of the tile: sinks in the sinks' chunks, then a run up to its
                // own position from the window's first slot on, and sinks that lie in those chunks
                const int hi_c = pos + 1 - key0;
                const int lo_c = pv.window > 0 ? pos + 1 - pv.window - key0 : -1;
                const int sk_c = min(pv.sinks - key0, hi_c);
                const int ch_c = sink_slots - v0, sc_c = min(ch_c, min(pv.sinks, pos + 1) - v0);
                uint32_t bits[4];
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    bits[w] = (((c_below(hi_c - 32 * w) & ~c_below(lo_c - 32 * w)) | c_below(sk_c - 32 * w)) &
                               ~c_below(ch_c - 32 * w)) | c_below(sc_c - 32 * w);
#pragma unroll
                for (int c = 0; c < kPagedTile; ++c)
                    sv[c] = (bits[c >> 5] & (1u << (c & 31))) ? sv[c] : 0xff800000u;  // -inf
            }
            float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kPagedTile; c += 2)
                mq[(c >> 1) & 3] = fmax3(mq[(c >> 1) & 3], __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            // rows past the set's tokens hold whatever shared memory held: they never move the
            // reference (no rescaling for their sake) and are never stored
            const float mt = used ? fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * c2 : -INFINITY;
            const bool move = (mt > m_ref + kCGap) || (m_ref == -INFINITY && mt > -INFINITY);
            const float m_old = m_ref;
            m_ref = move ? mt : m_ref;
            const float alpha = move ? (m_old == -INFINITY ? 0.f : c_ex2(m_old - mt)) : 1.f;
            const float mu = (m_ref == -INFINITY) ? 0.f : m_ref;
            const uint64_t c2x2 = f2_pack(c2, c2), nmu2 = f2_pack(-mu, -mu);
            uint64_t acc2[4] = {0, 0, 0, 0};  // packed zeros
            uint32_t pk[kPagedTile / 2];
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // 32 columns at a time, each step for all of them: element by element
                                           // they come out as chains of latencies
#pragma unroll
                for (int c = 16 * q; c < 16 * q + 16; ++c) {
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), c2x2, nmu2), x0, x1);
                    sv[2 * c] = __float_as_uint(x0);
                    sv[2 * c + 1] = __float_as_uint(x1);
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
                for (int cb = 0; cb < kCD; cb += 8) {  // (in small steps: it is rare, and registers are not)
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
            if (__builtin_expect(i < e_lo || i >= e_hi || !two, 0)) {
                alive &= mbar_wait_warp(&bar.vfull[i % kCStages], (i / kCStages) & 1, abort_flag);
                if (alive && !blk.range.seen(blk.range.slot(v0 + r), pv.sinks)) {
                    uint8_t *vr = ring + (size_t)(i % kCStages) * 2 * kCTile + kCTile + r * 128;
#pragma unroll 1
                    for (int ch = 0; ch < 16; ++ch)
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
                    float *pp = part + (((size_t)blk.slot * pv.Hkv + hk) * 2 + x) * (kCD + 2) * kCRows + r;
#pragma unroll 1
                    for (int cb = 0; cb < 4; ++cb) {
                        uint32_t ov[32];
                        tmem_ld32(o_t + cb * 32, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) pp[(size_t)(cb * 32 + e) * kCRows] = __uint_as_float(ov[e]);
                    }
                    pp[(size_t)kCD * kCRows] = m_ref;
                    pp[(size_t)(kCD + 1) * kCRows] = l;
                } else {
                    // o = O / l as bf16, staged in this set's Q tile (every S product is done), then rows
                    // of 256 bytes side by side
                    uint8_t *stg = sQ + x * kCTile;
                    // (a row whose scores are all -inf: 0 / 0, NaN as softmax has it)
                    const float inv = pos < 0 ? 0.f : 1.f / l;
#pragma unroll 1
                    for (int cb = 0; cb < 4; ++cb) {
                        uint32_t ov[32];
                        tmem_ld32(o_t + cb * 32, ov);
                        tmem_wait_ld();
                        if (__builtin_expect(pos < 0, 0)) {  // sees nothing: zero, though 0 times a value may be NaN
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
                    const int ch = r & 15;
                    const uint32_t by_g = 0x10000u / (uint32_t)G + 1;  // row / G for rows below 128
#pragma unroll 8
                    for (int k = 0; k < kCRows / 8; ++k) {
                        const int row = (r >> 4) + 8 * k, t = (int)((uint32_t)row * by_g >> 16);
                        const int tok = blk.row0 + x * TS + t, h = hk * G + row - t * G;
                        if (row >= toks * G || !YOCO_DCHECK(tok < rows && h < Hq, 0x68)) continue;
                        *reinterpret_cast<uint4 *>(O + ((size_t)tok * Hq + h) * kCD + ch * 8) =
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

cudaError_t paged_prefill_tc(const PagedArgs &a, const PagedGrid &g, cudaStream_t st) {
    const int G = a.Hq / a.cache->Hkv, TS = kCRows / G;
    CUtensorMap mq, mk, mv;
    // Q [rows, Hq, 128] by boxes of TS tokens x G heads x 64 channels
    const uint64_t dims[3] = {(uint64_t)kCD, (uint64_t)a.Hq, (uint64_t)a.rows};
    const uint64_t strides[2] = {(uint64_t)kCD * 2, (uint64_t)a.Hq * kCD * 2};
    const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)TS};
    if (!paged_map(&mq, a.Q, 3, dims, strides, box) || !paged_kv_map(&mk, a.cache->k, a.cache) ||
        !paged_kv_map(&mv, a.cache->v, a.cache))
        return cudaErrorInvalidValue;
    // the shared-memory opt-in is set on every launch (it belongs to the current device)
    cudaError_t e = cudaFuncSetAttribute(paged_prefill_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kCSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int64_t items = (int64_t)g.cap * a.cache->Hkv;
    if (items > 0x7fffffff) return cudaErrorInvalidValue;
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(items, g.slots));
    cfg.blockDim = dim3(kCThreads);
    cfg.dynamicSmemBytes = kCSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, paged_prefill_tc_kernel, mq, mk, mv, (bf16_t *)a.O, g.part, (PagedPlan *)g.plan,
                              (const PagedEntry *)g.entries, g.cap, a.rows, a.Hq, paged_view(a), a.scale * kCLog2e, a.err);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_prefill_tc)
