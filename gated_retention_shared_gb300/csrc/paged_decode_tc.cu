// paged_decode_tc.cu -- one new row per sequence over the paged cache on the tensor cores,
// bf16, head size 128, up to 16 query heads to a kv head.
//
// One block per SM walks an equal run of 128-key tiles (paged.cuh) through as many
// (sequence, kv head) units as the run covers, the tile rings running on across units.  Per
// tile, transposed so that the few query heads are the MMA's N:
//     S^T = K Q^T      M = 128 keys, N = 16 heads, K = 128       (TMEM)
//     p   = 2^(c s - m)       one thread per key, running maximum per head
//     O^T = V^T P^T    M = 128 dims, N = 16, K = 128 keys        (TMEM)
//     o   = o 2^(m_old - m_new) + O^T     one thread per head dim, fp32 registers
// p is rounded to bf16 for the second product (half a step, 2^-9 of each weight on average
// less, independent from key to key); its sum is kept in fp32 before that rounding.
//
// A tile's pages are separate TMA boxes (128 keys are 8 pages of 16, or part of a page),
// issued by as many lanes; the next tile's page numbers are fetched while this tile's slot
// is waited for.  A page that no row sees, or that the pool does not have, is asked for past
// the pool's end, which TMA fills with zeros without reading.  V rows that the row does not
// see are set to zero in shared memory before the product (their weights are 0, but 0 * NaN
// is not).
//
// Warps: 0 TMA producer, 1 MMA issuer, 2-5 softmax and sums (thread = TMEM lane = key of the
// tile / head dim), 6-7 the units' query rows into one of two shared-memory tiles.  A unit's
// last sums wait until the next unit's first weights are out, so that the tensor cores and
// the rings never stand still between units.  The softmax warps meet once a tile; every
// thread waits for what it reads itself, so no warp waits for another's wait as well.
//
// What bounds it: DRAM reads of K and V (32 sequences of 60 to 32000 keys 122 us, 6.2 TB/s;
// one of 10^6 keys 605 us, 7.1 TB/s).  With 16 query heads to a kv head the softmax shows: 32
// sequences of 60 to 30000 keys over 8 kv heads take 287 us with 3 heads each (6.8 TB/s), 291
// with 8 and 352 with 16 (5.6 TB/s).  Short calls (700 keys: 8.4 us) are the launch, two
// dependent tiles and the merge.  Four barriers a tile in place of one: 130 us for the first 32.
#include <cudaTypedefs.h>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "tc.cuh"

namespace yoco {

using namespace tc;

constexpr int kPD = 128;                   // head size = keys per tile
constexpr int kPN = 16;                    // MMA N: query heads (padded)
constexpr int kPStages = 3;
constexpr int kPTile = kPagedTile * kPD * 2;
constexpr int kPHalf = kPTile / 2;
constexpr int kPThreads = 256;
constexpr int kPQBytes = kPN * kPD * 2;
constexpr uint32_t kPColS = 0, kPColO = 32;
constexpr float kPLog2e = 1.4426950408889634f;

struct PagedDecSmem {
    uint64_t full_k[kPStages], full_v[kPStages], empty_k[kPStages], empty_v[kPStages];
    uint64_t s_full[2], s_free[2], p_ready[2], o_full[2], o_free[2], q_full[2], q_empty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    int sums[kPThreads / 32];
    int4 dead[2];             // per tile parity: softmax warps that have given up
    float wmax[2][4][kPN];    // per tile parity and softmax warp
    float wsum[4][kPN];
};

constexpr size_t kPTileBytes = (size_t)kPStages * 2 * kPTile + 4 * kPQBytes;  // K/V rings, 2 Q, 2 P
constexpr size_t paged_dec_smem(int B) { return kPTileBytes + sizeof(PagedDecSmem) + 1024 + ((size_t)B + 1) * sizeof(int); }
static_assert(paged_dec_smem(kPagedMaxB) <= 232448, "paged decode tiles must fit shared memory");

__device__ __forceinline__ void pbar(int n) {  // the softmax warps
    __syncwarp();
    asm volatile("bar.sync 1, %0;\n" ::"r"(n) : "memory");
}

__device__ __forceinline__ float pex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

template <int NQ>
__global__ void __launch_bounds__(kPThreads, 1)
paged_decode_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const bf16_t *__restrict__ Q, bf16_t *__restrict__ O, float *__restrict__ part,
                       PagedCut *__restrict__ cuts, int Hq, const PagedView pv, float c2, int keep_pages, int *err) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    uint8_t *tiles = smem_raw + pad;
    uint8_t *sQ = tiles + (size_t)kPStages * 2 * kPTile;
    uint8_t *sP = sQ + 2 * kPQBytes;
    PagedDecSmem &sm = *reinterpret_cast<PagedDecSmem *>(sP + 2 * kPQBytes);
    int *pre = reinterpret_cast<int *>(&sm + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = Hq / pv.Hkv, c = blockIdx.x;

    if (tid == 0) {
        for (int s = 0; s < kPStages; ++s) {
            mbar_init(&sm.full_k[s], 1);
            mbar_init(&sm.full_v[s], 1);
            mbar_init(&sm.empty_k[s], 1);
            mbar_init(&sm.empty_v[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.s_free[s], 4);   // one arrival per softmax warp
            mbar_init(&sm.p_ready[s], 4);
            mbar_init(&sm.o_full[s], 1);
            mbar_init(&sm.o_free[s], 4);
            mbar_init(&sm.q_full[s], 64);
            mbar_init(&sm.q_empty[s], 1);
        }
        mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // Q and P tiles zero: heads past G stay so
    for (int e = tid; e < 4 * kPQBytes / 16; e += kPThreads) reinterpret_cast<uint4 *>(sQ)[e] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 0) {
        tmem_alloc(&sm.tmem_base, 64);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    tc_fence_before();
    paged_prefix<kPThreads>(pv, pre, sm.sums, err);
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const int total = pre[pv.B] * pv.Hkv;
    const int each = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    const int from = (int)min((int64_t)c * each, (int64_t)total);
    const int to = (int)min((int64_t)(c + 1) * each, (int64_t)total);
    volatile int *abort_flag = &sm.abort_flag;
    auto fail = [&](int code) {
        *abort_flag = 1;
        paged_report(err, code);
    };
    PagedWalk w;
    bool more = w.start(pv, pre, from, to);

    if (warp == 0) {
        // -------------------------------------------------------------- TMA
        const int psz = min(1 << pv.shift, kPagedTile);  // slots of a box
        const int boxes = 2 * (kPagedTile / psz);        // per tile: (page, 64-channel half)
        const uint64_t pol_keep = l2_policy_evict_normal(), pol_stream = l2_policy_evict_first();
        PagedRange range{};
        int t = 0, slot = 0, page = 0;
        // this lane's box of the tile at (w, t): its page, or the one past the pool
        auto look_up = [&]() {
            const int v = t * kPagedTile + (lane >> 1) * psz;
            page = -1;
            if (lane < boxes && v < range.places) {
                slot = range.slot(v);
                page = paged_page(pv, w.b, slot >> pv.shift, err);
            }
            if (page < 0) page = pv.num_pages;
        };
        auto enter = [&]() {
            const int p = paged_len(pv, w.b, nullptr) - 1;
            range = paged_range(pv, p, p);
            t = w.t0;
        };
        if (more) {
            enter();
            look_up();
        }
        int i = 0;
        bool okp = true;
        for (; more; ++i) {
            const int s = i % kPStages;
            const uint32_t par = ((i / kPStages) + 1) & 1;
            const int my_page = page, my_row = slot & ((1 << pv.shift) - 1), hk = w.hk;
            if (++t == w.t1) {
                more = w.next(pv, pre);
                if (more) enter();
            }
            if (more) look_up();
            const uint64_t pol = my_page < keep_pages ? pol_keep : pol_stream;
            uint8_t *dst = tiles + (size_t)s * 2 * kPTile + (lane & 1) * kPHalf + (lane >> 1) * psz * 128;
            for (int is_v = 0; is_v < 2; ++is_v) {
                uint64_t *full = is_v ? &sm.full_v[s] : &sm.full_k[s];
                if (i >= kPStages) okp = mbar_wait(is_v ? &sm.empty_v[s] : &sm.empty_k[s], par, abort_flag);
                okp = __all_sync(0xffffffffu, okp);
                if (!okp) break;
                if (lane == 0) mbar_arrive_expect_tx(full, kPTile);
                __syncwarp();
                if (lane < boxes)
                    tma_load_4d_hint(dst + is_v * kPTile, is_v ? &tm_v : &tm_k, full, (lane & 1) * 64, my_row, hk, my_page,
                                     pol);
            }
            if (!okp) {
                if (lane == 0) fail(41);
                break;
            }
        }
        // leave no copy in flight (bounded by time only: an abort must still wait).  Where the
        // loop broke, tile i's K may be on its way too: its barrier is waited for all the same
        if (lane == 0) {
            volatile int no_abort = 0;
            for (int k = max(0, i - kPStages); k < i; ++k) {
                mbar_wait(&sm.full_k[k % kPStages], (k / kPStages) & 1, &no_abort, 200000000ull);
                mbar_wait(&sm.full_v[k % kPStages], (k / kPStages) & 1, &no_abort, 200000000ull);
            }
            if (!okp) mbar_wait(&sm.full_k[i % kPStages], (i / kPStages) & 1, &no_abort, 200000000ull);
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA
        if (lane == 0 && more) {
            const uint32_t id_s = idesc_bf16_f32(kPagedTile, kPN, false, false);  // A = K, B = Q (both K-major)
            const uint32_t id_o = idesc_bf16_f32(kPD, kPN, true, false);          // A = V^T (M-major), B = P^T (K-major)
            const int ntiles = to - from;
            int unit = 0, left = w.t1 - w.t0;
            bool enter = true;
            auto issue_s = [&](int i) -> bool {
                if (left == 0) {
                    (void)w.next(pv, pre);
                    left = w.t1 - w.t0;
                    ++unit;
                    enter = true;
                }
                const int s = i % kPStages;
                if (enter && !mbar_wait(&sm.q_full[unit & 1], (unit >> 1) & 1, abort_flag)) return false;
                enter = false;
                if (!mbar_wait(&sm.full_k[s], (i / kPStages) & 1, abort_flag)) return false;
                if (i >= 2 && !mbar_wait(&sm.s_free[i & 1], ((i / 2) - 1) & 1, abort_flag)) return false;
                tc_fence_after();
                const uint64_t dk = smem_desc_sw128(smem_u32(tiles + (size_t)s * 2 * kPTile), 16, 1024);
                const uint64_t dq = smem_desc_sw128(smem_u32(sQ + (unit & 1) * kPQBytes), 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(tmem + kPColS + 16 * (i & 1), dk + (uint64_t)(((kk >> 2) * kPHalf + (kk & 3) * 32) >> 4),
                           dq + (uint64_t)(((kk >> 2) * (kPN * 128) + (kk & 3) * 32) >> 4), id_s, kk > 0);
                mma_commit(&sm.s_full[i & 1]);
                mma_commit(&sm.empty_k[s]);
                if (--left == 0) mma_commit(&sm.q_empty[unit & 1]);
                return true;
            };
            bool ok = issue_s(0);
            for (int i = 0; i < ntiles && ok; ++i) {
                if (i + 1 < ntiles && !(ok = issue_s(i + 1))) break;
                const int s = i % kPStages;
                if (!(ok = mbar_wait(&sm.p_ready[i & 1], (i / 2) & 1, abort_flag))) break;
                if (i >= 2 && !(ok = mbar_wait(&sm.o_free[i & 1], ((i / 2) - 1) & 1, abort_flag))) break;
                if (!(ok = mbar_wait(&sm.full_v[s], (i / kPStages) & 1, abort_flag))) break;
                tc_fence_after();
                const uint64_t dv = smem_desc_sw128(smem_u32(tiles + (size_t)s * 2 * kPTile + kPTile), kPHalf, 1024);
                const uint64_t dp = smem_desc_sw128(smem_u32(sP + (i & 1) * kPQBytes), 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(tmem + kPColO + 16 * (i & 1), dv + (uint64_t)((kk * 2048) >> 4),
                           dp + (uint64_t)(((kk >> 2) * (kPN * 128) + (kk & 3) * 32) >> 4), id_o, kk > 0);
                mma_commit(&sm.o_full[i & 1]);
                mma_commit(&sm.empty_v[s]);
            }
            if (!ok) fail(42);
            mma_commit(&sm.drain);
            volatile int no_abort = 0;
            mbar_wait(&sm.drain, 0, &no_abort, 200000000ull);
        }
    } else if (warp >= 6) {
        // ------------------------------------------------------------ Q rows
        const int t = tid - 6 * 32;
        for (int unit = 0; more; ++unit, more = w.next(pv, pre)) {
            const bf16_t *src = Q + ((size_t)w.b * Hq + w.hk * G) * kPD;
            uint4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int e = t + 64 * x;  // 16-byte chunk e % 16 of head e / 16
                if (e < G * 16) v[x] = paged_ld16(src + (size_t)e * 8);
            }
            if (unit >= 2 && !mbar_wait(&sm.q_empty[unit & 1], ((unit >> 1) - 1) & 1, abort_flag)) {
                fail(43);
                break;
            }
            uint8_t *dst = sQ + (unit & 1) * kPQBytes;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int e = t + 64 * x;
                if (e < G * 16) *reinterpret_cast<uint4 *>(dst + sw128_offset(e >> 4, (e & 15) * 8, kPN)) = v[x];
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.q_full[unit & 1]);
        }
    } else {
        // ---------------------------------------------------- softmax and sums
        const int q4 = warp & 3;
        const int r = q4 * 32 + lane;  // key of the tile / head dim
        const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
        // sequences without a key: zeros
        for (int b = c; b < pv.B; b += gridDim.x)
            if (pre[b + 1] == pre[b])
                for (int h = 0; h < Hq; ++h) O[((size_t)b * Hq + h) * kPD + r] = 0;
        PagedCut cut{-1, 0, 0, 0};
        if (more && w.t0 > 0) cut = paged_cut(pv, pre, w, c, each);
        if (r == 0) cuts[c] = cut;
        float m[NQ], l[NQ], acc[NQ], corr[NQ], l_done[NQ], m_done[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) acc[n] = corr[n] = l_done[n] = m_done[n] = 0.f;
        int done_b = 0, done_hk = 0, done_slot = 0;  // the unit whose last tile is not added yet
        bool done_whole = false, alive = true;
        // acc = acc corr + O^T(i); corr belongs to tile i
        auto accumulate = [&](int i) {
            alive &= mbar_wait_warp(&sm.o_full[i & 1], (i / 2) & 1, abort_flag);
            __syncwarp();
            tc_fence_after();
            uint32_t o[16];
            tmem_ld16(tmem + kPColO + 16 * (i & 1) + lane_base, o);
            tmem_wait_ld();
#pragma unroll
            for (int n = 0; n < NQ; ++n) acc[n] = fmaf(acc[n], corr[n], __uint_as_float(o[n]));
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.o_free[i & 1]);
        };
        // the finished unit's output, or its partial result
        auto flush = [&]() {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float x = l_done[n];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
                if (lane == 0) sm.wsum[q4][n] = x;
            }
            pbar(128);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                if (n >= G) break;
                const float L = sm.wsum[0][n] + sm.wsum[1][n] + sm.wsum[2][n] + sm.wsum[3][n];
                if (!YOCO_DCHECK(done_b < pv.B && done_hk < pv.Hkv, 0x67)) continue;
                if (done_whole) {
                    O[((size_t)done_b * Hq + done_hk * G + n) * kPD + r] = from_f32<bf16_t>(acc[n] / L);
                } else {
                    float *pp = part + (((size_t)c * 2 + done_slot) * G + n) * (kPD + 2);
                    pp[r] = acc[n];
                    if (r == 0) {
                        pp[kPD] = m_done[n];
                        pp[kPD + 1] = L;
                    }
                }
            }
            pbar(128);  // wsum may be written again
        };
        // One barrier of the four warps a tile: it makes their maxima known, and with them which warps
        // have given up a wait, so that all leave together.
        int i = 0;
        bool all = true;
        for (int unit = 0; more && all; ++unit, more = w.next(pv, pre)) {
            const int p = paged_len(pv, w.b, nullptr) - 1;
            const PagedRange range = paged_range(pv, p, p);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                m[n] = -INFINITY;
                l[n] = 0.f;
            }
            for (int t = w.t0; t < w.t1; ++t, ++i) {
                alive &= mbar_wait_warp(&sm.s_full[i & 1], (i / 2) & 1, abort_flag);
                __syncwarp();
                tc_fence_after();
                uint32_t sv[16];
                tmem_ld16(tmem + kPColS + 16 * (i & 1) + lane_base, sv);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.s_free[i & 1]);
                const bool seen = range.seen(range.slot(t * kPagedTile + r), pv.sinks);
                float sc[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    sc[n] = seen && n < G ? c2 * __uint_as_float(sv[n]) : -INFINITY;
                    float x = sc[n];
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                    if (lane == 0) sm.wmax[i & 1][q4][n] = x;
                }
                // V rows out of sight: zero, once the tile has come (V(i - 3), the phase before, was used by
                // a product that this warp has seen the end of)
                if (range.edge(t, pv.sinks)) {
                    alive &= mbar_wait_warp(&sm.full_v[i % kPStages], (i / kPStages) & 1, abort_flag);
                    if (alive && !seen) {
                        uint8_t *vr = tiles + (size_t)(i % kPStages) * 2 * kPTile + kPTile + r * 128;
#pragma unroll
                        for (int ch = 0; ch < 16; ++ch)
                            *reinterpret_cast<uint4 *>(vr + (ch >> 3) * kPHalf + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                if (lane == 0) reinterpret_cast<int *>(&sm.dead[i & 1])[q4] = alive ? 0 : 1;
                pbar(128);
                const int4 dead = sm.dead[i & 1];
                if (dead.x | dead.y | dead.z | dead.w) {
                    all = false;
                    break;
                }
                uint8_t *pb = sP + (i & 1) * kPQBytes;
                float now[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const float(&wm)[4][kPN] = sm.wmax[i & 1];
                    const float mt = fmaxf(fmaxf(wm[0][n], wm[1][n]), fmaxf(wm[2][n], wm[3][n]));
                    const float mn = fmaxf(m[n], mt);
                    now[n] = (mn == -INFINITY) ? 1.f : pex2(m[n] - mn);
                    const float pe = (sc[n] == -INFINITY) ? 0.f : pex2(sc[n] - mn);
                    l[n] = fmaf(l[n], now[n], pe);
                    m[n] = mn;
                    if (n < G)
                        *reinterpret_cast<__nv_bfloat16 *>(pb + sw128_offset(n, r, kPN)) = __float2bfloat16_rn(pe);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_ready[i & 1]);
                if (i > 0) accumulate(i - 1);
                if (unit > 0 && t == w.t0) {
                    flush();
#pragma unroll
                    for (int n = 0; n < NQ; ++n) acc[n] = 0.f;
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n) corr[n] = now[n];
            }
            done_b = w.b;
            done_hk = w.hk;
            done_whole = w.whole();
            done_slot = unit > 0 ? 1 : 0;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                l_done[n] = l[n];
                m_done[n] = m[n];
            }
        }
        if (all && i > 0) {
            accumulate(i - 1);
            if (!alive) fail(45);
            flush();
        }
        if (!all && lane == 0) fail(44);
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 64);
}

}  // namespace yoco

namespace yoco_host {
using namespace yoco;

bool paged_map(CUtensorMap *m, const void *ptr, int rank, const uint64_t *dims, const uint64_t *strides,
               const uint32_t *box) {
    static PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)p;
    }();
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(ptr), dims, strides, box, es,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool paged_kv_map(CUtensorMap *m, const void *ptr, const yoco_paged_kv *c) {
    const uint64_t row = (uint64_t)c->d * 2, P = (uint64_t)c->page_size;
    const uint64_t dims[4] = {(uint64_t)c->d, P, (uint64_t)c->Hkv, (uint64_t)c->num_pages};
    const uint64_t strides[3] = {row, row * P, row * P * c->Hkv};
    const uint32_t box[4] = {64, (uint32_t)(c->page_size < kPagedTile ? c->page_size : kPagedTile), 1, 1};
    return paged_map(m, ptr, 4, dims, strides, box);
}

template <int NQ>
static cudaError_t launch(const CUtensorMap &mk, const CUtensorMap &mv, const PagedArgs &a, const PagedView &pv,
                          PagedCut *cuts, float *part, int keep, int blocks, cudaStream_t st) {
    // the shared-memory opt-in is set on every launch (it belongs to the current device)
    cudaError_t e = cudaFuncSetAttribute(paged_decode_tc_kernel<NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)paged_dec_smem(kPagedMaxB));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kPThreads);
    cfg.dynamicSmemBytes = paged_dec_smem(pv.B);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, paged_decode_tc_kernel<NQ>, mk, mv, (const bf16_t *)a.Q, (bf16_t *)a.O, part, cuts,
                              a.Hq, pv, a.scale * kPLog2e, keep, a.err);
}

cudaError_t paged_decode_tc(const PagedArgs &a, void *cuts, float *part, int blocks, cudaStream_t st) {
    CUtensorMap mk, mv;
    if (!paged_kv_map(&mk, a.cache->k, a.cache) || !paged_kv_map(&mv, a.cache->v, a.cache)) return cudaErrorInvalidValue;
    const PagedView pv = paged_view(a);
    // pages up to half the L2's size keep normal priority and stay cached for the next layer's
    // call over the same pool, the rest streams through
    const int64_t l2 = device_l2_bytes();
    const int64_t page_bytes = (int64_t)a.cache->page_size * a.cache->Hkv * kPD * 2 * 2;
    const int keep = (int)(l2 / 2 / page_bytes);
    const int G = a.Hq / pv.Hkv;
    PagedCut *pc = (PagedCut *)cuts;
    return G <= 4   ? launch<4>(mk, mv, a, pv, pc, part, keep, blocks, st)
           : G <= 8 ? launch<8>(mk, mv, a, pv, pc, part, keep, blocks, st)
                    : launch<16>(mk, mv, a, pv, pc, part, keep, blocks, st);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_decode_tc)
