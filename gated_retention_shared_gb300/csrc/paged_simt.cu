// paged_simt.cu -- attention over the paged cache on the CUDA cores, fp32 arithmetic: every
// type and head size the library has (the tensor-core kernels take bf16 at head size 128),
// and the merges of split keys that both paths share.
//
//   o = sum_m p_m v_m / sum_m p_m,   p_m = 2^(c q.k_m - r),  c = scale log2(e),
//
// over the slots m that the row sees, r a running maximum.  K and V of slots that no row
// of a block sees are never loaded, so what those hold (nothing yet, NaN, another
// sequence's rows) cannot reach a result.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace yoco {

constexpr float kPagedLog2e = 1.4426950408889634f;

// 4 or 8 consecutive elements (16 bytes) as floats
template <typename T> __device__ __forceinline__ void load16(const T *p, float (&x)[16 / sizeof(T)]) {
    const uint4 u = paged_ld16(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            x[i] = __uint_as_float(w[i]);
        }
    }
}

// ----------------------------------------------------------------- decode
//
// One row per sequence; a unit is one (sequence, kv head) with its G query heads.  Eight
// lanes hold one key (16-byte chunk j of the row in lane j % 8), four keys to a warp, 32 to
// the block: a key's score is summed over its lanes, and each group of eight lanes keeps a
// running maximum, sum and weighted sum of its own, merged at the end of the unit.  K and V
// go from global memory to registers once.  Groups with more than kDecQ heads take them
// kDecQ at a time, reading K and V again (from L2).  32 sequences of 60 to 30000 keys over 4 kv
// heads: fp32 x 128 282 us with one head each (6.9 TB/s, the read rate), 427 with four, 468 with
// eight; bf16 x 64 170, 223 and 440 us (2.9, 2.2 and 1.1 TB/s: the sums, not the reads).
constexpr int kDecThreads = 256;
constexpr int kDecWarps = kDecThreads / 32;
constexpr int kDecQ = 8;      // query heads at a time
constexpr int kDecKeys = 2;   // keys of a lane group in flight

template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kDecThreads)
paged_decode_simt_kernel(const T *__restrict__ Q, T *__restrict__ O, const T *__restrict__ K, const T *__restrict__ V,
                         float *__restrict__ part, PagedCut *__restrict__ cuts, int Hq, const PagedView pv, float c2,
                         int *err) {
    constexpr int EV = 16 / (int)sizeof(T);
    constexpr int NC = D / EV / 8;  // chunks of a key per lane
    constexpr int EL = NC * EV;     // elements of a key per lane
    static_assert(NC >= 1, "a key has at least one chunk per lane");
    extern __shared__ int pre[];
    __shared__ int sums[kDecWarps];
    __shared__ float qs[NQ][D];
    __shared__ float wm[kDecWarps][NQ], wl[kDecWarps][NQ], wo[kDecWarps][NQ][D];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j8 = lane & 7, grp = warp * 4 + (lane >> 3);
    const int G = Hq / pv.Hkv, c = blockIdx.x;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    paged_prefix<kDecThreads>(pv, pre, sums, err);
    const int total = pre[pv.B] * pv.Hkv;
    const int each = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    // sequences without a key: zeros
    for (int b = c; b < pv.B; b += gridDim.x)
        if (pre[b + 1] == pre[b])
            for (int e = tid; e < Hq * D; e += kDecThreads) O[(size_t)b * Hq * D + e] = from_f32<T>(0.f);
    PagedWalk w;
    PagedCut cut{-1, 0, 0, 0};
    bool more = w.start(pv, pre, (int)min((int64_t)c * each, (int64_t)total), (int)min((int64_t)(c + 1) * each, (int64_t)total));
    if (more && w.t0 > 0) cut = paged_cut(pv, pre, w, c, each);
    if (tid == 0) cuts[c] = cut;
    for (int seg = 0; more; ++seg, more = w.next(pv, pre)) {
        const int p = paged_len(pv, w.b, err) - 1;
        const PagedRange range = paged_range(pv, p, p);
        for (int g0 = 0; g0 < G; g0 += NQ) {
            const int nq = min(NQ, G - g0);
            const size_t qrow = (size_t)w.b * Hq + w.hk * G + g0;
            __syncthreads();
            for (int e = tid * EV; e < NQ * D; e += kDecThreads * EV) {
                float x[EV];
#pragma unroll
                for (int i = 0; i < EV; ++i) x[i] = 0.f;
                if (e < nq * D) load16(Q + qrow * D + e, x);
#pragma unroll
                for (int i = 0; i < EV; ++i) qs[e / D][e % D + i] = c2 * x[i];
            }
            __syncthreads();
            float m[NQ], l[NQ], acc[NQ][EL];
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
#pragma unroll
                for (int e = 0; e < EL; ++e) acc[i][e] = 0.f;
            }
            // this group's keys of the run: 4 of each 128-key tile
            const int steps = (w.t1 - w.t0) * (kPagedTile / 32);
            for (int st = 0; st < steps; st += kDecKeys) {
                float kx[kDecKeys][EL], vx[kDecKeys][EL];
                bool ok[kDecKeys];
#pragma unroll
                for (int x = 0; x < kDecKeys; ++x) {
                    const int key = range.slot(w.t0 * kPagedTile + (st + x) * 32 + grp);
                    ok[x] = range.seen(key, pv.sinks);
                    const int page = ok[x] ? paged_page(pv, w.b, key >> pv.shift, err) : -1;
                    const size_t at = (((size_t)max(page, 0) * pv.Hkv + w.hk) << pv.shift) + (key & ((1 << pv.shift) - 1));
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        float t[EV], u[EV];
#pragma unroll
                        for (int e = 0; e < EV; ++e) t[e] = u[e] = 0.f;
                        if (page >= 0) {
                            load16(K + at * D + (n * 8 + j8) * EV, t);
                            load16(V + at * D + (n * 8 + j8) * EV, u);
                        }
#pragma unroll
                        for (int e = 0; e < EV; ++e) {
                            kx[x][n * EV + e] = t[e];
                            vx[x][n * EV + e] = u[e];
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    float s[kDecKeys], top = m[i];
#pragma unroll
                    for (int x = 0; x < kDecKeys; ++x) {
                        float d = 0.f;
#pragma unroll
                        for (int e = 0; e < EL; ++e) d = fmaf(qs[i][(e / EV * 8 + j8) * EV + e % EV], kx[x][e], d);
#pragma unroll
                        for (int off = 4; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
                        s[x] = ok[x] ? d : -INFINITY;
                        top = fmaxf(top, s[x]);
                    }
                    // (no score yet, or NaN alone, which no maximum shows: the weights are 0 or NaN)
                    const float ref = top == -INFINITY ? 0.f : top;
                    const float old = exp2f(m[i] - ref);
                    m[i] = top;
                    l[i] *= old;
#pragma unroll
                    for (int e = 0; e < EL; ++e) acc[i][e] *= old;
#pragma unroll
                    for (int x = 0; x < kDecKeys; ++x) {
                        const float pe = exp2f(s[x] - ref);
                        l[i] += pe;
#pragma unroll
                        for (int e = 0; e < EL; ++e) acc[i][e] = fmaf(pe, vx[x][e], acc[i][e]);
                    }
                }
            }
            // the warp's four groups, then the eight warps
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                float M = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 8));
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
                const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - M);
                float L = l[i] * f;
                L += __shfl_xor_sync(0xffffffffu, L, 8);
                L += __shfl_xor_sync(0xffffffffu, L, 16);
                if (lane == 0) {
                    wm[warp][i] = M;
                    wl[warp][i] = L;
                }
#pragma unroll
                for (int e = 0; e < EL; ++e) {
                    float a = acc[i][e] * f;
                    a += __shfl_xor_sync(0xffffffffu, a, 8);
                    a += __shfl_xor_sync(0xffffffffu, a, 16);
                    if (lane < 8) wo[warp][i][(e / EV * 8 + j8) * EV + e % EV] = a;
                }
            }
            __syncthreads();
            for (int e = tid; e < nq * D; e += kDecThreads) {
                const int i = e / D, dd = e % D;
                float M = -INFINITY, L = 0.f, A = 0.f;
                for (int x = 0; x < kDecWarps; ++x) M = fmaxf(M, wm[x][i]);
                for (int x = 0; x < kDecWarps; ++x) {
                    const float f = wm[x][i] == -INFINITY ? 0.f : exp2f(wm[x][i] - M);
                    L += wl[x][i] * f;
                    A += wo[x][i][dd] * f;
                }
                if (!YOCO_DCHECK(w.b < pv.B && w.hk < pv.Hkv, 0x64)) continue;
                if (w.whole()) {
                    O[qrow * D + e] = from_f32<T>(A / L);
                } else {
                    float *pp = part + (((size_t)c * 2 + (seg > 0)) * G + g0 + i) * (D + 2);
                    pp[dd] = A;
                    if (dd == 0) {
                        pp[D] = M;
                        pp[D + 1] = L;
                    }
                }
            }
        }
    }
}

// Joins the partial results of a unit that several blocks share: block x of the grid looks
// at the cut before run x + 1, one query head per grid.y, thread = head dim.
constexpr int kMergeBatch = 16;

template <typename T, int D>
__global__ void __launch_bounds__(D)
paged_merge_kernel(const float *__restrict__ part, const PagedCut *__restrict__ cuts, T *__restrict__ O, int G) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int *note = reinterpret_cast<const int *>(cuts + blockIdx.x + 1);
    const PagedCut cut{paged_ld(note), paged_ld(note + 1), paged_ld(note + 2), paged_ld(note + 3)};
    if (cut.unit < 0) return;
    const int g = blockIdx.y, dd = threadIdx.x;
    float M = -INFINITY, L = 0.f, A = 0.f;
    for (int c0 = cut.c_first; c0 <= cut.c_last; c0 += kMergeBatch) {
        float m[kMergeBatch], l[kMergeBatch], a[kMergeBatch], top = M;
#pragma unroll
        for (int x = 0; x < kMergeBatch; ++x) {
            const int c = min(c0 + x, cut.c_last);
            const float *pp = part + (((size_t)c * 2 + (c == cut.c_first ? cut.slot_first : 0)) * G + g) * (D + 2);
            m[x] = __ldcg(pp + D);
            l[x] = __ldcg(pp + D + 1);
            a[x] = __ldcg(pp + dd);
            top = fmaxf(top, m[x]);
        }
        if (top == -INFINITY) {  // no score yet, or NaN alone, which no maximum shows: the sums are 0 or NaN
#pragma unroll
            for (int x = 0; x < kMergeBatch; ++x) L += l[x];
            continue;
        }
        const float old = exp2f(M - top);
        M = top;
        L *= old;
        A *= old;
#pragma unroll
        for (int x = 0; x < kMergeBatch; ++x) {
            const bool there = c0 + x <= cut.c_last;
            const float f = there ? exp2f(m[x] - top) : 0.f;
            L = fmaf(l[x], f, L);
            A = fmaf(there ? a[x] : 0.f, f, A);  // (a value may be infinite)
        }
    }
    O[((size_t)cut.unit * G + g) * D + dd] = from_f32<T>(A / L);
}

// ----------------------------------------------------------------- prefill
//
// 64 rows (tokens x the G query heads of one kv head) against 64-key steps, 256 threads as
// 16 x 16: thread (ty, tx) holds rows 4 ty .. and keys tx + 16 j of the scores, rows 4 ty ..
// and dims 4 tx + 64 j .. of the output.  Everything the products read is in shared memory
// as fp32: two blocks to an SM at head size 64, one at 128 (113 KB each).  K and V have one buffer each: the next step's K comes in
// while this step's softmax and P V run, its V while the next scores do (asynchronous copies
// for fp32, registers for bf16, which is widened on the way).  Bound by shared-memory reads and
// the fp32 pipe, about half of its peak (4096 fp32 rows, 8 over 4 heads x 64: 475 us, 36 TFLOP/s;
// x 128 998 us, 34; bf16, 16 over 4 heads x 64, 926 us, 37; 8 x 8 values to a thread and half the
// reads: 480 us for the first).  Four chunks of 99 to 470 rows, 31 us: the plan 3, two to four steps
// of 5 us each after 3 us of start, the merge 4.
constexpr int kPreRows = 64, kPreKeys = 64, kPreThreads = 256;
constexpr int kPreMinPiece = 1;       // tiles
constexpr float kPreSplitCost = .002f;
constexpr float kPreEntryCost = 1.f;  // a block's start and end take about as long as a tile

template <int D> __host__ __device__ constexpr size_t pre_smem() {
    return sizeof(float) * ((size_t)kPreRows * D + kPreKeys * (D + 4) + kPreKeys * D + kPreRows * kPreKeys);
}

// One 64-key step of K or V on its way from the pages to shared memory (rows PITCH floats apart)
template <typename T, int D, int PITCH> struct PreStage {
    static constexpr int EV = 16 / (int)sizeof(T), CH = D / EV, N = kPreKeys * CH / kPreThreads;
    uint4 r[sizeof(T) == 2 ? N : 1];
    // `at`: the step's slots, in rows of the pool, -1: not to be read
    __device__ __forceinline__ void issue(const T *src, float *dst, const int64_t *at) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int e = threadIdx.x + n * kPreThreads, row = e / CH, ch = e % CH;
            const int64_t o = at[row];
            if constexpr (sizeof(T) == 2) {
                r[n] = make_uint4(0, 0, 0, 0);
                if (o >= 0) r[n] = paged_ld16(src + o * D + ch * EV);
            } else {
                // 0 bytes are read and 16 zeros written where the slot is not to be read
                const unsigned s = (unsigned)__cvta_generic_to_shared(dst + row * PITCH + ch * EV);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(s), "l"(src + max(o, (int64_t)0) * D + ch * EV),
                             "r"(o >= 0 ? 16 : 0));
            }
        }
        asm volatile("cp.async.commit_group;\n" ::);
    }
    // all but the newest issue() of the two stages has come; the caller synchronises
    __device__ __forceinline__ void land(float *dst) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int e = threadIdx.x + n * kPreThreads, row = e / CH, ch = e % CH;
                const uint32_t w[4] = {r[n].x, r[n].y, r[n].z, r[n].w};
                float4 *p = reinterpret_cast<float4 *>(dst + row * PITCH + ch * EV);
                p[0] = make_float4(__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u),
                                   __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u));
                p[1] = make_float4(__uint_as_float(w[2] << 16), __uint_as_float(w[2] & 0xFFFF0000u),
                                   __uint_as_float(w[3] << 16), __uint_as_float(w[3] & 0xFFFF0000u));
            }
        } else {
            asm volatile("cp.async.wait_group 1;\n" ::: "memory");
        }
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kPreThreads, 2)
paged_prefill_simt_kernel(const T *__restrict__ Q, T *__restrict__ O, const T *__restrict__ K, const T *__restrict__ V,
                          float *__restrict__ part, const PagedPlan *__restrict__ plan,
                          const PagedEntry *__restrict__ entries, int rows, int Hq, const PagedView pv, float c2, int *err) {
    constexpr int EV = 16 / (int)sizeof(T), NJ = D / 64;
    extern __shared__ float4 smem4[];
    float *sq = reinterpret_cast<float *>(smem4);
    float *sk = sq + kPreRows * D, *sv = sk + kPreKeys * (D + 4), *sp = sv + kPreKeys * D;
    __shared__ PagedEntry blk;
    __shared__ int64_t at[2][kPreKeys];
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int G = Hq / pv.Hkv, TS = kPreRows / G;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int hk = blockIdx.x % pv.Hkv, entry = blockIdx.x / pv.Hkv;
    // (both loads at once: the list has room for every entry of the grid)
    const int word = tid < 16 ? paged_ld(reinterpret_cast<const int *>(entries + entry) + tid) : 0;
    if (entry >= paged_ld(&plan->entries)) return;
    if (tid < 16) reinterpret_cast<int *>(&blk)[tid] = word;
    __syncthreads();
    if (blk.nrow == 0) return;
    const int nr = blk.nrow * G;  // rows in use: (token, head) = (r / G, r % G)
    const size_t row_stride = (size_t)Hq * D;
    const int t0 = 2 * blk.i0, t1 = min(2 * blk.i1, (blk.range.places + kPreKeys - 1) / kPreKeys);
    auto look_up = [&](int t) {  // the slots of step t
        if (tid < kPreKeys) {
            const int key = blk.range.slot(t * kPreKeys + tid);
            int64_t o = -1;
            if (t < t1 && blk.range.seen(key, pv.sinks)) {
                const int page = paged_page(pv, blk.b, key >> pv.shift, err);
                if (page >= 0) o = (((int64_t)page * pv.Hkv + hk) << pv.shift) + (key & ((1 << pv.shift) - 1));
            }
            at[t & 1][tid] = o;
        }
    };
    look_up(t0);
    look_up(t0 + 1);
    __syncthreads();
    PreStage<T, D, D + 4> stage_k;
    PreStage<T, D, D> stage_v;
    if (t0 < t1) {
        stage_k.issue(K, sk, at[t0 & 1]);
        stage_v.issue(V, sv, at[t0 & 1]);
    }
    for (int e = tid; e < kPreRows * (D / EV); e += kPreThreads) {
        const int r = e / (D / EV), ch = e % (D / EV);
        float x[EV];
#pragma unroll
        for (int i = 0; i < EV; ++i) x[i] = 0.f;
        if (r < nr) load16(Q + (blk.row0 + r / G) * row_stride + (size_t)(hk * G + r % G) * D + ch * EV, x);
#pragma unroll
        for (int i = 0; i < EV; ++i) sq[r * D + ch * EV + i] = c2 * x[i];
    }
    float m[4], l[4], acc[4][4 * NJ];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 4 * NJ; ++e) acc[i][e] = 0.f;
    }
    for (int t = t0; t < t1; ++t) {
        const int v0 = t * kPreKeys;
        stage_k.land(sk);
        __syncthreads();
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[i][x] = 0.f;
#pragma unroll 8
        for (int dd = 0; dd < D; dd += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(sq + (4 * ty + i) * D + dd);
#pragma unroll
            for (int x = 0; x < 4; ++x) b[x] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * x) * (D + 4) + dd);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    s[i][x] = fmaf(a[i].x, b[x].x, fmaf(a[i].y, b[x].y, fmaf(a[i].z, b[x].z, fmaf(a[i].w, b[x].w, s[i][x]))));
        }
        __syncthreads();  // K read by everyone
        stage_k.issue(K, sk, at[(t + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pos = blk.pos0 + (4 * ty + i) / G;
            float top = m[i];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int key = blk.range.slot(v0 + tx + 16 * x);
                const bool seen = key <= pos && (pv.window <= 0 || key > pos - pv.window || key < pv.sinks);
                if (!seen) s[i][x] = -INFINITY;
                top = fmaxf(top, s[i][x]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float ref = top == -INFINITY ? 0.f : top;
            const float old = exp2f(m[i] - ref);
            m[i] = top;
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float pe = exp2f(s[i][x] - ref);
                sum += pe;
                sp[(4 * ty + i) * kPreKeys + tx + 16 * x] = pe;
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[i] = l[i] * old + sum;
#pragma unroll
            for (int e = 0; e < 4 * NJ; ++e) acc[i][e] *= old;
        }
        stage_v.land(sv);
        __syncthreads();  // V and P there
#pragma unroll 4
        for (int kk = 0; kk < kPreKeys; kk += 4) {
            float pr[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = *reinterpret_cast<const float4 *>(sp + (4 * ty + i) * kPreKeys + kk);
                pr[i][0] = f.x;
                pr[i][1] = f.y;
                pr[i][2] = f.z;
                pr[i][3] = f.w;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int n = 0; n < NJ; ++n) {
                    const float4 vv = *reinterpret_cast<const float4 *>(sv + (kk + x) * D + 64 * n + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[i][4 * n] = fmaf(pr[i][x], vv.x, acc[i][4 * n]);
                        acc[i][4 * n + 1] = fmaf(pr[i][x], vv.y, acc[i][4 * n + 1]);
                        acc[i][4 * n + 2] = fmaf(pr[i][x], vv.z, acc[i][4 * n + 2]);
                        acc[i][4 * n + 3] = fmaf(pr[i][x], vv.w, acc[i][4 * n + 3]);
                    }
                }
        }
        __syncthreads();  // V and P read by everyone
        stage_v.issue(V, sv, at[(t + 1) & 1]);
        look_up(t + 2);
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (blk.pieces > 1) {  // [slot][kv head][D + 2][row]
            float *pp = part + ((size_t)blk.slot * pv.Hkv + hk) * (D + 2) * kPreRows + r;
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) pp[(64 * n + 4 * tx + e) * kPreRows] = acc[i][4 * n + e];
            if (tx == 0) {
                pp[D * kPreRows] = m[i];
                pp[(D + 1) * kPreRows] = l[i];
            }
        } else if (r < nr) {
            const float inv = 1.f / l[i];            // (0 / 0 where every score is -inf: NaN, as softmax has it)
            const bool none = blk.pos0 + r / G < 0;  // sees nothing: zero, though 0 times a value may be NaN
            T *op = O + (blk.row0 + r / G) * row_stride + (size_t)(hk * G + r % G) * D;
            if (!YOCO_DCHECK(blk.row0 + r / G < rows && hk * G + r % G < Hq, 0x65)) continue;
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) op[64 * n + 4 * tx + e] = from_f32<T>(none ? 0.f : acc[i][4 * n + e] * inv);
        }
    }
}

// Joins the pieces of the row blocks that are cut: partials [slot][kv head][set][D + 2][R], a
// part of the work is (row block, kv head, set) and kMergeCols head dims, thread = row.
// kMergePieces pieces' maxima, sums and values come in at a time: a latency for so many pieces,
// not for each.  The grid does not grow with what the call might have cut, so a call that cuts
// nothing does not launch thousands of blocks to find that out.
constexpr int kMergeCols = 8, kMergePieces = 4, kMergeBlocks = 12;

template <typename T, int D, int R>
__global__ void __launch_bounds__(R)
paged_merge_rows_kernel(const float *__restrict__ part, T *__restrict__ O, const PagedPlan *__restrict__ plan,
                        const PagedEntry *__restrict__ cuts, int rows, int Hq, int Hkv, int sets) {
    const int r = threadIdx.x, G = Hq / Hkv, TS = R / G;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    // (the first part's row block and how many there are, in one latency)
    int row0, nrow, pos0, pieces, slot, stride;
    auto look_up = [&](int64_t w) {
        const int *c = reinterpret_cast<const int *>(cuts + w / (D / kMergeCols) / sets / Hkv);
        row0 = paged_ld(c + 1), nrow = paged_ld(c + 2), pos0 = paged_ld(c + 3), pieces = paged_ld(c + 6);
        slot = paged_ld(c + 7), stride = paged_ld(c + 8);
    };
    int64_t w = blockIdx.x;
    look_up(w);
    const int64_t parts = (int64_t)paged_ld(&plan->cut) * Hkv * sets * (D / kMergeCols);
    for (; w < parts; w += gridDim.x) {
        if (w != blockIdx.x) look_up(w);
        const int d0 = (int)(w % (D / kMergeCols)) * kMergeCols, unit = (int)(w / (D / kMergeCols));
        const int set = unit % sets, hk = unit / sets % Hkv;
        const int tok = set * TS + r / G;
        if (nrow == 0 || pieces == 1 || r >= TS * G || tok >= nrow) continue;
        const size_t step = (size_t)stride * Hkv * sets * (D + 2) * R;  // from piece to piece
        const float *pp = part + (((size_t)slot * Hkv + hk) * sets + set) * (D + 2) * R + r;
        float M = -INFINITY, L = 0.f, A[kMergeCols];
#pragma unroll
        for (int e = 0; e < kMergeCols; ++e) A[e] = 0.f;
        for (int s0 = 0; s0 < pieces; s0 += kMergePieces) {
            float m[kMergePieces], l[kMergePieces], x[kMergePieces][kMergeCols], top = M;
#pragma unroll
            for (int k = 0; k < kMergePieces; ++k) {
                const float *q = pp + min(s0 + k, pieces - 1) * step;
                m[k] = __ldcg(q + D * R);
                l[k] = __ldcg(q + (D + 1) * R);
#pragma unroll
                for (int e = 0; e < kMergeCols; ++e) x[k][e] = __ldcg(q + (d0 + e) * R);
            }
#pragma unroll
            for (int k = 0; k < kMergePieces; ++k) {
                if (s0 + k >= pieces) m[k] = -INFINITY, l[k] = 0.f;
                top = fmaxf(top, m[k]);
            }
            const float ref = top == -INFINITY ? 0.f : top, old = exp2f(M - ref);
            M = top;
            L *= old;
#pragma unroll
            for (int e = 0; e < kMergeCols; ++e) A[e] *= old;
#pragma unroll
            for (int k = 0; k < kMergePieces; ++k) {
                const float f = exp2f(m[k] - ref);
                // nothing seen in it, whatever it holds (where something was, it may be that every
                // score is NaN, which no maximum shows: the sum is NaN then)
                if (m[k] == -INFINITY && l[k] == 0.f) continue;
                L = fmaf(l[k], f, L);
#pragma unroll
                for (int e = 0; e < kMergeCols; ++e) A[e] = fmaf(x[k][e], f, A[e]);
            }
        }
        // a row that sees nothing: zero; one whose scores are all -inf: 0 / 0, NaN as softmax has it
        const float inv = pos0 + tok < 0 ? 0.f : 1.f / L;
        T *op = O + (size_t)(row0 + tok) * Hq * D + (size_t)(hk * G + r % G) * D + d0;
        if (!YOCO_DCHECK(row0 + tok < rows, 0x66)) continue;
#pragma unroll
        for (int e = 0; e < kMergeCols; e += 16 / (int)sizeof(T)) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(A[e + 2 * i] * inv, A[e + 2 * i + 1] * inv);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h2);
                } else {
                    w[i] = __float_as_uint(A[e + i] * inv);
                }
            }
            *reinterpret_cast<uint4 *>(op + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

}  // namespace yoco

namespace yoco_host {
using namespace yoco;

// workspace: status word and plan, then the cuts of a decode or the entries and cut row
// blocks of a prefill, then partial results
constexpr size_t kPagedPlanAt = 128;
constexpr size_t kPagedHead = 256;
constexpr size_t kPagedCuts = 16384;  // PagedCut per block of a decode grid
constexpr int kMaxDecodeBlocks = (int)(kPagedCuts / sizeof(PagedCut));

// the tensor-core kernels take what fits their tiles
static bool paged_on_tc(const yoco_paged_kv *c) { return c->dtype == YOCO_BF16 && c->d == 128; }

// blocks that a decode's grid has and a prefill's plan counts on: one per SM of the tensor-core
// kernels, two of the CUDA-core ones.  (Two are resident at head size 64 with up to four heads at a
// time and at 128 with up to two; the decode with more of them, and the prefill at 128, have one:
// the grid is then two rounds, and the plan's rounds are half as many as there are.)
static int paged_slots(const yoco_paged_kv *c) { return (paged_on_tc(c) ? 1 : 2) * device_sm_count(); }
static int paged_decode_blocks(const yoco_paged_kv *c) { return std::min(kMaxDecodeBlocks, paged_slots(c)); }

static size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// the plan of a prefill of `rows` rows, with offsets into the workspace for pointers; its bytes
static size_t prefill_grid(const yoco_paged_kv *c, int Hq, int rows, PagedGrid &g, char *ws) {
    const bool tc = paged_on_tc(c);
    const int G = Hq / c->Hkv;
    g.rows = tc ? 2 * (128 / G) : kPreRows / G;
    g.slots = paged_slots(c);
    g.min_piece = tc ? kPagedMinPiece : kPreMinPiece;
    g.entry_cost = tc ? kPagedEntryCost : kPreEntryCost;
    g.split_cost = tc ? kPagedSplitCost : kPreSplitCost;
    const int64_t blocks = std::max<int64_t>(
        1, c->B == 1 ? ((int64_t)rows + g.rows - 1) / g.rows : (int64_t)rows / g.rows + std::min(c->B, rows));
    // up to three rounds of pieces, however many row blocks there are: one of them may see far more than the rest
    const int64_t tiles = ((int64_t)c->max_pages * c->page_size + kPagedTile - 1) / kPagedTile;
    g.max_split = 0;
    if (tiles > g.min_piece)
        g.max_split = (int)std::min<int64_t>(3 * g.slots, blocks * c->Hkv * ((tiles + g.min_piece - 1) / g.min_piece));
    const int64_t split = g.max_split / c->Hkv;
    g.cap = (int)(blocks + split);
    size_t at = kPagedHead;
    g.plan = ws + kPagedPlanAt;
    g.entries = ws + at;
    at += align256((size_t)g.cap * sizeof(PagedEntry));
    g.cuts = ws + at;
    at += align256((size_t)(split / 2) * sizeof(PagedEntry));
    g.part = (float *)(ws + at);
    return at + (size_t)split * c->Hkv * (tc ? 256 : kPreRows) * (c->d + 2) * sizeof(float);
}

size_t paged_workspace(const yoco_paged_kv *c, int Hq, int rows) {
    PagedGrid g;
    const size_t dec = (size_t)paged_decode_blocks(c) * 2 * (Hq / c->Hkv) * (c->d + 2) * sizeof(float);
    return std::max(kPagedHead + kPagedCuts + dec, prefill_grid(c, Hq, rows, g, nullptr));
}

static void pdl_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, dim3 grid, int threads, size_t smem,
                       cudaStream_t st) {
    cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
}

template <typename T, int D, int NQ>
static cudaError_t decode_simt(const PagedArgs &a, const PagedView &pv, PagedCut *cuts, float *part, int blocks,
                               cudaStream_t st) {
    const size_t smem = ((size_t)pv.B + 1) * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(paged_decode_simt_kernel<T, D, NQ>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (kPagedMaxB + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    pdl_config(cfg, attr, dim3(blocks), kDecThreads, smem, st);
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, paged_decode_simt_kernel<T, D, NQ>, (const T *)a.Q, (T *)a.O, (const T *)a.cache->k,
                              (const T *)a.cache->v, part, cuts, a.Hq, pv, a.scale * kPagedLog2e, a.err);
}

template <typename T, int D>
static cudaError_t decode(const PagedArgs &a, cudaStream_t st) {
    const PagedView pv = paged_view(a);
    const int G = a.Hq / pv.Hkv, blocks = paged_decode_blocks(a.cache);
    PagedCut *cuts = (PagedCut *)((char *)a.ws + kPagedHead);
    float *part = (float *)((char *)a.ws + kPagedHead + kPagedCuts);
    cudaError_t e;
    if constexpr (sizeof(T) == 2 && D == 128)
        e = paged_decode_tc(a, cuts, part, blocks, st);
    else
        e = G <= 1   ? decode_simt<T, D, 1>(a, pv, cuts, part, blocks, st)
            : G <= 2 ? decode_simt<T, D, 2>(a, pv, cuts, part, blocks, st)
            : G <= 4 ? decode_simt<T, D, 4>(a, pv, cuts, part, blocks, st)
                     : decode_simt<T, D, kDecQ>(a, pv, cuts, part, blocks, st);
    if (e != cudaSuccess || blocks < 2) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    pdl_config(cfg, attr, dim3(blocks - 1, G), D, 0, st);
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, D>, (const float *)part, (const PagedCut *)cuts, (T *)a.O, G);
}

template <typename T, int D>
static cudaError_t prefill_simt(const PagedArgs &a, const PagedGrid &g, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(paged_prefill_simt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)pre_smem<D>());
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    const int64_t blocks = (int64_t)g.cap * a.cache->Hkv;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    pdl_config(cfg, attr, dim3((unsigned)blocks), kPreThreads, pre_smem<D>(), st);
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, paged_prefill_simt_kernel<T, D>, (const T *)a.Q, (T *)a.O, (const T *)a.cache->k,
                              (const T *)a.cache->v, g.part, (const PagedPlan *)g.plan, (const PagedEntry *)g.entries,
                              a.rows, a.Hq, paged_view(a), a.scale * kPagedLog2e, a.err);
}

template <typename T, int D>
static cudaError_t prefill(const PagedArgs &a, cudaStream_t st) {
    constexpr bool tc = sizeof(T) == 2 && D == 128;
    constexpr int R = tc ? 128 : kPreRows, sets = tc ? 2 : 1;
    PagedGrid g{};
    (void)prefill_grid(a.cache, a.Hq, a.rows, g, (char *)a.ws);
    cudaError_t e = paged_plan(a, g, st);
    if (e != cudaSuccess) return e;
    if constexpr (tc) e = paged_prefill_tc(a, g, st);
    else e = prefill_simt<T, D>(a, g, st);
    const int64_t cut = g.max_split / a.cache->Hkv / 2;  // what is cut has two pieces or more
    if (e != cudaSuccess || cut == 0) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    pdl_config(cfg, attr, dim3((unsigned)std::min<int64_t>(cut * a.cache->Hkv * sets * (D / kMergeCols), kMergeBlocks * g.slots)), R, 0, st);
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, paged_merge_rows_kernel<T, D, R>, (const float *)g.part, (T *)a.O,
                              (const PagedPlan *)g.plan, (const PagedEntry *)g.cuts, a.rows, a.Hq, a.cache->Hkv, sets);
}

cudaError_t paged_decode(const PagedArgs &a, cudaStream_t st) {
    if (a.cache->dtype == YOCO_BF16) return a.cache->d == 64 ? decode<bf16_t, 64>(a, st) : decode<bf16_t, 128>(a, st);
    return a.cache->d == 64 ? decode<float, 64>(a, st) : decode<float, 128>(a, st);
}

cudaError_t paged_prefill(const PagedArgs &a, cudaStream_t st) {
    if (a.cache->dtype == YOCO_BF16) return a.cache->d == 64 ? prefill<bf16_t, 64>(a, st) : prefill<bf16_t, 128>(a, st);
    return a.cache->d == 64 ? prefill<float, 64>(a, st) : prefill<float, 128>(a, st);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_simt)
