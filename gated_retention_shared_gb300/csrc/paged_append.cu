// paged_append.cu -- new rows into the paged cache: k turned by its position and written,
// with v, to its slot; q (optional) turned by the same angle.
//
// Channel pair (2i, 2i+1) of the row at position p turns by p theta_i, theta_i =
// base^(-2i/d).  The angle is kept in turns as 64-bit fixed point: theta_i / 2 pi is a
// fraction F_i of 2^64 (formed once on the host in fp64), p F_i wraps modulo one turn by
// itself, and its top 32 bits, as a signed number, are the angle in [-pi, pi): exact to
// p 2^-53 turns however far the position, with one integer product and no fp64 on the
// device.
//
// A warp takes one row (or, where there are few rows, a part of a row's heads, so that a
// step of a few sequences still fills the GPU): it finds the row's sequence, 32 bounds at a
// time, and page once, holds the cosines and sines of its 16-byte chunk in registers, and
// copies head by head with kUnroll loads in flight.  Bound by HBM: each value is read and
// written once.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "rope.cuh"
#include "rope_units.cuh"

namespace yoco {

struct PagedAppend {
    const uint8_t *k, *v, *q;
    int64_t k_row, k_head, v_row, v_head, q_row, q_head;  // strides in bytes
    uint8_t *kc, *vc, *q_out;
    const int32_t *cu;
    int rows, Hq;
    bool turn;
    int *err;
};

constexpr int kAppendWarps = 4;
constexpr int kUnroll = 5, kRopeHalvesUnroll = 4;

// Finds the sequences that have `row` and calls put(pos, b, turn_q) for each, all lanes together.
template <typename Put>
__device__ __forceinline__ void append_row(const PagedAppend &a, const PagedView &pv, int row, int lane, Put put) {
    bool turn_q = a.q != nullptr;
    // The sequences that have this row: cu[b] <= row < cu[b + 1] with bounds within [0, rows].  Bounds
    // that do not decrease give it to one at most; where some fall back, two may have it, and the
    // first one turns q.
    int b = row, first = row, n = 1;
    bool bad = false;
    for (int from = 0, left = 1; left > 0; --left, from = b + 1) {
        if (a.cu) {
            int hits = 0, mine = pv.B;
            const unsigned rows = (unsigned)a.rows;  // (as unsigned numbers, those below 0 are past every bound)
#pragma unroll 8
            for (int seq = from + lane; seq < pv.B; seq += 32) {
                const unsigned c0 = (unsigned)a.cu[seq], c1 = (unsigned)a.cu[seq + 1];
                const bool sound = c0 <= c1 && c1 <= rows, has = sound && (unsigned)row - c0 < c1 - c0;
                bad |= !sound;
                mine = min(mine, has ? seq : pv.B);
                hits += has;
            }
            if (from == 0) left = __reduce_add_sync(0xffffffffu, hits);
            if (bad && from == 0) paged_report(a.err, kErrPagedRows);
            if (left == 0) return;  // between or behind the sequences
            b = __reduce_min_sync(0xffffffffu, mine);
            first = a.cu[b];
            n = a.cu[b + 1] - first;
        }
        const int pos = paged_len(pv, b, a.err) - n + (row - first);
        if (pos < 0) continue;
        put(pos, b, turn_q);
        turn_q = false;
    }
}

// byte offset of the slot of position pos of sequence b for kv head 0, or -1
template <typename T, int D>
__device__ __forceinline__ int64_t append_slot(const PagedAppend &a, const PagedView &pv, int pos, int b, int nkv) {
    if (!nkv) return -1;
    const int64_t head_bytes = ((int64_t)D * sizeof(T)) << pv.shift;
    const int page = paged_page(pv, b, pos >> pv.shift, a.err);
    if (page < 0) return -1;
    return (int64_t)page * pv.Hkv * head_bytes + (int64_t)(pos & ((1 << pv.shift) - 1)) * D * sizeof(T);
}

template <typename T, int D>
__global__ void __launch_bounds__(kAppendWarps * 32)
paged_append_kernel(const PagedAppend a, const PagedView pv, int parts, const RopeTurns turns) {
    constexpr int EV = 16 / (int)sizeof(T);  // elements per 16-byte chunk
    constexpr int PC = EV / 2;               // pairs per chunk
    constexpr int CH = D / EV;               // chunks per head
    constexpr int HS = 32 / CH;              // heads a warp covers at a time
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const int row = (int)(item / parts), part = (int)(item % parts);
    if (row >= a.rows) return;
    const int ch = lane % CH;
    append_row(a, pv, row, lane, [&](int pos, int b, bool turn_q) {
        float c[PC], s[PC];
        if (a.turn) {
#pragma unroll
            for (int i = 0; i < PC; ++i) {
                const uint64_t u = (uint64_t)pos * turns.f[ch * PC + i];
                sincospif((float)(int32_t)(u >> 32) * 0x1p-31f, &s[i], &c[i]);
            }
        }
        // heads in the order k, v, q
        const int nkv = a.k ? pv.Hkv : 0, heads = 2 * nkv + (turn_q ? a.Hq : 0);
        const int64_t slot = append_slot<T, D>(a, pv, pos, b, nkv);
        const int64_t head_bytes = ((int64_t)D * sizeof(T)) << pv.shift;
        for (int h0 = part * HS + lane / CH; h0 < heads; h0 += parts * HS * kUnroll) {
            uint4 u[kUnroll];
#pragma unroll
            for (int x = 0; x < kUnroll; ++x) {
                const int h = h0 + x * parts * HS;
                if (h >= heads) break;
                const uint8_t *src = h < nkv       ? a.k + row * a.k_row + h * a.k_head
                                     : h < 2 * nkv ? a.v + row * a.v_row + (h - nkv) * a.v_head
                                                   : a.q + row * a.q_row + (h - 2 * nkv) * a.q_head;
                u[x] = *reinterpret_cast<const uint4 *>(src + ch * 16);
            }
#pragma unroll
            for (int x = 0; x < kUnroll; ++x) {
                const int h = h0 + x * parts * HS;
                if (h >= heads) break;
                const bool is_v = h >= nkv && h < 2 * nkv;
                if (a.turn && !is_v) {
                    uint32_t w[4] = {u[x].x, u[x].y, u[x].z, u[x].w};
#pragma unroll
                    for (int i = 0; i < PC; ++i) {
                        if constexpr (sizeof(T) == 2) {
                            float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xFFFF0000u);
                            rope_turn(x0, x1, c[i], s[i]);
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(x0, x1);
                            w[i] = *reinterpret_cast<const uint32_t *>(&h2);
                        } else {
                            float x0 = __uint_as_float(w[2 * i]), x1 = __uint_as_float(w[2 * i + 1]);
                            rope_turn(x0, x1, c[i], s[i]);
                            w[2 * i] = __float_as_uint(x0);
                            w[2 * i + 1] = __float_as_uint(x1);
                        }
                    }
                    u[x] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                uint8_t *dst;
                if (h < 2 * nkv) {
                    if (slot < 0) continue;
                    if (!YOCO_DCHECK(b < pv.B && slot / head_bytes < (int64_t)pv.num_pages * pv.Hkv, 0x63)) continue;
                    dst = (is_v ? a.vc : a.kc) + slot + (is_v ? h - nkv : h) * head_bytes;
                } else {
                    dst = a.q_out + ((int64_t)row * a.Hq + (h - 2 * nkv)) * (int64_t)(D * sizeof(T));
                }
                *reinterpret_cast<uint4 *>(dst + ch * 16) = u[x];
            }
        }
    });
}

// The same with a rotation as yoco_rope describes it: a lane has a unit of the head (rope_units.cuh).
// The first heads' loads go before the row's place is looked up, which takes three latencies (11924
// rows of 8 sequences, half of each head turned, 55 -> 43 us with that and units of one size, 5.7 TB/s).
template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kAppendWarps * 32)
paged_append_rope_kernel(const PagedAppend a, const PagedView pv, int parts, const __grid_constant__ RopeScaled r) {
    constexpr int U = HALVES ? kRopeHalvesUnroll : kUnroll;  // heads in flight
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const int row = (int)(item / parts), part = (int)(item % parts);
    if (row >= a.rows) return;
    RopeUnit<T, D, HALVES> u;
    constexpr int step = 32 / u.N;  // heads at a time
    const int unit = lane % u.N, h_first = part * step + lane / u.N;
    const int nkv = a.k ? pv.Hkv : 0, all = 2 * nkv + (a.q ? a.Hq : 0);
    u.place(r, unit);
    uint4 v[U], w[U];
    auto load = [&](int h0, int heads) {  // heads h0, h0 + parts step .. in the order k, v, q
#pragma unroll
        for (int x = 0; x < U; ++x) {
            const int h = h0 + x * parts * step;
            if (h >= heads) break;
            u.load(h < nkv       ? a.k + row * a.k_row + h * a.k_head
                   : h < 2 * nkv ? a.v + row * a.v_row + (h - nkv) * a.v_head
                                 : a.q + row * a.q_row + (h - 2 * nkv) * a.q_head,
                   v[x], w[x]);
        }
    };
    load(h_first, all);  // on its way while the row's place is looked up
    bool there = true;
    append_row(a, pv, row, lane, [&](int pos, int b, bool turn_q) {
        const int heads = turn_q ? all : min(all, 2 * nkv);
        u.turn_by(r, unit, pos);
        const int64_t slot = append_slot<T, D>(a, pv, pos, b, nkv);
        const int64_t head_bytes = ((int64_t)D * sizeof(T)) << pv.shift;
        for (int h0 = h_first; h0 < heads; h0 += parts * step * U) {
            if (!there) load(h0, heads);
            there = false;
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int h = h0 + x * parts * step;
                if (h >= heads) break;
                const bool is_v = h >= nkv && h < 2 * nkv;
                if (u.turns && !is_v) u.turn(v[x], w[x]);
                if (h < 2 * nkv) {
                    if (slot < 0) continue;
                    if (!YOCO_DCHECK(b < pv.B && slot / head_bytes < (int64_t)pv.num_pages * pv.Hkv, 0x6A)) continue;
                    u.store((is_v ? a.vc : a.kc) + slot + (is_v ? h - nkv : h) * head_bytes, v[x], w[x]);
                } else {
                    u.store(a.q_out + ((int64_t)row * a.Hq + (h - 2 * nkv)) * (int64_t)(D * sizeof(T)), v[x], w[x]);
                }
            }
        }
        there = false;
    });
}

}  // namespace yoco

namespace yoco_host {
using namespace yoco;

PagedView paged_view(const PagedArgs &a) {
    PagedView v{};
    v.table = a.cache->page_table;
    v.lens = a.cache->seq_lens;
    v.B = a.cache->B;
    v.Hkv = a.cache->Hkv;
    v.max_pages = a.cache->max_pages;
    v.num_pages = a.cache->num_pages;
    v.shift = 0;
    while ((1 << v.shift) < a.cache->page_size) ++v.shift;
    v.window = a.window;
    v.sinks = a.window > 0 ? a.sinks : 0;
    return v;
}

PagedMod paged_mod(const PagedArgs &a) {
    PagedMod m{};
    const float cap = a.scores ? a.scores->softcap : 0.f;
    m.qk = cap > 0.f ? a.scale / cap : a.scale * kPagedLog2E;
    if (!a.scores) return m;
    m.slopes = a.scores->slopes;
    m.prefix = a.scores->prefix;
    m.doc = a.scores->doc_first;
    m.cap2 = cap * kPagedLog2E;
    if (cap > 0.f) {
        const double k = m.qk, c = m.cap2;
        struct Fit {  // of tanh(x) / x in x^2: up to |x| = reach; a product of `far` / k gets weight 0
            int degree;
            double reach, far, a[6];
        };
        static const Fit fits[3] = {
            {2, 0.26, -0x1p20, {0.999999501, -0.333200077, 0.128027106}},  // (the last term is positive: it falls towards -s^5)
            {3, 0.5, 0x1p15, {0.999999456, -0.33326318, 0.131902967, -0.0444022262}},
            {5, 1.0, 0x1p10, {0.999999414, -0.333290425, 0.132814342, -0.0516056791, 0.016743118, -0.00306706059}}};
        // (head size 64 makes do with two of them)
        const Fit &fit = fits[cap < kWideCap ? 2 : cap < kShortCap || a.cache->d == 64 ? 1 : 0];
        m.degree = fit.degree;
        m.quick = (float)std::min(fit.reach / k, kQuickScore / (c * k));
        m.hidden = (float)(fit.far / k);  // (there the polynomial is some -2^100 C)
        for (int i = 0; i <= m.degree; ++i) {
            const double x = c * std::pow(k, 2 * i + 1) * fit.a[i];
            m.a[i] = (float)x;
            // (caps that 32 bits cannot follow that way go the exact way)
            if (!(std::fabs(x) > 1e-36 && std::fabs(x) < 1e36)) m.quick = -1.f;
        }
        if (!(m.quick < 1e18f)) m.quick = -1.f;
    }
    return m;
}

// warps to a row: one, or up to one per group of heads (hs of them) while that leaves the SMs
// with fewer than 16 warps each; blocks: those that makes
static int append_parts(const PagedAppend &p, const PagedView &pv, int hs, int64_t &blocks) {
    const int heads = (p.k ? 2 * pv.Hkv : 0) + (p.q ? p.Hq : 0);
    const int64_t want = (int64_t)device_sm_count() * 16;
    const int parts = (int)std::max<int64_t>(1, std::min<int64_t>((heads + hs - 1) / hs, want / p.rows));
    blocks = ((int64_t)p.rows * parts + kAppendWarps - 1) / kAppendWarps;
    return parts;
}

template <typename T, int D>
static cudaError_t append_launch(const PagedAppend &p, const PagedView &pv, const RopeTurns &t, cudaStream_t st) {
    int64_t blocks;
    const int parts = append_parts(p, pv, 32 / (D * (int)sizeof(T) / 16), blocks);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    count_launches(1);
    paged_append_kernel<T, D><<<(unsigned)blocks, kAppendWarps * 32, 0, st>>>(p, pv, parts, t);
    return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t append_rope_launch(const PagedAppend &p, const PagedView &pv, const yoco_rope &rope, cudaStream_t st) {
    const RopeScaled &r = rope_scaled(rope, D, 16 / (int)sizeof(T));
    const bool halves = rope.layout == YOCO_ROPE_HALVES;
    int64_t blocks;
    const int parts = append_parts(p, pv, 32 / (halves ? RopeUnit<T, D, true>::N : RopeUnit<T, D, false>::N), blocks);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    count_launches(1);
    if (halves) paged_append_rope_kernel<T, D, true><<<(unsigned)blocks, kAppendWarps * 32, 0, st>>>(p, pv, parts, r);
    else paged_append_rope_kernel<T, D, false><<<(unsigned)blocks, kAppendWarps * 32, 0, st>>>(p, pv, parts, r);
    return cudaGetLastError();
}

// The turns of a base and head size; a thread keeps the last ones (64 powers take longer
// than the rest of the call).  base 0: none, nothing is turned.
static const RopeTurns &rope_turns(float base, int d) {
    static thread_local RopeTurns t{};
    static thread_local float t_base = 0.f;
    static thread_local int t_d = 0;
    if (base > 0.f && (base != t_base || d != t_d)) {
        const RopeFreq f = make_rope_freq(base, d);
        for (int i = 0; i < 64; ++i) t.f[i] = (uint64_t)std::ldexp(f.theta[i] / kRopeTwoPi, 64);
        t_base = base;
        t_d = d;
    }
    return t;
}

cudaError_t paged_append(const PagedArgs &a, const PagedSource &s, const yoco_rope *rope, cudaStream_t st) {
    const int es = a.cache->dtype == YOCO_BF16 ? 2 : 4, d = a.cache->d;
    PagedAppend p{};
    p.k = (const uint8_t *)s.k;
    p.v = (const uint8_t *)s.v;
    p.q = (const uint8_t *)a.Q;
    p.k_row = s.k_row * es;
    p.k_head = s.k_head * es;
    p.v_row = s.v_row * es;
    p.v_head = s.v_head * es;
    p.q_row = s.q_row * es;
    p.q_head = s.q_head * es;
    p.kc = (uint8_t *)a.cache->k;
    p.vc = (uint8_t *)a.cache->v;
    p.q_out = (uint8_t *)a.O;
    p.cu = a.cu;
    p.rows = a.rows;
    p.Hq = a.Hq;
    p.err = a.err;
    const PagedView pv = paged_view(a);
    if (rope) {
        if (es == 2)
            return d == 64 ? append_rope_launch<bf16_t, 64>(p, pv, *rope, st) : append_rope_launch<bf16_t, 128>(p, pv, *rope, st);
        return d == 64 ? append_rope_launch<float, 64>(p, pv, *rope, st) : append_rope_launch<float, 128>(p, pv, *rope, st);
    }
    p.turn = a.cache->rope_base > 0.f;
    const RopeTurns &t = rope_turns(a.cache->rope_base, d);
    if (es == 2) return d == 64 ? append_launch<bf16_t, 64>(p, pv, t, st) : append_launch<bf16_t, 128>(p, pv, t, st);
    return d == 64 ? append_launch<float, 64>(p, pv, t, st) : append_launch<float, 128>(p, pv, t, st);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_append)
