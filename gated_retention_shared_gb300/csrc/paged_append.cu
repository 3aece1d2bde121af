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

namespace yoco {

struct RopeTurns {
    uint64_t f[64];  // theta_i / 2 pi in 2^-64 turns; all 0: no rotary encoding
};

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
constexpr int kUnroll = 5;

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
        turn_q = false;
        int64_t slot = -1;  // byte offset of the slot's kv head 0
        const int64_t head_bytes = ((int64_t)D * sizeof(T)) << pv.shift;
        if (nkv) {
            const int page = paged_page(pv, b, pos >> pv.shift, a.err);
            if (page >= 0)
                slot = (int64_t)page * pv.Hkv * head_bytes + (int64_t)(pos & ((1 << pv.shift) - 1)) * D * sizeof(T);
        }
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
    }
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

template <typename T, int D>
static cudaError_t append_launch(const PagedAppend &p, const PagedView &pv, const RopeTurns &t, cudaStream_t st) {
    constexpr int HS = 32 / (D * (int)sizeof(T) / 16);
    const int heads = (p.k ? 2 * pv.Hkv : 0) + (p.q ? p.Hq : 0);
    // a warp per row, or up to one per group of heads while that leaves the SMs with fewer
    // than 16 warps each
    const int64_t want = (int64_t)device_sm_count() * 16;
    const int parts = (int)std::max<int64_t>(1, std::min<int64_t>((heads + HS - 1) / HS, want / p.rows));
    const int64_t blocks = ((int64_t)p.rows * parts + kAppendWarps - 1) / kAppendWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    count_launches(1);
    paged_append_kernel<T, D><<<(unsigned)blocks, kAppendWarps * 32, 0, st>>>(p, pv, parts, t);
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

cudaError_t paged_append(const PagedArgs &a, const PagedSource &s, cudaStream_t st) {
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
    p.turn = a.cache->rope_base > 0.f;
    const RopeTurns &t = rope_turns(a.cache->rope_base, d);
    const PagedView pv = paged_view(a);
    if (es == 2) return d == 64 ? append_launch<bf16_t, 64>(p, pv, t, st) : append_launch<bf16_t, 128>(p, pv, t, st);
    return d == 64 ? append_launch<float, 64>(p, pv, t, st) : append_launch<float, 128>(p, pv, t, st);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(paged_append)
