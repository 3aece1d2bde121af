// rope_scaled.cu -- rotary encoding of strided rows at given positions (yoco_rope): pairs or
// halves of a part of each head, frequencies scaled for long contexts.  rope_units.cuh has the
// mathematics and what a lane does.
//
// A warp takes one row, or, where there are few rows, a part of a row's heads, so that a step of a
// few sequences still fills the GPU; it holds its units' cosines and sines in registers and goes
// head by head with a few heads' loads in flight, the first of them before the angles are formed.
// Bound by HBM: each value is read and written once (12000 rows of 32 heads x 128 31.5 us, 6.2 TB/s;
// 64 rows 3.0 us in a graph, a launch).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "kernels.h"
#include "rope_units.cuh"

namespace yoco {

struct RopeRows {
    const uint8_t *x;
    uint8_t *out;
    int64_t x_row, x_head, out_row, out_head;  // strides in bytes
    const int32_t *positions;
    int64_t pos0;
    int rows, H;
};

constexpr int kRopeWarps = 4;

template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kRopeWarps * 32)
rope_scaled_kernel(const RopeRows a, int parts, const __grid_constant__ RopeScaled r) {
    constexpr int U = HALVES ? 3 : 4;  // heads in flight
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    const int row = (int)(item / parts), part = (int)(item % parts);
    if (row >= a.rows) return;
    RopeUnit<T, D, HALVES> u;
    constexpr int step = 32 / u.N;  // heads at a time
    const int unit = lane % u.N;
    u.place(r, unit);
    const uint8_t *x = a.x + row * a.x_row;
    uint8_t *out = a.out + row * a.out_row;
    uint4 v[U], w[U];
    auto load = [&](int h0) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = h0 + k * parts * step;
            if (h < a.H) u.load(x + h * a.x_head, v[k], w[k]);
        }
    };
    int h0 = part * step + lane / u.N;
    load(h0);  // on its way while the angles are formed
    u.turn_by(r, unit, a.positions ? a.positions[row] : a.pos0 + row);
    for (;;) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = h0 + k * parts * step;
            if (h >= a.H) break;
            if (u.turns) u.turn(v[k], w[k]);
            if (!YOCO_DCHECK(h < a.H && row < a.rows && u.far < D, 0x69)) continue;
            u.store(out + h * a.out_head, v[k], w[k]);
        }
        h0 += parts * step * U;
        if (h0 >= a.H) break;
        load(h0);
    }
}

}  // namespace yoco

namespace yoco_host {
using namespace yoco;

const RopeScaled &rope_scaled(const yoco_rope &rope, int d, int per16) {
    static thread_local RopeScaled t{};
    static thread_local yoco_rope of{};
    static thread_local int of_d = 0, of_per = 0;
    if (of_d == d && of_per == per16 && std::memcmp(&of, &rope, sizeof(rope)) == 0) return t;
    const int r = rope.rotary_dim ? rope.rotary_dim : d, n = r / 2;
    double base = rope.base;
    const double factor = rope.factor;
    if (rope.scaling == YOCO_ROPE_NTK) base *= std::pow(factor, (double)r / (r - 2));
    for (int i = 0; i < 64; ++i) t.turns.f[i] = 0;
    for (int i = 0; i < n; ++i) {
        double theta = std::exp2(-2.0 * i / r * std::log2(base));
        if (rope.scaling == YOCO_ROPE_LINEAR) theta /= factor;
        if (rope.scaling == YOCO_ROPE_BY_PARTS) {
            const double turns = rope.original * theta / kRopeTwoPi;
            const double w = std::min(1.0, std::max(0.0, (turns - rope.low) / ((double)rope.high - rope.low)));
            theta *= w + (1.0 - w) / factor;
        }
        t.turns.f[i] = (uint64_t)std::ldexp(theta / kRopeTwoPi, 64);
    }
    t.magnitude = rope.magnitude;
    t.paired = r / per16 / (rope.layout == YOCO_ROPE_HALVES ? 2 : 1);
    of = rope;
    of_d = d;
    of_per = per16;
    return t;
}

template <typename T, int D, bool HALVES>
static cudaError_t rope_launch(const RopeRows &a, const RopeScaled &r, cudaStream_t st) {
    // a warp per row, or up to one per group of heads while that leaves the SMs with fewer than
    // 16 warps each
    constexpr int step = 32 / RopeUnit<T, D, HALVES>::N;
    const int64_t want = (int64_t)device_sm_count() * 16;
    const int parts = (int)std::max<int64_t>(1, std::min<int64_t>((a.H + step - 1) / step, want / a.rows));
    const int64_t blocks = ((int64_t)a.rows * parts + kRopeWarps - 1) / kRopeWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    count_launches(1);
    rope_scaled_kernel<T, D, HALVES><<<(unsigned)blocks, kRopeWarps * 32, 0, st>>>(a, parts, r);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t rope_rows(const RopeRows &a, int d, const yoco_rope &rope, cudaStream_t st) {
    const RopeScaled &r = rope_scaled(rope, d, 16 / (int)sizeof(T));
    if (rope.layout == YOCO_ROPE_HALVES)
        return d == 64 ? rope_launch<T, 64, true>(a, r, st) : rope_launch<T, 128, true>(a, r, st);
    return d == 64 ? rope_launch<T, 64, false>(a, r, st) : rope_launch<T, 128, false>(a, r, st);
}

cudaError_t rope_apply_scaled(const RopeArgs &s, const yoco_rope &rope, cudaStream_t st) {
    const int es = s.dt == YOCO_BF16 ? 2 : 4;
    const RopeRows a{(const uint8_t *)s.x, (uint8_t *)s.out, s.x_row * es, s.x_head * es, s.out_row * es, s.out_head * es,
                     s.positions, s.pos0, s.rows, s.H};
    return s.dt == YOCO_BF16 ? rope_rows<bf16_t>(a, s.d, rope, st) : rope_rows<float>(a, s.d, rope, st);
}

}  // namespace yoco_host

YOCO_DEBUG_TU(rope_scaled)
