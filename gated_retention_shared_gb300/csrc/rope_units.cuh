// rope_units.cuh -- rotary encoding of a part of each head, in pairs or halves, with scaled
// frequencies (yoco_rope), as the strided pass (rope_scaled.cu) and the paged append
// (paged_append.cu) do it.
//
// A head is cut into units that one lane turns alone: with pairs (2i, 2i+1) one 16-byte chunk of
// the channels, with halves (i, i + r/2) the two chunks whose channels turn together, so no lane
// needs another's values and a row may be turned in place.  Past the r channels a unit is as many
// chunks, which are copied: all lanes have the same to move (with units of one chunk there, half a
// head turned took 46 us in place of 32, 12000 rows of 32 heads).  A lane keeps its unit from head to
// head, so the cosines and sines of a row are formed once.
//
// The angle p theta_i is kept in turns as 64-bit fixed point: theta_i / 2 pi is a fraction F_i of
// 2^64 (formed on the host in fp64), p F_i wraps modulo one turn by itself, and its top 32 bits,
// as a signed number, are the angle in [-pi, pi): exact to p 2^-53 + 2^-32 turns.
#pragma once

#include "common.cuh"
#include "rope.cuh"

namespace yoco {

struct RopeTurns {
    uint64_t f[64];  // theta_i / 2 pi in 2^-64 turns; all 0: no rotary encoding
};

struct RopeScaled {
    RopeTurns turns;
    float magnitude;
    int paired;  // of a head's units, those that turn: the first ones
};

template <typename T, int D, bool HALVES> struct RopeUnit {
    static constexpr int EV = 16 / (int)sizeof(T);     // channels of a chunk
    static constexpr int R = HALVES ? EV : EV / 2;     // pairs of a unit
    static constexpr int N = D / EV / (HALVES ? 2 : 1);  // units of a head, a lane each
    float c[R], s[R];
    int at, far;  // first channel of the chunk, and of the other one (halves; else at)
    bool turns;
    __device__ __forceinline__ void place(const RopeScaled &r, int unit) {
        turns = unit < r.paired;
        at = EV * (HALVES && !turns ? 2 * unit : unit);
        far = !HALVES ? at : at + EV * (turns ? r.paired : 1);
    }
    __device__ __forceinline__ void turn_by(const RopeScaled &r, int unit, int64_t pos) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            c[i] = 1.f;
            s[i] = 0.f;
            if (turns) {
                const uint64_t u = (uint64_t)pos * r.turns.f[min(unit * R + i, 63)];
                sincospif((float)(int32_t)(u >> 32) * 0x1p-31f, &s[i], &c[i]);
                c[i] *= r.magnitude;
                s[i] *= r.magnitude;
            }
        }
    }
    __device__ __forceinline__ void load(const uint8_t *head, uint4 &a, uint4 &b) const {
        a = *reinterpret_cast<const uint4 *>(head + at * sizeof(T));
        if constexpr (HALVES) b = *reinterpret_cast<const uint4 *>(head + far * sizeof(T));
    }
    __device__ __forceinline__ void turn(uint4 &a, uint4 &b) const {
        uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
        if constexpr (HALVES) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if constexpr (sizeof(T) == 2) {
                    float x0 = __uint_as_float(x[w] << 16), x1 = __uint_as_float(x[w] & 0xFFFF0000u);
                    float y0 = __uint_as_float(y[w] << 16), y1 = __uint_as_float(y[w] & 0xFFFF0000u);
                    rope_turn(x0, y0, c[2 * w], s[2 * w]);
                    rope_turn(x1, y1, c[2 * w + 1], s[2 * w + 1]);
                    const __nv_bfloat162 hx = __floats2bfloat162_rn(x0, x1), hy = __floats2bfloat162_rn(y0, y1);
                    x[w] = *reinterpret_cast<const uint32_t *>(&hx);
                    y[w] = *reinterpret_cast<const uint32_t *>(&hy);
                } else {
                    float x0 = __uint_as_float(x[w]), y0 = __uint_as_float(y[w]);
                    rope_turn(x0, y0, c[w], s[w]);
                    x[w] = __float_as_uint(x0);
                    y[w] = __float_as_uint(y0);
                }
            }
            b = make_uint4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if constexpr (sizeof(T) == 2) {
                    float x0 = __uint_as_float(x[i] << 16), x1 = __uint_as_float(x[i] & 0xFFFF0000u);
                    rope_turn(x0, x1, c[i], s[i]);
                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(x0, x1);
                    x[i] = *reinterpret_cast<const uint32_t *>(&h2);
                } else {
                    float x0 = __uint_as_float(x[2 * i]), x1 = __uint_as_float(x[2 * i + 1]);
                    rope_turn(x0, x1, c[i], s[i]);
                    x[2 * i] = __float_as_uint(x0);
                    x[2 * i + 1] = __float_as_uint(x1);
                }
            }
        }
        a = make_uint4(x[0], x[1], x[2], x[3]);
    }
    __device__ __forceinline__ void store(uint8_t *head, const uint4 &a, const uint4 &b) const {
        *reinterpret_cast<uint4 *>(head + at * sizeof(T)) = a;
        if constexpr (HALVES) *reinterpret_cast<uint4 *>(head + far * sizeof(T)) = b;
    }
};

}  // namespace yoco

namespace yoco_host {
// frequencies and units of `rope` (checked before) for heads of d channels of 16 / per16 bytes; a
// thread keeps the last ones
const yoco::RopeScaled &rope_scaled(const yoco_rope &rope, int d, int per16);
}  // namespace yoco_host
