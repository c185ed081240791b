// chunk_rows.cuh -- rows of new tokens: narrowing to e and the rotation by position.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_internal.cuh"

namespace kvq {

// Two floats rounded to e, the first in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

template <bool BF16>
__device__ __forceinline__ float2 widen_pair(uint32_t v) {
    if constexpr (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// x cos - y sin and y cos + x sin, each operation rounded on its own (no contraction, which the packed
// forms of two products or sums do not rule out): the rotated key decides codes, so every
// evaluation of the formula has to agree on its bits.
__device__ __forceinline__ float turn_x(float x, float y, float c, float s) {
    return __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}
__device__ __forceinline__ float turn_y(float x, float y, float c, float s) {
    return __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// A row as units of one or two 8-channel vectors, each rotated by one thread: with channels
// (i, i + rot/2) a unit is a pair of vectors rot/2 apart, so that a thread writes what it alone
// has read (rows may be rotated in place); elsewhere a unit is one vector.
struct RowUnits {
    int pairs;                   // units 0 .. pairs-1: vectors u and u + pairs
    int n;                       // then vector u + pairs each
};
__device__ __forceinline__ RowUnits row_units(int d, const RopeArgs &r) {
    const int pairs = r.cos && !r.pairs ? r.rot / 16 : 0;
    return {pairs, d / 8 - pairs};
}

__device__ __forceinline__ uint4 read_once(const uint16_t *src, int v) {
    return __ldcs(reinterpret_cast<const uint4 *>(src) + v);
}

// Unit u of the row at src: vectors va, and vb when vb >= 0.
struct LoadedUnit {
    uint4 a, b;
    int va, vb;
};
__device__ __forceinline__ LoadedUnit load_unit(const uint16_t *src, int u, const RowUnits &ru) {
    LoadedUnit x;
    const bool pair = u < ru.pairs;
    x.va = pair ? u : u + ru.pairs;
    x.vb = pair ? u + ru.pairs : -1;
    x.a = read_once(src, x.va);
    if (pair) x.b = read_once(src, x.vb);
    return x;
}

// Token tok's angles for a unit whose first vector is va: of its eight channels, or of its four pairs of
// neighbours.
struct UnitAngles {
    float4 c[2], s[2];
    bool on;
};
__device__ __forceinline__ UnitAngles unit_angles(int va, bool pair, int64_t tok, const RopeArgs &r) {
    UnitAngles x;
    x.on = r.cos && 8 * va < r.rot;
    if (!x.on) return x;
    const int64_t at = (tok < r.positions ? tok : r.positions - 1) * (r.rot / 2);   // the host has refused later ones
    const int first = pair ? 8 * va : 4 * va;
    const float4 *c = reinterpret_cast<const float4 *>(r.cos + at + first);
    const float4 *s = reinterpret_cast<const float4 *>(r.sin + at + first);
    x.c[0] = c[0];
    x.s[0] = s[0];
    if (pair) {
        x.c[1] = c[1];
        x.s[1] = s[1];
    }
    return x;
}

// The unit rotated by these angles.
template <bool BF16>
__device__ __forceinline__ void turn_unit(LoadedUnit &unit, const UnitAngles &g) {
    if (!g.on) return;
    uint32_t x[4] = {unit.a.x, unit.a.y, unit.a.z, unit.a.w};
    if (unit.vb >= 0) {
        uint32_t y[4] = {unit.b.x, unit.b.y, unit.b.z, unit.b.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 c4 = g.c[k / 2], s4 = g.s[k / 2];
            const float2 c = k % 2 ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
            const float2 s = k % 2 ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y);
            const float2 p = widen_pair<BF16>(x[k]), q = widen_pair<BF16>(y[k]);
            x[k] = narrow2<BF16>(turn_x(p.x, q.x, c.x, s.x), turn_x(p.y, q.y, c.y, s.y));
            y[k] = narrow2<BF16>(turn_y(p.x, q.x, c.x, s.x), turn_y(p.y, q.y, c.y, s.y));
        }
        unit.b = make_uint4(y[0], y[1], y[2], y[3]);
    } else {                                       // neighbouring channels: rot is a multiple of 16
        const float cs[4] = {g.c[0].x, g.c[0].y, g.c[0].z, g.c[0].w}, sn[4] = {g.s[0].x, g.s[0].y, g.s[0].z, g.s[0].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 p = widen_pair<BF16>(x[k]);
            x[k] = narrow2<BF16>(turn_x(p.x, p.y, cs[k], sn[k]), turn_y(p.x, p.y, cs[k], sn[k]));
        }
    }
    unit.a = make_uint4(x[0], x[1], x[2], x[3]);
}

// The unit rotated by token tok's angles.
template <bool BF16>
__device__ __forceinline__ void rotate_unit(LoadedUnit &unit, int64_t tok, const RopeArgs &r) {
    turn_unit<BF16>(unit, unit_angles(unit.va, unit.vb >= 0, tok, r));
}

// The slot whose rows offsets[slot] .. offsets[slot + 1] - 1 hold row i (0 <= i < offsets[B]);
// slots without rows are passed over.
__device__ __forceinline__ int slot_of(const int32_t *offsets, int B, int64_t i) {
    int lo = 0, hi = B;                            // offsets[lo] <= i < offsets[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace kvq
