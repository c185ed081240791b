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

// x cos - y sin and y cos + x sin, each operation rounded on its own (no contraction): the
// rotated key decides codes, so every evaluation of the formula has to agree on its bits.
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

// The unit rotated by token tok's angles.
template <bool BF16>
__device__ __forceinline__ void rotate_unit(LoadedUnit &unit, int64_t tok, const RopeArgs &r) {
    uint4 &a = unit.a, &b = unit.b;
    const int va = unit.va;
    const bool pair = unit.vb >= 0;
    if (!r.cos || 8 * va >= r.rot) return;
    const int half = r.rot / 2;
    const int64_t at = tok < r.positions ? tok : r.positions - 1;   // the host has refused later ones
    const uint32_t x[4] = {a.x, a.y, a.z, a.w};
    uint32_t ox[4];
    if (pair) {
        const uint32_t y[4] = {b.x, b.y, b.z, b.w};
        uint32_t oy[4];
        const float4 *c4 = reinterpret_cast<const float4 *>(r.cos + at * half + 8 * va);
        const float4 *s4 = reinterpret_cast<const float4 *>(r.sin + at * half + 8 * va);
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            const float4 c = c4[k2], s = s4[k2];
            const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = 2 * k2 + j;
                const float2 p = widen_pair<BF16>(x[k]), q = widen_pair<BF16>(y[k]);
                ox[k] = narrow2<BF16>(turn_x(p.x, q.x, cs[2 * j], sn[2 * j]),
                                      turn_x(p.y, q.y, cs[2 * j + 1], sn[2 * j + 1]));
                oy[k] = narrow2<BF16>(turn_y(p.x, q.x, cs[2 * j], sn[2 * j]),
                                      turn_y(p.y, q.y, cs[2 * j + 1], sn[2 * j + 1]));
            }
        }
        b = make_uint4(oy[0], oy[1], oy[2], oy[3]);
    } else {                                       // neighbouring channels: rot is a multiple of 16
        const float4 c = *reinterpret_cast<const float4 *>(r.cos + at * half + 4 * va);
        const float4 s = *reinterpret_cast<const float4 *>(r.sin + at * half + 4 * va);
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 p = widen_pair<BF16>(x[k]);
            ox[k] = narrow2<BF16>(turn_x(p.x, p.y, cs[k], sn[k]), turn_y(p.x, p.y, cs[k], sn[k]));
        }
    }
    a = make_uint4(ox[0], ox[1], ox[2], ox[3]);
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
