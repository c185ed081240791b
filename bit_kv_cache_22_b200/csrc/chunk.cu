// chunk.cu -- several new tokens of each sequence at once: the rows that stay in the residual,
// the rotation of the queries, and reading a chunk's tokens back.  (The blocks a chunk fills are
// quantized by quantize.cu, its attention is in attend_narrow.cu and attend_wide.cu.)
#include <cstdint>

#include "chunk_rows.cuh"
#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kRowThreads = 128;

// The residual rows (keys rotated) of the new tokens behind their slots' last whole blocks, R floor(end /
// R); those before were quantized by the launch before.  SLOTS: CTA (b, i) has the i-th such token of slot b.
// Otherwise one CTA per new token, which also turns its queries unless the launch before did.  A
// slot's first CTA sets the slot's length, which no CTA reads.
// Bound by memory: each row is read and written once, 16 bytes a thread; queries of 32768 tokens and 32
// heads alone, 0.54 GB, in 109 us.  Behind quantized blocks little is left: 3 to 6 us.
template <bool BF16, bool SLOTS>
__global__ void __launch_bounds__(kRowThreads) chunk_rows_kernel(const PagedView c, const ChunkTable t, const Rows k,
                                                                 const Rows v, const RopeArgs rope, const Rows q,
                                                                 const Rows q_out) {
    const int b = SLOTS ? static_cast<int>(blockIdx.y) : slot_of(t.offsets, t.B, blockIdx.x);
    const int64_t first = t.offsets[b], start = t.starts[b], end = start + t.offsets[b + 1] - first;
    if (SLOTS && end == start) return;
    const int64_t kept = max(start, end / c.R * c.R);          // the first that stays in the residual
    const int64_t row = SLOTS ? first + kept - start + blockIdx.x : blockIdx.x, tok = start + row - first;
    if (start < 0 || end < start || first < 0 || first + end - start > t.tokens || row < first ||
        (!SLOTS && tok >= end)) {                 // not this library's table
        if (threadIdx.x == 0) atomicOr(c.status, 8u);
        return;
    }
    if (threadIdx.x == 0 && (SLOTS ? blockIdx.x == 0 : row == first)) c.seq_len[b] = static_cast<int32_t>(end);
    if (SLOTS && tok >= end) return;
    const RowUnits ru = row_units(c.d, rope), plain = {0, c.d / 8};
    const int n_k = tok >= kept ? c.Hkv * ru.n : 0, n_v = n_k ? c.Hkv * plain.n : 0;
    const int n_q = q.p ? c.Hq * ru.n : 0;
    const int64_t res_row = static_cast<int64_t>(b) * c.Hkv * c.R + tok % c.R;
    for (int i0 = threadIdx.x; i0 < n_k + n_v + n_q; i0 += 2 * kRowThreads) {
        LoadedUnit unit[2];
        uint16_t *dst[2];
        bool turn[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {              // two units' loads in flight
            const int i = i0 + x * kRowThreads;
            dst[x] = nullptr;
            if (i >= n_k + n_v + n_q) continue;
            const bool is_k = i < n_k, is_q = i >= n_k + n_v;
            const int j = is_k ? i : is_q ? i - n_k - n_v : i - n_k;
            turn[x] = is_k || is_q;
            const RowUnits &of = turn[x] ? ru : plain;
            const int h = j / of.n, u = j - h * of.n;
            const Rows &in = is_k ? k : is_q ? q : v;
            dst[x] = is_q ? q_out.p + row * q_out.ts + h * q_out.hs
                          : (is_k ? c.kr : c.vr) + (res_row + static_cast<int64_t>(h) * c.R) * c.d;
            unit[x] = load_unit(in.p + row * in.ts + h * in.hs, u, of);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (!dst[x]) continue;
            if (turn[x]) rotate_unit<BF16>(unit[x], tok, rope);
            __stcs(reinterpret_cast<uint4 *>(dst[x]) + unit[x].va, unit[x].a);
            if (unit[x].vb >= 0) __stcs(reinterpret_cast<uint4 *>(dst[x]) + unit[x].vb, unit[x].b);
        }
    }
}

// One warp per (16-token tile of a slot that meets its chunk, kv head, keys or values): the tile's
// tokens as e.  A quantized tile's words are unpacked from the fragment layout (include/kvq.h): each
// lane holds two tokens x four channels per chunk of keys, two channels x four tokens of values; the
// elements go through shared memory so that rows leave in 16-byte vectors.  Bound by instruction issue (74%
// of the cycles) and the latency of a warp's chain (offsets, page, codes, parameters), so keys and values
// are warps of their own: 43 us for four prompts of 8192 tokens (8 kv heads, d = 128, 2-bit; 0.16 GB moved), 50 us with both in one.
// Rows turned about vector by vector instead of padded have no bank conflicts but more address
// arithmetic: 48 us.
constexpr int kReadWarps = 4;

template <int D, int N, bool BF16>
__global__ void __launch_bounds__(32 * kReadWarps) chunk_read_kernel(const PagedView c, const ChunkTable t,
                                                                     const Rows k_out, const Rows v_out) {
    __shared__ __align__(16) uint16_t tile_s[kReadWarps][16][D + 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kReadWarps + warp) / 2;
    const bool is_v = warp & 1;
    if (unit >= static_cast<int64_t>(t.n_tiles) * c.Hkv) return;
    const int64_t ti = unit / c.Hkv;
    const int h = static_cast<int>(unit % c.Hkv);
    const int b = slot_of(t.tiles, t.B, ti);
    const int64_t first = t.offsets[b], start = t.starts[b], end = start + t.offsets[b + 1] - first;
    const int64_t tok0 = (start / 16 + ti - t.tiles[b]) * 16;
    const int len = c.seq_len[b];
    const int64_t tq = len > 0 ? len / c.R * c.R : 0;
    if (start < 0 || end > len) {                  // the slot holds less than the host knew
        if (lane == 0) atomicOr(c.status, 8u);
        return;
    }
    uint16_t(*tile)[D + 8] = tile_s[warp];
    if (tok0 >= tq) {
        const uint16_t *res = is_v ? c.vr : c.kr;
        for (int i = lane; i < 16 * (D / 8); i += 32) {
            const int r = i / (D / 8), v = i % (D / 8);
            const int64_t tok = tok0 + r;
            if (tok >= start && tok < end)
                reinterpret_cast<uint4 *>(tile[r])[v] = reinterpret_cast<const uint4 *>(
                    res + ((static_cast<int64_t>(b) * c.Hkv + h) * c.R + tok % c.R) * D)[v];
        }
    } else {
        const int64_t pi = tok0 / c.P;
        const int page = pi < c.max_pages ? c.page_table[static_cast<int64_t>(b) * c.max_pages + pi] : -1;
        if (page < 0 || page >= c.num_pages) {
            if (lane == 0) atomicOr(c.status, 2u);
            return;
        }
        constexpr int W = D * N / 64, TW = D * N / 2, B = 4 / N;
        const int64_t slice = static_cast<int64_t>(page) * c.Hkv + h, pt = tok0 - pi * c.P;
        const uint32_t *words = (is_v ? c.vc : c.kc) + (slice * (c.P / 16) + pt / 16) * TW + lane * W;
        constexpr uint32_t kMask = 0x01010101u * ((1u << N) - 1);
        constexpr float kHalf = static_cast<float>(1 << (N - 1));
        uint32_t code[W];
#pragma unroll
        for (int i = 0; i < W; i += 2) {
            const uint2 x = reinterpret_cast<const uint2 *>(words)[i / 2];
            code[i] = x.x;
            code[i + 1] = x.y;
        }
        // four codes (the bytes of b), minus z, times s
        auto values = [](uint32_t b, const float (&z)[4], const float (&s)[4], float (&f)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {          // (2^23 + code) - (2^23 + z) is exact
                const float x = __uint_as_float(__byte_perm(b, 0x4b000000u, 0x7540 + e));
                f[e] = __fmul_rn(__fadd_rn(x, z[e]), s[e]);
            }
        };
        float f[4];
        if (!is_v) {
            const float *s_k = c.ks + (slice * (c.P / c.G) + pt / c.G) * D;
            const int16_t *z_k = c.kz + (slice * (c.P / c.G) + pt / c.G) * D;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const float4 s4 = reinterpret_cast<const float4 *>(s_k)[4 * j + (lane & 3)];
                const float sk[4] = {s4.x, s4.y, s4.z, s4.w};
                float zk[4] = {-8388608.0f - kHalf, -8388608.0f - kHalf, -8388608.0f - kHalf, -8388608.0f - kHalf};
                if (!c.sym) {
                    const uint2 z4 = reinterpret_cast<const uint2 *>(z_k)[4 * j + (lane & 3)];
                    zk[0] = -8388608.0f - static_cast<float>(static_cast<int16_t>(z4.x & 0xffffu));
                    zk[1] = -8388608.0f - static_cast<float>(static_cast<int>(z4.x) >> 16);
                    zk[2] = -8388608.0f - static_cast<float>(static_cast<int16_t>(z4.y & 0xffffu));
                    zk[3] = -8388608.0f - static_cast<float>(static_cast<int>(z4.y) >> 16);
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    values((code[j / B] >> (N * (2 * (j % B) + half))) & kMask, zk, sk, f);
                    *reinterpret_cast<uint2 *>(&tile[(lane >> 2) + 8 * half][16 * j + 4 * (lane & 3)]) =
                        make_uint2(narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]));
                }
            }
        } else {
            const int ngv = D / c.Gv;
            const float *s_v = c.vs + (slice * c.P + pt) * ngv;
            const int16_t *z_v = c.vz + (slice * c.P + pt) * ngv;
            float sv[4], zv[4];
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                if (j == 0 || ((16 * j) & (c.Gv - 1)) == 0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int g = (4 * (lane & 3) + e) * ngv + 16 * j / c.Gv;
                        sv[e] = s_v[g];
                        zv[e] = -8388608.0f - (c.sym ? kHalf : static_cast<float>(z_v[g]));
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    values((code[j / B] >> (N * (2 * (j % B) + half))) & kMask, zv, sv, f);
                    const int ch = 16 * j + (lane >> 2) + 8 * half;
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const uint32_t two = narrow2<BF16>(f[e], f[e + 1]);
                        tile[4 * (lane & 3) + e][ch] = static_cast<uint16_t>(two);
                        tile[4 * (lane & 3) + e + 1][ch] = static_cast<uint16_t>(two >> 16);
                    }
                }
            }
        }
    }
    __syncwarp();
    const Rows &out = is_v ? v_out : k_out;
    for (int i = lane; i < 16 * (D / 8); i += 32) {
        const int r = i / (D / 8), v = i % (D / 8);
        const int64_t tok = tok0 + r, row = first + tok - start;
        if (tok < start || tok >= end || row < 0 || row >= t.tokens) continue;
        reinterpret_cast<uint4 *>(out.p + row * out.ts + h * out.hs)[v] = reinterpret_cast<uint4 *>(tile[r])[v];
    }
}

// Packed query rows of slots with one new token each to dense [B][Hq][d] (TO_SLOTS; slots without one
// get zeros), or dense fp32 outputs [B][Hq][d] to packed rows of e.  One CTA a slot.
template <bool TO_SLOTS, bool BF16>
__global__ void __launch_bounds__(kRowThreads) slot_rows_kernel(const ChunkTable t, const Rows rows, uint16_t *q,
                                                                const float *out, int Hq, int d) {
    const int b = blockIdx.x;
    const int64_t row = t.offsets[b];
    const bool has = t.offsets[b + 1] > row && row >= 0 && row < t.tokens;
    const int vec = d / 8;
    for (int i = threadIdx.x; i < Hq * vec; i += kRowThreads) {
        const int h = i / vec, v = i - h * vec;
        const int64_t at = (static_cast<int64_t>(b) * Hq + h) * vec + v;
        uint4 *packed = reinterpret_cast<uint4 *>(rows.p + row * rows.ts + h * rows.hs) + v;
        if constexpr (TO_SLOTS) {
            reinterpret_cast<uint4 *>(q)[at] = has ? *packed : make_uint4(0u, 0u, 0u, 0u);
        } else if (has) {
            const float4 x = reinterpret_cast<const float4 *>(out)[2 * at], y = reinterpret_cast<const float4 *>(out)[2 * at + 1];
            *packed = make_uint4(narrow2<BF16>(x.x, x.y), narrow2<BF16>(x.z, x.w), narrow2<BF16>(y.x, y.y),
                                 narrow2<BF16>(y.z, y.w));
        }
    }
}

template <int D, int N>
void read_launch(const PagedView &c, const ChunkTable &t, const Rows &k, const Rows &v, unsigned grid, cudaStream_t s) {
    if (c.bf16) chunk_read_kernel<D, N, true><<<grid, 32 * kReadWarps, 0, s>>>(c, t, k, v);
    else chunk_read_kernel<D, N, false><<<grid, 32 * kReadWarps, 0, s>>>(c, t, k, v);
}

}  // namespace

cudaError_t launch_chunk_rows(const PagedView &c, const ChunkTable &t, const Rows &k, const Rows &v,
                              const RopeArgs &rope, const Rows &q, const Rows &q_out, cudaStream_t s) {
    if (t.tokens == 0) return cudaSuccess;
    const Rows none{};
    const bool turned = t.n_blocks > 0;            // the quantizer's launch did
    // long chunks leave little behind their blocks: the smaller grid
    if (turned && t.tokens > static_cast<int64_t>(c.R) * t.B) {
        const dim3 grid(static_cast<unsigned>(c.R), static_cast<unsigned>(t.B));
        if (c.bf16) chunk_rows_kernel<true, true><<<grid, kRowThreads, 0, s>>>(c, t, k, v, rope, none, none);
        else chunk_rows_kernel<false, true><<<grid, kRowThreads, 0, s>>>(c, t, k, v, rope, none, none);
    } else {
        const unsigned grid = static_cast<unsigned>(t.tokens);
        if (c.bf16) chunk_rows_kernel<true, false><<<grid, kRowThreads, 0, s>>>(c, t, k, v, rope, turned ? none : q, q_out);
        else chunk_rows_kernel<false, false><<<grid, kRowThreads, 0, s>>>(c, t, k, v, rope, turned ? none : q, q_out);
    }
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_rows_to_slots(const ChunkTable &t, const Rows &q, uint16_t *dense, int Hq, int d, cudaStream_t s) {
    slot_rows_kernel<true, true><<<static_cast<unsigned>(t.B), kRowThreads, 0, s>>>(t, q, dense, nullptr, Hq, d);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_slots_to_rows(const ChunkTable &t, const float *dense, const Rows &o, int Hq, int d, bool bf16,
                                 cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(t.B);
    if (bf16) slot_rows_kernel<false, true><<<grid, kRowThreads, 0, s>>>(t, o, nullptr, dense, Hq, d);
    else slot_rows_kernel<false, false><<<grid, kRowThreads, 0, s>>>(t, o, nullptr, dense, Hq, d);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_chunk_read(const PagedView &c, const ChunkTable &t, const Rows &k, const Rows &v, cudaStream_t s) {
    if (t.n_tiles == 0) return cudaSuccess;
    const int64_t units = 2 * static_cast<int64_t>(t.n_tiles) * c.Hkv;
    const unsigned grid = static_cast<unsigned>((units + kReadWarps - 1) / kReadWarps);
    if (c.d == 64 && c.bits == 2) read_launch<64, 2>(c, t, k, v, grid, s);
    else if (c.d == 64) read_launch<64, 4>(c, t, k, v, grid, s);
    else if (c.bits == 2) read_launch<128, 2>(c, t, k, v, grid, s);
    else read_launch<128, 4>(c, t, k, v, grid, s);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace kvq
