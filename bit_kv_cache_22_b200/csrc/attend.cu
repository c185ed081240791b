// attend.cu -- causal attention of a chunk of new tokens: over packed prompts, or over the paged
// low-bit cache that already holds them.
#include <cstdint>

#include "chunk_rows.cuh"
#include "kvq_internal.cuh"

namespace kvq {
namespace {

// One warp per (query row, query head): an online softmax over the tokens the row sees, 32 at a
// time: lane l takes token 32 i + l's logit (its whole dot product), then the warp's lanes take
// d / 32 channels each of the weighted sum.
constexpr int kRowWarps = 4;

// Element (token tok, channel c) of keys (V false) or values (V true) of head h.
template <int D, bool BF16, bool CACHE, bool V>
__device__ __forceinline__ float held(const AttendArgs &a, int b, int h, int64_t row0, int64_t tok, int64_t tq, int c) {
    if constexpr (!CACHE) {
        const Rows &r = V ? a.v : a.k;
        return widen(r.p[(row0 + tok) * r.ts + h * r.hs + c], BF16);
    } else {
        const PagedView &p = a.cache;
        if (tok >= tq)
            return widen((V ? p.vr : p.kr)[((static_cast<int64_t>(b) * p.Hkv + h) * p.R + tok % p.R) * D + c], BF16);
        const int64_t pi = tok / p.P;
        int page = pi < p.max_pages ? p.page_table[static_cast<int64_t>(b) * p.max_pages + pi] : -1;
        if (page < 0 || page >= p.num_pages) {
            atomicOr(p.status, 2u);
            page = 0;
        }
        const int n = p.bits, B = 4 / n, W = D * n / 64;
        const int64_t slice = static_cast<int64_t>(page) * p.Hkv + h, pt = tok - pi * p.P;
        const int ti = static_cast<int>(pt % 16), ci = c % 16, j = c / 16;
        const int row = V ? ci : ti, col = V ? ti : ci;
        const uint32_t *words = (V ? p.vc : p.kc) + (slice * (p.P / 16) + pt / 16) * (D * n / 2);
        const uint32_t word = words[(4 * (row % 8) + col / 4) * W + j / B];
        const int code = (word >> (8 * (col % 4) + n * (2 * (j % B) + row / 8))) & ((1 << n) - 1);
        const int64_t mi = V ? (slice * p.P + pt) * (D / p.Gv) + c / p.Gv : (slice * (p.P / p.G) + pt / p.G) * D + c;
        const int z = p.sym ? 1 << (n - 1) : (V ? p.vz : p.kz)[mi];
        return static_cast<float>(code - z) * (V ? p.vs : p.ks)[mi];
    }
}

template <int D, bool BF16, bool CACHE>
__global__ void __launch_bounds__(32 * kRowWarps) attend_rows_kernel(const AttendArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp;
    if (unit >= a.t.tokens * a.Hq) return;
    const int64_t row = unit / a.Hq;
    const int hq = static_cast<int>(unit % a.Hq), h = hq / (a.Hq / a.Hkv);
    const int b = slot_of(a.t.offsets, a.t.B, row);
    const int64_t first = a.t.offsets[b], start = CACHE ? a.t.starts[b] : 0;
    int64_t seen = first >= 0 && start >= 0 ? start + row - first + 1 : 0, tq = 0;
    if constexpr (CACHE) {
        const int64_t len = a.cache.seq_len[b] > 0 ? a.cache.seq_len[b] : 0;
        tq = len / a.cache.R * a.cache.R;
        seen = seen < len ? seen : len;
    }
    __shared__ float qs[kRowWarps][D];
    const uint16_t *q = a.q.p + row * a.q.ts + hq * a.q.hs;
    for (int c = lane; c < D; c += 32) qs[warp][c] = widen(q[c], BF16) * a.scale;
    __syncwarp();
    float m = -INFINITY, l = 0.0f, o[D / 32] = {};
    for (int64_t t0 = 0; t0 < seen; t0 += 32) {
        const int64_t tok = t0 + lane;
        float y = -INFINITY;
        if (tok < seen) {
            y = 0.0f;
            for (int c = 0; c < D; ++c) y = fmaf(qs[warp][c], held<D, BF16, CACHE, false>(a, b, h, first, tok, tq, c), y);
        }
        float mx = fmaxf(m, y);
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float p = tok < seen ? exp2f(y - mx) : 0.0f, alpha = exp2f(m - mx);
        m = mx;
        l = l * alpha + p;
        for (int e = 0; e < D / 32; ++e) o[e] *= alpha;
        const int n = static_cast<int>(seen - t0 < 32 ? seen - t0 : 32);
        for (int i = 0; i < n; ++i) {
            const float w = __shfl_sync(0xffffffffu, p, i);
            for (int e = 0; e < D / 32; ++e)
                o[e] = fmaf(w, held<D, BF16, CACHE, true>(a, b, h, first, t0 + i, tq, lane + 32 * e), o[e]);
        }
    }
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    uint16_t *out = a.o.p + row * a.o.ts + hq * a.o.hs;
    for (int e = 0; e < D / 32; ++e)
        out[lane + 32 * e] = static_cast<uint16_t>(narrow2<BF16>(seen > 0 ? o[e] / l : 0.0f, 0.0f));
}

template <int D>
void rows_launch(const AttendArgs &a, unsigned grid, cudaStream_t s) {
    if (a.cache.kc) {
        if (a.bf16) attend_rows_kernel<D, true, true><<<grid, 32 * kRowWarps, 0, s>>>(a);
        else attend_rows_kernel<D, false, true><<<grid, 32 * kRowWarps, 0, s>>>(a);
    } else {
        if (a.bf16) attend_rows_kernel<D, true, false><<<grid, 32 * kRowWarps, 0, s>>>(a);
        else attend_rows_kernel<D, false, false><<<grid, 32 * kRowWarps, 0, s>>>(a);
    }
}

}  // namespace

cudaError_t launch_attend_cache(const AttendArgs &a, cudaStream_t s) {
    if (a.t.tokens == 0) return cudaSuccess;
    const unsigned grid = static_cast<unsigned>((a.t.tokens * a.Hq + kRowWarps - 1) / kRowWarps);
    if (a.d == 64) rows_launch<64>(a, grid, s);
    else rows_launch<128>(a, grid, s);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace kvq
