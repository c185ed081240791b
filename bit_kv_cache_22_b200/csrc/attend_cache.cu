// attend_cache.cu -- attention of a chunk of new tokens over the paged low-bit cache, on the tensor
// cores.
//
// Query row i of a slot, at position p, sees tokens 0 .. p of its sequence: o_i = sum_{j <= p}
// p_ij v_j with p_i = softmax_j(q_i . k_j / sqrt(d)), k_j and v_j as the cache holds them: (code - z) s
// for tokens below Tq, the residual rows behind.  One pass with a running maximum and sum per row.
//
// A CTA serves one kv head and up to two tiles of 128 query rows (tokens x the query heads of that
// kv head).  Eight warps turn each tile of 128 tokens' codes into fp16 operands in shared memory,
// once for all rows; S = Q K^T and O += P V run on tcgen05 with both accumulators and P in tensor
// memory, and four warps per query tile take the softmax.  Where one query tile holds all rows
// (decode steps, short chunks) the two halves of the CTA take alternate key tiles of it and meet at
// the end.
//
//   warps 0-3, 4-7   softmax of stream 0, 1: thread = row
//   warps 8-15       operands: warp w the tokens 16w .. 16w+15 of each key tile
//   warp 16          issues the MMAs
//
// Operands in fp16 for caches of either type: (code - z) s is computed in fp32 and rounded once to
// 11 bits (bf16 would leave 8, a rounding as large as the output's own).  What fp16 lacks is range,
// so operands carry powers of two of their own: a query row that of its largest channel, a key
// tile that of a bound on its elements, 2^14 <= largest < 2^15, undone in the logits' scale; value
// tiles the largest such exponent so far in the CTA's pass, undone at the end (the sums in tensor
// memory are rescaled when it grows).  An element far below its tile's largest loses bits under
// 2^-40 of that largest.
#include <algorithm>
#include <cstdint>

#include "chunk_rows.cuh"
#include "kvq_internal.cuh"
#include "tensor_core.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 544;
constexpr int kRows = 128;                 // rows of a query tile, tokens of a key tile
constexpr int kStages = 2;                 // key and value operand tiles, each
constexpr int kUnpackWarps = 8;
constexpr int kExps = 8;                   // key tiles whose exponents are kept (at most kStages + 1 are live)
constexpr float kLazyMax = 8.0f;           // the running maximum is raised when a logit passes it by this
constexpr float kNoMax = -1e30f;           // the maximum of no logits: finite, so differences stay numbers
constexpr int kMaxTokens = 0x7fffffff - 1024;   // of a sequence (the planner refuses more)
constexpr int kMinExp = -112;              // exponents of operand scales: 2^e and 2^-e stay normal

template <int D>
struct CacheSmem {
    static constexpr int kTileBytes = kRows * D * 2;
    static constexpr int q = 0;                                   // two tiles
    static constexpr int k = q + 2 * kTileBytes;
    static constexpr int v = k + kStages * kTileBytes;
    static constexpr int meta = v + kStages * kTileBytes;         // per unpacking warp: s, z of keys and values
    static constexpr int kMetaFloats = 2 * D + 2 * 128;
    static constexpr int row_scale = meta + kUnpackWarps * kMetaFloats * 4;   // [2][128]
    static constexpr int bars = row_scale + 2 * kRows * 4;
    // one CTA an SM: it holds all of the tensor memory
    static constexpr int bytes = (bars + 256 > 120 * 1024 ? bars + 256 : 120 * 1024) + 1024;
};

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// the exponent e with bound 2^-e in [2^14, 2^15), as far as kMinExp allows
__device__ __forceinline__ int operand_exp(uint32_t bound_bits) {
    return max(static_cast<int>(bound_bits >> 23) - 127 - 14, kMinExp);
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// byte e of w as 2^23 + byte
template <int E>
__device__ __forceinline__ float byte_plus_2_23(uint32_t w) {
    return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 + E));
}

// What one unpacking warp needs of a tile's 16 tokens: the code words of its lanes, and the scales
// and zeros it spreads over shared memory.
template <int D, int N>
struct Fetched {
    static constexpr int W = D * N / 64;   // words per lane
    uint32_t kw[W], vw[W];
    float4 ks;                             // keys: channels 4 lane .. 4 lane + 3 (lanes below D / 4)
    uint2 kz;
    float vs[4];                           // values: entries lane + 32 i of [16 tokens][D / Gv]
    int vz[4];
    int kind;                              // 0: no tokens, 1: quantized, 2: residual
};

template <int D, int N, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) attend_cache_kernel(const AttendArgs a) {
    using L = CacheSmem<D>;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (tc::smem_addr(raw) + 1023u) & ~1023u;
    unsigned char *smem = raw + (base - tc::smem_addr(raw));
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    __shared__ int exp_k[kExps], exp_v[kExps];
    __shared__ uint32_t bounds[2][2][kUnpackWarps];   // [tile parity][keys, values][warp]
    const PagedView &c = a.cache;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;

    // the work item: up to 2 * tpt tokens of one slot's chunk from q0 on, split s of n over their keys
    const int h = blockIdx.x % a.Hkv;
    const int4 item = a.t.items[blockIdx.x / a.Hkv];
    const int hg = a.Hq / a.Hkv, tpt = kRows / hg;
    const int slot = item.x, q0 = item.y, split = item.z & 0xffff, n_splits = item.z >> 16;
    int first = 0, count = 0, start = 0;
    bool good = slot >= 0 && slot < a.t.B && q0 >= 0 && split < n_splits && item.w >= 0;
    if (good) {
        first = a.t.offsets[slot];
        count = a.t.offsets[slot + 1] - first;
        start = a.t.starts[slot];
        good = first >= 0 && count > q0 && start >= 0 && start <= kMaxTokens - count && static_cast<int64_t>(first) + count <= a.t.tokens;
        if (n_splits > 1 &&
            item.w + static_cast<int64_t>(n_splits) * (count - q0 <= tpt ? 1 : 2) > a.part_tiles)
            good = false;
    }
    if (!good) {                                   // not this library's table
        if (threadIdx.x == 0) atomicOr(a.status, 8u);
        return;
    }
    // (positions stay below 2^31 - 1024, so a tile's tokens are 32-bit numbers)
    const int len = min(max(c.seq_len[slot], 0), kMaxTokens), tq = len / c.R * c.R;
    const int n_tok = min(2 * tpt, count - q0);
    const bool alternate = n_tok <= tpt;           // one query tile, alternate key tiles
    // key tiles: those the item's last row sees, this split's share [tile0, tile0 + n)
    const int all = (min(start + q0 + n_tok, len) + kRows - 1) / kRows;
    const int share = all / n_splits, extra = all % n_splits;      // the first splits take a tile more
    const int tile0 = share * split + min(split, extra), n = share + (split < extra);
    // stream t takes tiles first_of(t), + stride, ... below end_of(t)
    const int stride = alternate ? 2 : 1;
    int ends[2];
    ends[1] = n;
    if (alternate) {
        ends[0] = n;
    } else {
        ends[0] = max(0, min(n, (min(start + q0 + tpt, len) + kRows - 1) / kRows - tile0));
    }

    const uint32_t bars = base + L::bars;
    auto bar = [&](int i) { return bars + 8u * i; };
    enum { kQFull = 0, kKFull = 1, kVFull = kKFull + kStages, kKEmpty = kVFull + kStages, kVEmpty = kKEmpty + kStages,
           kSFull = kVEmpty + kStages, kPFull = kSFull + 2, kOFull = kPFull + 2, kDrain = kOFull + 2, kBars };
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < kBars; ++i) {
            const bool unpacked = i < kKEmpty;     // kQFull, kKFull, kVFull
            tc::bar_init(bar(i), unpacked ? kUnpackWarps : i == kPFull || i == kPFull + 1 ? 4 : 1);
        }
        tc::fence_barrier_init();
    }
    if (warp == 16) tc::tmem_alloc(tc::smem_addr(&tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    float *row_scale = reinterpret_cast<float *>(smem + L::row_scale);

    if (warp >= 8 && warp < 16) {
        // ------------------------------ operands ---------------------------
        const int w = warp - 8;
        // queries: a warp turns a row at a time, four (d = 128) or two channels a lane
        for (int r = w; r < (alternate ? kRows : 2 * kRows); r += kUnpackWarps) {
            const int t = r / kRows, rr = r % kRows, tok = q0 + t * tpt + rr / hg;
            constexpr int E = D / 32;
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = 0.0f;
            if (rr < hg * tpt && tok < count) {
                const uint16_t *src = a.q.p + static_cast<int64_t>(first + tok) * a.q.ts +
                                      static_cast<int64_t>(h * hg + rr % hg) * a.q.hs + lane * E;
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 p = widen_pair<BF16>(reinterpret_cast<const uint32_t *>(src)[e / 2]);
                    x[e] = p.x;
                    x[e + 1] = p.y;
                }
            }
            float big = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) big = fmaxf(big, fabsf(x[e]));
            const int ex = operand_exp(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
            const float down = pow2(-ex);
            if (lane == 0) row_scale[r] = pow2(ex) * a.scale;
            const int col = lane * E;              // channel: 128-byte rows of 64 channels, swizzled
            unsigned char *dst = smem + L::q + t * L::kTileBytes + (col / 64) * (kRows * 128) + rr * 128 +
                                 ((((col % 64) / 8) ^ (rr & 7)) << 4) + (col % 8) * 2;
#pragma unroll
            for (int e = 0; e < E; e += 2)
                reinterpret_cast<uint32_t *>(dst)[e / 2] = half2_bits(x[e] * down, x[e + 1] * down);
        }
        tc::fence_async_proxy();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar(kQFull));

        float *meta = reinterpret_cast<float *>(smem + L::meta) + w * L::kMetaFloats;
        float *ks_s = meta, *kz_s = meta + D, *vs_s = meta + 2 * D, *vz_s = vs_s + 128;
        const int gv_shift = __ffs(c.Gv) - 1, g_shift = __ffs(c.G) - 1;      // powers of two
        const int ngv = D >> gv_shift, ngv_shift = __ffs(ngv) - 1;
        constexpr int B = 4 / N, W = D * N / 64, TW = D * N / 2;
        constexpr uint32_t kMask = 0x01010101u * ((1u << N) - 1);
        constexpr float kTop = static_cast<float>((1 << N) - 1);

        const int32_t *pages = c.page_table + static_cast<int64_t>(slot) * c.max_pages;
        // this warp's place in the pages: of the tile to fetch (page index and token in it), whose page
        // number is loaded a tile ahead
        int at_page = ((tile0 * kRows) + 16 * w) / c.P, at_tok = ((tile0 * kRows) + 16 * w) % c.P;
        auto page_at = [&](int j, int pi) -> int {
            return j < n && (tile0 + j) * kRows + 16 * w < tq && pi < c.max_pages ? pages[pi] : -1;
        };
        auto advance = [&] {
            at_tok += kRows;
            while (at_tok >= c.P) {
                at_tok -= c.P;
                ++at_page;
            }
        };
        Fetched<D, N> f;
        auto fetch = [&](int j, int page) {
            const int tok = (tile0 + j) * kRows + 16 * w;
            f.kind = j >= n || tok >= len ? 0 : tok < tq ? 1 : 2;
            if (f.kind != 1) return;
            if (page < 0 || page >= c.num_pages) {
                if (lane == 0) atomicOr(a.status, 2u);
                page = 0;
            }
            const int64_t slice = static_cast<int64_t>(page) * a.Hkv + h;
            const int pt = at_tok;
            const int64_t words = (slice * (c.P >> 4) + (pt >> 4)) * TW + lane * W;
#pragma unroll
            for (int i = 0; i < W; i += W >= 4 ? 4 : 2) {
                if constexpr (W >= 4) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(c.kc + words + i);
                    const uint4 y = *reinterpret_cast<const uint4 *>(c.vc + words + i);
                    f.kw[i] = x.x; f.kw[i + 1] = x.y; f.kw[i + 2] = x.z; f.kw[i + 3] = x.w;
                    f.vw[i] = y.x; f.vw[i + 1] = y.y; f.vw[i + 2] = y.z; f.vw[i + 3] = y.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(c.kc + words);
                    const uint2 y = *reinterpret_cast<const uint2 *>(c.vc + words);
                    f.kw[0] = x.x; f.kw[1] = x.y;
                    f.vw[0] = y.x; f.vw[1] = y.y;
                }
            }
            const int64_t km = (slice * (c.P >> g_shift) + (pt >> g_shift)) * D + 4 * lane;
            if (4 * lane < D) {
                f.ks = *reinterpret_cast<const float4 *>(c.ks + km);
                if (!c.sym) f.kz = *reinterpret_cast<const uint2 *>(c.kz + km);
            }
            const int64_t vm = (slice * c.P + pt) << ngv_shift;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane + 32 * i < 16 * ngv) {
                    f.vs[i] = c.vs[vm + lane + 32 * i];
                    f.vz[i] = c.sym ? 1 << (N - 1) : c.vz[vm + lane + 32 * i];
                }
        };
        const uint16_t *res_k = c.kr + (static_cast<int64_t>(slot) * a.Hkv + h) * c.R * D;
        const uint16_t *res_v = c.vr + (static_cast<int64_t>(slot) * a.Hkv + h) * c.R * D;
        auto z4 = [&](int (&z)[4]) {
            z[0] = static_cast<int16_t>(f.kz.x & 0xffffu); z[1] = static_cast<int>(f.kz.x) >> 16;
            z[2] = static_cast<int16_t>(f.kz.y & 0xffffu); z[3] = static_cast<int>(f.kz.y) >> 16;
            if (c.sym) z[0] = z[1] = z[2] = z[3] = 1 << (N - 1);
        };
        // bounds on the magnitude of this warp's tokens of tile j, left for all unpacking warps
        auto bound = [&](int j) {
            float bk = 0.0f, bv = 0.0f;
            if (f.kind == 1) {
                if (4 * lane < D) {
                    int z[4];
                    z4(z);
                    const float s[4] = {f.ks.x, f.ks.y, f.ks.z, f.ks.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float zf = static_cast<float>(z[e]);
                        bk = fmaxf(bk, s[e] * fmaxf(fabsf(zf), fabsf(kTop - zf)));
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (lane + 32 * i < 16 * ngv) {
                        const float zf = static_cast<float>(f.vz[i]);
                        bv = fmaxf(bv, f.vs[i] * fmaxf(fabsf(zf), fabsf(kTop - zf)));
                    }
            } else if (f.kind == 2) {
                const int tok = (tile0 + j) * kRows + 16 * w;
                for (int i = lane; i < 16 * D / 2; i += 32) {
                    const int tk = tok + i / (D / 2);
                    if (tk < len) {
                        const int64_t at = static_cast<int64_t>(tk - tq) * (D / 2) + i % (D / 2);
                        const float2 x = widen_pair<BF16>(reinterpret_cast<const uint32_t *>(res_k)[at]);
                        const float2 y = widen_pair<BF16>(reinterpret_cast<const uint32_t *>(res_v)[at]);
                        bk = fmaxf(bk, fmaxf(fabsf(x.x), fabsf(x.y)));
                        bv = fmaxf(bv, fmaxf(fabsf(y.x), fabsf(y.y)));
                    }
                }
            }
            const uint32_t mk = __reduce_max_sync(0xffffffffu, __float_as_uint(bk));
            const uint32_t mv = __reduce_max_sync(0xffffffffu, __float_as_uint(bv));
            if (lane == 0) {
                bounds[j & 1][0][w] = mk;
                bounds[j & 1][1][w] = mv;
            }
        };
        int ev = kMinExp;
        bool go = true;
        // lane's place in an operand tile: row l / 4 (+ 8), 8 bytes l % 4 of a 32-byte step, swizzled
        const uint32_t place = (lane >> 2) * 128 + ((((lane & 3) >> 1) ^ (lane >> 2)) << 4) + (lane & 1) * 8;

        fetch(0, page_at(0, at_page));
        advance();
        int page = page_at(1, at_page);
        bound(0);
        for (int j = 0; j < n; ++j) {
            asm volatile("bar.sync 1, %0;" ::"r"(32 * kUnpackWarps) : "memory");
            uint32_t mk = 0, mv = 0;
#pragma unroll
            for (int i = 0; i < kUnpackWarps; ++i) {
                mk = max(mk, bounds[j & 1][0][i]);
                mv = max(mv, bounds[j & 1][1][i]);
            }
            const int ek = operand_exp(mk);
            ev = max(ev, operand_exp(mv));
            const float down_k = pow2(-ek), down_v = pow2(-ev);
            if (w == 0 && lane == 0) {
                exp_k[j % kExps] = ek;
                exp_v[j % kExps] = ev;
            }
            const int kind = f.kind;
            uint32_t kw[W], vw[W];
            if (kind == 1) {
                __syncwarp();                      // the tile before is unpacked
                if (4 * lane < D) {
                    int z[4];
                    z4(z);
                    reinterpret_cast<float4 *>(ks_s)[lane] =
                        make_float4(f.ks.x * down_k, f.ks.y * down_k, f.ks.z * down_k, f.ks.w * down_k);
                    reinterpret_cast<float4 *>(kz_s)[lane] =
                        make_float4(-8388608.0f - static_cast<float>(z[0]), -8388608.0f - static_cast<float>(z[1]),
                                    -8388608.0f - static_cast<float>(z[2]), -8388608.0f - static_cast<float>(z[3]));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (lane + 32 * i < 16 * ngv) {
                        const int tk = (lane + 32 * i) >> ngv_shift, g = (lane + 32 * i) & (ngv - 1);
                        vs_s[g * 16 + tk] = f.vs[i] * down_v;
                        vz_s[g * 16 + tk] = -8388608.0f - static_cast<float>(f.vz[i]);
                    }
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    kw[i] = f.kw[i];
                    vw[i] = f.vw[i];
                }
                __syncwarp();
            }
            fetch(j + 1, page);
            advance();
            page = page_at(j + 2, at_page);

            const int s = j % kStages, phase = (j / kStages) & 1;
            const int tok = (tile0 + j) * kRows + 16 * w;
            // four codes at a time: bytes to fp32, minus z, times s, rounded to fp16
            auto four = [&](uint32_t b, const float4 &sc, const float4 &zr, uint32_t dst) {
                const float2 x = tc::mul2(tc::add2(make_float2(byte_plus_2_23<0>(b), byte_plus_2_23<1>(b)),
                                                   make_float2(zr.x, zr.y)), make_float2(sc.x, sc.y));
                const float2 y = tc::mul2(tc::add2(make_float2(byte_plus_2_23<2>(b), byte_plus_2_23<3>(b)),
                                                   make_float2(zr.z, zr.w)), make_float2(sc.z, sc.w));
                tc::store_shared(dst, half2_bits(x.x, x.y), half2_bits(y.x, y.y));
            };
            // ---- keys: rows = tokens, channels along a row
            // (a warp whose wait gave up keeps step with the others, which meet at the barrier above)
            if (j >= kStages) go = go && tc::bar_wait_warp(bar(kKEmpty + s), phase ^ 1, &gave_up);
            const uint32_t kt = base + L::k + s * L::kTileBytes + 16 * w * 128;
            if (!go) {
            } else if (kind == 1) {
                const float4 *s4 = reinterpret_cast<const float4 *>(ks_s) + (lane & 3);
                const float4 *r4 = reinterpret_cast<const float4 *>(kz_s) + (lane & 3);
                float4 sc = s4[0], zr = r4[0];
#pragma unroll
                for (int ch = 0; ch < D / 16; ++ch) {      // the next chunk's scales before this one's stores
                    float4 sc1 = sc, zr1 = zr;
                    if (ch + 1 < D / 16) {
                        sc1 = s4[4 * (ch + 1)];
                        zr1 = r4[4 * (ch + 1)];
                    }
                    const uint32_t dst = kt + (ch / 4) * (kRows * 128) + (place ^ ((ch % 4) << 5));
                    four((kw[ch / B] >> (N * 2 * (ch % B))) & kMask, sc, zr, dst);
                    four((kw[ch / B] >> (N * 2 * (ch % B) + N)) & kMask, sc, zr, dst + 1024);
                    sc = sc1;
                    zr = zr1;
                }
            } else {
                for (int i = lane; i < 16 * (D / 8); i += 32) {
                    const int r = i / (D / 8), v = i % (D / 8);
                    uint32_t o[4] = {0u, 0u, 0u, 0u};
                    if (kind == 2 && tok + r < len) {
                        const uint4 x = reinterpret_cast<const uint4 *>(res_k + static_cast<int64_t>(tok + r - tq) * D)[v];
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 p = widen_pair<BF16>(xw[e]);
                            o[e] = half2_bits(p.x * down_k, p.y * down_k);
                        }
                    }
                    tc::store_shared(kt + (v / 8) * (kRows * 128) + r * 128 + (((v % 8) ^ (r & 7)) << 4), o);
                }
            }
            tc::fence_async_proxy();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(bar(kKFull + s));
            // ---- values: rows = channels, tokens along a row
            if (j >= kStages) go = go && tc::bar_wait_warp(bar(kVEmpty + s), phase ^ 1, &gave_up);
            const uint32_t vt = base + L::v + s * L::kTileBytes + (w / 4) * (D * 128);
            if (!go) {
            } else if (kind == 1) {
                const float4 *s4 = reinterpret_cast<const float4 *>(vs_s) + (lane & 3);
                const float4 *r4 = reinterpret_cast<const float4 *>(vz_s) + (lane & 3);
                float4 sc = s4[0], zr = r4[0];
#pragma unroll
                for (int ch = 0; ch < D / 16; ++ch) {
                    float4 sc1 = sc, zr1 = zr;
                    if (ch + 1 < D / 16) {
                        const int g = (16 * (ch + 1)) >> gv_shift;
                        sc1 = s4[4 * g];
                        zr1 = r4[4 * g];
                    }
                    const uint32_t dst = vt + 16 * ch * 128 + (place ^ ((w % 4) << 5));
                    four((vw[ch / B] >> (N * 2 * (ch % B))) & kMask, sc, zr, dst);
                    four((vw[ch / B] >> (N * 2 * (ch % B) + N)) & kMask, sc, zr, dst + 1024);
                    sc = sc1;
                    zr = zr1;
                }
            } else {
                for (int cp = lane; cp < D / 2; cp += 32) {           // channels 2 cp, 2 cp + 1: 16 tokens each
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t o[2][4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float2 p[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int tk = tok + 8 * i + 2 * k + e;
                                p[e] = make_float2(0.0f, 0.0f);
                                if (kind == 2 && tk < len)
                                    p[e] = widen_pair<BF16>(reinterpret_cast<const uint32_t *>(
                                        res_v + static_cast<int64_t>(tk - tq) * D)[cp]);
                            }
                            o[0][k] = half2_bits(p[0].x * down_v, p[1].x * down_v);
                            o[1][k] = half2_bits(p[0].y * down_v, p[1].y * down_v);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int r = 2 * cp + e;
                            tc::store_shared(vt + r * 128 + (((2 * (w % 4) + i) ^ (r & 7)) << 4), o[e]);
                        }
                    }
                }
            }
            tc::fence_async_proxy();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(bar(kVFull + s));
            bound(j + 1);
        }
    } else if (warp == 16) {
        // ------------------------------ MMAs -------------------------------
        if (lane == 0 && n > 0) {
            constexpr uint32_t kDescS = tc::mma_desc(kRows, kRows, false, false);
            constexpr uint32_t kDescO = tc::mma_desc(kRows, D, false, false);
            auto issue_s = [&](int t, int s) {
                const uint64_t qd = tc::desc_k_major(base + L::q + (alternate ? 0 : t) * L::kTileBytes);
                const uint64_t kd = tc::desc_k_major(base + L::k + s * L::kTileBytes);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint64_t step = (i / 4) * (kRows * 128 / 16) + (i % 4) * 2;
                    tc::mma_ss(tmem + t * 128, qd + step, kd + step, kDescS, i > 0);
                }
                tc::mma_commit(bar(kSFull + t));
            };
            bool go = tc::bar_wait(bar(kQFull), 0, &gave_up);
            for (int t = 0; t < 2 && go; ++t) {
                const int j = alternate ? t : 0;   // the stream's first tile
                if (j < ends[t]) {
                    go = tc::bar_wait(bar(kKFull + j % kStages), (j / kStages) & 1, &gave_up);
                    if (go) issue_s(t, j % kStages);
                }
                if (go && (alternate ? j < n : t == 1)) tc::mma_commit(bar(kKEmpty + j % kStages));
            }
            for (int j = 0; j < n && go; ++j) {
                const int s = j % kStages, next = j + stride, s1 = next % kStages;
                go = tc::bar_wait(bar(kVFull + s), (j / kStages) & 1, &gave_up);
                for (int t = 0; t < 2 && go; ++t) {
                    if (j >= ends[t] || (alternate && (j & 1) != t)) continue;
                    const int i = alternate ? j / 2 : j;       // how many tiles the stream has had
                    go = tc::bar_wait(bar(kPFull + t), i & 1, &gave_up);
                    if (!go) break;
                    tc::fence_after_sync();
                    const uint64_t vd = tc::desc_k_major(base + L::v + s * L::kTileBytes);
#pragma unroll
                    for (int k = 0; k < kRows / 16; ++k)
                        tc::mma_ts(tmem + 256 + t * 128, tmem + t * 128 + 8 * k,
                                   vd + (k / 4) * (D * 128 / 16) + (k % 4) * 2, kDescO, i > 0 || k > 0);
                    if (next < ends[t]) {
                        go = tc::bar_wait(bar(kKFull + s1), (next / kStages) & 1, &gave_up);
                        if (go) issue_s(t, s1);
                    } else {
                        tc::mma_commit(bar(kOFull + t));
                    }
                }
                if (go) {
                    tc::mma_commit(bar(kVEmpty + s));
                    if (next < n) tc::mma_commit(bar(kKEmpty + s1));
                }
            }
            volatile int never = 0;                // MMAs in flight end before tensor memory is freed
            tc::mma_commit(bar(kDrain));
            tc::bar_wait(bar(kDrain), 0, &never);
        }
    } else if (warp < 8) {
        // ------------------------------ softmax ----------------------------
        const int t = warp >> 2, r = threadIdx.x & 127;
        const int qt = alternate ? 0 : t;          // the query tile
        const int tok = q0 + qt * tpt + r / hg;
        const bool mine = r < hg * tpt && tok < count;
        const bool any = __any_sync(0xffffffffu, mine);      // a warp without rows only keeps step
        // tokens row r sees, from tile0 on
        const int seen0 = min(start + tok + 1, len) - tile0 * kRows;
        const int seen_least = __reduce_min_sync(0xffffffffu, mine ? seen0 : 0x7fffffff);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
        float m = kNoMax, l = 0.0f, row_s = 0.0f;
        int e_ref = kMinExp;
        bool go = n == 0 || tc::bar_wait_warp(bar(kQFull), 0, &gave_up);
        if (go && n > 0) row_s = row_scale[qt * kRows + r];
        int i = 0;                                 // tiles this stream has had
        for (int j = alternate ? t : 0; j < ends[t] && go; j += stride, ++i) {
            go = tc::bar_wait_warp(bar(kSFull + t), i & 1, &gave_up);
            if (!go) break;
            tc::fence_after_sync();
            if (any) {
                const float scale = row_s * pow2(exp_k[j % kExps]);
                const int ev = exp_v[j % kExps];
                const int seen = seen0 - j * kRows;
                const bool masked = seen_least < (j + 1) * kRows;
                auto logits = [&](int cc, uint32_t(&x)[32]) {
                    tc::tmem_load(ts + 32 * cc, x);
                    tc::tmem_arrived(x);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * cc + e >= seen) x[e] = 0xff800000u;
                    }
                };
                float mx = kNoMax;
#pragma unroll 1
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t x[32];
                    logits(cc, x);
                    float m4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) m4[e] = __uint_as_float(x[e]);
#pragma unroll
                    for (int e = 4; e < 32; ++e) m4[e % 4] = fmaxf(m4[e % 4], __uint_as_float(x[e]));
                    mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale);
                }
                if (i == 0) {
                    m = mx;
                    e_ref = ev;
                } else if (ev != e_ref || __any_sync(0xffffffffu, mx > m + kLazyMax)) {
                    // O holds every tile of the stream before j: S_j was committed after its last MMA
                    const float mn = fmaxf(m, mx), alpha = tc::ex2(m - mn);
                    const float alpha_o = alpha * tc::ex2(static_cast<float>(e_ref - ev));
                    m = mn;
                    l *= alpha;
                    e_ref = ev;
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        tc::tmem_load(to + 32 * cc, o);
                        tc::tmem_arrived(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha_o);
                        tc::tmem_store(to + 32 * cc, o);
                    }
                }
                float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t x[32], p[16];
                    logits(cc, x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 y = tc::fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                                  make_float2(scale, scale), make_float2(-m, -m));
                        const float2 wt = make_float2(tc::ex2(y.x), tc::ex2(y.y));
                        l2[e % 2] = tc::add2(l2[e % 2], wt);
                        p[e] = half2_bits(wt.x, wt.y);
                    }
                    tc::tmem_store16(ts + 16 * cc, p);   // over logits that both passes have read
                }
                tc::tmem_stored();
                l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(bar(kPFull + t));
        }
        const bool had = i > 0;                    // O holds something
        if (go && had) go = tc::bar_wait_warp(bar(kOFull + t), 0, &gave_up);
        if (alternate) {
            // stream 1 hands its sums over through the key tiles' shared memory, which the tensor
            // core is done with once stream 0's last MMA is
            float *ml = reinterpret_cast<float *>(smem + L::v), *ox = reinterpret_cast<float *>(smem + L::k);
            if (t == 1) {
                if (go && n > 0) go = tc::bar_wait_warp(bar(kOFull), 0, &gave_up);
                tc::fence_after_sync();
                if (any && go) {
                    ml[r] = m;
                    ml[kRows + r] = l;
                    const float up = pow2(e_ref);
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        if (had) {
                            tc::tmem_load(to + 32 * cc, o);
                            tc::tmem_arrived(o);
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ox[(32 * cc + e) * kRows + r] = had ? __uint_as_float(o[e]) * up : 0.0f;
                    }
                }
            }
            asm volatile("bar.sync 2, 256;" ::: "memory");
            if (t == 0 && any && go) {
                tc::fence_after_sync();
                const float m1 = ml[r], l1 = ml[kRows + r];
                const float mn = fmaxf(m, m1), w0 = tc::ex2(m - mn), w1 = tc::ex2(m1 - mn);
                const float sum = l * w0 + l1 * w1, inv = n_splits > 1 ? 1.0f : sum > 0.0f ? __fdividef(1.0f, sum) : 0.0f;
                const float f0 = w0 * inv * pow2(e_ref), f1 = w1 * inv;
                uint16_t *out = a.o.p + static_cast<int64_t>(first + tok) * a.o.ts +
                                static_cast<int64_t>(h * hg + r % hg) * a.o.hs;
                const int64_t tile = (static_cast<int64_t>(item.w) + split) * a.Hkv + h;
                float *part = a.part_o + (tile * kRows + r) * D;
                if (n_splits > 1 && mine) {
                    a.part_ml[tile * 2 * kRows + r] = mn;
                    a.part_ml[(tile * 2 + 1) * kRows + r] = sum;
                }
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    __syncwarp();
                    if (had) {
                        tc::tmem_load(to + 32 * cc, o);
                        tc::tmem_arrived(o);
                    }
                    if (!mine) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            y[k] = (had ? __uint_as_float(o[e + k]) * f0 : 0.0f) + ox[(32 * cc + e + k) * kRows + r] * f1;
                        if (n_splits > 1) {
                            reinterpret_cast<float4 *>(part + 32 * cc + e)[0] = make_float4(y[0], y[1], y[2], y[3]);
                            reinterpret_cast<float4 *>(part + 32 * cc + e)[1] = make_float4(y[4], y[5], y[6], y[7]);
                        } else {
                            *reinterpret_cast<uint4 *>(out + 32 * cc + e) =
                                make_uint4(narrow2<BF16>(y[0], y[1]), narrow2<BF16>(y[2], y[3]),
                                           narrow2<BF16>(y[4], y[5]), narrow2<BF16>(y[6], y[7]));
                        }
                    }
                }
            }
        } else if (any && go) {
            tc::fence_after_sync();
            const float f0 = (n_splits > 1 ? 1.0f : l > 0.0f ? __fdividef(1.0f, l) : 0.0f) * pow2(e_ref);
            uint16_t *out = a.o.p + static_cast<int64_t>(first + tok) * a.o.ts +
                            static_cast<int64_t>(h * hg + r % hg) * a.o.hs;
            const int64_t tile = (static_cast<int64_t>(item.w) + 2 * split + t) * a.Hkv + h;
            float *part = a.part_o + (tile * kRows + r) * D;
            if (n_splits > 1 && mine) {
                a.part_ml[tile * 2 * kRows + r] = m;
                a.part_ml[(tile * 2 + 1) * kRows + r] = l;
            }
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                __syncwarp();
                if (had) {
                    tc::tmem_load(to + 32 * cc, o);
                    tc::tmem_arrived(o);
                }
                if (!mine) continue;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] = had ? __uint_as_float(o[e + k]) * f0 : 0.0f;
                    if (n_splits > 1) {
                        reinterpret_cast<float4 *>(part + 32 * cc + e)[0] = make_float4(y[0], y[1], y[2], y[3]);
                        reinterpret_cast<float4 *>(part + 32 * cc + e)[1] = make_float4(y[4], y[5], y[6], y[7]);
                    } else {
                        *reinterpret_cast<uint4 *>(out + 32 * cc + e) =
                            make_uint4(narrow2<BF16>(y[0], y[1]), narrow2<BF16>(y[2], y[3]), narrow2<BF16>(y[4], y[5]),
                                       narrow2<BF16>(y[6], y[7]));
                    }
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && gave_up) atomicOr(a.status, 1u);
    if (warp == 16) {
        tc::fence_after_sync();
        tc::tmem_free(tmem, 512);
    }
}

// Joins an item's splits: one warp per (query token, query head) of its rows, o = sum_s 2^(m_s - M)
// o_s / sum_s 2^(m_s - M) l_s, in the splits' order.  merges: [n][4] = (slot, first query token, splits,
// first partial tile).
constexpr int kMergeWarps = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_splits_kernel(const AttendArgs a) {
    const int4 item = a.t.merges[blockIdx.y];
    const int hg = a.Hq / a.Hkv, tpt = kRows / hg;
    const int slot = item.x, q0 = item.y, n_splits = item.z;
    if (slot < 0 || slot >= a.t.B || q0 < 0 || n_splits < 1 || item.w < 0) {
        if (threadIdx.x == 0) atomicOr(a.status, 8u);
        return;
    }
    const int first = a.t.offsets[slot], count = a.t.offsets[slot + 1] - first;
    const int n_tok = min(2 * tpt, count - q0), nt = n_tok <= tpt ? 1 : 2;
    if (first < 0 || n_tok < 1 || static_cast<int64_t>(first) + count > a.t.tokens ||
        static_cast<int64_t>(item.w) + static_cast<int64_t>(n_splits) * nt > a.part_tiles) {
        if (threadIdx.x == 0) atomicOr(a.status, 8u);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int u = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (u >= n_tok * a.Hq) return;
    const int tok = u / a.Hq, hq = u % a.Hq, h = hq / hg;
    const int t = tok / tpt, r = (tok % tpt) * hg + hq % hg;
    auto tile = [&](int s) { return (static_cast<int64_t>(item.w) + s * nt + t) * a.Hkv + h; };
    float M = kNoMax;
    for (int s = lane; s < n_splits; s += 32) M = fmaxf(M, a.part_ml[tile(s) * 2 * kRows + r]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    constexpr int E = D / 32;
    float o[E] = {}, l = 0.0f;
    for (int s = 0; s < n_splits; ++s) {
        const float w = tc::ex2(a.part_ml[tile(s) * 2 * kRows + r] - M);
        l = fmaf(w, a.part_ml[(tile(s) * 2 + 1) * kRows + r], l);
        const float *p = a.part_o + (tile(s) * kRows + r) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 x = *reinterpret_cast<const float2 *>(p + e);
            o[e] = fmaf(w, x.x, o[e]);
            o[e + 1] = fmaf(w, x.y, o[e + 1]);
        }
    }
    const float inv = l > 0.0f ? __fdividef(1.0f, l) : 0.0f;
    uint16_t *out = a.o.p + static_cast<int64_t>(first + q0 + tok) * a.o.ts + static_cast<int64_t>(hq) * a.o.hs + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        reinterpret_cast<uint32_t *>(out)[e / 2] = narrow2<BF16>(o[e] * inv, o[e + 1] * inv);
}

template <int D, int N, bool BF16>
cudaError_t launch_instance(const AttendArgs &a, cudaStream_t s) {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(attend_cache_kernel<D, N, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 CacheSmem<D>::bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = true;
    }
    attend_cache_kernel<D, N, BF16><<<static_cast<unsigned>(a.t.n_items) * a.Hkv, kThreads, CacheSmem<D>::bytes, s>>>(a);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.t.n_merges == 0) return e;
    // the grid covers the largest item's rows; smaller items leave warps idle
    const int hg = a.Hq / a.Hkv, rows = std::min<int64_t>(2 * (kRows / hg), a.most_tokens) * a.Hq;
    const dim3 grid(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps), static_cast<unsigned>(a.t.n_merges));
    merge_splits_kernel<D, BF16><<<grid, 32 * kMergeWarps, 0, s>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_cache(const AttendArgs &a, cudaStream_t s) {
    if (a.t.n_items == 0) return cudaSuccess;
    if (a.d == 64) {
        if (a.cache.bits == 2) return a.bf16 ? launch_instance<64, 2, true>(a, s) : launch_instance<64, 2, false>(a, s);
        return a.bf16 ? launch_instance<64, 4, true>(a, s) : launch_instance<64, 4, false>(a, s);
    }
    if (a.cache.bits == 2) return a.bf16 ? launch_instance<128, 2, true>(a, s) : launch_instance<128, 2, false>(a, s);
    return a.bf16 ? launch_instance<128, 4, true>(a, s) : launch_instance<128, 4, false>(a, s);
}

}  // namespace kvq
