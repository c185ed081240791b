// attend_narrow.cu -- attention over the paged low-bit cache for slots with few new tokens (decode
// steps, drafts): one query tile of 128 rows holds all of a slot's rows, so each code is used by one
// tile only and is unpacked where it is used.
//
//   warps 0, 4       softmax of stream 0, 1: alternate key tiles, at most 32 rows (the warps that
//                    reach the tensor memory of rows 0-31)
//   warps 1, 16      the queries' operands (rows 32 to 127 of the tile stay as they lie: a row of the tile
//                    reaches its own row of the logits and the sums, and those are not read)
//   warp 1           then issues the MMAs
//   the others       sixteen that unpack, keys or values, each 32 tokens of every other key tile: two on
//                    the SM quarter of the softmax warps (0, 4, ...), four and five on the others
//
// Bound by instruction issue (busy 63% of the cycles), nearly all of it unpacking (about 1200 instructions a
// warp for 32 tokens x 128 channels), and by a stream's chain: product, 128 logits of a row by one thread,
// product, some 5000 cycles for every other key tile.  One new token for each of 31 slots of 512 to 15872
// tokens (32 query / 8 kv heads, d = 128, 2-bit; 0.23 GB): 259 us, 1.8 us a key tile and CTA; four new
// tokens for each of 32: 267 us.  With eight unpacking
// warps, and registers moved from them to eight softmax warps, of which six had no rows, it took 289
// us, with the sixteen spread evenly over the SM's quarters 269 us, with 64 logits read at a time instead
// of 32 269 us.  (The decode kernel, whose operands are smaller, takes 156 us, so steps of single newest
// tokens go there.)  Three slots of 100 to 400 tokens with up to six new ones: 14 us, a launch and one
// CTA's chain: 1 us for the table and tensor memory, 3.5 us until the first keys are unpacked, 2.7 us a
// tile and stream.
#include <algorithm>
#include <cstdint>

#include "attend_cache.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 640;
constexpr int kTurns = 2;                  // key tiles in hand at a time
constexpr int kUnpackWarps = 2 * kTurns * kUnits;
constexpr int kMostRows = 32;              // of a slot here
constexpr int kQueryWarps = 2;

template <int D>
struct NarrowSmem {
    static constexpr int kTileBytes = kRows * D * 2;
    static constexpr int q = 0;
    static constexpr int k = q + kTileBytes;
    static constexpr int v = k + kStages * kTileBytes;
    static constexpr int meta = v + kStages * kTileBytes;
    static constexpr int row_scale = meta + kUnpackWarps * kMetaBytes;     // [128]
    static constexpr int bars = row_scale + kRows * 4;
    // one CTA an SM: it holds all of the tensor memory
    static constexpr int bytes = (bars + 256 > 120 * 1024 ? bars + 256 : 120 * 1024) + 1024;
};

template <int D, bool BF16, class L>
__device__ __forceinline__ void emit_queries_of(const AttendArgs &a, const CacheItem &work, unsigned char *smem,
                                                uint32_t base, int w, int lane) {
    const int hg = work.hg, rows = hg * min(work.tpt, work.count - work.q0);
    const uint16_t *src = a.q.p + static_cast<int64_t>(work.first + work.q0) * a.q.ts +
                          static_cast<int64_t>(work.h) * hg * a.q.hs;
    emit_queries<D, BF16>(
        kMostRows, w, kQueryWarps, lane,
        [&](int r) -> const uint16_t * {
            return r < rows ? src + static_cast<int64_t>(r / hg) * a.q.ts + static_cast<int64_t>(r % hg) * a.q.hs : nullptr;
        },
        SharedPut{base + L::q}, [&](int r, float scale) { reinterpret_cast<float *>(smem + L::row_scale)[r] = scale; });
    tc::fence_async_proxy();
    __syncwarp();
    if (lane == 0) tc::bar_arrive(base + L::bars + 8u * kQFull);
}

// Warp of those that unpack keys (kv 0) or values (1): unit u of key tiles `turn`, turn + kTurns, ...,
// fetched a tile ahead, its page number two.  Each tile is a chain -- parameters, shared memory, codes,
// stores -- that a warp cannot hide from itself.
template <int D, int N, bool BF16, class L>
__device__ __forceinline__ void unpack_role(const AttendArgs &a, const CacheItem &work, TileExps *exps,
                                            unsigned char *smem, uint32_t base, int kv, int turn, int u, int lane,
                                            volatile int &gave_up) {
    const PagedView &c = a.cache;
    unsigned char *meta = smem + L::meta + (kUnits * (kTurns * kv + turn) + u) * kMetaBytes;
    const int n = work.n;
    constexpr int W = D * N / 64;
    const UnitSource<D> src(c, kv, work.slot, work.h, work.len, work.tq);
    const int32_t *pages = c.page_table + static_cast<int64_t>(work.slot) * c.max_pages;
    int tok = (work.tile0 + turn) * kRows + 32 * u;         // of the tile in hand
    int at_page = tok / c.P, at_tok = tok % c.P;   // of the tile to fetch
    auto page_at = [&](int t) { return t < src.tq && at_page < c.max_pages ? pages[at_page] : -1; };
    auto advance = [&] {
        at_tok += kTurns * kRows;
        while (at_tok >= c.P) {
            at_tok -= c.P;
            ++at_page;
        }
    };
    Fetched<D, N> f;
    fetch_unit<D, N>(f, c, src, page_at(tok), at_tok, tok, turn < n, lane);
    advance();
    int page = page_at(tok + kTurns * kRows);
    for (int j = turn; j < n; j += kTurns, tok += kTurns * kRows) {
        if (kCheck && !kv && blockIdx.x == 0 && j + 1 == a.stall_tile) break;
        const int s = j % kStages, kind0 = f.kind[0], kind1 = f.kind[1];
        int ex;
        const bool narrow = prepare_unit<D, N, BF16>(f, c, src, tok, lane, meta, ex);
        uint32_t words[2][W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            words[0][i] = f.w[0][i];
            words[1][i] = f.w[1][i];
        }
        fetch_unit<D, N>(f, c, src, page, at_tok, tok + kTurns * kRows, j + kTurns < n, lane);
        advance();
        page = page_at(tok + 2 * kTurns * kRows);
        if (j >= kStages &&
            !tc::bar_wait_warp(base + L::bars + 8u * ((kv ? kVEmpty : kKEmpty) + s), ((j / kStages) & 1) ^ 1, &gave_up))
            break;
        if (lane == 0) {
            if (kv) exps[j % kExps].exp_v[u] = static_cast<float>(ex);
            else exps[j % kExps].scale_k[u] = pow2(ex);
        }
        emit_unit<D, N, BF16>(words, kind0, kind1, narrow, c, src, tok, pow2(-ex), u, lane, meta,
                              SharedPut{base + (kv ? L::v : L::k) + s * L::kTileBytes});
        tc::fence_async_proxy();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(base + L::bars + 8u * ((kv ? kVFull : kKFull) + s));
    }
}

template <int D, int N, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) attend_narrow_kernel(const AttendArgs a) {
    using L = NarrowSmem<D>;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (tc::smem_addr(raw) + 1023u) & ~1023u;
    unsigned char *smem = raw + (base - tc::smem_addr(raw));
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    __shared__ CacheItem work;                     // in shared memory: each role keeps what it needs of it
    __shared__ TileExps exps[kExps];
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) work = cache_item<false>(a, a.t.items[a.t.n_wide + blockIdx.x / a.Hkv], blockIdx.x % a.Hkv);
    if (threadIdx.x == 64) {
        gave_up = 0;
        init_bars(base + L::bars, kQueryWarps, kUnits, 1);
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_addr(&tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;

    if (!work.good || work.count > kMostRows / work.hg) { // not this library's table
        if (threadIdx.x == 0) atomicOr(a.status, 8u);
    } else if (warp == 0 || warp == 4) {
        softmax_role<D, BF16, false, L>(a, work, exps, smem, base, tmem, warp, lane, gave_up);
    } else if (warp == 1) {
        emit_queries_of<D, BF16, L>(a, work, smem, base, 0, lane);
        if (work.n > 0) mma_role<D, false, L>(work, base, tmem, gave_up);
    } else if (warp == 16) {
        emit_queries_of<D, BF16, L>(a, work, smem, base, 1, lane);
    } else {
        const int i = warp - 2 - (warp > 4) - (warp > 16);     // 0 .. 15
        unpack_role<D, N, BF16, L>(a, work, exps, smem, base, i / (kTurns * kUnits), i / kUnits % kTurns, i % kUnits, lane,
                                   gave_up);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && gave_up) atomicOr(a.status, 1u);
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_free(tmem, 512);
    }
}

// Joins an item's splits: one warp per (query token, query head) of its rows, o = sum_s w_s o_s /
// sum_s w_s with w_s = 2^(m_s - M) l_s, in the splits' order (o_s: the split's own output; weighed by shares of 1, so that
// no sum passes the range of the values).  merges: [n][4] = (slot, first query token, splits,
// first partial tile).  Bound by memory: 0.14 GB of partial sums (2048 tokens x 32 heads in four splits,
// d = 128) in 48 us.
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
    float l = 0.0f;
    for (int s = lane; s < n_splits; s += 32)
        l = fmaf(tc::ex2(a.part_ml[tile(s) * 2 * kRows + r] - M), a.part_ml[(tile(s) * 2 + 1) * kRows + r], l);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    const float inv = l > 0.0f ? __fdividef(1.0f, l) : 0.0f;
    constexpr int E = D / 32;
    float o[E] = {};
    for (int s0 = 0; s0 < n_splits; s0 += 32) {    // a lane has the share of split s0 + lane
        float share = 0.0f;
        if (s0 + lane < n_splits)
            share = tc::ex2(a.part_ml[tile(s0 + lane) * 2 * kRows + r] - M) *
                    a.part_ml[(tile(s0 + lane) * 2 + 1) * kRows + r] * inv;
        const int n = min(32, n_splits - s0);
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const float w = __shfl_sync(0xffffffffu, share, s);
            const float *p = a.part_o + (tile(s0 + s) * kRows + r) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 x = *reinterpret_cast<const float2 *>(p + e);
                o[e] = fmaf(w, x.x, o[e]);
                o[e + 1] = fmaf(w, x.y, o[e + 1]);
            }
        }
    }
    uint16_t *out = a.o.p + static_cast<int64_t>(first + q0 + tok) * a.o.ts + static_cast<int64_t>(hq) * a.o.hs + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        reinterpret_cast<uint32_t *>(out)[e / 2] = narrow2<BF16>(o[e], o[e + 1]);
}

template <int D, int N, bool BF16>
cudaError_t launch_instance(const AttendArgs &a, cudaStream_t s) {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(attend_narrow_kernel<D, N, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 NarrowSmem<D>::bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = true;
    }
    const unsigned grid = static_cast<unsigned>(a.t.n_items - a.t.n_wide) * a.Hkv;
    attend_narrow_kernel<D, N, BF16><<<grid, kThreads, NarrowSmem<D>::bytes, s>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_narrow(const AttendArgs &a, cudaStream_t s) {
    if (a.t.n_items == a.t.n_wide) return cudaSuccess;
    if (a.d == 64) {
        if (a.cache.bits == 2) return a.bf16 ? launch_instance<64, 2, true>(a, s) : launch_instance<64, 2, false>(a, s);
        return a.bf16 ? launch_instance<64, 4, true>(a, s) : launch_instance<64, 4, false>(a, s);
    }
    if (a.cache.bits == 2) return a.bf16 ? launch_instance<128, 2, true>(a, s) : launch_instance<128, 2, false>(a, s);
    return a.bf16 ? launch_instance<128, 4, true>(a, s) : launch_instance<128, 4, false>(a, s);
}

cudaError_t launch_merge_splits(const AttendArgs &a, cudaStream_t s) {
    if (a.t.n_merges == 0) return cudaSuccess;
    // the grid covers the largest item's rows; smaller items leave warps idle
    const int hg = a.Hq / a.Hkv;
    const int64_t rows = std::min<int64_t>(2 * (kRows / hg), a.most_tokens) * a.Hq;
    const dim3 grid(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps), static_cast<unsigned>(a.t.n_merges));
    if (a.d == 64) {
        if (a.bf16) merge_splits_kernel<64, true><<<grid, 32 * kMergeWarps, 0, s>>>(a);
        else merge_splits_kernel<64, false><<<grid, 32 * kMergeWarps, 0, s>>>(a);
    } else {
        if (a.bf16) merge_splits_kernel<128, true><<<grid, 32 * kMergeWarps, 0, s>>>(a);
        else merge_splits_kernel<128, false><<<grid, 32 * kMergeWarps, 0, s>>>(a);
    }
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace kvq
