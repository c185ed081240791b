// attend_wide.cu -- attention over the paged low-bit cache for slots with many new tokens (chunked
// prefill): several query tiles use each code, so a first kernel unpacks every slot's keys and values
// once, as the operand tiles themselves (swizzled, 64 KB per 128 tokens and kv head at d = 128), and
// the queries, into the workspace; the attention kernel copies whole tiles.
//
//   warps 0-3, 4-7   softmax of query tile 0, 1 (a slot's last CTA may have one: alternate key tiles)
//   warp 8           issues the MMAs
//   warp 9           copies (warps 10, 11 fill the warpgroup, which gives its registers to the
//                    softmax: 2 x 128 x 208 + 128 x 80 <= 384 x 168)
//
// Bound by the tensor cores, at the clock that the power limit leaves: 2048 tokens behind 126976 (32
// query / 8 kv heads, d = 128, 2-bit; 4.29 TFLOP) take 3.74 ms in a burst, 1147 TFLOP/s, with 0.12 ms of
// staging before and 0.05 ms of joining splits behind.  With the codes unpacked in the attention kernel,
// anew for each 256 query rows and beside the softmax, an earlier form took 11.8 ms.  Six chunks of 66 to
// 613 tokens behind 586 to 2557 (32 / 32 heads, 4-bit; 45 GFLOP): 95 us, after 63 us of staging.  There
// pieces of fewer than 256 rows leave tensor core rows idle (1.35 times the operations), and CTAs of 7 to
// 21 key tiles start 2.6 times on each SM, each with its table, its tensor memory and its first tiles.
#include <cstdint>

#include "attend_cache.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 384;
constexpr int kStageThreads = 32 * kUnits;

template <int D>
struct WideSmem {
    static constexpr int kTileBytes = kRows * D * 2;
    static constexpr int q = 0;                                   // two tiles
    static constexpr int k = q + 2 * kTileBytes;
    static constexpr int v = k + kStages * kTileBytes;
    static constexpr int exps = v + kStages * kTileBytes;
    static constexpr int row_scale = exps + kExps * static_cast<int>(sizeof(TileExps));       // [2][128]
    static constexpr int bars = row_scale + 2 * kRows * 4;
    // one CTA an SM: it holds all of the tensor memory
    static constexpr int bytes = (bars + 256 > 120 * 1024 ? bars + 256 : 120 * 1024) + 1024;
};

// The workspace: operand tiles [key tile][kv head][keys, values], [query tile][kv head], then the key
// tiles' powers of two and the query rows' [..][128].
template <int D>
struct Staged {
    static constexpr int64_t kTileBytes = kRows * D * 2;
    unsigned char *kv, *q;
    TileExps *exps;
    float *row_scale;
    __device__ explicit Staged(const AttendArgs &a) {
        kv = a.staged;
        q = kv + a.t.n_kv_tiles * a.Hkv * 2 * kTileBytes;
        exps = reinterpret_cast<TileExps *>(q + a.t.n_q_tiles * a.Hkv * kTileBytes);
        row_scale = reinterpret_cast<float *>(exps + a.t.n_kv_tiles * a.Hkv);
    }
};

// CTA (x, h): keys (x even) or values of key tile x / 2 of the wide slots, or query tile x - 2 n_kv_tiles.
// The tile is put together in shared memory and leaves in one copy.  Bound by the latency of a tile's
// chain -- page, codes and scales, parameters through shared memory -- (issue 50% of the cycles, memory 43%
// of its rate), so tiles are CTAs of four warps, five or more an SM: 0.18 GB of tiles in 63 us (keys and values of 11243 tokens, 32 heads, d = 128,
// 4-bit).  With both in one CTA of eight warps whose lanes store their 8 bytes to global memory, 73
// us; with CTAs of four heads that fetch the next head's codes ahead, but hold 96 registers, 94 us.
template <int D, int N, bool BF16>
__global__ void __launch_bounds__(kStageThreads) stage_kernel(const AttendArgs a) {
    extern __shared__ __align__(128) unsigned char tile_s[];
    constexpr int kTileBytes = kRows * D * 2;
    const Staged<D> st(a);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
    const SharedPut put{tc::smem_addr(tile_s)};
    unsigned char *out;
    if (blockIdx.x < 2u * a.t.n_kv_tiles) {
        const int x = blockIdx.x / 2, kv = blockIdx.x % 2, slot = slot_of(a.t.kv_tiles, a.t.B, x);
        const int tok0 = (x - a.t.kv_tiles[slot]) * kRows;
        if (tok0 < 0) return;
        const int64_t at = static_cast<int64_t>(x) * a.Hkv + h;
        const PagedView &c = a.cache;
        const int len = min(max(c.seq_len[slot], 0), kMaxTokens), tq = len / c.R * c.R;
        const int tok = tok0 + 32 * w, pi = tok / c.P;
        const int page = tok < tq && pi < c.max_pages ? c.page_table[static_cast<int64_t>(slot) * c.max_pages + pi] : -1;
        const UnitSource<D> src(c, kv, slot, h, len, tq);
        Fetched<D, N> f;
        fetch_unit<D, N>(f, c, src, page, tok % c.P, tok, true, lane);
        int ex;
        unsigned char *meta = tile_s + kTileBytes + w * kMetaBytes;
        const bool narrow = prepare_unit<D, N, BF16>(f, c, src, tok, lane, meta, ex);
        if (lane == 0) {
            if (kv) st.exps[at].exp_v[w] = static_cast<float>(ex);
            else st.exps[at].scale_k[w] = pow2(ex);
        }
        emit_unit<D, N, BF16>(f.w, f.kind[0], f.kind[1], narrow, c, src, tok, pow2(-ex), w, lane, meta, put);
        out = st.kv + (at * 2 + kv) * kTileBytes;
    } else {
        const int x = blockIdx.x - 2 * a.t.n_kv_tiles, slot = slot_of(a.t.q_tiles, a.t.B, x);
        const int hg = a.Hq / a.Hkv, tpt = kRows / hg;
        const int first = a.t.offsets[slot], count = a.t.offsets[slot + 1] - first;
        const int q0 = (x - a.t.q_tiles[slot]) * tpt;
        if (first < 0 || q0 < 0 || static_cast<int64_t>(first) + count > a.t.tokens) return;
        const int64_t at = static_cast<int64_t>(x) * a.Hkv + h;
        emit_queries<D, BF16>(
            kRows, w, kUnits, lane,
            [&](int r) -> const uint16_t * {
                const int tok = q0 + r / hg;
                if (r >= hg * tpt || tok >= count) return nullptr;
                return a.q.p + static_cast<int64_t>(first + tok) * a.q.ts + static_cast<int64_t>(h * hg + r % hg) * a.q.hs;
            },
            put, [&](int r, float scale) { st.row_scale[at * kRows + r] = scale; });
        out = st.q + at * kTileBytes;
    }
    tc::fence_async_proxy();
    __syncthreads();
    if (threadIdx.x == 0) {
        tc::bulk_store(out, tc::smem_addr(tile_s), kTileBytes);
        tc::bulk_store_read();
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) attend_wide_kernel(const AttendArgs a) {
    using L = WideSmem<D>;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (tc::smem_addr(raw) + 1023u) & ~1023u;
    unsigned char *smem = raw + (base - tc::smem_addr(raw));
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    __shared__ CacheItem work;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) work = cache_item<true>(a, a.t.items[blockIdx.x / a.Hkv], blockIdx.x % a.Hkv);
    if (threadIdx.x == 32) {
        gave_up = 0;
        init_bars(base + L::bars, 1, 1, 4);
    }
    if (warp == 8) tc::tmem_alloc(tc::smem_addr(&tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    const bool good = work.good;                   // else not this library's table
    if (!good && threadIdx.x == 0) atomicOr(a.status, 8u);
    auto bar = [&](int i) { return base + L::bars + 8u * i; };

    if (warp >= 8) {
        tc::regs_give<80>();
        if (warp == 9 && lane == 0 && good && work.n > 0) {
            // ------------------------------ copies -------------------------
            const Staged<D> st(a);
            const int n = work.n, h = work.h, q_tiles = work.alternate ? 1 : 2;
            const int64_t q_at = static_cast<int64_t>(work.q_at + work.q0 / work.tpt);
            tc::bar_expect(bar(kQFull), q_tiles * (L::kTileBytes + kRows * 4));
            for (int t = 0; t < q_tiles; ++t) {
                const int64_t at = (q_at + t) * a.Hkv + h;
                tc::bulk_load(base + L::q + t * L::kTileBytes, st.q + at * L::kTileBytes, L::kTileBytes, bar(kQFull));
                tc::bulk_load(base + L::row_scale + t * kRows * 4, st.row_scale + at * kRows, kRows * 4, bar(kQFull));
            }
            int64_t at = static_cast<int64_t>(work.kv_at + work.tile0) * a.Hkv + h;
            int keys = 0, values = 0;
            for (int j = 0; j < n; ++j, at += a.Hkv) {
                const int s = j % kStages, phase = (j / kStages) & 1;
                const unsigned char *tile = st.kv + at * 2 * L::kTileBytes;
                if (kCheck && blockIdx.x == 0 && j + 1 == a.stall_tile) break;
                if (j >= kStages && !tc::bar_wait(bar(kKEmpty + s), phase ^ 1, &gave_up)) break;
                tc::bar_expect(bar(kKFull + s), L::kTileBytes + static_cast<int>(sizeof(TileExps)));
                tc::bulk_load(base + L::k + s * L::kTileBytes, tile, L::kTileBytes, bar(kKFull + s));
                tc::bulk_load(base + L::exps + (j % kExps) * static_cast<int>(sizeof(TileExps)), st.exps + at,
                              sizeof(TileExps), bar(kKFull + s));
                keys = j + 1;
                if (j >= kStages && !tc::bar_wait(bar(kVEmpty + s), phase ^ 1, &gave_up)) break;
                tc::bar_expect(bar(kVFull + s), L::kTileBytes);
                tc::bulk_load(base + L::v + s * L::kTileBytes, tile + L::kTileBytes, L::kTileBytes, bar(kVFull + s));
                values = j + 1;
            }
            tc::bar_drain(bar(kQFull), 0);         // copies in flight land before the CTA leaves
            for (int j = max(0, keys - kStages); j < keys; ++j) tc::bar_drain(bar(kKFull + j % kStages), (j / kStages) & 1);
            for (int j = max(0, values - kStages); j < values; ++j)
                tc::bar_drain(bar(kVFull + j % kStages), (j / kStages) & 1);
        } else if (warp == 8 && good && work.n > 0) {
            mma_role<D, true, L>(work, base, tmem, gave_up);
        }
    } else {
        tc::regs_take<208>();
        if (good)
            softmax_role<D, BF16, true, L>(a, work, reinterpret_cast<const TileExps *>(smem + L::exps), smem, base, tmem, warp,
                                       lane, gave_up);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && gave_up) atomicOr(a.status, 1u);
    if (warp == 8) {
        tc::fence_after_sync();
        tc::tmem_free(tmem, 512);
    }
}

template <int D, int N, bool BF16>
cudaError_t launch_instance(const AttendArgs &a, cudaStream_t s) {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(attend_wide_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 WideSmem<D>::bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = true;
    }
    const dim3 grid(static_cast<unsigned>(2 * a.t.n_kv_tiles + a.t.n_q_tiles), static_cast<unsigned>(a.Hkv));
    constexpr int kStageBytes = kRows * D * 2 + kUnits * kMetaBytes;       // at most 40 KB
    stage_kernel<D, N, BF16><<<grid, kStageThreads, kStageBytes, s>>>(a);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    attend_wide_kernel<D, BF16><<<static_cast<unsigned>(a.t.n_wide) * a.Hkv, kThreads, WideSmem<D>::bytes, s>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

int64_t staged_bytes(int64_t kv_tiles, int64_t q_tiles, int kv_heads, int d) {
    const int64_t tile = static_cast<int64_t>(kRows) * d * 2;
    return kv_heads * (kv_tiles * (2 * tile + static_cast<int64_t>(sizeof(TileExps))) + q_tiles * (tile + kRows * 4));
}

cudaError_t launch_attend_wide(const AttendArgs &a, cudaStream_t s) {
    if (a.t.n_wide == 0) return cudaSuccess;
    if (a.d == 64) {
        if (a.cache.bits == 2) return a.bf16 ? launch_instance<64, 2, true>(a, s) : launch_instance<64, 2, false>(a, s);
        return a.bf16 ? launch_instance<64, 4, true>(a, s) : launch_instance<64, 4, false>(a, s);
    }
    if (a.cache.bits == 2) return a.bf16 ? launch_instance<128, 2, true>(a, s) : launch_instance<128, 2, false>(a, s);
    return a.bf16 ? launch_instance<128, 4, true>(a, s) : launch_instance<128, 4, false>(a, s);
}

}  // namespace kvq
