// attend_prompt.cu -- causal attention over packed prompts on the tensor cores.
//
// o_i = sum_{j <= i} p_ij v_j, p_i = softmax_j(q_i . k_j / sqrt(d)), one pass over the keys with a
// running maximum m and sum l per row: with y = log2(e) q.k / sqrt(d), weights 2^(y - m) meet the
// values as they come, and the sums are rescaled when m rises.
//
// A CTA serves one kv head and two tiles of 128 query rows; the rows of a tile are tokens x the
// query heads of that kv head, so keys and values are fetched once for all of them.  Key and value
// tiles of 128 tokens stream through shared memory by TMA; S = Q K^T and O += P V run on tcgen05
// with both accumulators in tensor memory, and P never leaves tensor memory: a row's thread reads
// its logits there, and writes its weights, as e, over them.  While one tile's threads take the
// exponentials the tensor core works for the other tile.
//
//   warps 0-3, 4-7   softmax of tile 0, 1: thread = row
//   warp 8           issues the MMAs
//   warp 9           TMA loads (warps 10, 11 fill the warpgroup, which gives its registers to the
//                    softmax: 2 x 128 x 208 + 128 x 80 <= 384 x 168)
//
// Tensor memory (512 columns): S0 | S1 | O0 | O1, P over the first half of its S.
//
// Bound by the tensor cores and, under a lasting load, by the power limit.  One prompt of 8192 tokens (32
// query / 8 kv heads, d = 128, bf16; 0.55 TFLOP): 418 us in a burst, 1315 TFLOP/s, and 485 us where
// calls follow one another for a second.  Two of 4096 (32 / 32 heads, fp16): 255 and 303 us.  Twelve of
// 32 to 2048 (32 / 8 heads; 0.12 TFLOP): 137 and 156 us; with a CTA a piece instead of persistent ones
// 156 us in a burst.  A few of up to 160 (2 heads, d = 64): 8 us.  What short jobs cost is their border, where
// the first product of the next job waits for both streams' last of this one: the twelve are 1424 jobs of
// 6 key tiles on average, whose padding (1.13) and dealing (1.05) explain little of the way from 72 us.
#include <cuda.h>

#include <cstdint>

#include "chunk_rows.cuh"
#include "kvq_internal.cuh"
#include "tensor_core.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 384;
constexpr int kRows = 128;                 // rows of a query tile, tokens of a key tile
constexpr int kStages = 2;                 // key and value tiles in flight, each

template <int D>
struct PromptSmem {
    static constexpr int kTileBytes = kRows * D * 2;
    static constexpr int q = 0;                                  // two tiles
    static constexpr int k = q + 2 * kTileBytes;
    static constexpr int v = k + kStages * kTileBytes;
    static constexpr int bars = v + kStages * kTileBytes;
    // one CTA an SM: it holds all of the tensor memory
    static constexpr int bytes = (bars + 256 > 120 * 1024 ? bars + 256 : 120 * 1024) + 1024;
};

// The running maximum is raised when a logit passes it by this: weights grow by up to 2^8 over that of
// the maximum, and the sums are rescaled rarely.
constexpr float kLazyMax = 8.0f;
// The weight of the maximum is 2^kTopWeight.  fp16 holds weights up to 2^15, so that those far below the
// maximum keep their bits (with 2^0 instead of 2^7 a hundred thousand weights of 2^-26 would be lost).
// bf16 has bits to spare below, and its values may be as large as fp32 goes: their sum over 2^16 tokens
// stays in range before it is divided.
template <bool BF16>
constexpr float kTopWeight = BF16 ? -24.0f : 7.0f;
constexpr float kNoMax = -3.4e38f;         // below it: no logits

// A CTA's piece of work: up to 2 * tpt tokens of one slot's prompt from token q0 on, for kv head h.
struct Job {
    int first, count, q0, h;                       // the prompt's first row and tokens
    int tiles[2];                                  // key tiles each query tile sees (0: the tile has no tokens)
    __device__ __forceinline__ int most() const { return max(tiles[0], tiles[1]); }
};

// Job i of the CTA; tiles {0, 0} when there is none.  The jobs lie longest first, and the CTAs take
// them to and fro, so that their sums come out alike.
__device__ __forceinline__ Job prompt_job(const AttendArgs &a, int i) {
    Job w{};
    const int n_ctas = gridDim.x;
    const int64_t at = static_cast<int64_t>(i) * n_ctas +
                       (i & 1 ? n_ctas - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x));
    if (at >= static_cast<int64_t>(a.t.n_items) * a.Hkv) return w;
    const int4 item = a.t.items[at / a.Hkv];
    w.h = static_cast<int>(at % a.Hkv);
    w.q0 = item.y;
    if (item.x >= 0 && item.x < a.t.B && w.q0 >= 0) {
        w.first = a.t.offsets[item.x];
        w.count = a.t.offsets[item.x + 1] - w.first;
        if (w.first >= 0 && w.count > w.q0 && static_cast<int64_t>(w.first) + w.count <= a.t.tokens) {
            const int tpt = kRows / (a.Hq / a.Hkv);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tok = w.q0 + t * tpt;
                w.tiles[t] = tok < w.count ? (min(tok + tpt, w.count) + kRows - 1) / kRows : 0;
            }
            return w;
        }
    }
    if (a.status) atomicOr(a.status, 8u);          // not this library's table
    return w;
}

// Persistent: the roles go from job to job on their own, so that a job's first loads and products run
// while the one before is divided and written out.  Tiles, stages and phases are counted over all
// of the CTA's jobs.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) attend_prompt_kernel(const __grid_constant__ CUtensorMap map_q,
                                                                   const __grid_constant__ CUtensorMap map_k,
                                                                   const __grid_constant__ CUtensorMap map_v,
                                                                   const AttendArgs a) {
    using L = PromptSmem<D>;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (tc::smem_addr(raw) + 1023u) & ~1023u;
    unsigned char *smem = raw + (base - tc::smem_addr(raw));
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const int hg = a.Hq / a.Hkv, tpt = kRows / hg;
    const int64_t n_jobs = static_cast<int64_t>(a.t.n_items) * a.Hkv;
    const int rounds = static_cast<int>((n_jobs + gridDim.x - 1) / gridDim.x);

    const uint32_t bars = base + L::bars;
    auto bar = [&](int i) { return bars + 8u * i; };
    // kPFull: [half of the tile's tokens][stream].  kVFixed: [stage], so that kVEmpty of the stage, committed
    // behind the wait for it, comes between two of its arrivals (short jobs may follow one another while the
    // MMA warp waits for a query tile).
    enum { kQFull = 0, kQEmpty = 2, kKFull = 4, kKEmpty = 6, kVFull = 8, kVEmpty = 10, kSFull = 12, kPFull = 14,
           kOFull = 18, kVFixed = 20, kDrain = 22, kBars = 23 };
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < kBars; ++i) tc::bar_init(bar(i), i >= kPFull && i < kPFull + 4 ? 4 : 1);
        tc::fence_barrier_init();
    }
    if (warp == 8) tc::tmem_alloc(tc::smem_addr(&tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;

    if (warp >= 8) {
        tc::regs_give<80>();
        if (warp == 9) {
            // ------------------------------ loads --------------------------
            const uint32_t q_bytes = static_cast<uint32_t>(hg * tpt * D * 2);
            const uint32_t leader = tc::elect_leader();
            auto load = [&](const CUtensorMap *map, uint32_t dst, int head, int tok, uint32_t b, uint32_t bytes) {
                if (!leader) return;
                tc::bar_expect(b, bytes);
#pragma unroll
                for (int p = 0; p < D / 64; ++p) tc::tma_load_3d(dst + p * kRows * 128, map, 64 * p, head, tok, b);
            };
            bool go = true;
            int keys = 0, values = 0, queries[2] = {0, 0};     // tiles asked for
            auto load_keys = [&](const Job &w, int j) {
                if (kCheck && blockIdx.x == 0 && keys + 1 == a.stall_tile) go = false;
                if (!go) return;
                const int s = keys % kStages;
                if (keys >= kStages) go = go && tc::bar_wait_warp(bar(kKEmpty + s), ((keys / kStages) & 1) ^ 1, &gave_up);
                if (!go) return;
                load(&map_k, base + L::k + s * L::kTileBytes, w.h, w.first + j * kRows, bar(kKFull + s), L::kTileBytes);
                ++keys;
            };
            Job next = prompt_job(a, 0);
            for (int i = 0; i < rounds && go; ++i) {
                const Job w = next;
                next = prompt_job(a, i + 1);
                const int n = w.most();
                for (int t = 0; t < 2 && go; ++t) {
                    if (w.tiles[t]) {
                        if (queries[t] > 0) go = tc::bar_wait_warp(bar(kQEmpty + t), (queries[t] - 1) & 1, &gave_up);
                        if (!go) break;
                        load(&map_q, base + L::q + t * L::kTileBytes, w.h * hg, w.first + w.q0 + t * tpt, bar(kQFull + t),
                             q_bytes);
                        ++queries[t];
                    }
                    if (t == 0 && n > 0) load_keys(w, 0);
                }
                for (int j = 0; j < n && go; ++j) {
                    if (j > 0) load_keys(w, j);
                    const int s = values % kStages;
                    if (values >= kStages)
                        go = go && tc::bar_wait_warp(bar(kVEmpty + s), ((values / kStages) & 1) ^ 1, &gave_up);
                    if (!go) break;
                    load(&map_v, base + L::v + s * L::kTileBytes, w.h, w.first + j * kRows, bar(kVFull + s), L::kTileBytes);
                    ++values;
                }
                // The last value tile may reach past the sequence, into rows that are another's or
                // anything: their weights are 0, but 0 times an infinity is not, so they are cleared.
                const int left = w.count - (n - 1) * kRows;
                if (go && n > 0 && left < kRows) {
                    const int s = (values - 1) % kStages;
                    go = tc::bar_wait_warp(bar(kVFull + s), ((values - 1) / kStages) & 1, &gave_up);
                    unsigned char *v = smem + L::v + s * L::kTileBytes;
                    for (int k = lane; go && k < (kRows - left) * 8; k += 32)  // whole 128-byte rows: the swizzle stays inside
#pragma unroll
                        for (int p = 0; p < D / 64; ++p)
                            *reinterpret_cast<uint4 *>(v + p * kRows * 128 + left * 128 + 16 * k) = make_uint4(0, 0, 0, 0);
                    tc::fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) tc::bar_arrive(bar(kVFixed + s));
                }
            }
            for (int t = 0; t < 2; ++t)            // copies in flight land before the CTA leaves
                if (queries[t]) tc::bar_drain(bar(kQFull + t), (queries[t] - 1) & 1);
            for (int k = max(0, keys - kStages); k < keys; ++k) tc::bar_drain(bar(kKFull + k % kStages), (k / kStages) & 1);
            for (int k = max(0, values - kStages); k < values; ++k)
                tc::bar_drain(bar(kVFull + k % kStages), (k / kStages) & 1);
        } else if (warp == 8) {
            // ------------------------------ MMAs ---------------------------
            const uint32_t leader = tc::elect_leader();
            constexpr uint32_t kDescS = tc::mma_desc(kRows, kRows, BF16, false);
            constexpr uint32_t kDescO = tc::mma_desc(kRows, D, BF16, true);
            auto issue_s = [&](int t, int s, bool last) {
                const uint64_t qd = tc::desc_k_major(base + L::q + t * L::kTileBytes);
                const uint64_t kd = tc::desc_k_major(base + L::k + s * L::kTileBytes);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint64_t step = (i / 4) * (kRows * 128 / 16) + (i % 4) * 2;
                    tc::mma_ss(tmem + t * 128, qd + step, kd + step, kDescS, i > 0, leader);
                }
                tc::mma_commit(bar(kSFull + t), leader);
                if (last) tc::mma_commit(bar(kQEmpty + t), leader);
            };
            bool go = true;
            int at = 0, queries[2] = {0, 0}, weights[2] = {0, 0}, fixed = 0;   // key tiles, and the rest, before this job; kVFixed's phases
            Job next = prompt_job(a, 0);
            for (int i = 0; i < rounds && go; ++i) {
                const Job w = next;
                next = prompt_job(a, i + 1);
                const int n = w.most();
                if (n == 0) continue;
                go = tc::bar_wait_warp(bar(kKFull + at % kStages), (at / kStages) & 1, &gave_up);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!go || w.tiles[t] == 0) continue;
                    go = tc::bar_wait_warp(bar(kQFull + t), queries[t] & 1, &gave_up);
                    if (go) issue_s(t, at % kStages, w.tiles[t] == 1);
                    ++queries[t];
                }
                if (go) tc::mma_commit(bar(kKEmpty + at % kStages), leader);
                for (int j = 0; j < n && go; ++j, ++at) {
                    const int s = at % kStages, s1 = (at + 1) % kStages;
                    go = tc::bar_wait_warp(bar(kVFull + s), (at / kStages) & 1, &gave_up);
                    if (go && j == n - 1 && w.count - j * kRows < kRows) {
                        go = tc::bar_wait_warp(bar(kVFixed + s), (fixed >> s) & 1, &gave_up);
                        fixed ^= 1 << s;
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!go || j >= w.tiles[t]) continue;
                        const uint64_t vd = tc::desc_mn_major(base + L::v + s * L::kTileBytes, kRows * 128);
#pragma unroll
                        for (int half = 0; half < 2; ++half) { // the first weights while the others are taken
                            go = go && tc::bar_wait_warp(bar(kPFull + 2 * half + t), weights[t] & 1, &gave_up);
                            if (!go) break;
                            tc::fence_after_sync();
#pragma unroll
                            for (int k = 4 * half; k < 4 * half + 4; ++k)
                                tc::mma_ts(tmem + 256 + t * 128, tmem + t * 128 + 8 * k, vd + k * (2048 / 16), kDescO,
                                           j > 0 || k > 0, leader);
                        }
                        if (!go) continue;
                        ++weights[t];
                        if (j + 1 < w.tiles[t]) {
                            go = tc::bar_wait_warp(bar(kKFull + s1), ((at + 1) / kStages) & 1, &gave_up);
                            if (go) issue_s(t, s1, j + 2 == w.tiles[t]);
                        } else {
                            tc::mma_commit(bar(kOFull + t), leader);
                        }
                    }
                    if (go) {
                        tc::mma_commit(bar(kVEmpty + s), leader);
                        if (j + 1 < n) tc::mma_commit(bar(kKEmpty + s1), leader);
                    }
                }
            }
            // MMAs in flight end before tensor memory is freed
            tc::mma_commit(bar(kDrain), leader);
            tc::bar_drain(bar(kDrain), 0);
        }
    } else {
        tc::regs_take<208>();
        // ------------------------------ softmax ----------------------------
        const int t = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
        const float scale = a.scale;
        bool go = true;
        int at = 0, outputs = 0;                   // this stream's tiles and outputs before this job
        Job next = prompt_job(a, 0);
        for (int i = 0; i < rounds && go; ++i) {
            const Job w = next;
            next = prompt_job(a, i + 1);
            const int n = t ? w.tiles[1] : w.tiles[0];
            if (n == 0) continue;
            const int tok0 = w.q0 + t * tpt, tok = tok0 + r / hg;
            float m = 0.0f, l = 0.0f;
            for (int j = 0; j < n && go; ++j, ++at) {
                go = tc::bar_wait_warp(bar(kSFull + t), at & 1, &gave_up);
                if (!go) break;
                tc::fence_after_sync();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::tmem_load(ts + 32 * c, s[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::tmem_arrived(s[c]);
                if ((j + 1) * kRows > tok0 + 1) {  // tokens ahead of some row
                    const int seen = tok + 1 - j * kRows;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * c + e >= seen) s[c][e] = 0xff800000u;
                }
                float mxs[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mxs[c] = __uint_as_float(s[c][0]);
#pragma unroll
                    for (int e = 1; e < 32; ++e) mxs[c] = fmaxf(mxs[c], __uint_as_float(s[c][e]));
                }
                const float mx = fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3])) * scale;
                const bool far = fabsf(mx) > kFarLogit && mx > kNoMax;
                bool careful = false;
                if (j == 0) {
                    m = mx - kTopWeight<BF16>;
                    careful = __any_sync(0xffffffffu, far);
                } else if (__any_sync(0xffffffffu, mx - m > kLazyMax + kTopWeight<BF16> || far)) {
                    careful = __any_sync(0xffffffffu, far);
                    // O holds every tile before j: S_j was committed after its last MMA
                    const float mn = fmaxf(m, mx - kTopWeight<BF16>), alpha = tc::ex2(m - mn);
                    m = mn;
                    l *= alpha;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tc::tmem_load(to + 32 * c, o);
                        tc::tmem_arrived(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tc::tmem_store(to + 32 * c, o);
                    }
                }
                if (careful)
#pragma unroll
                    for (int c = 0; c < 4; ++c) subtract_rounded<32>(s[c], scale, m);
                const float sc = careful ? 1.0f : scale, from = careful ? 0.0f : m;
                float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t(&p)[32] = s[2 * half];    // a weight takes the place of a logit read before
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t *src = &s[2 * half + e / 16][2 * (e % 16)];
                        const float2 y = tc::fma2(make_float2(__uint_as_float(src[0]), __uint_as_float(src[1])),
                                                  make_float2(sc, sc), make_float2(-from, -from));
                        const float2 wt = make_float2(tc::ex2(y.x), tc::ex2(y.y));
                        l2[e % 2] = tc::add2(l2[e % 2], wt);
                        p[e] = narrow2<BF16>(wt.x, wt.y);
                    }
                    tc::tmem_store(ts + 32 * half, p);
                    tc::tmem_stored();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::bar_arrive(bar(kPFull + 2 * half + t));
                }
                l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
            }
            if (go) go = tc::bar_wait_warp(bar(kOFull + t), outputs & 1, &gave_up);
            if (!go) break;
            ++outputs;
            tc::fence_after_sync();
            const float inv = __fdividef(1.0f, l);
            const bool mine = r < hg * tpt && tok < w.count;
            uint16_t *out = a.o.p + static_cast<int64_t>(w.first + tok) * a.o.ts +
                            static_cast<int64_t>(w.h * hg + r % hg) * a.o.hs;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                __syncwarp();
                tc::tmem_load(to + 32 * c, o);
                tc::tmem_arrived(o);
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[k] = narrow2<BF16>(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                                 __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                        reinterpret_cast<uint4 *>(out + 32 * c)[e] = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            __syncwarp();
            tc::fence_before_sync();               // O is read: the next job's weights may change it
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && gave_up && a.status) atomicOr(a.status, 1u);
    if (warp == 8) {
        tc::fence_after_sync();
        tc::tmem_free(tmem, 512);
    }
}

// The tensor map of packed rows [tokens][heads][d], boxes of 64 channels x box_heads x box_tokens
// in 128-byte rows with the 128-byte swizzle; rows outside the tensor read as zeros.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

bool rows_map(CUtensorMap *map, const Rows &r, int64_t tokens, int heads, int d, bool bf16, int box_heads,
              int box_tokens) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    // the stride of a dimension of one entry is never followed: any valid one
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? r.hs : d) * 2,
                                   static_cast<cuuint64_t>(tokens > 1 ? r.ts : d) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
    const cuuint32_t one[3] = {1, 1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, r.p, dims, strides,
                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16>
cudaError_t launch_instance(const AttendArgs &a, cudaStream_t s) {
    const int hg = a.Hq / a.Hkv, tpt = kRows / hg;
    CUtensorMap mq, mk, mv;
    if (!rows_map(&mq, a.q, a.t.tokens, a.Hq, D, BF16, hg, tpt) ||
        !rows_map(&mk, a.k, a.t.tokens, a.Hkv, D, BF16, 1, kRows) ||
        !rows_map(&mv, a.v, a.t.tokens, a.Hkv, D, BF16, 1, kRows))
        return cudaErrorInvalidValue;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(attend_prompt_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PromptSmem<D>::bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = true;
    }
    static int sms[64] = {};
    if (dev < 64 && sms[dev] == 0) {
        e = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
    }
    const int64_t jobs = static_cast<int64_t>(a.t.n_items) * a.Hkv, ctas = dev < 64 ? sms[dev] : 148;
    attend_prompt_kernel<D, BF16><<<static_cast<unsigned>(jobs < ctas ? jobs : ctas), kThreads, PromptSmem<D>::bytes, s>>>(
        mq, mk, mv, a);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_prompt(const AttendArgs &a, cudaStream_t s) {
    if (a.t.n_items == 0) return cudaSuccess;
    if (a.d == 64) return a.bf16 ? launch_instance<64, true>(a, s) : launch_instance<64, false>(a, s);
    return a.bf16 ? launch_instance<128, true>(a, s) : launch_instance<128, false>(a, s);
}

}  // namespace kvq
