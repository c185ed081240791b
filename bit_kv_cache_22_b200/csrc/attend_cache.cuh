// attend_cache.cuh -- what the two kernels that attend a chunk over the paged low-bit cache share
// (attend_narrow.cu: few query rows a slot, attend_wide.cu: many): the operands' form, their
// unpacking, the MMA and softmax roles.
//
// Query row i of a slot, at position p, sees tokens 0 .. p of its sequence: o_i = sum_{j <= p}
// p_ij v_j with p_i = softmax_j(q_i . k_j / sqrt(d)), k_j and v_j as the cache holds them: (code - z) s
// for tokens below Tq, the residual rows behind.  One pass with a running maximum and sum per row.
//
// A CTA serves one kv head and up to two tiles of 128 query rows (tokens x the query heads of that
// kv head).  Key and value tiles of 128 tokens lie in shared memory as fp16 operands; S = Q K^T and
// O += P V run on tcgen05 with both accumulators and P in tensor memory, and four warps per query
// tile take the softmax (thread = row).  Where one query tile holds all rows the two halves of the
// CTA take alternate key tiles of it and meet at the end.
//
// Operands in fp16 for caches of either type: (code - z) s is rounded to 11 bits (bf16 would leave 8,
// a rounding as large as the output's own).  What fp16 lacks is range, so operands carry powers of
// two of their own: a query row that of its largest channel, 32 tokens' keys and values those of
// bounds on their elements, so that the largest lies in [2^14, 2^15) -- values' in steps of 2^4.
// They are undone in the logits' scale, and for the values in the weights: a row's sums stand for
// 2^(m + e) of what they hold, and a weight that meets values under 2^ev enters as 2^(y - m) 2^(ev - e).  e
// follows, as m follows the logits, the largest weight x 2^ev that 32 tokens brought the row, so that a
// weight is rounded by what it adds: to 11 bits, and its token's share by at most 2^-26 of (the largest
// weight x the largest value) of some 32 tokens.  (That weight lies at 2^5 or above, where others are
// off by 2^-25; operands reach 2^15, and bounds lie 2^11 or more above 2^ev.)  Large values that hardly
// weigh, or that the row does not see, cost it nothing unless they lie among the 32 tokens of one that
// weighs.
// An element far below the largest of its 32 tokens loses bits under 2^-36 of it.
//
// Unpacking is bound by the integer pipe, so codes stay in 16-bit pairs: bytes 0 and 2 (1 and 3) of a
// word's slot, OR 0x6400, are the fp16 numbers 1024 + code; minus (1024 + z), exact for |z| <= 1024,
// times s -- in fp16 caches in two fp16 parts, lest s's own rounding double the element's; next to a
// bf16 output s goes as one.  Keys carry nearly all of the error, since a logit's error grows with its
// terms: with one channel ten times the others, d = 128, outputs are off 64 bits by 0.0009 in fp16 (the
// output's own rounding: 0.0002) and by 0.0020 in bf16 (0.0017).
//
// The order of channels in keys and queries, and of tokens in keys and values, is free as long as
// both agree.  A lane unpacks four neighbouring channels (tokens) at a time, which lie in the operand as
// 0, 2, 1, 3, as the pairs come; and of 64 channels (tokens) c, eight to a 16-byte step of a 128-byte
// row, step c/16 + 4 ((c/8) mod 2) holds c's eight, so that the stores of a warp -- eight rows, four
// lanes along each -- meet every bank once (in plain order each bank twice).
#pragma once

#include <cstdint>

#include "chunk_rows.cuh"
#include "kvq_internal.cuh"
#include "tensor_core.cuh"

namespace kvq {
namespace {

constexpr int kRows = 128;                 // rows of a query tile, tokens of a key tile
constexpr int kStages = 2;                 // key and value operand tiles, each
constexpr int kUnits = 4;                  // of 32 tokens in a key tile: a warp's work for keys or values
constexpr int kExps = 8;                   // key tiles whose exponents are kept (at most kStages + 1 are live)
constexpr int kValueStep = 4;              // values' exponents are multiples of this: they rarely differ
// Weights, as they meet the values, lie below 2^(kTopWeight + kLazyMax); where the maximum, or e, is raised
// the largest becomes about 2^kTopWeight.
constexpr float kTopWeight = 7.0f, kLazyMax = 8.0f;
constexpr float kNoMax = -1e30f;           // the maximum of no logits: finite, so differences stay numbers
constexpr int kMaxTokens = 0x7fffffff - 1024;   // of a sequence (the planner refuses more)
// Least exponents of operands: values' 2^e and 2^-e stay normal; those of queries and keys keep
// their product, the logits' scale, above 0 (what they cost a logit is below 2^-60 of the other).
constexpr int kMinExp = -112, kMinLogitExp = -56;      // kMinExp: a multiple of kValueStep

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// the exponent e with bound 2^-e in [2^14, 2^15), as far as `least` allows
__device__ __forceinline__ int operand_exp(uint32_t bound_bits, int least) {
    return max(static_cast<int>(bound_bits >> 23) - 127 - 14, least);
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

// place of element i of four in an operand: 0, 2, 1, 3
__host__ __device__ constexpr int mixed(int i) { return (i & ~3) | ((i & 1) << 1) | ((i >> 1) & 1); }
// 16-byte step of 64 elements that holds the eight of element c
__host__ __device__ constexpr int step_of(int c) { return (c / 16) % 4 + 4 * ((c / 8) % 2); }
// the token of column c of a key tile, and the unit of 32 it is in
__host__ __device__ constexpr int token_of(int c) {
    return c / 64 * 64 + (c / 8) % 4 * 16 + (c / 32) % 2 * 8 + mixed(c % 8);
}
static_assert(step_of(token_of(77)) == 77 / 8 % 8 && mixed(token_of(77) % 8) == 77 % 8, "token_of inverts the places");

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2 *>(&v); }
__device__ __forceinline__ uint32_t as_bits(__half2 v) { return *reinterpret_cast<const uint32_t *>(&v); }

// The parameters of four elements, in pairs (0, 2) and (1, 3): -(1024 + z), and s in two parts (the
// second in fp16 caches only).
struct Quad {
    uint2 z, hi, lo;
};

// Four codes of N bits in the bytes of b (above them anything): (code - z) s.
template <int N, bool BF16>
__device__ __forceinline__ uint2 unpack_four(uint32_t b, const Quad &q) {
    constexpr uint32_t kMask = 0x00010001u * ((1u << N) - 1);
    const __half2 x = __hadd2(as_half2((b & kMask) | 0x64006400u), as_half2(q.z.x));
    const __half2 y = __hadd2(as_half2(((b >> 8) & kMask) | 0x64006400u), as_half2(q.z.y));
    if constexpr (BF16)
        return make_uint2(as_bits(__hmul2(x, as_half2(q.hi.x))), as_bits(__hmul2(y, as_half2(q.hi.y))));
    return make_uint2(as_bits(__hfma2(x, as_half2(q.hi.x), __hmul2(x, as_half2(q.lo.x)))),
                      as_bits(__hfma2(y, as_half2(q.hi.y), __hmul2(y, as_half2(q.lo.y)))));
}
// The same in fp32, for zeros that 1024 + z does not hold.
__device__ __forceinline__ uint2 unpack_four_wide(uint32_t b, const float4 &s, const float4 &z) {
    const float2 x = tc::mul2(tc::add2(make_float2(byte_plus_2_23<0>(b), byte_plus_2_23<2>(b)), make_float2(z.x, z.z)),
                              make_float2(s.x, s.z));
    const float2 y = tc::mul2(tc::add2(make_float2(byte_plus_2_23<1>(b), byte_plus_2_23<3>(b)), make_float2(z.y, z.w)),
                              make_float2(s.y, s.w));
    return make_uint2(half2_bits(x.x, x.y), half2_bits(y.x, y.y));
}

// What one unpacking warp needs of a unit's keys or values: the code words of its lanes, and four
// scales and zeros a lane twice, which it spreads over shared memory -- keys: channels 4 lane .. of the
// halves' groups (one group of 32 tokens or more: the first only); values: entries 4 lane .. and 128 +
// 4 lane .. of [32 tokens][D / Gv].
template <int D, int N>
struct Fetched {
    static constexpr int W = D * N / 64;   // words per lane and half
    uint32_t w[2][W];
    float4 s[2];
    uint2 z[2];
    int kind[2];                           // of each 16 tokens; 0: none, 1: quantized, 2: residual
};

// Where a warp unpacks: keys (kv 0) or values (1) of a slot's kv head.  One code serves both: the
// narrow kernel's roles together have to stay in the SM's instruction cache.
template <int D>
struct UnitSource {
    const uint32_t *words;
    const float *scales;
    const int16_t *zeros;
    const uint16_t *res;                   // the slot's residual rows: token tq's first
    int kv, h, len, tq;
    int tokens_shift, entries_shift;       // entries of parameters: (token >> tokens_shift) << entries_shift
    int first, second, apart;              // a unit's: how many, how many more `apart` on
    __device__ __forceinline__ UnitSource(const PagedView &c, int kv_, int slot, int h_, int len_, int tq_)
        : kv(kv_), h(h_), len(len_), tq(tq_) {
        words = kv ? c.vc : c.kc;
        scales = kv ? c.vs : c.ks;
        zeros = kv ? c.vz : c.kz;
        res = (kv ? c.vr : c.kr) + (static_cast<int64_t>(slot) * c.Hkv + h) * c.R * D;
        const int ngv_shift = __ffs(D) - __ffs(c.Gv);      // G, Gv, D: powers of two
        tokens_shift = kv ? 0 : __ffs(c.G) - 1;
        entries_shift = kv ? ngv_shift : __ffs(D) - 1;
        first = kv ? min(32 << ngv_shift, 128) : D;
        second = kv ? (32 << ngv_shift) - first : c.G == 16 ? D : 0;
        apart = kv ? 128 : D;
    }
};

__device__ __forceinline__ void widen_zeros(uint2 z, bool sym, int half_levels, float (&f)[4]) {
    f[0] = static_cast<float>(sym ? half_levels : static_cast<int>(static_cast<int16_t>(z.x & 0xffffu)));
    f[1] = static_cast<float>(sym ? half_levels : static_cast<int>(z.x) >> 16);
    f[2] = static_cast<float>(sym ? half_levels : static_cast<int>(static_cast<int16_t>(z.y & 0xffffu)));
    f[3] = static_cast<float>(sym ? half_levels : static_cast<int>(z.y) >> 16);
}

// The powers of two of a key tile's units: 2^e of the keys, then e of the values.
struct TileExps {
    float scale_k[kUnits];
    float exp_v[kUnits];
};

// Fetches the 32 tokens tok .. ; at_tok: the first one's place in its page.
template <int D, int N>
__device__ __forceinline__ void fetch_unit(Fetched<D, N> &f, const PagedView &c, const UnitSource<D> &src, int page,
                                           int at_tok, int tok, bool on, int lane) {
    constexpr int W = D * N / 64, TW = D * N / 2;
#pragma unroll
    for (int p = 0; p < 2; ++p) f.kind[p] = !on || tok + 16 * p >= src.len ? 0 : tok + 16 * p < src.tq ? 1 : 2;
    if (f.kind[0] != 1) return;
    if (page < 0 || page >= c.num_pages) {
        if (lane == 0) atomicOr(c.status, 2u);
        page = 0;
    }
    const int64_t slice = static_cast<int64_t>(page) * c.Hkv + src.h;
    const uint32_t *words = src.words + (slice * (c.P >> 4) + (at_tok >> 4)) * TW + lane * W;
#pragma unroll
    for (int p = 0; p < 2; ++p) {                  // pages hold whole units: a half behind tq is read for nothing
        if constexpr (W >= 4) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(words + p * TW + i);
                f.w[p][i] = x.x; f.w[p][i + 1] = x.y; f.w[p][i + 2] = x.z; f.w[p][i + 3] = x.w;
            }
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(words + p * TW);
            f.w[p][0] = x.x; f.w[p][1] = x.y;
        }
    }
    const int64_t at =
        ((slice * (c.P >> src.tokens_shift) + (at_tok >> src.tokens_shift)) << src.entries_shift) + 4 * lane;
    if (4 * lane < src.first) {
        f.s[0] = *reinterpret_cast<const float4 *>(src.scales + at);
        if (!c.sym) f.z[0] = *reinterpret_cast<const uint2 *>(src.zeros + at);
    }
    if (4 * lane < src.second) {
        f.s[1] = *reinterpret_cast<const float4 *>(src.scales + at + src.apart);
        if (!c.sym) f.z[1] = *reinterpret_cast<const uint2 *>(src.zeros + at + src.apart);
    }
}

// A warp's shared memory for the parameters of its unit.
constexpr int kMetaBytes = 2048;

// The unit's power of two e, and its parameters spread over shared memory for the lanes that use them;
// false: in fp32, for zeros that 1024 + z does not hold.
//   keys: [half's group][z, hi, lo][D / 4] pairs of pairs; values: [z, hi, lo][D / Gv][32] halves, in mixed order
//   in fp32: [s, z], keys [half's group][D], values [D / Gv][32]
template <int D, int N, bool BF16>
__device__ __forceinline__ bool prepare_unit(const Fetched<D, N> &f, const PagedView &c, const UnitSource<D> &src,
                                             int tok, int lane, unsigned char *meta, int &ex) {
    constexpr float kTop = static_cast<float>((1 << N) - 1);
    const int ngv_shift = src.entries_shift, ngv = 1 << ngv_shift;     // (of values)
    float big = 0.0f, z[2][4];
    bool on[2], over = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int half = src.kv ? (4 * lane + 128 * x) >> (ngv_shift + 4) : x;
        on[x] = 4 * lane < (x ? src.second : src.first) && (half ? f.kind[1] : f.kind[0]) == 1;
        if (!on[x]) continue;
        widen_zeros(f.z[x], c.sym, 1 << (N - 1), z[x]);
        const float s[4] = {f.s[x].x, f.s[x].y, f.s[x].z, f.s[x].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            big = fmaxf(big, s[e] * fmaxf(fabsf(z[x][e]), fabsf(kTop - z[x][e])));
            over = over || fabsf(z[x][e]) > 1024.0f;
        }
    }
    if (f.kind[0] == 2 || f.kind[1] == 2) {        // rows of one token are D / 8 vectors
        const int from = max(tok, src.tq);
#pragma unroll 4
        for (int i = lane; i < 32 * (D / 8); i += 32) {
            const int tk = tok + i / (D / 8);
            if (tk < from || tk >= src.len) continue;
            const uint4 v = reinterpret_cast<const uint4 *>(src.res)[static_cast<int64_t>(tok - src.tq) * (D / 8) + i];
            const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 y = widen_pair<BF16>(vw[e]);
                big = fmaxf(big, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
        }
    }
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
    ex = src.kv ? (operand_exp(bits, kMinExp) + kValueStep - 1) & ~(kValueStep - 1) : operand_exp(bits, kMinLogitExp);
    if (f.kind[0] != 1) return true;
    const float down = pow2(-ex);
    const bool wide = __any_sync(0xffffffffu, over);       // (and the unit before is unpacked)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if (!on[x]) continue;
        const float s[4] = {f.s[x].x * down, f.s[x].y * down, f.s[x].z * down, f.s[x].w * down};
        float lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) lo[e] = s[e] - __half2float(__float2half_rn(s[e]));
        if (!src.kv) {
            if (!wide) {
                uint2 *m = reinterpret_cast<uint2 *>(meta) + x * (3 * D / 4) + lane;
                m[0] = make_uint2(half2_bits(-1024.0f - z[x][0], -1024.0f - z[x][2]),
                                  half2_bits(-1024.0f - z[x][1], -1024.0f - z[x][3]));
                m[D / 4] = make_uint2(half2_bits(s[0], s[2]), half2_bits(s[1], s[3]));
                if (!BF16) m[D / 2] = make_uint2(half2_bits(lo[0], lo[2]), half2_bits(lo[1], lo[3]));
            } else {
                float4 *m = reinterpret_cast<float4 *>(meta) + x * (2 * D / 4) + lane;
                m[0] = make_float4(s[0], s[1], s[2], s[3]);
                m[D / 4] = make_float4(-8388608.0f - z[x][0], -8388608.0f - z[x][1], -8388608.0f - z[x][2],
                                       -8388608.0f - z[x][3]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * lane + 128 * x + e, g = (i & (ngv - 1)) * 32, tk = i >> ngv_shift;
                if (!wide) {
                    uint16_t *m = reinterpret_cast<uint16_t *>(meta) + g + mixed(tk);
                    m[0] = __half_as_ushort(__float2half_rn(-1024.0f - z[x][e]));
                    m[256] = __half_as_ushort(__float2half_rn(s[e]));
                    if (!BF16) m[512] = __half_as_ushort(__float2half_rn(lo[e]));
                } else {
                    float *m = reinterpret_cast<float *>(meta) + g + tk;
                    m[0] = s[e];
                    m[256] = -8388608.0f - z[x][e];
                }
            }
        }
    }
    __syncwarp();
    return !wide;
}

// put for a tile in shared memory
struct SharedPut {
    uint32_t tile;
    __device__ __forceinline__ void operator()(int offset, uint32_t x, uint32_t y) const {
        tc::store_shared(tile + offset, x, y);
    }
    __device__ __forceinline__ void operator()(int offset, const uint32_t (&v)[4]) const { tc::store_shared(tile + offset, v); }
};

// Unit u of a key tile as operands: keys, rows = tokens, channels along a row; values, rows =
// channels, tokens along a row.  put(offset, a, b) stores 8 bytes of the tile, put(offset, v) 16.
// words are used up.
template <int D, int N, bool BF16, class Put>
__device__ __forceinline__ void emit_unit(uint32_t (&words)[2][D * N / 64], int kind0, int kind1, bool narrow,
                                          const PagedView &c, const UnitSource<D> &src, int tok, float down, int u,
                                          int lane, const unsigned char *meta, const Put &put) {
    constexpr int B = 4 / N, W = D * N / 64;
    const int kv = src.kv;
    if (kind0 == 1) {
        // the lane's place: a row, a step along it (swizzled), eight bytes of that; then the same for the
        // next chunks of 16 channels, for the second of a slot's two codes (eight channels or tokens
        // on) and the second half's tokens
        const int row = kv ? lane >> 2 : 64 * (u / 2) + 16 * (u % 2) + mixed(lane >> 2);
        const int line = (kv ? (u / 2) * (D * 128) : 0) + row * 128 + (lane & 1) * 8;
        const int far = 4 * ((lane >> 1) & 1) + (kv ? 2 * (u % 2) : 0);
        int at[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) at[x] = line + (((far + (kv ? 0 : x)) ^ (row & 7)) << 4) + (kv ? x * 2048 : 0);
        const int code2 = kv ? 1024 : 4096;
        const int half2 = kv ? (((far + 1) ^ (row & 7)) - (far ^ (row & 7))) << 4 : 1024;
        const bool both = kind1 == 1;
        const int shift = kv ? __ffs(c.Gv) - 5 : 0;            // chunk -> group of parameters
        if (narrow) {
            // per group (kv) or chunk, and half: z, hi, lo `next` apart
            const int next = kv ? 64 : D / 4, per = kv ? 3 : 2, other = kv ? 4 : c.G == 16 ? 3 * D / 4 : 0;
            const uint2 *pm = reinterpret_cast<const uint2 *>(meta) + (lane & 3);
            auto quad = [&](int ch, int from) {
                const uint2 *q = pm + ((ch >> shift) << per) + from;
                return Quad{q[0], q[next], BF16 ? make_uint2(0u, 0u) : q[2 * next]};
            };
            Quad q0 = quad(0, 0), q1 = quad(0, other);
#pragma unroll 1
            for (int ch0 = 0; ch0 < D / 16; ch0 += 4) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {      // the next chunk's parameters before this one's stores
                    const int more = ch0 + x + 1 < D / 16 ? ch0 + x + 1 : 0;
                    const Quad n0 = quad(more, 0), n1 = quad(more, other);
                    const uint32_t b0 = words[0][x / B] >> (N * 2 * (x % B)), b1 = words[1][x / B] >> (N * 2 * (x % B));
                    const uint2 x0 = unpack_four<N, BF16>(b0, q0), y0 = unpack_four<N, BF16>(b0 >> N, q0);
                    const uint2 x1 = unpack_four<N, BF16>(b1, q1), y1 = unpack_four<N, BF16>(b1 >> N, q1);
                    put(at[x], x0.x, x0.y);
                    put(at[x] + code2, y0.x, y0.y);
                    if (both) {
                        put(at[x] + half2, x1.x, x1.y);
                        put(at[x] + half2 + code2, y1.x, y1.y);
                    }
                    at[x] += kv ? 4 * 2048 : kRows * 128;
                    q0 = n0;
                    q1 = n1;
                }
#pragma unroll
                for (int i = 0; i + 4 / B < W; ++i) {
                    words[0][i] = words[0][i + 4 / B];
                    words[1][i] = words[1][i + 4 / B];
                }
            }
        } else {
            constexpr uint32_t kMask = 0x01010101u * ((1u << N) - 1);
            const int next = kv ? 64 : D / 4, per = kv ? 3 : 2, other = kv ? 4 : c.G == 16 ? 2 * D / 4 : 0;
            const float4 *pm = reinterpret_cast<const float4 *>(meta) + (lane & 3);
#pragma unroll 1
            for (int i = 0; i < D / 8; ++i) {      // chunk i / 2 of half i % 2
                const int ch = i / 2, p = i % 2;
                if (p == 0 || both) {
                    const float4 *from = pm + ((ch >> shift) << per) + (p ? other : 0);
                    const float4 sc = from[0], z = from[next];
                    const uint32_t b = (p ? words[1][0] : words[0][0]) >> (N * 2 * (ch % B));
                    const uint2 x = unpack_four_wide(b & kMask, sc, z), y = unpack_four_wide((b >> N) & kMask, sc, z);
                    const int to = (ch & 2 ? ch & 1 ? at[3] : at[2] : ch & 1 ? at[1] : at[0]) + (p ? half2 : 0) +
                                   (ch / 4) * (kv ? 4 * 2048 : kRows * 128);
                    put(to, x.x, x.y);
                    put(to + code2, y.x, y.y);
                }
                if (p == 1 && ch % B == B - 1)
#pragma unroll
                    for (int k = 0; k + 1 < W; ++k) {
                        words[0][k] = words[0][k + 1];
                        words[1][k] = words[1][k + 1];
                    }
            }
        }
        if (both) return;
    }
    // the rest: residual rows, zeros behind the last token
    const int from = kind0 == 1 ? 16 : 0;
    if (!kv) {
#pragma unroll 4
        for (int i = lane; i < (32 - from) * (D / 8); i += 32) {
            const int t = from + i / (D / 8), v = i % (D / 8);
            const int rm = 64 * (u / 2) + 16 * (u % 2) + 8 * (t / 16) + 32 * ((t / 8) % 2) + mixed(t % 8);
            uint32_t o[4] = {0u, 0u, 0u, 0u};
            if (tok + t < src.len) {
                const uint4 x = reinterpret_cast<const uint4 *>(src.res + static_cast<int64_t>(tok + t - src.tq) * D)[v];
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 p = widen_pair<BF16>(xw[e]), q = widen_pair<BF16>(xw[e + 1]);
                    o[e] = half2_bits(p.x * down, q.x * down);
                    o[e + 1] = half2_bits(p.y * down, q.y * down);
                }
            }
            put((v / 8) * (kRows * 128) + rm * 128 + ((step_of(8 * v) ^ (rm & 7)) << 4), o);
        }
    } else {
#pragma unroll 2
        for (int i = lane; i < (4 - from / 8) * (D / 2); i += 32) {    // channels 2 cp, 2 cp + 1: eight tokens
            const int cp = i % (D / 2), t0 = from + 8 * (i / (D / 2));
            uint32_t o[2][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 p[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tk = tok + t0 + mixed(2 * k + e);
                    p[e] = make_float2(0.0f, 0.0f);
                    if (tk < src.len)
                        p[e] = widen_pair<BF16>(
                            reinterpret_cast<const uint32_t *>(src.res + static_cast<int64_t>(tk - src.tq) * D)[cp]);
                }
                o[0][k] = half2_bits(p[0].x * down, p[1].x * down);
                o[1][k] = half2_bits(p[0].y * down, p[1].y * down);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * cp + e;
                put((u / 2) * (D * 128) + r * 128 + ((step_of(32 * (u % 2) + t0) ^ (r & 7)) << 4), o[e]);
            }
        }
    }
}

// Query rows r (tokens x heads) of a tile as operands, by warp w of n_warps: four channels a lane,
// kBatch rows of loads in flight.  row(r) is a row's elements, or NULL; put(offset, a, b) as above;
// put_scale(r, 2^e).
template <int D, bool BF16, class Row, class Put, class PutScale>
__device__ __forceinline__ void emit_queries(int rows, int w, int n_warps, int lane, const Row &row, const Put &put,
                                             const PutScale &put_scale) {
    constexpr int kLanes = D / 4, kPer = 32 / kLanes, kBatch = 4;      // lanes a row, rows at a time
    const int col = (lane % kLanes) * 4, step = n_warps * kPer;
#pragma unroll 1
    for (int r0 = w * kPer + lane / kLanes; r0 < rows; r0 += kBatch * step) {
        uint2 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = r0 + k * step;
            const uint16_t *src = r < rows ? row(r) : nullptr;
            x[k] = src ? *reinterpret_cast<const uint2 *>(src + col) : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = r0 + k * step;
            const float2 p = widen_pair<BF16>(x[k].x), q = widen_pair<BF16>(x[k].y);
            float big = fmaxf(fmaxf(fabsf(p.x), fabsf(p.y)), fmaxf(fabsf(q.x), fabsf(q.y)));
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
            const int ex = operand_exp(__float_as_uint(big), kMinLogitExp);
            const float down = pow2(-ex);
            if (r >= rows) continue;
            if (col == 0) put_scale(r, pow2(ex));
            put((col / 64) * (kRows * 128) + r * 128 + ((step_of(col) ^ (r & 7)) << 4) + (col % 8) * 2,
                half2_bits(p.x * down, q.x * down), half2_bits(p.y * down, q.y * down));
        }
    }
}

// A CTA's work: up to 2 * tpt tokens of one slot's chunk from q0 on, for kv head h, over split
// `split` of n_splits of the key tiles their last token sees: tiles tile0 .. tile0 + n - 1.
struct CacheItem {
    int slot, h, q0, count, first, start;          // the slot's chunk: tokens, first row, first position
    int hg, tpt;                                   // query heads of the kv head, tokens of a query tile
    int len, tq;                                   // tokens of the slot, quantized ones
    int tile0, n;
    int end0;                                      // tiles below it concern stream 0 (stream 1: n)
    int split, n_splits, part;                     // first partial tile
    int kv_at, q_at;                               // STAGED: the slot's first staged key and query tile
    bool alternate;                                // one query tile, alternate key tiles
    bool good;
};

// Every load of the table is under way before the first check (a CTA waits for two in a row, not five).
template <bool STAGED>
__device__ __forceinline__ CacheItem cache_item(const AttendArgs &a, const int4 item, int h) {
    const int slot = min(max(item.x, 0), a.t.B - 1);
    const int first = a.t.offsets[slot], behind = a.t.offsets[slot + 1], start = a.t.starts[slot];
    const int len = a.cache.seq_len[slot];
    int kv[2] = {0, 0}, q[2] = {0, 0};
    if constexpr (STAGED) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            kv[e] = a.t.kv_tiles[slot + e];
            q[e] = a.t.q_tiles[slot + e];
        }
    }
    CacheItem w{};
    w.h = h;
    w.hg = a.Hq / a.Hkv;
    w.tpt = kRows / w.hg;
    w.slot = item.x;
    w.q0 = item.y;
    w.split = item.z & 0xffff;
    w.n_splits = item.z >> 16;
    w.part = item.w;
    w.good = w.slot >= 0 && w.slot < a.t.B && w.q0 >= 0 && w.split < w.n_splits && w.part >= 0;
    if (!w.good) return w;
    w.first = first;
    w.count = behind - first;
    w.start = start;
    w.alternate = w.count - w.q0 <= w.tpt;
    w.good = w.first >= 0 && w.count > w.q0 && w.start >= 0 && w.start <= kMaxTokens - w.count &&
             static_cast<int64_t>(w.first) + w.count <= a.t.tokens &&
             (w.n_splits == 1 ||
              w.part + static_cast<int64_t>(w.n_splits) * (w.alternate ? 1 : 2) <= a.part_tiles);
    if (!w.good) return w;
    // (positions stay below 2^31 - 1024, so a tile's tokens are 32-bit numbers)
    w.len = min(max(len, 0), kMaxTokens);
    w.tq = w.len / a.cache.R * a.cache.R;
    const int last = min(w.q0 + 2 * w.tpt, w.count);
    const int all = (min(w.start + last, w.len) + kRows - 1) / kRows;
    const int share = all / w.n_splits, extra = all % w.n_splits;      // the first splits take a tile more
    w.tile0 = share * w.split + min(w.split, extra);
    w.n = share + (w.split < extra);
    w.end0 = w.n;
    if (!w.alternate)
        w.end0 = max(0, min(w.n, (min(w.start + w.q0 + w.tpt, w.len) + kRows - 1) / kRows - w.tile0));
    if constexpr (STAGED) {
        w.kv_at = kv[0];
        w.q_at = q[0];
        w.good = kv[0] >= 0 && kv[0] <= a.t.n_kv_tiles && kv[0] + w.tile0 + w.n <= kv[1] && kv[1] <= a.t.n_kv_tiles &&
                 q[0] >= 0 && q[0] <= a.t.n_q_tiles && q[0] + (w.count + w.tpt - 1) / w.tpt <= q[1] &&
                 q[1] <= a.t.n_q_tiles;
    }
    return w;
}

// The CTA's barriers; kPFull: [half of the tile's tokens][stream].
enum { kQFull = 0, kKFull = 1, kVFull = kKFull + kStages, kKEmpty = kVFull + kStages, kVEmpty = kKEmpty + kStages,
       kSFull = kVEmpty + kStages, kPFull = kSFull + 2, kOFull = kPFull + 4, kDrain = kOFull + 2, kBars };

// queries, filled, weighed: arrivals that fill the queries, a tile's keys or values, half its weights
__device__ __forceinline__ void init_bars(uint32_t bars, int queries, int filled, int weighed) {
    for (int i = 0; i < kBars; ++i)
        tc::bar_init(bars + 8u * i,
                     i == kQFull ? queries : i < kKEmpty ? filled : i >= kPFull && i < kPFull + 4 ? weighed : 1);
    tc::fence_barrier_init();
}

// Tensor memory (512 columns): S0 | S1 | O0 | O1, P over the first half of its S.

// Issues the CTA's MMAs (a whole warp).  WIDE: unrolled, for the kernel whose other code is small.
template <int D, bool WIDE, class L>
__device__ __forceinline__ void mma_role(const CacheItem &work, uint32_t base, uint32_t tmem, volatile int &gave_up) {
    const uint32_t bars = base + L::bars;
    auto bar = [&](int i) { return bars + 8u * i; };
    const uint32_t leader = tc::elect_leader();
    const int n = work.n;
    const bool alternate = work.alternate;
    const int stride = alternate ? 2 : 1;          // of a stream's tiles
    constexpr uint32_t kDescS = tc::mma_desc(kRows, kRows, false, false);
    constexpr uint32_t kDescO = tc::mma_desc(kRows, D, false, false);
    auto issue_s = [&](int t, int s) {
        uint32_t qa = base + L::q + (alternate ? 0 : t) * L::kTileBytes, ka = base + L::k + s * L::kTileBytes;
#pragma unroll(WIDE ? D / 64 : 1)
        for (int i = 0; i < D / 64; ++i, qa += kRows * 128, ka += kRows * 128)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                tc::mma_ss(tmem + t * 128, tc::desc_k_major(qa + 32 * k), tc::desc_k_major(ka + 32 * k), kDescS, i + k > 0, leader);
        tc::mma_commit(bar(kSFull + t), leader);
    };
    bool go = tc::bar_wait_warp(bar(kQFull), 0, &gave_up);
#pragma unroll 1
    for (int t = 0; t < 2 && go; ++t) {
        const int j = alternate ? t : 0;   // the stream's first tile
        if (j < (t ? n : work.end0)) {
            go = tc::bar_wait_warp(bar(kKFull + j % kStages), (j / kStages) & 1, &gave_up);
            if (go) issue_s(t, j % kStages);
        }
        if (go && (alternate ? j < n : t == 1)) tc::mma_commit(bar(kKEmpty + j % kStages), leader);
    }
    for (int j = 0; j < n && go; ++j) {
        const int s = j % kStages, next = j + stride, s1 = next % kStages;
        go = tc::bar_wait_warp(bar(kVFull + s), (j / kStages) & 1, &gave_up);
#pragma unroll(WIDE ? 2 : 1)
        for (int t = 0; t < 2 && go; ++t) {
            if (j >= (t ? n : work.end0) || (alternate && (j & 1) != t)) continue;
            const int i = alternate ? j / 2 : j;       // how many tiles the stream has had
            const uint32_t va = base + L::v + s * L::kTileBytes;
#pragma unroll(WIDE ? 2 : 1)
            for (int half = 0; half < 2; ++half) {         // the first weights while the others are taken
                go = tc::bar_wait_warp(bar(kPFull + 2 * half + t), i & 1, &gave_up);
                if (!go) break;
                tc::fence_after_sync();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_ts(tmem + 256 + t * 128, tmem + t * 128 + 32 * half + 8 * k,
                               tc::desc_k_major(va + half * (D * 128) + k * 32), kDescO, i > 0 || half > 0 || k > 0, leader);
            }
            if (!go) break;
            if (next < (t ? n : work.end0)) {
                go = tc::bar_wait_warp(bar(kKFull + s1), (next / kStages) & 1, &gave_up);
                if (go) issue_s(t, s1);
            } else {
                tc::mma_commit(bar(kOFull + t), leader);
            }
        }
        if (go) {
            tc::mma_commit(bar(kVEmpty + s), leader);
            if (next < n) tc::mma_commit(bar(kKEmpty + s1), leader);
        }
    }
    // MMAs in flight end before tensor memory is freed
    tc::mma_commit(bar(kDrain), leader);
    tc::bar_drain(bar(kDrain), 0);
}

// The softmax of one query row a thread, warps 0-3 for stream 0, 4-7 for stream 1; then the row's
// output, or its part of it.  WHOLE: a row's 128 logits are held in registers at once; else they are
// read twice, 32 at a time, by rolled loops, and the rows are at most 32, of warps 0 and 4.
template <int D, bool BF16, bool WHOLE, class L>
__device__ __forceinline__ void softmax_role(const AttendArgs &a, const CacheItem &work, const TileExps *exps,
                                             unsigned char *smem, uint32_t base, uint32_t tmem, int warp, int lane,
                                             volatile int &gave_up) {
    const uint32_t bars = base + L::bars;
    auto bar = [&](int i) { return bars + 8u * i; };
    const float *row_scale = reinterpret_cast<const float *>(smem + L::row_scale);
    const int t = warp >> 2, r = threadIdx.x & 127;
    const bool alternate = work.alternate;
    const int qt = alternate ? 0 : t;          // the query tile
    // tokens row r sees, from tile0 on; a warp without rows only keeps step
    int seen0;
    bool mine, any;
    {
        const int hg = work.hg, tok = work.q0 + qt * work.tpt + r / hg;
        mine = r < hg * work.tpt && tok < work.count;
        any = __any_sync(0xffffffffu, mine);
        seen0 = min(work.start + tok + 1, work.len) - work.tile0 * kRows;
    }
    const int seen_least = __reduce_min_sync(0xffffffffu, mine ? seen0 : 0x7fffffff);
    const int stride = alternate ? 2 : 1, n = work.n;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
    // weights are 2^(y - m) with sum l; O holds the sums of 2^(y - m) v 2^-e_ref
    float m = kNoMax, l = 0.0f, row_s = 0.0f, e_ref = kMinExp;
    bool go = n == 0 || tc::bar_wait_warp(bar(kQFull), 0, &gave_up);
    if (go && n > 0) row_s = row_scale[qt * kRows + r] * a.scale;
    const int end = t == 0 ? work.end0 : n;
    int i = 0;                                 // tiles this stream has had
    for (int j = alternate ? t : 0; j < end && go; j += stride, ++i) {
        go = tc::bar_wait_warp(bar(kSFull + t), i & 1, &gave_up);
        if (!go) break;
        tc::fence_after_sync();
        if (any) {
            const float *scales = exps[j % kExps].scale_k;
            const int seen = seen0 - j * kRows;
            const bool masked = seen_least < (j + 1) * kRows;
            // the tile's columns from 32 k on; column e is token token_of(e)
            auto logits = [&](int k, uint32_t(&x)[32]) {
                tc::tmem_arrived(x);
                if (masked) {
                    const int past = seen - 64 * (k / 2) - 8 * (k % 2);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (token_of(e) >= past) x[e] = 0xff800000u;
                }
            };
            // 16 columns from 32 k + 16 g on are of one unit
            auto unit = [&](int k, int g) { return 2 * (k / 2) + g; };
            float big[kUnits] = {kNoMax, kNoMax, kNoMax, kNoMax};      // the units' largest logits
            auto largest = [&](int k, const uint32_t(&x)[32]) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float m2[2] = {__uint_as_float(x[16 * g]), __uint_as_float(x[16 * g + 1])};
#pragma unroll
                    for (int e = 2; e < 16; ++e) m2[e % 2] = fmaxf(m2[e % 2], __uint_as_float(x[16 * g + e]));
                    const float y = fmaxf(m2[0], m2[1]) * (row_s * scales[unit(k, g)]);
                    if constexpr (WHOLE) {
                        if (k < 2) big[g] = fmaxf(big[g], y);
                        else big[2 + g] = fmaxf(big[2 + g], y);
                    } else {                       // (rolled: no branch)
                        big[g] = fmaxf(big[g], k < 2 ? y : kNoMax);
                        big[2 + g] = fmaxf(big[2 + g], k < 2 ? kNoMax : y);
                    }
                }
            };
            constexpr int kHeld = WHOLE ? 4 : 1;
            uint32_t x[kHeld][32];
            if constexpr (WHOLE) {
#pragma unroll
                for (int k = 0; k < 4; ++k) tc::tmem_load(ts + 32 * k, x[k]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    logits(k, x[k]);
                    largest(k, x[k]);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    tc::tmem_load(ts + 32 * k, x[0]);
                    logits(k, x[0]);
                    largest(k, x[0]);
                }
            }
            if constexpr (!WHOLE) {                // the values' powers come with the values
                go = tc::bar_wait_warp(bar(kVFull + j % kStages), (j / kStages) & 1, &gave_up);
                if (!go) break;
            }
            const float *evs = exps[j % kExps].exp_v;
            const float mx = fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));
            const bool far = fabsf(mx) > kFarLogit && mx > kNoMax;
            // the row's largest weight, times 2^ev, where weights are 2^(y - from)
            auto share = [&](float from) {
                return fmaxf(fmaxf(big[0] - from + evs[0], big[1] - from + evs[1]),
                             fmaxf(big[2] - from + evs[2], big[3] - from + evs[3]));
            };
            auto level = [&] { return evs[0] == e_ref && evs[1] == e_ref && evs[2] == e_ref && evs[3] == e_ref; };
            bool careful = false, even = __all_sync(0xffffffffu, level());
            if (i == 0 || __any_sync(0xffffffffu, fmaxf(mx - m, even ? kNoMax : share(m) - e_ref) > kTopWeight + kLazyMax || far)) {
                careful = __any_sync(0xffffffffu, far);
                const float mn = fmaxf(m, mx - kTopWeight), down = m - mn;
                // in steps of the values' own exponents, so that it comes to equal them
                const float er = fmaxf(rintf(fmaxf(down + e_ref, share(mn) - kTopWeight) * (1.0f / kValueStep)) * kValueStep,
                                       kMinExp);
                const float alpha_o = tc::ex2(down + (e_ref - er));
                m = mn;
                l *= tc::ex2(down);
                e_ref = er;
                even = __all_sync(0xffffffffu, level());
                // O holds every tile of the stream before j: S_j was committed after its last MMA
#pragma unroll 1
                for (int cc = i == 0 ? D / 32 : 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    tc::tmem_load(to + 32 * cc, o);
                    tc::tmem_arrived(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha_o);
                    tc::tmem_store(to + 32 * cc, o);
                }
            }
            float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            // the weights of 32 columns, packed, take the place of their first logits
            auto weights = [&](int k, uint32_t(&x)[32], uint32_t *p) {
                if (careful)
#pragma unroll
                    for (int g = 0; g < 2; ++g) subtract_rounded<16>(&x[16 * g], row_s * scales[unit(k, g)], m);
                const float from = careful ? 0.0f : m;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float sc = careful ? 1.0f : row_s * scales[unit(k, g)];
                    const float down = even ? 1.0f : tc::ex2(fminf(evs[unit(k, g)] - e_ref, 126.0f));
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t *y = &x[16 * g + 2 * e];
                        const float2 z = tc::fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])),
                                                  make_float2(sc, sc), make_float2(-from, -from));
                        float2 wt = make_float2(tc::ex2(z.x), tc::ex2(z.y));
                        l2[e % 2] = tc::add2(l2[e % 2], wt);
                        if (!even) wt = tc::mul2(wt, make_float2(down, down));
                        p[8 * g + e] = half2_bits(wt.x, wt.y);
                    }
                }
            };
            auto handed = [&](int half) {
                tc::tmem_stored();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::bar_arrive(bar(kPFull + 2 * half + t));
            };
            if constexpr (WHOLE) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t(&p)[32] = x[2 * half];
                    weights(2 * half, x[2 * half], p);
                    weights(2 * half + 1, x[2 * half + 1], p + 16);
                    tc::tmem_store(ts + 32 * half, p);         // over logits that have been read
                    handed(half);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    uint32_t p[16];
                    tc::tmem_load(ts + 32 * k, x[0]);
                    logits(k, x[0]);
                    weights(k, x[0], p);
                    tc::tmem_store16(ts + 16 * k, p);
                    if (k & 1) handed(k / 2);
                }
            }
            l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
        } else {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                tc::bar_arrive(bar(kPFull + t));
                tc::bar_arrive(bar(kPFull + 2 + t));
            }
        }
    }
    const bool had = i > 0;                    // O holds something
    const int h = work.h, first = work.first, split = work.split, n_splits = work.n_splits, hg = work.hg;
    const int tok = work.q0 + qt * work.tpt + r / hg;
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
                // divided by its own sum of weights: a sum of large values may pass the range of fp32
                const float inv = l > 0.0f ? __fdividef(1.0f, l) : 0.0f, up = tc::ex2(e_ref);
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    if (had) {
                        tc::tmem_load(to + 32 * cc, o);
                        tc::tmem_arrived(o);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        ox[(32 * cc + e) * kRows + r] = had ? __uint_as_float(o[e]) * inv * up : 0.0f;
                }
            }
        }
        if constexpr (WHOLE) asm volatile("bar.sync 2, 256;" ::: "memory");
        else asm volatile("bar.sync 2, 64;" ::: "memory");
        if (t == 0 && any && go) {
            tc::fence_after_sync();
            const float m1 = ml[r], l1 = ml[kRows + r];
            const float mn = fmaxf(m, m1), w0 = tc::ex2(m - mn), w1 = tc::ex2(m1 - mn);
            const float sum = l * w0 + l1 * w1, inv = sum > 0.0f ? __fdividef(1.0f, sum) : 0.0f;
            const float f0 = w0 * inv, f1 = l1 * w1 * inv, up = tc::ex2(e_ref);
            uint16_t *out = a.o.p + static_cast<int64_t>(first + tok) * a.o.ts +
                            static_cast<int64_t>(h * hg + r % hg) * a.o.hs;
            const int64_t tile = (static_cast<int64_t>(work.part) + split) * a.Hkv + h;
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
                        y[k] = (had ? __uint_as_float(o[e + k]) * f0 * up : 0.0f) + ox[(32 * cc + e + k) * kRows + r] * f1;
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
        const float inv = l > 0.0f ? __fdividef(1.0f, l) : 0.0f, up = tc::ex2(e_ref);
        uint16_t *out = a.o.p + static_cast<int64_t>(first + tok) * a.o.ts +
                        static_cast<int64_t>(h * hg + r % hg) * a.o.hs;
        const int64_t tile = (static_cast<int64_t>(work.part) + 2 * split + t) * a.Hkv + h;
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
                for (int k = 0; k < 8; ++k) y[k] = had ? __uint_as_float(o[e + k]) * inv * up : 0.0f;
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

}  // namespace
}  // namespace kvq
