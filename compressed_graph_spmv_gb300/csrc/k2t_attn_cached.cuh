// k2t_attn_cached.cuh -- hop-biased attention over the 8-bit cache of node
// states (k2t_cache.cuh) on tcgen05.
//
// The forward pass of k2t_attn_fwd.cuh with its layout: rows of all heads that
// share a key/value head, nodes of a head split over blocks, one block an SM,
// tiles of 128 nodes through rings in shared memory, S = Q K^T and O = P V in
// tensor memory, two groups of softmax threads that take alternate tiles, few
// rows repeated down the 128 lanes with a part of the nodes for each copy.
// What differs:
//
// S is a product of 8-bit operands: the cached bytes are the operand as they
// lie.  A query goes in as three e5m2 terms, each what the ones before leave
// of it; bf16 and fp16 values are three such terms exactly, down to 2^-31 of
// the row's largest (the row is scaled by a power of two that brings that to
// 2^14), so that nothing of the query is rounded.
//
// V is turned into fp16, exactly, by four warps on the way to the second
// product; weights are fp16 as in an fp16 call there.
//
// A block of 32 nodes has a power of two for keys, 2^ek, which multiplies its
// scores, and one for values, 2^ev, which is added to the exponent of its
// weights: with the running maximum m of s + ev a weight is 2^(s + ev - m), the
// sum takes it times 2^-ev, and no value is multiplied.  Where scores are so
// large that fp32 does not hold s + ev (a soft mask of -1e9 on all that a row
// sees), s and m are against an origin, a whole number near the row's scores:
// (s - origin) is exact and small, and ev is added to that.
//
// Two threads have a row, one each half of the nodes, and go through them 32 at
// a time, once: m is a whole number and trails the maximum by at most 2^8 in
// the weights; when a score exceeds that, the thread multiplies its weights of
// the tile so far by a power of two and goes on against a larger m, and at the
// tile's end both take the larger of theirs, with O and the sums.
//
// Hops are turned into bucket bytes by a kernel before, once for all heads and
// rows (30 us of the 400 below; a form where each block turned its own and a row had one thread took 37 us more).
//
// Roles of the 24 warps: 16 softmax, four V -> fp16, one brings keys, one values,
// one issues the products, in a fixed order, one copies bucket bytes.  Each slot
// of a ring is filled by one warp in order.
//
// Measured, 2^20 nodes, 4 key/value heads of 128, 32 queries of 16 heads, bf16:
// 400 us, with the hop table and the cache read once 130 us at the copy rate.
// What bounds it: the latency of a tile's steps (scores, weights, values, one
// after another in two groups) and no one unit; of about 3500 clocks a tile
// shared memory is busy 2300, the tensor cores 1280, the exponential unit 1024.
// One query term instead of three saves 5 %, so the terms stay.  1024 tokens over
// 16384 nodes: 146 us.  Origins cost 2 % of each (393 and 142 us without).
#pragma once

#include "k2t_attn.cuh"
#include "k2t_attn_fwd.cuh"
#include "k2t_cache.cuh"

namespace k2t {

struct CachedParams : AttnParams {
    uint32_t pitch;                       // bytes of a cached row
    uint64_t scale_pitch, cached;         // of a head's scales; nodes of the cache
    const uint8_t *kc, *vc, *ks, *vs;
    uint8_t *hop_tiles;                   // bucket bytes of the nodes, tile by tile: attn_hops_kernel
    uint32_t hop_tile;                    // bytes of a tile: [n_sources + 1][kTcPitch], then which nodes are seen, 4 words
};

inline uint32_t hop_tile_bytes(uint32_t sources) { return ((sources + 1) * kTcPitch + 16 + 127) / 128 * 128; }

constexpr float kCachedUp = 7.0f;         // weights are at most 2^(8 + 7)

// A row's origin: 0, and where what a larger m comes from is kCachedFar or more away from it, another whole number.  m, a
// whole number below 2^23, and m - ev are then exact.  The halves of a row take the higher of theirs: fp32 holds the
// difference wherever a weight against the other is not 0.
constexpr float kCachedFar = 0x1p22f;
__device__ __forceinline__ float origin_near(float top) { return fabsf(top) >= kCachedFar && fabsf(top) < INFINITY ? rintf(top) : 0.0f; }
// What the sums of a row are against, without its origin: a whole number near the logarithm of the sum of the weights, so
// that rounding it costs neither that sum its range nor another part of the row its share.  Returns what the sums are to be
// multiplied by for it.
__device__ __forceinline__ float without_origin(float &against, float origin, float sum)
{
    if (origin == 0.0f || sum == 0.0f) return 1.0f;
    const float all = rintf(origin + (against + log2f(sum))), f = ex2(origin - all + against);
    against = all;
    return f;
}

template <int DP> struct CachedSmem {
    static constexpr int kTile = kTcTile * 128;               // 128 rows of 128 bytes
    static constexpr int kKeys = DP == 64 ? 4 : 3;            // slots of keys, of values, of values in fp16
    static constexpr int kValues = DP == 64 ? 4 : 2;
    static constexpr int kWide = DP == 64 ? 3 : 2;
    // Warps: 0-15 softmax, then four for values -> fp16, one for keys, one for values, products, bucket bytes.
    static constexpr int kWiden = 16, kLoad = 20, kMma = kLoad + 2, kThreads = (kMma + 2) * 32;
    // Bucket tiles.  An even number, so that a buffer's tiles are all of one group, which has waited for each of them: a wait
    // for a buffer that the other group's tile was in would pass while that one's copy is still under way.
    static constexpr int kBufs = 4;
    static_assert(kBufs % 2 == 0);
    static constexpr int kValueSlot = kTcTile * DP, kWideSlot = kTile * (DP / 64);
    static constexpr int kQ = 0;                              // three terms
    static constexpr int kK = kQ + 3 * kTile;
    static constexpr int kWideAt = kK + kKeys * kTile;
    static constexpr int kV = kWideAt + kWide * kWideSlot;
    static constexpr int kBuckets = kV + kValues * kValueSlot;
    static constexpr int kCtl = kBuckets + kBufs * 33 * kTcPitch;
    struct Ctl {
        uint64_t k_full[kKeys], k_empty[kKeys], v_full[kValues], v_empty[kValues], w_full[kWide], w_empty[kWide];
        uint64_t hop_full[kBufs], hop_empty[kBufs], s_full[2], p_full[2], o_full[2], drained;
        uint32_t tmem, gave_up, far, pad;      // far: a row has, or had, an origin that is not 0
        float row_scale[128];             // what multiplies a row's scores
        float most[2][2][128];            // [group][half][lane]: a thread's origin; at votes its m, at the end what rounding added to its sum
    };
    static constexpr int kLut = kCtl + (int)((sizeof(Ctl) + 15) / 16 * 16);
    static_assert(kLut + kTcLutAlign + (K2T_ATTN_MAX_BUCKETS + 2) * K2T_ATTN_MAX_GROUP * 4 <= 232448, "every call's fits an SM");
    static size_t bytes(const AttnParams &p) { return kLut + kTcLutAlign + (size_t)(p.buckets + 2) * p.group2 * 4; }
};

// kind::f8f6f4 with fp32 accumulators, A e5m2, B e4m3, M = 128, N = n, both K-major.
__device__ __forceinline__ uint32_t idesc_e5m2_e4m3(uint32_t n) { return (1u << 4) | (1u << 7) | ((n >> 3) << 17) | ((128u >> 4) << 24); }
__device__ __forceinline__ void mma8_ss(bool lead, uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add)
{
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"((uint32_t)add), "r"((uint32_t)lead) : "memory");
}
// Two values as e5m2, to nearest even, a in the low byte.
__device__ __forceinline__ uint32_t to_e5m2(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// e5m2 is the upper half of fp16.
__device__ __forceinline__ float2 from_e5m2(uint32_t two)
{
    const uint32_t h = __byte_perm(two, 0, 0x1404);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Biases of 16 nodes, whose bucket bytes lie at shared-memory address bt: see bias_scores.
__device__ __forceinline__ void look_up(float (&bias)[16], uint32_t bt, uint32_t lg, uint32_t shift)
{
    const uint32_t mask = 255u << shift;
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(bt) : "memory");
#pragma unroll
    for (int y = 0; y < 16; y += 2) {
        const uint32_t v = w[y >> 2];
        const uint32_t i0 = (y & 3) ? v >> (16 - shift) : v << shift, i1 = (y & 3) ? v >> (24 - shift) : v >> (8 - shift);
        bias[y] = table((i0 & mask) | lg), bias[y + 1] = table((i1 & mask) | lg);
    }
}
// 16 scores of N, from `from` on, in units of log2 with them, and their maximum with `top`.
template <int N> __device__ __forceinline__ float add_bias(uint32_t (&s)[N], int from, float scale, const float (&bias)[16], float top)
{
    const float2 sc = make_float2(scale, scale);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        const float2 x = fma2(make_float2(__uint_as_float(s[from + e]), __uint_as_float(s[from + e + 1])), sc, make_float2(bias[e], bias[e + 1]));
        s[from + e] = __float_as_uint(x.x), s[from + e + 1] = __float_as_uint(x.y);
        top = max3(top, x.x, x.y);
    }
    return top;
}

// As weights() in fp16, with the sum of the weights as rounded in `kept`.  A weight is rounded to 11 bits here (y 2^13 + y takes
// the others' place and leaves), so that below fp16's normal range, where it has fewer, the sum does not follow.
template <int N>
__device__ __forceinline__ void weights_kept(uint32_t (&out)[N / 2], const uint32_t (&s)[N], float m, float2 (&sum)[2], float2 (&kept)[2])
{
    const float2 nm = make_float2(-m, -m), up = make_float2(8193.0f, 8193.0f), zero = make_float2(0.0f, 0.0f), minus = make_float2(-1.0f, -1.0f);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
        const float2 x = add2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), nm);
        const float2 y = make_float2(ex2(x.x), ex2(x.y));
        const float2 c = fma2(y, up, zero), r = fma2(fma2(y, minus, c), minus, c);
        sum[e & 1] = add2(sum[e & 1], y);
        kept[e & 1] = add2(kept[e & 1], r);
        out[e] = Elem<__half>::pack(r.x, r.y);
    }
}

// Whether any thread of the two warps that share barrier `id` says so.
__device__ __forceinline__ bool pair_any(int id, bool yes)
{
    uint32_t any;
    __syncwarp();
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.aligned.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"(id), "r"((uint32_t)yes) : "memory");
    return any;
}

// Bucket bytes of the block's tiles -> shared memory.
template <int DP, typename Ctl>
__device__ __forceinline__ void hop_copies(const CachedParams &p, Ctl *ctl, uint32_t sm, uint32_t tiles, uint32_t split, volatile uint32_t *gave_up)
{
    using S = CachedSmem<DP>;
    const bool lead = tc::elect();
    const uint32_t size = (p.sources + 1) * kTcPitch;
    const uint8_t *from = p.hop_tiles + (uint64_t)split * p.hop_tile;
    uint32_t t = 0;
    for (; t < tiles; ++t, from += (uint64_t)p.splits * p.hop_tile) {
        const uint32_t buf = t % S::kBufs;
        if (t >= S::kBufs && !__all_sync(~0u, tc::bar_wait(&ctl->hop_empty[buf], (t / S::kBufs - 1) & 1, gave_up))) break;
        if (lead) {
            const uint32_t bar = tc::saddr(&ctl->hop_full[buf]);
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(size) : "memory");
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(sm + S::kBuckets + buf * 33 * kTcPitch),
                         "l"(from), "r"(size), "r"(bar) : "memory");
        }
        __syncwarp();
    }
    if (t < tiles)         // copies in flight end before the block does
        for (uint32_t u = t < S::kBufs ? 0 : t - S::kBufs; u < t; ++u) {
            const long long start = clock64();
            while (!tc::bar_peek(&ctl->hop_full[u % S::kBufs], (u / S::kBufs) & 1) && clock64() - start < (1ll << 28)) {}
        }
}

// Byte offset of chunk c of row r in a slot of values: odd rows of 128 bytes have their halves exchanged, so that the eight
// lanes that read four chunks of two rows meet no bank twice.
template <int DP> __device__ __forceinline__ uint32_t value_chunk(uint32_t r, uint32_t c) { return r * DP + (DP == 128 ? c ^ (r & 1) << 2 : c) * 16; }

// Keys (VALUES: values) of every tile's seen nodes -> slots, by one warp: all warps a part of every tile are each held up by
// every tile's waits, and with a warp for some of the tiles one could wait for a slot's phase but one, which a barrier does
// not tell from the last.
template <int DP, int SLOTS, bool VALUES, typename Ctl>
__device__ __forceinline__ void cached_node_warp(const CachedParams &p, Ctl *ctl, uint32_t sm, int lane, uint32_t hk,
                                                 uint32_t tiles, uint32_t split, volatile uint32_t *gave_up)
{
    using S = CachedSmem<DP>;
    constexpr int C = DP / 16, RP = 32 / C, kTurn = VALUES ? 1 : 8 / RP;   // chunks of 16 bytes a row, rows a pass, passes until the swizzle repeats
    constexpr int kRow = VALUES ? DP : 128;
    const uint32_t c = lane % C, r0 = lane / C, chunks = p.pitch / 16, fill = VALUES ? C : (chunks + 1) & ~1u;
    uint64_t *full = VALUES ? ctl->v_full : ctl->k_full, *empty = VALUES ? ctl->v_empty : ctl->k_empty;
    constexpr uint32_t kSlot = VALUES ? S::kValueSlot : S::kTile;
    uint32_t to[kTurn];
#pragma unroll
    for (int k = 0; k < kTurn; ++k) {
        const uint32_t r = r0 + k * RP;         // RP is even: a lane's rows of values all have their chunk at the same place
        to[k] = VALUES ? sm + S::kV + value_chunk<DP>(r, c) : sm + S::kK + r * 128 + ((c ^ (r & 7)) << 4) - k * RP * 128;
    }
    const uint8_t *head = (VALUES ? p.vc : p.kc) + (uint64_t)hk * p.cached * p.pitch + (uint64_t)r0 * p.pitch + c * 16;
    const uint32_t step = RP * p.pitch;
    auto tile_at = [&](uint32_t i) { return split + (uint64_t)i * p.splits; };
    auto seen_of = [&](uint32_t i) {
        uint4 w = make_uint4(~0u, ~0u, ~0u, ~0u);
        if (i >= tiles) return w;
        if (p.sources) return __ldg(reinterpret_cast<const uint4 *>(p.hop_tiles + tile_at(i) * p.hop_tile + (p.sources + 1) * kTcPitch));
        const uint64_t left = p.n - tile_at(i) * kTcTile;
        if (left < kTcTile) {
            uint32_t m[4];
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) m[q] = left >= q * 32 + 32 ? ~0u : left > q * 32 ? (1u << (left - q * 32)) - 1 : 0;
            w = make_uint4(m[0], m[1], m[2], m[3]);
        }
        return w;
    };
    uint4 next = seen_of(0), after = seen_of(1);
    uint32_t slot = 0, use = 0;
    for (uint32_t i = 0; i < tiles; ++i) {
        // a node that no query sees, or past n, or a chunk past the row: zeros, and nothing is read
        uint32_t seen[4] = {next.x >> r0, next.y >> r0, next.z >> r0, next.w >> r0};
        if (c >= chunks) seen[0] = seen[1] = seen[2] = seen[3] = 0;
        next = after, after = seen_of(i + 2);
        const uint8_t *src = head + tile_at(i) * kTcTile * p.pitch;
        if (!__all_sync(~0u, !use || tc::bar_wait(&empty[slot], (use - 1) & 1, gave_up))) break;
        if (c < fill) {
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                const uint32_t bits = q == 0 ? seen[0] : q == 1 ? seen[1] : q == 2 ? seen[2] : seen[3], at = slot * kSlot + q * 32 * kRow;
#pragma unroll
                for (int k = 0; k < 32 / RP; ++k, src += step) cp16(to[k % kTurn] + at + k * RP * kRow, src, bits >> (k * RP) & 1 ? 16 : 0);
            }
        }
        tc::cp_arrive(&full[slot]);
        if (++slot == SLOTS) slot = 0, ++use;
    }
    cp_commit();
    cp_wait<0>();
}

// Values in 8 bits -> fp16 in the second product's layout; tid is 0..127.
template <int DP, typename Ctl>
__device__ __forceinline__ void widen_warps(Ctl *ctl, uint8_t *smem, int tid, uint32_t tiles, volatile uint32_t *gave_up)
{
    using S = CachedSmem<DP>;
    const uint32_t c0 = tid % 4, r0 = tid / 4;                  // four chunks of 32 rows a pass
    for (uint32_t i = 0; i < tiles; ++i) {
        const uint32_t vs = i % S::kValues, ws = i % S::kWide;
        bool ok = tc::bar_wait(&ctl->v_full[vs], (i / S::kValues) & 1, gave_up);
        if (ok && i >= S::kWide) ok = tc::bar_wait(&ctl->w_empty[ws], (i / S::kWide - 1) & 1, gave_up);
        if (!__all_sync(~0u, ok)) break;
#pragma unroll
        for (int h = 0; h < DP / 64; ++h) {                     // chunks 4 h .. 4 h + 3 are one panel
            const uint8_t *from = smem + S::kV + vs * S::kValueSlot + value_chunk<DP>(r0, c0 + 4 * h);
            uint8_t *to = smem + S::kWideAt + ws * S::kWideSlot + h * S::kTile;
            const uint32_t at0 = tc::chunk(r0, 2 * c0, 0), at1 = tc::chunk(r0, 2 * c0 + 1, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {                       // 32 rows on, the swizzle is the same
                const uint4 u = *reinterpret_cast<const uint4 *>(from + k * 32 * DP);
                *reinterpret_cast<uint4 *>(to + at0 + k * 32 * 128) =
                    make_uint4(from_e4m3(u.x & 0xffffu), from_e4m3(u.x >> 16), from_e4m3(u.y & 0xffffu), from_e4m3(u.y >> 16));
                *reinterpret_cast<uint4 *>(to + at1 + k * 32 * 128) =
                    make_uint4(from_e4m3(u.z & 0xffffu), from_e4m3(u.z >> 16), from_e4m3(u.w & 0xffffu), from_e4m3(u.w >> 16));
            }
        }
        tc::fence_async();
        __syncwarp();
        if ((tid & 31) == 0) tc::bar_arrive(&ctl->v_empty[vs]), tc::bar_arrive(&ctl->w_full[ws]);
    }
}

// Row `row` of the queries as three e5m2 terms, tiles of 128-byte rows `next` bytes apart, its row `l` of them; this thread's
// are values [16 c, 16 c + 16), and a warp's are those of four rows.  Returns what multiplies the row's scores.
template <typename T>
__device__ __forceinline__ float query_terms_of(const CachedParams &p, uint32_t row, uint32_t c, uint32_t hk, uint8_t *to, uint32_t next, uint32_t l)
{
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.0f;
    if (row < p.rows && c * 16 < p.d) {
        const uint32_t t = row / p.group, g = row - t * p.group;
        const T *src = static_cast<const T *>(p.q) + (int64_t)t * p.q_row + (int64_t)(hk * p.group + g) * p.q_head + c * 16;
        Eight<T> a;
        a.load(src);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = a.v[e];
        if (c * 16 + 8 < p.d) {
            a.load(src + 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[8 + e] = a.v[e];
        }
    }
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const uint32_t u = __float_as_uint(x[e]) & 0x7fffffffu;
        top = max(top, u < 0x7f800000u ? u : 0);
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
    const int e0 = min(max((int)(top >> 23) - 127 - 14, -112), 112);        // 2^14 <= largest < 2^15
    const float down = power_of_two(-e0);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = fmaf(x[e], down, x[e] * 0.0f);      // an infinite value becomes NaN
#pragma unroll
    for (int term = 0; term < 3; ++term) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t a = to_e5m2(x[4 * e], x[4 * e + 1]), b = to_e5m2(x[4 * e + 2], x[4 * e + 3]);
            w[e] = a | b << 16;
            const float2 y = from_e5m2(a), z = from_e5m2(b);
            x[4 * e] -= y.x, x[4 * e + 1] -= y.y, x[4 * e + 2] -= z.x, x[4 * e + 3] -= z.y;
        }
        *reinterpret_cast<uint4 *>(to + term * next + l * 128 + ((c ^ (l & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return p.scale_log2 * power_of_two(e0);
}

// Queries of a block; lane l holds row row0 + l % KW.  Eight threads a row.
template <typename T, int DP, int KW, typename Ctl>
__device__ __forceinline__ void query_terms(const CachedParams &p, Ctl *ctl, uint8_t *smem, int tid, uint32_t row0, uint32_t hk)
{
    using S = CachedSmem<DP>;
    for (int i = tid; i < 128 * 8; i += S::kThreads) {        // whole warps: the count is a multiple of 32
        const uint32_t l = i / 8;
        const float scale = query_terms_of<T>(p, row0 + l % KW, i % 8, hk, smem + S::kQ, S::kTile, l);
        if (i % 8 == 0) ctl->row_scale[l] = scale;
    }
}

template <typename T, int DP, int KW>
__global__ void __launch_bounds__(CachedSmem<DP>::kThreads, 1) attn_cached_kernel(const __grid_constant__ CachedParams p)
{
    using S = CachedSmem<DP>;
    using Ctl = typename S::Ctl;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + S::kCtl);
    const uint32_t sm = tc::saddr(smem);
    const uint32_t lut_at = (sm + S::kLut + kTcLutAlign - 1) & ~(uint32_t)(kTcLutAlign - 1);
    float *lut = reinterpret_cast<float *>(smem + (lut_at - sm));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t hk = blockIdx.y, split = blockIdx.x % p.splits;
    const uint32_t row0 = blockIdx.x / p.splits * KW;
    const uint32_t tiles = (uint32_t)(split < p.tiles ? (p.tiles - split + p.splits - 1) / p.splits : 0);
    auto tile_at = [&](uint32_t i) { return split + (uint64_t)i * p.splits; };

    // ---- set-up ----
    if (warp == S::kMma) tc::alloc(&ctl->tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < S::kKeys; ++i) tc::bar_init(&ctl->k_full[i], 32), tc::bar_init(&ctl->k_empty[i], 1);
        for (int i = 0; i < S::kValues; ++i) tc::bar_init(&ctl->v_full[i], 32), tc::bar_init(&ctl->v_empty[i], 4);
        for (int i = 0; i < S::kWide; ++i) tc::bar_init(&ctl->w_full[i], 4), tc::bar_init(&ctl->w_empty[i], 1);
        for (int i = 0; i < S::kBufs; ++i) tc::bar_init(&ctl->hop_full[i], 1), tc::bar_init(&ctl->hop_empty[i], 8);
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(&ctl->s_full[i], 1);
            tc::bar_init(&ctl->p_full[i], 8);
            tc::bar_init(&ctl->o_full[i], 1);
        }
        tc::bar_init(&ctl->drained, 1);
        ctl->gave_up = ctl->far = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc::grid_wait();
    fill_bias<T>(lut, p, hk, tid, p.group2);
    query_terms<T, DP, KW>(p, ctl, smem, tid, row0, hk);
    tc::fence_async();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    tc::grid_next();
    const uint32_t tm = ctl->tmem;                       // S of group w at w * 128, O at 256 + w * DP
    volatile uint32_t *gave_up = &ctl->gave_up;

    if (warp >= S::kWiden && warp < S::kLoad) {
        widen_warps<DP>(ctl, smem, tid - S::kWiden * 32, tiles, gave_up);
    } else if (warp == S::kLoad) {
        cached_node_warp<DP, S::kKeys, false>(p, ctl, sm, lane, hk, tiles, split, gave_up);
    } else if (warp == S::kLoad + 1) {
        cached_node_warp<DP, S::kValues, true>(p, ctl, sm, lane, hk, tiles, split, gave_up);
    } else if (warp == S::kMma + 1) {
        if (p.sources) hop_copies<DP>(p, ctl, sm, tiles, split, gave_up);
        else if (tiles && tile_at(tiles - 1) == p.tiles - 1 && p.n % kTcTile) {
            // without a table: the bytes of the last tile, which has nodes past the end
            uint8_t *bt = smem + S::kBuckets + (tiles - 1) % S::kBufs * 33 * kTcPitch;
            for (uint32_t j = lane; j < kTcTile; j += 32) bt[j] = j < p.n % kTcTile;
            __syncwarp();
            if (lane == 0) tc::bar_arrive(&ctl->hop_full[(tiles - 1) % S::kBufs]);
        }
    } else if (warp == S::kMma) {
        // ---- products: tile u belongs to group u & 1 ----
        const bool lead = tc::elect();
        const uint32_t id_s = idesc_e5m2_e4m3(kTcTile);
        const uint32_t dn = (p.d + 15) & ~15u, id_o = tc::idesc(false, dn, false, true);
        // Scores run two tiles ahead of the outputs, in a fixed order: S of tile u + 2 takes the place of the weights of tile
        // u, so that it follows their product anyway.
        auto scores = [&](uint32_t u) {
            const uint32_t slot = u % S::kKeys;
            if (!__all_sync(~0u, tc::bar_wait(&ctl->k_full[slot], (u / S::kKeys) & 1, gave_up))) return false;
            tc::fence_async();       // the copies were made by threads, the product reads through the async proxy
            tc::fence_after();
            const uint64_t k = tc::desc(sm + S::kK + slot * S::kTile, S::kTile);
#pragma unroll
            for (uint32_t term = 0; term < 3; ++term) {
                const uint64_t q = tc::desc(sm + S::kQ + term * S::kTile, S::kTile);
#pragma unroll
                for (uint32_t kk = 0; kk < DP / 32; ++kk)
                    if (kk * 32 < p.pitch) mma8_ss(lead, tm + (u & 1) * 128, q + kk * 2, k + kk * 2, id_s, term + kk > 0);
            }
            tc::commit(lead, &ctl->s_full[u & 1]);
            tc::commit(lead, &ctl->k_empty[slot]);
            return true;
        };
        bool ok = (tiles < 1 || scores(0)) && (tiles < 2 || scores(1));
        uint32_t done = 0;
        for (; ok && done < tiles; ++done) {
            const uint32_t w = done & 1, slot = done % S::kWide;
            ok = __all_sync(~0u, tc::bar_wait(&ctl->w_full[slot], (done / S::kWide) & 1, gave_up) && tc::bar_wait(&ctl->p_full[w], (done >> 1) & 1, gave_up));
            if (!ok) break;
            tc::fence_async();
            tc::fence_after();
            const uint64_t v = tc::desc(sm + S::kWideAt + slot * S::kWideSlot, S::kTile);
#pragma unroll
            for (uint32_t kk = 0; kk < kTcTile / 16; ++kk)
                tc::mma_ts(lead, tm + 256 + w * DP, tm + w * 128 + (kk >> 1) * 32 + (kk & 1) * (KW == 32 ? 16 : 8), v, kk * 2048, id_o, done > 1 || kk > 0);
            tc::commit(lead, &ctl->w_empty[slot]);
            if (done + 2 >= tiles) tc::commit(lead, &ctl->o_full[w]);
            else ok = scores(done + 2);
        }
        if (done != tiles) tc::drain(lead, &ctl->drained, 0);
        __syncwarp();
    } else {
        // ---- softmax: a thread has a lane of tensor memory, and of every other tile half of its copy's nodes ----
        // Biases are looked up while the scores are on their way, the first ones before they are there: 32 queries over 2^20
        // nodes, 8 heads of 64, 356 us, all afterwards 392 (fp16 376 and 413; with 64 rows a head of 128 277 and 287).  With
        // 128 rows a head of 128 afterwards: 400 us, early 420.
        constexpr bool kEarly = DP == 64 || KW < 128;
        constexpr int HW = KW / 2, CH = HW < 32 ? HW : 32;            // nodes of a thread's part of a tile, of them at a time
        const int w = warp >> 3, half = warp >> 2 & 1, l = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // lane field of this warp's tensor memory
        const uint32_t row = row0 + l % KW;
        const int copy = l / KW, key0 = copy * KW + half * HW;        // this thread's part of a tile
        const uint32_t col = p.sources && row < p.rows ? row_column(p, row) : 0;
        const uint32_t G = p.group, shift = p.group2_log + 2;
        const uint32_t lg = lut_at | (row < p.rows ? row % G : 0) * 4;
        const uint32_t s_at = tm + lanes + w * 128 + key0;            // the scores of its nodes
        auto o_at = [&] { return ctl->tmem + ((uint32_t)(threadIdx.x >> 5 & 3) << 21) + 256 + w * DP + (threadIdx.x >> 7 & 1) * (DP / 2); };
        const uint32_t bt0 = sm + S::kBuckets + col * kTcPitch + key0;
        const uint8_t *ks = p.ks + hk * p.scale_pitch + key0 / 32 + split * 4;
        // the tile with nodes past the end, without a table
        const uint32_t tail = !p.sources && tiles && tile_at(tiles - 1) == p.tiles - 1 && p.n % kTcTile ? tiles - 1 : ~0u;
        const int pair = w * 4 + (warp & 3) + 2;                      // barrier of the two warps that share rows
        const float row_scale = ctl->row_scale[l];
        float m = -INFINITY;                                          // both halves' alike, as is the origin
        // Origins are 0 but for very large scores: they are kept in shared memory.
        auto place = [&](int of) -> float & { return (&ctl->most[0][0][0])[threadIdx.x ^ of]; };    // of 128: the other half's
        bool shifted = false;                                         // one of the warp's is another
        place(0) = 0.0f;
        LongSum sum;
        // fp16: what rounding added to the weights.  O over the sum of the weights as they were multiplied: a row of one node is
        // that node's value, and of a few what all weights were off by cancels.  (In bf16 such a value's 4 bits survive it.)
        // It costs 32 queries over 2^20 nodes, 128 rows a head of 128, 46 us: 446, in bf16 400.
        constexpr bool kKeep = std::is_same<T, __half>::value;
        float off = 0.0f;
        bool ok = true;
        uint32_t mine = 0;                                            // tiles of this group done
        uint32_t kb = 0, vb = 0;                                      // the next tile's scale bytes
        auto scales = [&](uint32_t i) {
            if (i < tiles) {
                const uint8_t *at = ks + (uint64_t)i * p.splits * 4, *av = at + (p.vs - p.ks);
                if constexpr (HW == 64) {
                    kb = __ldg(reinterpret_cast<const uint16_t *>(at)), vb = __ldg(reinterpret_cast<const uint16_t *>(av));
                } else {
                    kb = __ldg(at), vb = __ldg(av);
                }
            }
        };
        // this tile's weights so far, [0, to) of the thread's nodes, times f
        auto scale_weights = [&](float f, int to) {
            const __half2 hf = __float2half2_rn(f);
            tc::wait_st();
#pragma unroll 1
            for (int c = 0; c < to; c += 16) {
                uint32_t x[8];
                const uint32_t at = s_at + (HW == 16 ? 0 : c / 32 * 32 + (c % 32) / 2);
                tc::ld8(x, at);
                tc::wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x[e]), hf);
                    x[e] = *reinterpret_cast<const uint32_t *>(&y);
                }
                tc::st8(at, x);
            }
        };
        scales(w);
        for (uint32_t i = w; i < tiles; i += 2, ++mine) {
            const uint32_t buf = i % S::kBufs;
            // a table, or nodes past the end; after a wait that ran out the bytes are none: they may index past the table
            bool bytes = p.sources || i == tail;
            uint32_t kb0 = kb, vb0 = vb;
            const uint32_t bt = bt0 + buf * 33 * kTcPitch;
            float bias[16];
            if constexpr (kEarly) {
                ok = !bytes || tc::bar_wait(&ctl->hop_full[buf], p.sources ? (i / S::kBufs) & 1 : 0, gave_up);
                bytes = bytes && ok;
                if (bytes) {
                    look_up(bias, bt, lg, shift);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) bias[e] = 0.0f;
                }
                ok = tc::bar_wait(&ctl->s_full[w], mine & 1, gave_up) && ok;
            } else {
                // even lanes wait for the scores, odd ones for the bucket bytes
                ok = lane & 1 ? !bytes || tc::bar_wait(&ctl->hop_full[buf], p.sources ? (i / S::kBufs) & 1 : 0, gave_up) : tc::bar_wait(&ctl->s_full[w], mine & 1, gave_up);
            }
            ok = __all_sync(~0u, ok);
            bytes = bytes && ok;
            __syncwarp();
            scales(i + 2);
            tc::fence_after();
            float tile_sum = 0.0f, tile_off = 0.0f, mt = m;                            // of this tile's weights, and what they are against
#pragma unroll 1
            for (int b = 0; b < HW; b += CH) {
                uint32_t s[CH];
                tc::load(s, s_at + b);
                if constexpr (kEarly) {
                    if (b && bytes) look_up(bias, bt + b, lg, shift);
                }
                const float sc = row_scale * power_of_two((int)(kb0 & 255) - kScaleBias);
                const int ev = (int)(vb0 & 255) - kScaleBias;
                tc::wait_ld();
                float top;
                if constexpr (kEarly) {
                    top = add_bias(s, 0, sc, bias, -INFINITY);
                    if constexpr (CH == 32) {
                        if (bytes) look_up(bias, bt + b + 16, lg, shift);
                        top = add_bias(s, 16, sc, bias, top);
                    }
                } else {
                    top = bias_scores(s, sc, !bytes, smem + (bt - sm) + b, lg, shift, -INFINITY);
                }
                float near = top + ev;
                if (__any_sync(~0u, near > mt + kTcLag || shifted)) {
                    if (shifted) near = top - place(0) + ev;
                    const bool grow = near > mt + kTcLag;             // mt = -inf: of a node that is seen
                    if (__any_sync(~0u, grow && fabsf(near) >= kCachedFar)) {
                        float to = place(0);
                        if (grow && fabsf(near) >= kCachedFar) {
                            const float by = to - origin_near(top);
                            to = origin_near(top);
                            m += by, mt += by, near = top - to + ev;
                            place(0) = to;
                            ctl->far = 1;
                        }
                        shifted = __any_sync(~0u, to != 0.0f);
                    }
                    if (shifted) {
                        const float from = place(0);
#pragma unroll
                        for (int e = 0; e < CH; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) - from);
                    }
                    const float next = grow ? ceilf(near) : mt;
                    const float f = mt == -INFINITY ? 0.0f : ex2(mt - next);    // mt = -inf: nothing was summed yet
                    mt = next;
                    tile_sum *= f, tile_off *= f;
                    scale_weights(f, b);
                }
                // weights over the scores they come from, two a word
                float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                uint32_t out[CH / 2];
                const float against = mt == -INFINITY ? 0.0f : mt - kCachedUp - ev;
                if constexpr (kKeep) {
                    float2 kept[2] = {part[0], part[1]};
                    weights_kept<CH>(out, s, against, part, kept);
                    tile_off = fmaf((kept[0].x - part[0].x + (kept[0].y - part[0].y)) + (kept[1].x - part[1].x + (kept[1].y - part[1].y)),
                                    power_of_two(-ev), tile_off);
                } else {
                    weights<__half, CH>(out, s, against, part);
                }
                tc::store(s_at + b, out);
                kb0 >>= 8, vb0 >>= 8;
                tile_sum = fmaf((part[0].x + part[0].y) + (part[1].x + part[1].y), power_of_two(-ev), tile_sum);
            }
            // After a wait that ran out the warp goes on to the vote, where both leave.
            if (pair_any(pair, !ok || mt != m)) {                     // an origin moves only where m grows
                float from = place(0);
                place(0) = mt;
                ok = !pair_any(pair, !ok);
                if (!ok) break;
                float other = place(128);
                if (__builtin_expect(pair_any(pair, from != 0.0f), 0)) {       // the higher origin of the halves that saw something
                    place(0) = from;
                    pair_any(pair, false);
                    const float theirs = place(128);
                    pair_any(pair, false);
                    float to = fmaxf(mt == -INFINITY ? -INFINITY : from, other == -INFINITY ? -INFINITY : theirs);
                    if (to == -INFINITY) to = 0.0f;
                    m += from - to, mt += from - to, other += theirs - to;
                    from = to;
                }
                place(0) = from;
                shifted = __any_sync(~0u, from != 0.0f);
                const float next = fmaxf(mt, other);
                const float f = m == -INFINITY ? 0.0f : ex2(m - next), ft = mt == -INFINITY ? 0.0f : ex2(mt - next);
                m = next;
                sum.sum *= f, sum.rest *= f, off *= f, tile_sum *= ft, tile_off *= ft;
                scale_weights(ft, HW);
                if (mine > 0) {
                    // the products issued before these scores are done, so O is at rest; each half takes half of it
#pragma unroll 1
                    for (int c = 0; c < DP / 2; c += 8) {
                        uint32_t o[8];
                        tc::ld8(o, o_at() + c);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::st8(o_at() + c, o);
                    }
                }
            }
            if (KW < 128) {                                           // nodes of the other copies' parts weigh nothing
                const uint32_t zero[HW / 2] = {};
#pragma unroll
                for (int j = 0; j < 128 / KW; ++j)
                    if (j != copy) tc::store(s_at + (j - copy) * KW, zero);
            }
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                tc::bar_arrive(&ctl->p_full[w]);
                if (p.sources) tc::bar_arrive(&ctl->hop_empty[buf]);
            }
            sum.add(tile_sum);
            off += tile_off;
        }
        // ---- join the copies and groups through the freed slots: [group][lane][DP + 4] ----
        if (ok && mine > 0) {
            ok = tc::bar_wait(&ctl->o_full[w], 0, gave_up);
            tc::fence_after();
        }
        asm volatile("bar.sync 1, 512;" ::: "memory");
        ok = !*gave_up;
        constexpr int P = DP + 4;
        static_assert(256 * P * 4 <= S::kBuckets, "the exchange fits the slots and queries");
        float *ex = reinterpret_cast<float *>(smem);
        if (ok) {
            float *at = ex + (size_t)(w * 128 + l) * P;
#pragma unroll 1
            for (int c = 0; c < DP / 2; c += 16) {
                uint32_t o[16];
                if (mine > 0) {
                    tc::load(o, o_at() + c);
                    tc::wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0;
                }
#pragma unroll
                for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4 *>(at + half * (DP / 2) + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
            if (half == 0) at[DP] = m - kCachedUp, at[DP + 3] = place(0);
            at[DP + 1 + half] = sum.total();
            if constexpr (kKeep) ctl->most[w][half][l] = off;
        }
        asm volatile("bar.sync 1, 512;" ::: "memory");
        constexpr int kSets = 2 * (128 / KW), Q4 = DP / 4;
        if (ok)
            for (int i = tid; i < KW * Q4; i += 512) {
                const int r = i / Q4, c = (i % Q4) * 4;
                const uint32_t rw = row0 + r;
                if (rw >= p.rows || c >= (int)p.d) continue;
                const float *e0 = ex + (size_t)r * P;
                float mx = -INFINITY, origin = 0.0f, of[kSets];
#pragma unroll
                for (int k = 0; k < kSets; ++k) of[k] = e0[(size_t)k * KW * P + DP], mx = fmaxf(mx, of[k]);
                if (__builtin_expect(ctl->far && mx > -INFINITY, 0)) {
                    // against the highest origin of those that saw something
                    origin = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kSets; ++k)
                        if (of[k] > -INFINITY) origin = fmaxf(origin, e0[(size_t)k * KW * P + DP + 3]);
                    mx = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kSets; ++k) of[k] += e0[(size_t)k * KW * P + DP + 3] - origin, mx = fmaxf(mx, of[k]);
                }
                const float ux = mx == -INFINITY ? 0.0f : mx;
                float ls = 0.0f, added = 0.0f;
                float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kSets; ++k) {
                    const float *e = e0 + (size_t)k * KW * P;
                    const float f = ex2(of[k] - ux);
                    const float4 x = *reinterpret_cast<const float4 *>(e + c);
                    ls += f * (e[DP + 1] + e[DP + 2]);
                    if constexpr (kKeep) {
                        const int at = k * KW + r;
                        added += f * (ctl->most[at >> 7][0][at & 127] + ctl->most[at >> 7][1][at & 127]);
                    }
                    acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
                }
                if (origin != 0.0f) {
                    const float f = without_origin(mx, origin, ls);
                    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f, ls *= f, added *= f;
                }
                const uint32_t t = rw / G, hd = hk * G + rw - t * G;
                if (p.splits > 1) {
                    const uint64_t at = ((uint64_t)split * p.T + t) * p.hq + hd;
                    if (kKeep && ls != 0.0f) {             // the parts are joined over the sums of the weights that were not rounded
                        const float f = ls / (ls + added);
                        acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
                    }
                    *reinterpret_cast<float4 *>(p.part + at * p.d + c) = acc;
                    if (c == 0) *reinterpret_cast<float2 *>(p.part_ml + at * 2) = make_float2(mx, ls);
                } else {
                    const float inv = ls == 0.0f ? 0.0f : 1.0f / (ls + added);     // 0: nothing was seen; a row that is no number says so
                    uint2 o2;
                    o2.x = Elem<T>::pack(acc.x * inv, acc.y * inv);
                    o2.y = Elem<T>::pack(acc.z * inv, acc.w * inv);
                    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (int64_t)t * p.out_row + (int64_t)hd * p.out_head + c) = o2;
                    if (c == 0) p.lse[(uint64_t)t * p.hq + hd] = ls == 0.0f ? -INFINITY : (mx + log2f(ls)) * kLn2;
                }
            }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == S::kMma) tc::dealloc(tm, 512);
    if (tid == 0 && *gave_up) atomicOr(p.status, K2T_STATUS_WAIT_TIMEOUT);
}

}  // namespace k2t
