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
// of it; bf16 and fp16 values are three such terms exactly, down to 2^-32 of
// the row's largest (the row is scaled by a power of two that brings that to
// 2^14), so that nothing of the query is rounded.
//
// V is turned into fp16, exactly, by four warps on the way to the second
// product; weights are fp16 as in an fp16 call there.
//
// A block of 32 nodes has a power of two for keys, 2^ek, which multiplies its
// scores, and one for values, 2^ev, which is added to the exponent of its
// weights: with the running maximum m of s + ev a weight is 2^(s + ev - m), the
// sum takes it times 2^-ev, and no value is multiplied.
//
// A thread has a row and goes through its part of a tile 32 nodes at a time,
// once: m is a whole number and trails the maximum by at most 2^8 in the
// weights; when a score exceeds that, O, the sum and the weights of the tile
// so far are multiplied by a power of two.
#pragma once

#include "k2t_attn.cuh"
#include "k2t_attn_fwd.cuh"
#include "k2t_cache.cuh"

namespace k2t {

struct CachedParams : AttnParams {
    uint32_t pitch;                       // bytes of a cached row
    uint64_t scale_pitch, cached;         // of a head's scales; nodes of the cache
    const uint8_t *kc, *vc, *ks, *vs;
};

// Warps: 0-7 softmax, 8-11 hops -> bucket bytes, 12-15 states -> slots, 16-19 values -> fp16, 20 products.
constexpr int kCachedThreads = 672;
constexpr float kCachedUp = 7.0f;         // weights are at most 2^(8 + 7)

template <int DP> struct CachedSmem {
    static constexpr int kTile = kTcTile * 128;               // 128 rows of 128 bytes
    static constexpr int kKeys = DP == 64 ? 4 : 3;            // slots of keys, of values, of values in fp16
    static constexpr int kValues = DP == 64 ? 4 : 2;
    static constexpr int kWide = DP == 64 ? 3 : 2;
    static constexpr int kBufs = DP == 64 ? 4 : 3;            // bucket tiles
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
        uint32_t tmem, gave_up, columns, all;
        uint32_t seen[kBufs][4];
        float row_scale[128];             // what multiplies a row's scores
        uint8_t byte_of[257 + 15];
    };
    static constexpr int kLut = kCtl + (int)((sizeof(Ctl) + 15) / 16 * 16);
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

// Byte offset of chunk c of row r in a slot of values: odd rows of 128 bytes have their halves exchanged, so that the eight
// lanes that read four chunks of two rows meet no bank twice.
template <int DP> __device__ __forceinline__ uint32_t value_chunk(uint32_t r, uint32_t c) { return r * DP + (DP == 128 ? c ^ (r & 1) << 2 : c) * 16; }

// States of a tile's seen nodes -> slots, keys then values; this warp brings nodes [32 cw, 32 cw + 32).
template <int DP, typename Ctl>
__device__ __forceinline__ void cached_node_warps(const CachedParams &p, Ctl *ctl, uint32_t sm, int cw, int lane, uint32_t hk,
                                                  uint32_t tiles, uint32_t split, volatile uint32_t *gave_up)
{
    using S = CachedSmem<DP>;
    constexpr int C = DP / 16, RP = 32 / C;                    // chunks of 16 bytes a row, rows a pass
    constexpr int kTurn = 8 / RP;                              // passes until the key slots' swizzle repeats
    const uint32_t c = lane % C, r0 = cw * 32 + lane / C, chunks = p.pitch / 16, fill = (chunks + 1) & ~1u;
    uint32_t k_at[kTurn];
#pragma unroll
    for (int k = 0; k < kTurn; ++k) k_at[k] = sm + S::kK + (r0 + k * RP) * 128 + ((c ^ ((r0 + k * RP) & 7)) << 4) - k * RP * 128;
    const uint32_t v_at = sm + S::kV + value_chunk<DP>(r0, c);   // RP is even: the same for all of a lane's rows
    const uint64_t first = (uint64_t)hk * p.cached * p.pitch + ((uint64_t)split * kTcTile + r0) * p.pitch + c * 16;
    const uint32_t step = RP * p.pitch;
    const uint64_t stride = (uint64_t)p.splits * kTcTile * p.pitch;
    const uint8_t *kc = p.kc + first, *vc = p.vc + first;
    bool ok = true;
    for (uint32_t i = 0; i < tiles && ok; ++i, kc += stride, vc += stride) {
        const uint32_t buf = i % S::kBufs, ks = i % S::kKeys, vs = i % S::kValues;
        ok = __all_sync(~0u, tc::bar_wait(&ctl->hop_full[buf], (i / S::kBufs) & 1, gave_up));
        if (!ok) break;
        // a node that no query sees, or past n, or a chunk past the row: zeros, and nothing is read
        const uint32_t seen = c < chunks ? ctl->seen[buf][cw] >> (lane / C) : 0;
        if (i >= S::kKeys) ok = __all_sync(~0u, tc::bar_wait(&ctl->k_empty[ks], (i / S::kKeys - 1) & 1, gave_up));
        if (!ok) break;
        if (c < fill) {
#pragma unroll
            for (int k = 0; k < 32 / RP; ++k) cp16(k_at[k % kTurn] + ks * S::kTile + k * RP * 128, kc + k * step, seen >> (k * RP) & 1 ? 16 : 0);
        }
        tc::cp_arrive(&ctl->k_full[ks]);
        if (i >= S::kValues) ok = __all_sync(~0u, tc::bar_wait(&ctl->v_empty[vs], (i / S::kValues - 1) & 1, gave_up));
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 32 / RP; ++k) cp16(v_at + vs * S::kValueSlot + k * RP * DP, vc + k * step, seen >> (k * RP) & 1 ? 16 : 0);
        tc::cp_arrive(&ctl->v_full[vs]);
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
    for (int i = tid; i < 128 * 8; i += kCachedThreads) {        // whole warps: the count is a multiple of 32
        const uint32_t l = i / 8;
        const float scale = query_terms_of<T>(p, row0 + l % KW, i % 8, hk, smem + S::kQ, S::kTile, l);
        if (i % 8 == 0) ctl->row_scale[l] = scale;
    }
}

template <typename T, int DP, int KW>
__global__ void __launch_bounds__(kCachedThreads, 1) attn_cached_kernel(const __grid_constant__ CachedParams p)
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
    if (warp == 20) tc::alloc(&ctl->tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < S::kKeys; ++i) tc::bar_init(&ctl->k_full[i], 128), tc::bar_init(&ctl->k_empty[i], 1);
        for (int i = 0; i < S::kValues; ++i) tc::bar_init(&ctl->v_full[i], 128), tc::bar_init(&ctl->v_empty[i], 4);
        for (int i = 0; i < S::kWide; ++i) tc::bar_init(&ctl->w_full[i], 4), tc::bar_init(&ctl->w_empty[i], 1);
        for (int i = 0; i < S::kBufs; ++i) tc::bar_init(&ctl->hop_full[i], 4), tc::bar_init(&ctl->hop_empty[i], 4);
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(&ctl->s_full[i], 1);
            tc::bar_init(&ctl->p_full[i], 128);
            tc::bar_init(&ctl->o_full[i], 1);
        }
        tc::bar_init(&ctl->drained, 1);
        ctl->gave_up = ctl->columns = ctl->all = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (p.sources)
        for (int i = tid; i < 257; i += kCachedThreads) ctl->byte_of[i] = i ? p.bucket_of[i - 1] + 1 : 0;
    tc::grid_wait();
    fill_bias<T>(lut, p, hk, tid, p.group2);
    query_terms<T, DP, KW>(p, ctl, smem, tid, row0, hk);
    tc::fence_async();
    __syncthreads();
    if (p.sources)
        for (int i = tid; i < KW; i += kCachedThreads)
            if (row0 + i < p.rows) {
                const uint32_t c = row_column(p, row0 + i);
                if (c < p.sources) atomicOr(&ctl->columns, 1u << c);
                else ctl->all = 1;
            }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    tc::grid_next();
    const uint32_t tm = ctl->tmem;                       // S of group w at w * 128, O at 256 + w * DP
    volatile uint32_t *gave_up = &ctl->gave_up;

    if (warp >= 8 && warp < 12) {
        hop_warps<S::kBufs>(p, ctl, smem + S::kBuckets, warp - 8, lane, tiles, split, gave_up);
    } else if (warp >= 12 && warp < 16) {
        cached_node_warps<DP>(p, ctl, sm, warp - 12, lane, hk, tiles, split, gave_up);
    } else if (warp >= 16 && warp < 20) {
        widen_warps<DP>(ctl, smem, tid - 16 * 32, tiles, gave_up);
    } else if (warp == 20) {
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
                tc::mma_ts(lead, tm + 256 + w * DP, tm + w * 128 + (kk >> 1) * 32 + (kk & 1) * 8, v, kk * 2048, id_o, done > 1 || kk > 0);
            tc::commit(lead, &ctl->w_empty[slot]);
            if (done + 2 >= tiles) tc::commit(lead, &ctl->o_full[w]);
            else ok = scores(done + 2);
        }
        if (done != tiles) tc::drain(lead, &ctl->drained, 0);
        __syncwarp();
    } else {
        // ---- softmax: a thread has a lane of tensor memory, and of every other tile its copy's nodes ----
        const int w = warp >> 2, l = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // lane field of this warp's tensor memory
        const uint32_t row = row0 + l % KW;
        const int copy = l / KW, key0 = copy * KW;                    // this thread's part of a tile
        const uint32_t col = row < p.rows ? row_column(p, row) : 0;
        const uint32_t G = p.group, shift = p.group2_log + 2;
        const uint32_t lg = lut_at | (row < p.rows ? row % G : 0) * 4;
        const uint32_t s_at = tm + lanes + w * 128, o_at = tm + lanes + 256 + w * DP;
        const uint8_t *bt0 = smem + S::kBuckets + col * kTcPitch + key0;
        const float row_scale = ctl->row_scale[l];
        const uint8_t *ks = p.ks + hk * p.scale_pitch, *vs = p.vs + hk * p.scale_pitch;
        float m = -INFINITY;
        LongSum sum;
        bool ok = true;
        uint32_t mine = 0;                                            // tiles of this group done
        uint32_t kb = 0, vb = 0;                                      // the next tile's scale bytes
        auto scales = [&](uint32_t i) {
            if (i < tiles) {
                kb = __ldg(reinterpret_cast<const uint32_t *>(ks + tile_at(i) * 4));
                vb = __ldg(reinterpret_cast<const uint32_t *>(vs + tile_at(i) * 4));
            }
        };
        scales(w);
        for (uint32_t i = w; i < tiles; i += 2, ++mine) {
            const uint32_t buf = i % S::kBufs;
            const uint32_t kb0 = kb >> (copy * KW / 4), vb0 = vb >> (copy * KW / 4);
            ok = tc::bar_wait(&ctl->hop_full[buf], (i / S::kBufs) & 1, gave_up) && tc::bar_wait(&ctl->s_full[w], mine & 1, gave_up);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            scales(i + 2);
            tc::fence_after();
            const bool plain = !p.sources && (tile_at(i) + 1) * kTcTile <= p.n;   // no table, no node past the end
            const uint8_t *bt = bt0 + buf * 33 * kTcPitch;
            float tile_sum = 0.0f;
#pragma unroll 1
            for (int b = 0; b < KW; b += 32) {
                uint32_t s[32];
                tc::load(s, s_at + key0 + b);
                const float sc = row_scale * power_of_two((int)(kb0 >> (b / 4) & 255) - kScaleBias);
                const int ev = (int)(vb0 >> (b / 4) & 255) - kScaleBias;
                tc::wait_ld();
                const float top = bias_scores(s, sc, plain, bt + b, lg, shift, -INFINITY) + ev;
                const bool grow = top > m + kTcLag || (m == -INFINITY && top > -INFINITY);
                if (__any_sync(~0u, grow)) {
                    const float next = grow ? ceilf(top) : m;
                    const float f = m == -INFINITY ? 0.0f : ex2(m - next);      // m = -inf: nothing was summed yet
                    m = next;
                    sum.sum *= f, sum.rest *= f, tile_sum *= f;
                    const __half2 hf = __float2half2_rn(f);
#pragma unroll 1
                    for (int c = 0; c < b; c += 32) {                           // this tile's weights so far
                        uint32_t x[16];
                        tc::load(x, s_at + key0 + c);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x[e]), hf);
                            x[e] = *reinterpret_cast<const uint32_t *>(&y);
                        }
                        tc::store(s_at + key0 + c, x);
                    }
                    if (mine > 0) {
                        // the products issued before these scores are done, so O is at rest
#pragma unroll 1
                        for (int c = 0; c < DP; c += 16) {
                            uint32_t o[16];
                            tc::load(o, o_at + c);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc::store(o_at + c, o);
                        }
                    }
                    tc::wait_st();
                }
                // weights over the scores they come from, two a word
                float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                uint32_t out[16];
                weights<__half, 32>(out, s, m == -INFINITY ? 0.0f : m - kCachedUp - ev, part);
                tc::store(s_at + key0 + b, out);
                tile_sum = fmaf((part[0].x + part[0].y) + (part[1].x + part[1].y), power_of_two(-ev), tile_sum);
            }
            if (KW < 128) {                                           // nodes of the other copies weigh nothing
                const uint32_t zero[16] = {};
#pragma unroll
                for (int c = 0; c < 128; c += 32)
                    if (c / KW != copy) tc::store(s_at + c, zero);
            }
            tc::wait_st();
            tc::fence_before();
            tc::bar_arrive(&ctl->p_full[w]);
            __syncwarp();
            if (lane == 0) tc::bar_arrive(&ctl->hop_empty[buf]);
            sum.add(tile_sum);
        }
        // ---- join the copies and groups through the freed slots: [group][lane][DP + 4] ----
        if (ok && mine > 0) {
            ok = tc::bar_wait(&ctl->o_full[w], 0, gave_up);
            tc::fence_after();
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        ok = !*gave_up;
        constexpr int P = DP + 4;
        static_assert(256 * P * 4 <= S::kBuckets, "the exchange fits the slots and queries");
        float *ex = reinterpret_cast<float *>(smem);
        if (ok) {
            float *at = ex + (size_t)(w * 128 + l) * P;
#pragma unroll 1
            for (int c = 0; c < DP; c += 16) {
                uint32_t o[16];
                if (mine > 0) {
                    tc::load(o, o_at + c);
                    tc::wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0;
                }
#pragma unroll
                for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4 *>(at + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
            at[DP] = m - kCachedUp;
            at[DP + 1] = sum.total();
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        constexpr int kSets = 2 * (128 / KW), Q4 = DP / 4;
        if (ok)
            for (int i = tid; i < KW * Q4; i += 256) {
                const int r = i / Q4, c = (i % Q4) * 4;
                const uint32_t rw = row0 + r;
                if (rw >= p.rows || c >= (int)p.d) continue;
                const float *e0 = ex + (size_t)r * P;
                float mx = -INFINITY;
#pragma unroll
                for (int k = 0; k < kSets; ++k) mx = fmaxf(mx, e0[(size_t)k * KW * P + DP]);
                const float ux = mx == -INFINITY ? 0.0f : mx;
                float ls = 0.0f;
                float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kSets; ++k) {
                    const float *e = e0 + (size_t)k * KW * P;
                    const float f = ex2(e[DP] - ux);
                    const float4 x = *reinterpret_cast<const float4 *>(e + c);
                    ls += f * e[DP + 1];
                    acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
                }
                const uint32_t t = rw / G, hd = hk * G + rw - t * G;
                if (p.splits > 1) {
                    const uint64_t at = ((uint64_t)split * p.T + t) * p.hq + hd;
                    *reinterpret_cast<float4 *>(p.part + at * p.d + c) = acc;
                    if (c == 0) *reinterpret_cast<float2 *>(p.part_ml + at * 2) = make_float2(mx, ls);
                } else {
                    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;     // 0: nothing was seen; a row that is no number says so
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
    if (warp == 20) tc::dealloc(tm, 512);
    if (tid == 0 && *gave_up) atomicOr(p.status, K2T_STATUS_WAIT_TIMEOUT);
}

}  // namespace k2t
