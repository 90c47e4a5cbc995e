// k2t_attn_few.cuh -- attention over the 8-bit cache for at most 16 rows of a
// key/value head (a few queries at a time), on tcgen05 with the products
// turned round.
//
// k2t_attn_cached.cuh repeats few rows down the 128 lanes of tensor memory and
// reads every operand from shared memory for all of them: with 4 rows a head
// that traffic (S alone 96 KB a tile) and the instructions of turning values
// into fp16 take longer than the memory.  Here nodes lie along the lanes and
// rows along the columns:
//   S^T = K Q^T   (128 nodes x 16 rows)
//   O^T = V^T P   (head_dim x rows, nodes summed)
// Both products read the cached bytes as they lie, keys and values alike as
// the 8-bit A operand, and their cost goes with the few rows.  A query is
// three e5m2 terms, as there.  A weight is four e5m2 terms, each of what the
// ones before leave, 2^3 times larger, and each with columns of its own, so
// that together they hold 2^-12 of a weight and what is 2^-41 of the largest;
// the columns are put together in fp32 at the end.
//
// A thread has a node, and its warp's 32 are one block of the cache: both its
// scales are the warp's.  The reference m of a row's weights (a whole number
// that trails the maximum of s + ev by at most 2^8) is the block's: tiles are
// taken by two groups of threads in turn, and a group releases its tile's
// weights only when the one before has, so that whoever has to raise m does it
// alone: it waits for the products so far, multiplies O by powers of two and
// forms its weights again.  Whoever used the m of before does so too.
//
// What bounds it: memory.
#pragma once

#include "k2t_attn_cached.cuh"

namespace k2t {

// Warps: 0-7 softmax (two groups), 8-11 hops -> bucket bytes, 12-15 states -> slots, 16 products.
constexpr int kFewThreads = 544;
constexpr int kFewRows = 16;              // rows of the score product
constexpr int kFewTerms = 4;              // of a weight

struct FewSmem {
    static constexpr int kTile = kTcTile * 128;               // 128 rows of 128 bytes
    static constexpr int kSlots = 9, kBufs = 4;               // keys and values alternate; bucket tiles
    static constexpr int kP = kSlots * kTile;                 // weights of both groups
    static constexpr int kQ = kP + 2 * kTile;                 // three terms of 16 rows of 128 bytes
    static constexpr int kBuckets = kQ + 3 * kFewRows * 128;
    static constexpr int kCtl = kBuckets + kBufs * 33 * kTcPitch;
    struct Row { float scale; uint32_t at; };                 // what multiplies the row's scores; its column of bytes and head
    struct Ctl {
        uint64_t full[kSlots], empty[kSlots], hop_full[kBufs], hop_empty[kBufs];
        uint64_t s_full[2], s_empty[2], p_full[2], p_done[2], token[2], drained;
        uint32_t tmem, gave_up, columns, all, version, pad[3];
        uint32_t seen[kBufs][4];
        Row row[kFewRows];
        float m[2][kFewRows];             // of this version and of the one before
        float tops[4][kFewRows];
        float sums[8][kFewRows];
        uint8_t byte_of[257 + 15];
    };
    static constexpr int kLut = kCtl + (int)((sizeof(Ctl) + 15) / 16 * 16);
    static size_t bytes(const AttnParams &p) { return kLut + kTcLutAlign + (size_t)(p.buckets + 2) * p.group2 * 4; }
};

// kind::f8f6f4 with fp32 accumulators, A e4m3, B e5m2, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_e4m3_e5m2(uint32_t n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// States of a tile's seen nodes -> slots, keys then values, both in the products' 128-byte rows.
template <int C>
__device__ __forceinline__ void few_node_warps(const CachedParams &p, FewSmem::Ctl *ctl, uint32_t sm, int cw, int lane, uint32_t hk,
                                               uint32_t tiles, uint32_t split, volatile uint32_t *gave_up)
{
    using S = FewSmem;
    constexpr int RP = 32 / C, kTurn = 8 / RP;                 // rows a pass; passes until the swizzle repeats
    const uint32_t c = lane % C, r0 = cw * 32 + lane / C, chunks = p.pitch / 16, fill = (chunks + 1) & ~1u;
    uint32_t to[kTurn];
#pragma unroll
    for (int k = 0; k < kTurn; ++k) to[k] = sm + (r0 + k * RP) * 128 + ((c ^ ((r0 + k * RP) & 7)) << 4) - k * RP * 128;
    const uint64_t first = (uint64_t)hk * p.cached * p.pitch + ((uint64_t)split * kTcTile + r0) * p.pitch + c * 16;
    const uint32_t step = RP * p.pitch;
    const uint64_t stride = (uint64_t)p.splits * kTcTile * p.pitch;
    const uint8_t *kc = p.kc + first, *vc = p.vc + first;
    uint32_t slot = 0, use = 0;
    bool ok = true;
    auto bring = [&](const uint8_t *src, uint32_t seen) {
        if (use) ok = __all_sync(~0u, tc::bar_wait(&ctl->empty[slot], (use - 1) & 1, gave_up));
        if (!ok) return;
        if (c < fill) {
#pragma unroll
            for (int k = 0; k < 32 / RP; ++k) cp16(to[k % kTurn] + slot * S::kTile + k * RP * 128, src + k * step, seen >> (k * RP) & 1 ? 16 : 0);
        }
        tc::cp_arrive(&ctl->full[slot]);
        if (++slot == S::kSlots) slot = 0, ++use;
    };
    for (uint32_t i = 0; i < tiles && ok; ++i, kc += stride, vc += stride) {
        const uint32_t buf = i % S::kBufs;
        ok = __all_sync(~0u, tc::bar_wait(&ctl->hop_full[buf], (i / S::kBufs) & 1, gave_up));
        if (!ok) break;
        // a node that no query sees, or past n, or a chunk past the row: zeros, and nothing is read
        const uint32_t seen = c < chunks ? ctl->seen[buf][cw] >> (lane / C) : 0;
        bring(kc, seen);
        if (ok) bring(vc, seen);
    }
    cp_commit();
    cp_wait<0>();
}

// Whether any of a group's 128 threads says so; a barrier of theirs.
__device__ __forceinline__ bool group_any(int w, bool yes)
{
    uint32_t any;
    __syncwarp();
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.aligned.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"(w + 1), "r"((uint32_t)yes) : "memory");
    return any;
}

template <int N> __device__ __forceinline__ void load_columns(uint32_t (&r)[N], uint32_t at)
{
    if constexpr (N == 16) {
        tc::ld16(r, at);
    } else {
        uint32_t x[8];
        tc::ld8(x, at);
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = x[i];
    }
}

// T: queries, bias and outputs; NR: rows, 4, 8 or 16.
template <typename T, int NR>
__global__ void __launch_bounds__(kFewThreads, 1) attn_few_kernel(const __grid_constant__ CachedParams p)
{
    using S = FewSmem;
    extern __shared__ __align__(1024) uint8_t smem[];
    S::Ctl *ctl = reinterpret_cast<S::Ctl *>(smem + S::kCtl);
    const uint32_t sm = tc::saddr(smem);
    const uint32_t lut_at = (sm + S::kLut + kTcLutAlign - 1) & ~(uint32_t)(kTcLutAlign - 1);
    float *lut = reinterpret_cast<float *>(smem + (lut_at - sm));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t hk = blockIdx.y, split = blockIdx.x;
    const uint32_t tiles = (uint32_t)(split < p.tiles ? (p.tiles - split + p.splits - 1) / p.splits : 0);
    auto tile_at = [&](uint32_t i) { return split + (uint64_t)i * p.splits; };
    constexpr uint32_t kO = 32, kON = kFewTerms * NR;          // columns of tensor memory: S of group w at 16 w, O behind

    // ---- set-up ----
    if (warp == 16) tc::alloc(&ctl->tmem, 128);
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) tc::bar_init(&ctl->full[i], 128), tc::bar_init(&ctl->empty[i], 1);
        for (int i = 0; i < S::kBufs; ++i) tc::bar_init(&ctl->hop_full[i], 4), tc::bar_init(&ctl->hop_empty[i], 4);
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(&ctl->s_full[i], 1);
            tc::bar_init(&ctl->s_empty[i], 4);
            tc::bar_init(&ctl->p_full[i], 1);
            tc::bar_init(&ctl->p_done[i], 1);
            tc::bar_init(&ctl->token[i], 1);
        }
        tc::bar_init(&ctl->drained, 1);
        ctl->gave_up = ctl->columns = ctl->all = ctl->version = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid < kFewRows) ctl->m[0][tid] = -INFINITY;
    if (p.sources)
        for (int i = tid; i < 257; i += kFewThreads) ctl->byte_of[i] = i ? p.bucket_of[i - 1] + 1 : 0;
    tc::grid_wait();
    fill_bias<T>(lut, p, hk, tid, p.group2);
    if (warp < 4) {                                            // queries: eight threads a row, 16 values each
        const uint32_t r = tid / 8, c = tid % 8;
        const float scale = query_terms_of<T>(p, r, c, hk, smem + S::kQ, kFewRows * 128, r);
        if (c == 0) {
            const uint32_t col = r < p.rows ? row_column(p, r) : 0;
            ctl->row[r] = S::Row{scale, col * kTcPitch << 8 | (r < p.rows ? r % p.group : 0) * 4};
        }
    }
    tc::fence_async();
    __syncthreads();
    if (p.sources && tid < NR && (uint32_t)tid < p.rows) {
        const uint32_t c = row_column(p, tid);
        if (c < p.sources) atomicOr(&ctl->columns, 1u << c);
        else ctl->all = 1;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    tc::grid_next();
    const uint32_t tm = ctl->tmem;
    volatile uint32_t *gave_up = &ctl->gave_up;

    if (warp >= 8 && warp < 12) {
        hop_warps<S::kBufs>(p, ctl, smem + S::kBuckets, warp - 8, lane, tiles, split, gave_up);
    } else if (warp >= 12 && warp < 16) {
        if (p.pitch <= 64) few_node_warps<4>(p, ctl, sm, warp - 12, lane, hk, tiles, split, gave_up);
        else few_node_warps<8>(p, ctl, sm, warp - 12, lane, hk, tiles, split, gave_up);
    } else if (warp == 16) {
        // ---- products: tile u belongs to group u & 1; scores two tiles ahead of the outputs ----
        const bool lead = tc::elect();
        const uint32_t id_s = idesc_e4m3_e5m2(kFewRows, false, false), id_o = idesc_e4m3_e5m2(kON, true, true);
        auto scores = [&](uint32_t u) {
            const uint32_t w = u & 1, item = 2 * u, slot = item % S::kSlots;
            bool ok = u < 2 || tc::bar_wait(&ctl->s_empty[w], ((u >> 1) - 1) & 1, gave_up);
            ok = ok && tc::bar_wait(&ctl->full[slot], (item / S::kSlots) & 1, gave_up);
            if (!__all_sync(~0u, ok)) return false;
            tc::fence_async();       // the copies were made by threads, the product reads through the async proxy
            tc::fence_after();
            const uint64_t k = tc::desc(sm + slot * S::kTile, S::kTile);
#pragma unroll
            for (uint32_t term = 0; term < 3; ++term) {
                const uint64_t q = tc::desc(sm + S::kQ + term * kFewRows * 128, S::kTile);
#pragma unroll
                for (uint32_t kk = 0; kk < 4; ++kk)
                    if (kk * 32 < p.pitch) mma8_ss(lead, tm + w * 16, k + kk * 2, q + kk * 2, id_s, term + kk > 0);
            }
            tc::commit(lead, &ctl->s_full[w]);
            tc::commit(lead, &ctl->empty[slot]);
            return true;
        };
        bool ok = (tiles < 1 || scores(0)) && (tiles < 2 || scores(1));
        uint32_t done = 0;
        while (ok && done < tiles) {
            const uint32_t w = done & 1, item = 2 * done + 1, slot = item % S::kSlots;
            if (done + 2 < tiles) ok = scores(done + 2);
            ok = ok && tc::bar_wait(&ctl->full[slot], (item / S::kSlots) & 1, gave_up) && tc::bar_wait(&ctl->p_full[w], (done >> 1) & 1, gave_up);
            if (!__all_sync(~0u, ok)) break;
            tc::fence_async();
            tc::fence_after();
            const uint64_t v = tc::desc(sm + slot * S::kTile, S::kTile), q = tc::desc(sm + S::kP + w * S::kTile, S::kTile);
#pragma unroll
            for (uint32_t kk = 0; kk < kTcTile / 32; ++kk) mma8_ss(lead, tm + kO, v + kk * 256, q + kk * 256, id_o, done + kk > 0);
            tc::commit(lead, &ctl->empty[slot]);
            tc::commit(lead, &ctl->p_done[w]);
            ++done;
        }
        if (done != tiles) tc::drain(lead, &ctl->drained, 0);
        __syncwarp();
    } else {
        // ---- softmax: thread = node of every other tile ----
        const int w = warp >> 2, l = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // lane field of this warp's tensor memory
        const uint32_t shift = p.group2_log + 2;
        const uint8_t *ks = p.ks + hk * p.scale_pitch + (warp & 3), *vs = p.vs + hk * p.scale_pitch + (warp & 3);
        float sum[NR], rest[NR];                                      // of the weights times 2^(kCachedUp - m)
#pragma unroll
        for (int r = 0; r < NR; ++r) sum[r] = rest[r] = 0.0f;
        uint32_t version = 0, mine = 0;
        bool ok = true;
        int kb = 0, vb = 0;                                           // the next tile's scale bytes
        auto scales = [&](uint32_t i) {
            if (i < tiles) kb = __ldg(ks + tile_at(i) * 4), vb = __ldg(vs + tile_at(i) * 4);
        };
        // weights of the scores x against m, as terms into the group's part of P; sums onto `part`
        auto release = [&](const float (&x)[NR], const float *m, int ev, float (&part)[NR]) {
            uint32_t words[NR];
#pragma unroll
            for (int r = 0; r < NR; r += 4) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float ref = m[r + e];
                    y[e] = ex2(x[r + e] - (ref == -INFINITY ? 0.0f : ref - kCachedUp));
                    part[r + e] = y[e] * power_of_two(-ev);
                }
#pragma unroll
                for (int term = 0; term < kFewTerms; ++term) {
                    const uint32_t a = to_e5m2(y[0], y[1]), b = to_e5m2(y[2], y[3]);
                    words[term * (NR / 4) + r / 4] = a | b << 16;
                    const float2 c = from_e5m2(a), d = from_e5m2(b);
                    y[0] = (y[0] - c.x) * 8.0f, y[1] = (y[1] - c.y) * 8.0f, y[2] = (y[2] - d.x) * 8.0f, y[3] = (y[3] - d.y) * 8.0f;
                }
            }
            uint8_t *to = smem + S::kP + w * S::kTile + l * 128;
#pragma unroll
            for (int j = 0; j < NR / 4; ++j)
                *reinterpret_cast<uint4 *>(to + ((j ^ (l & 7)) << 4)) = make_uint4(words[4 * j], words[4 * j + 1], words[4 * j + 2], words[4 * j + 3]);
            tc::fence_async();
        };
        // the sums from one version's m to another's
        auto rescale = [&](const float *from, const float *to) {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float f = from[r] == -INFINITY ? 0.0f : ex2(from[r] - to[r]);
                sum[r] *= f, rest[r] *= f;
            }
        };
        scales(w);
        for (uint32_t i = w; i < tiles; i += 2, ++mine) {
            const uint32_t buf = i % S::kBufs;
            const int ek = kb - kScaleBias, ev = vb - kScaleBias;
            ok = tc::bar_wait(&ctl->hop_full[buf], (i / S::kBufs) & 1, gave_up) && tc::bar_wait(&ctl->s_full[w], mine & 1, gave_up);
            // after a wait that ran out the warp goes on to the group's next vote, where all leave together
            scales(i + 2);
            tc::fence_after();
            __syncwarp();
            uint32_t s[NR];
            load_columns(s, tm + lanes + w * 16);
            tc::wait_ld();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(&ctl->s_empty[w]);
            const bool plain = !p.sources && (tile_at(i) + 1) * kTcTile <= p.n;   // no table, no node past the end
            const uint8_t *bt = smem + S::kBuckets + buf * 33 * kTcPitch + l;
            const float pk = power_of_two(ek), fe = (float)ev;
            float x[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const S::Row row = ctl->row[r];
                float bias = fe;
                if (!plain) bias += table(((uint32_t)bt[row.at >> 8] << shift) | lut_at | (row.at & 255));
                x[r] = fmaf(__uint_as_float(s[r]), row.scale * pk, bias);
            }
            __syncwarp();
            if (lane == 0) tc::bar_arrive(&ctl->hop_empty[buf]);
            const float *m = ctl->m[version & 1];
            bool grow = false;
#pragma unroll
            for (int r = 0; r < NR; ++r) grow |= x[r] > m[r] + kTcLag || (m[r] == -INFINITY && x[r] > -INFINITY);
            ok = ok && (mine == 0 || tc::bar_wait(&ctl->p_done[w], (mine - 1) & 1, gave_up));        // this part of P is free
            float part[NR];
            release(x, m, ev, part);
            ok = ok && (i == 0 || tc::bar_wait(&ctl->token[w], (w ? mine : mine - 1) & 1, gave_up));
            if (group_any(w, !ok || grow || *(volatile uint32_t *)&ctl->version != version)) {
                ok = !group_any(w, !ok);
                if (!ok) break;
                const uint32_t now = *(volatile uint32_t *)&ctl->version;
                if (now != version) rescale(m, ctl->m[now & 1]);
                version = now, m = ctl->m[version & 1];
                // the tile's largest of each row
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float top = x[r];
#pragma unroll
                    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                    if (lane == 0) ctl->tops[warp & 3][r] = top;
                }
                group_any(w, false);
                bool raise = false;
                float f[NR], next[NR];
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float top = fmaxf(fmaxf(ctl->tops[0][r], ctl->tops[1][r]), fmaxf(ctl->tops[2][r], ctl->tops[3][r]));
                    const bool up = top > m[r] + kTcLag || (m[r] == -INFINITY && top > -INFINITY);
                    next[r] = up ? ceilf(top) : m[r];
                    f[r] = m[r] == -INFINITY ? 0.0f : ex2(m[r] - next[r]);
                    raise |= up;
                }
                if (raise) {                                           // the same in all of the group's threads
                    if (i > 0) {
                        ok = tc::bar_wait(&ctl->p_done[w ^ 1], ((i - 1) >> 1) & 1, gave_up);     // O is at rest
                        tc::fence_after();
                    }
                    if (group_any(w, !ok)) {
                        ok = false;
                        break;
                    }
                    if (i > 0) {
#pragma unroll 1
                        for (int term = 0; term < kFewTerms; ++term) {
                            uint32_t o[NR < 8 ? 8 : NR];              // of four rows, two terms at a time
                            const uint32_t at = tm + lanes + kO + term * NR;
                            if (NR == 4 && (term & 1)) continue;
                            load_columns(o, at);
                            tc::wait_ld();
#pragma unroll
                            for (int r = 0; r < (NR < 8 ? 8 : NR); ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r % NR]);
                            if constexpr (NR == 16) tc::store(at, o);
                            else tc::st8(at, o);
                        }
                        tc::wait_st();
                    }
#pragma unroll
                    for (int r = 0; r < NR; ++r) sum[r] *= f[r], rest[r] *= f[r];
                    ++version;
                    if (l < NR) {
                        float mine_next = next[0];
#pragma unroll
                        for (int r = 1; r < NR; ++r) mine_next = l == r ? next[r] : mine_next;
                        ctl->m[version & 1][l] = mine_next;
                    }
                    if (l == 0) ctl->version = version;
                    m = ctl->m[version & 1];
                }
                group_any(w, false);
                release(x, m, ev, part);
                tc::fence_before();
                group_any(w, false);
            }
            if (l == 0) {
                tc::bar_arrive(&ctl->p_full[w]);
                if (i + 1 < tiles) tc::bar_arrive(&ctl->token[w ^ 1]);
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {      // what an addition cuts off is kept: very many small terms count beside a large one
                const float y = part[r] + rest[r], a = sum[r] + y, back = a - sum[r];
                rest[r] = (sum[r] - (a - back)) + (y - back);
                sum[r] = a;
            }
        }
        // ---- the block's sums and O, which both groups' tiles are in ----
        for (int k = 0; k < 2 && ok; ++k) {
            const uint32_t of = (tiles + 1 - k) / 2;                  // tiles of group k
            if (of) ok = tc::bar_wait(&ctl->p_done[k], (of - 1) & 1, gave_up);
        }
        tc::fence_after();
        asm volatile("bar.sync 3, 256;" ::: "memory");
        ok = !*gave_up;
        const float *m = ctl->m[ctl->version & 1];
        if (ctl->version != version) rescale(ctl->m[version & 1], m);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float a = sum[r] + rest[r];
#pragma unroll
            for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(~0u, a, o);
            if (lane == 0) ctl->sums[warp][r] = a;
        }
        asm volatile("bar.sync 3, 256;" ::: "memory");
        if (ok && w == 0) {
            uint32_t o[kFewTerms][NR < 8 ? 8 : NR];
#pragma unroll
            for (int term = 0; term < kFewTerms; ++term) {
                if (NR == 4 && (term & 1)) continue;
                load_columns(o[term], tm + lanes + kO + term * NR);
            }
            tc::wait_ld();
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                if ((uint32_t)r >= p.rows) break;
                float acc = 0.0f, ls = 0.0f;
                if (tiles) {
#pragma unroll
                    for (int term = kFewTerms - 1; term >= 0; --term)
                        acc = fmaf(acc, 0.125f, __uint_as_float(NR == 4 ? o[term & ~1][(term & 1) * 4 + r] : o[term][r]));
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) ls += ctl->sums[k][r];
                const uint32_t t = r / p.group, hd = hk * p.group + r - t * p.group;
                const float mr = m[r] - kCachedUp;
                if (p.splits > 1) {
                    const uint64_t at = ((uint64_t)split * p.T + t) * p.hq + hd;
                    if (l < (int)p.d) p.part[at * p.d + l] = acc;
                    if (l == 0) *reinterpret_cast<float2 *>(p.part_ml + at * 2) = make_float2(mr, ls);
                } else {
                    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;     // 0: nothing was seen; a row that is no number says so
                    if (l < (int)p.d) static_cast<T *>(p.out)[(int64_t)t * p.out_row + (int64_t)hd * p.out_head + l] = Elem<T>::from_float(acc * inv);
                    if (l == 0) p.lse[(uint64_t)t * p.hq + hd] = ls == 0.0f ? -INFINITY : (mr + log2f(ls)) * kLn2;
                }
            }
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 16) tc::dealloc(tm, 128);
    if (tid == 0 && *gave_up) atomicOr(p.status, K2T_STATUS_WAIT_TIMEOUT);
}

}  // namespace k2t
