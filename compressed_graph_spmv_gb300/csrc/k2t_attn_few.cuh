// k2t_attn_few.cuh -- attention over the 8-bit cache for at most 8 rows of a
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
// three e5m2 terms, as there.  A weight is four such terms (three in a bf16
// call), each of 8 times what the one before leaves, which is where the next
// bits of a large weight are and keeps those of a small one above the least
// e5m2: they hold it to 2^-12 (2^-9), and to 2^-32 (2^-29) of the largest where
// that is more.  Each has columns of its own, which are added in fp32 at the end.
//
// A thread has four rows of a node, and its warp's 32 nodes are one block of
// the cache: both its scales are the warp's.  The reference m of a row's weights (a whole number
// that trails the maximum of s + ev by at most 2^8) is the block's: tiles are
// taken by two or three groups of threads in turn, and a group releases its tile's
// weights only when the one before has, so that whoever has to raise m does it
// alone: it waits for the products so far, multiplies O by powers of two and
// forms its weights again.  Whoever used the m of before does so too.
//
// Very large scores (see origins in k2t_attn_cached.cuh): a row with an origin
// sends its group the way of a raise with every tile.
//
// What bounds it: memory with up to 4 rows a head of 128 (2^20 nodes, 4 key/value
// heads, bf16: one query of 16 heads 161 us, where its bytes take 159 at the copy
// rate; two, which are 8 rows, 179); with heads of 64, whose tiles are half the
// bytes, and with 5 to 8 rows of them the softmax threads (8 heads, one query
// 223 us, five 312, eight 326).
#pragma once

#include "k2t_attn_cached.cuh"

namespace k2t {

// Warps: softmax (three groups of four with up to 4 rows, two of eight with up to 8), four for states -> slots, two for products.
template <int RS> struct FewPlan {
    static constexpr int kGroups = RS == 1 ? 3 : 2, kThreads = 128 * RS;     // of a group
    static constexpr int kSoft = kGroups * 4 * RS, kAll = (kSoft + 6) * 32;
};
constexpr int kFewRows = 16;              // columns of the score product, of which 8 at most are rows
// More rows go to the general kernel.  Both over 2^20 nodes, bf16: 8 rows a head of 128 179 us (2 queries, 4 heads) and 193 (8
// queries), general 231 and 234; of 64 (8 heads) 5 rows 312 us and 8 rows 326, general 335; of 32 326 and 331.  With short
// calls of 5 to 8 rows the general one is ahead: 8 queries, 8 heads of 64, 16384 nodes, 20.6 us, general 18.7.
constexpr uint32_t kFewMost = 8;
constexpr float kTermUp = 8.0f;           // a weight's term is of what the one before left, times this
constexpr int kFewHops = 258;             // masked, hops 0 .. 255, no hop information

struct FewSmem {
    static constexpr int kTile = kTcTile * 128;               // 128 rows of 128 bytes
    static constexpr int kKeys = 4, kValues = 6;              // slots: keys are done with long before values
    static constexpr int kV = kKeys * kTile;
    static constexpr int kP = kV + kValues * kTile;           // weights of the groups, 128 rows of 32 bytes
    static constexpr int kWeights = kTcTile * 32;
    static constexpr int kQ = kP + 3 * kWeights;              // three terms of 16 rows of 128 bytes
    static constexpr int kCtl = kQ + 3 * kFewRows * 128;
    struct Row { float scale; int32_t col; uint32_t head, query; }; // what multiplies the row's scores; its column of hops or -1; 4 g; t
    struct Ctl {
        uint64_t k_full[kKeys], k_empty[kKeys], v_full[kValues], v_empty[kValues];
        uint64_t s_full[3], s_empty[3], p_full[3], p_done[3], token[3], drained[2];
        uint32_t tmem, gave_up, version, pad[1];
        Row row[8];
        float m[4][8], origin[4][8];      // of this version and of the three before
        float tops[4][8];
        float sums[16][4];
    };
    static constexpr int kLut = kCtl + (int)((sizeof(Ctl) + 15) / 16 * 16);
    // Tiles of hops, [query][node]: brought when the tile kKeys before has its slots, so that the tile another kValues before is
    // done with.
    static constexpr int kHopTiles = kKeys + kValues;
    static __host__ __device__ uint32_t hops_at(const AttnParams &p) { return kLut + (kFewHops * p.group2 * 4 + 15) / 16 * 16; }
    static size_t bytes(const AttnParams &p) { return hops_at(p) + (p.sources ? kHopTiles * p.T * kTcTile * 4 : 0); }
};

// Operand rows of 32 bytes (32-byte swizzle: the chunks of rows 4 to 7 of 8 are exchanged), K along the rows.
__device__ __forceinline__ uint64_t desc32(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | (1ull << 16) | ((uint64_t)(256 >> 4) << 32) | (1ull << 46) | (6ull << 61);
}

// kind::f8f6f4 with fp32 accumulators, A e4m3, B e5m2, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_e4m3_e5m2(uint32_t n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// States of a tile's seen nodes -> slots, keys then values, both in the products' 128-byte rows; warp cw of kKeys brings the
// tiles cw, cw + kKeys, .. by itself (all warps a part of every tile were each held up by every tile's waits: 193 us for one
// query over 2^20 nodes, 4 rows a head of 128).  The hops of its next tile come first: behind a full queue of loads they take
// as long as the states.
template <int C>
__device__ __forceinline__ void few_node_warps(const CachedParams &p, FewSmem::Ctl *ctl, uint8_t *smem, uint32_t sm, int cw, int lane, uint32_t hk,
                                               uint32_t tiles, uint32_t split, volatile uint32_t *gave_up)
{
    using S = FewSmem;
    constexpr int RP = 32 / C, kTurn = 8 / RP;                 // rows a pass; passes until the swizzle repeats
    const uint32_t c = lane % C, r0 = lane / C, chunks = p.pitch / 16, fill = (chunks + 1) & ~1u;
    uint32_t to[kTurn];
#pragma unroll
    for (int k = 0; k < kTurn; ++k) to[k] = sm + (r0 + k * RP) * 128 + ((c ^ ((r0 + k * RP) & 7)) << 4) - k * RP * 128;
    const uint32_t step = RP * p.pitch;
    const uint64_t head = (uint64_t)hk * p.cached * p.pitch + (uint64_t)r0 * p.pitch + c * 16;
    bool all = !p.sources;                                     // a query that sees every node
    for (uint32_t r = 0; r < p.rows; ++r) all |= ctl->row[r].col < 0;
    const uint32_t T = p.sources ? p.T : 0, hop_tile = p.T * kTcTile * 4, hops_at = S::hops_at(p) + lane * 4;
    auto bring_hops = [&](uint32_t i) {
        if (i < tiles) {
            const uint64_t node = (split + (uint64_t)i * p.splits) * kTcTile + lane;
            const uint32_t at = sm + hops_at + i % S::kHopTiles * hop_tile;
            for (uint32_t t = 0; t < T; ++t) {
                const int32_t *src = p.hops + node * p.sources + max(ctl->row[t * p.group].col, 0);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at + (t * kTcTile + q * 32) * 4),
                                 "l"(src + q * 32 * p.sources), "r"(node + q * 32 < p.n ? 4 : 0) : "memory");
            }
        }
        cp_commit();
    };
    bring_hops(cw);
    for (uint32_t i = cw, n = 0; i < tiles; i += S::kKeys, ++n) {
        const uint64_t node = (split + (uint64_t)i * p.splits) * kTcTile;
        const uint32_t vs = i % S::kValues, v_use = i / S::kValues;
        // even lanes wait for the slot of the keys, odd ones for that of the values
        const bool ok = lane & 1 ? !v_use || tc::bar_wait(&ctl->v_empty[vs], (v_use - 1) & 1, gave_up) : !n || tc::bar_wait(&ctl->k_empty[cw], (n - 1) & 1, gave_up);
        if (!__all_sync(~0u, ok)) break;
        if (n) cp_wait<1>();                                   // this tile's hops, which came before the last one's states
        else cp_wait<0>();
        __syncwarp();
        // a node that no query sees, or past n, or a chunk past the row: zeros, and nothing is read
        uint32_t seen[4];
        int32_t most[4];                                       // the sign tells whether a query sees the node
#pragma unroll
        for (int q = 0; q < 4; ++q) most[q] = all ? 0 : -1;
        const uint8_t *hops = smem + hops_at + i % S::kHopTiles * hop_tile;
        for (uint32_t t = 0; t < T; ++t, hops += kTcTile * 4)
#pragma unroll
            for (int q = 0; q < 4; ++q) most[q] = max(most[q], *reinterpret_cast<const int32_t *>(hops + q * 32 * 4));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            seen[q] = __ballot_sync(~0u, most[q] >= 0 && node + q * 32 + lane < p.n);
            seen[q] = c < chunks ? seen[q] >> r0 : 0;
        }
        bring_hops(i + S::kKeys);
        const uint8_t *kc = p.kc + head + node * p.pitch, *vc = p.vc + head + node * p.pitch;
        if (c < fill) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int k = 0; k < 32 / RP; ++k, kc += step)
                    cp16(to[k % kTurn] + cw * S::kTile + (q * 32 + k * RP) * 128, kc, seen[q] >> (k * RP) & 1 ? 16 : 0);
        }
        tc::cp_arrive(&ctl->k_full[cw]);
        if (c < fill) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int k = 0; k < 32 / RP; ++k, vc += step)
                    cp16(to[k % kTurn] + S::kV + vs * S::kTile + (q * 32 + k * RP) * 128, vc, seen[q] >> (k * RP) & 1 ? 16 : 0);
        }
        tc::cp_arrive(&ctl->v_full[vs]);
        cp_commit();
    }
    cp_wait<0>();
}

// Whether any of a group's N threads says so; a barrier of theirs.
template <int N> __device__ __forceinline__ bool group_any(int w, bool yes)
{
    uint32_t any;
    __syncwarp();
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.aligned.pred q, %1, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"(w + 1), "r"((uint32_t)yes), "n"(N) : "memory");
    return any;
}

// T: queries, bias and outputs; up to 4 RS rows.
template <typename T, int RS>
__global__ void __launch_bounds__(FewPlan<RS>::kAll, 1) attn_few_kernel(const __grid_constant__ CachedParams p)
{
    using S = FewSmem;
    using Plan = FewPlan<RS>;
    constexpr int kTerms = std::is_same<T, __half>::value ? 4 : 3;
    constexpr uint32_t G = Plan::kGroups;
    extern __shared__ __align__(1024) uint8_t smem[];
    S::Ctl *ctl = reinterpret_cast<S::Ctl *>(smem + S::kCtl);
    const uint32_t sm = tc::saddr(smem);
    float *lut = reinterpret_cast<float *>(smem + S::kLut);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t hk = blockIdx.y, split = blockIdx.x;
    const uint32_t tiles = (uint32_t)(split < p.tiles ? (p.tiles - split + p.splits - 1) / p.splits : 0);
    auto tile_at = [&](uint32_t i) { return split + (uint64_t)i * p.splits; };
    // Columns of tensor memory: S of group w at 48 w, [term][row]: a product takes as long for 16 columns as for 48 (64 clocks,
    // its nodes' bytes), so that all terms are in one.  O behind, [row / 4][term][row % 4].
    constexpr uint32_t kSN = 3 * kFewRows, kO = 3 * kSN, kON = 16 * RS;

    // ---- set-up ----
    if (warp == Plan::kSoft + 4) tc::alloc(&ctl->tmem, 256);
    if (tid == 0) {
        for (int i = 0; i < S::kKeys; ++i) tc::bar_init(&ctl->k_full[i], 32), tc::bar_init(&ctl->k_empty[i], 1);
        for (int i = 0; i < S::kValues; ++i) tc::bar_init(&ctl->v_full[i], 32), tc::bar_init(&ctl->v_empty[i], 1);
        for (int i = 0; i < 3; ++i) {
            tc::bar_init(&ctl->s_full[i], 1);
            tc::bar_init(&ctl->s_empty[i], 4 * RS);
            tc::bar_init(&ctl->p_full[i], 1);
            tc::bar_init(&ctl->p_done[i], 1);
            tc::bar_init(&ctl->token[i], 1);
        }
        for (int i = 0; i < 2; ++i) tc::bar_init(&ctl->drained[i], 1);
        ctl->gave_up = ctl->version = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid < 8) ctl->m[0][tid] = -INFINITY, ctl->origin[0][tid] = 0.0f;
    tc::grid_wait();
    for (uint32_t i = tid; i < kFewHops * p.group2; i += Plan::kAll) {     // bias in units of log2, by hops + 1 and head
        const uint32_t b = i >> p.group2_log, g = i & (p.group2 - 1);
        float v = b ? 0.0f : -INFINITY;
        if (b && b < kFewHops - 1 && p.bias && g < p.group) {
            v = Elem<T>::to_float(static_cast<const T *>(p.bias)[(uint64_t)(hk * p.group + g) * p.buckets + p.bucket_of[b - 1]]);
            v = v <= Elem<T>::kMasked ? -INFINITY : v * kLog2e;
        }
        lut[i] = v;
    }
    if (warp < 4) {                                            // queries: eight threads a row, 16 values each
        const uint32_t r = tid / 8, c = tid % 8;
        const float scale = query_terms_of<T>(p, r, c, hk, smem + S::kQ, kFewRows * 128, r);
        if (c == 0 && r < 8) {
            const uint32_t col = r < p.rows ? row_column(p, r) : 0;
            ctl->row[r] = S::Row{scale, col < p.sources ? (int32_t)col : -1, (r < p.rows ? r % p.group : 0) * 4, r < p.rows ? r / p.group : 0};
        }
    }
    tc::fence_async();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    tc::grid_next();
    const uint32_t tm = ctl->tmem;
    volatile uint32_t *gave_up = &ctl->gave_up;

    if (warp >= Plan::kSoft && warp < Plan::kSoft + 4) {
        if (p.pitch <= 64) few_node_warps<4>(p, ctl, smem, sm, warp - Plan::kSoft, lane, hk, tiles, split, gave_up);
        else few_node_warps<8>(p, ctl, smem, sm, warp - Plan::kSoft, lane, hk, tiles, split, gave_up);
    } else if (warp == Plan::kSoft + 4) {
        // ---- scores: tile u's go to group u mod G ----
        const bool lead = tc::elect();
        const uint32_t id = idesc_e4m3_e5m2(kSN, false, false);
        uint32_t slot = 0, use = 0, u = 0, w = 0, turn = 0;
        for (; u < tiles; ++u) {
            // even lanes wait for the keys, odd ones for the group to have read its last scores
            const bool odd = lane & 1;
            const bool ok = odd ? !turn || tc::bar_wait(&ctl->s_empty[w], (turn - 1) & 1, gave_up) : tc::bar_wait(&ctl->k_full[slot], use & 1, gave_up);
            if (!__all_sync(~0u, ok)) break;
            __syncwarp();            // what one lane's wait has seen, for all of them
            tc::fence_async();       // the copies were made by threads, the product reads through the async proxy
            tc::fence_after();
            const uint64_t k = tc::desc(sm + slot * S::kTile, S::kTile);
            const uint64_t q = tc::desc(sm + S::kQ, S::kTile);
#pragma unroll
            for (uint32_t kk = 0; kk < 4; ++kk)
                if (kk * 32 < p.pitch) mma8_ss(lead, tm + w * kSN, k + kk * 2, q + kk * 2, id, kk > 0);
            tc::commit(lead, &ctl->s_full[w]);
            tc::commit(lead, &ctl->k_empty[slot]);
            if (++slot == S::kKeys) slot = 0, ++use;
            if (++w == G) w = 0, ++turn;
        }
        if (u != tiles) tc::drain(lead, &ctl->drained[0], 0);
        __syncwarp();
    } else if (warp == Plan::kSoft + 5) {
        // ---- outputs ----
        const bool lead = tc::elect();
        const uint32_t id = idesc_e4m3_e5m2(kON, true, true);
        uint32_t slot = 0, use = 0, u = 0, w = 0, turn = 0;
        for (; u < tiles; ++u) {
            const bool ok = lane & 1 ? tc::bar_wait(&ctl->p_full[w], turn & 1, gave_up) : tc::bar_wait(&ctl->v_full[slot], use & 1, gave_up);
            if (!__all_sync(~0u, ok)) break;
            __syncwarp();            // what one lane's wait has seen, for all of them
            tc::fence_async();       // the copies were made by threads, the product reads through the async proxy
            tc::fence_after();
            const uint64_t v = tc::desc(sm + S::kV + slot * S::kTile, S::kTile), q = desc32(sm + S::kP + w * S::kWeights);
#pragma unroll
            for (uint32_t kk = 0; kk < kTcTile / 32; ++kk) mma8_ss(lead, tm + kO, v + kk * 256, q + kk * 64, id, u + kk > 0);
            tc::commit(lead, &ctl->p_done[w]);
            tc::commit(lead, &ctl->v_empty[slot]);
            if (++slot == S::kValues) slot = 0, ++use;
            if (++w == G) w = 0, ++turn;
        }
        if (u != tiles) tc::drain(lead, &ctl->drained[1], 0);
        __syncwarp();
    } else {
        // ---- softmax: thread = four rows of a node of the group's tiles ----
        const int w = warp / (4 * RS), rs = warp / 4 % RS, l = (warp & 3) * 32 + lane;
        const bool first_thread = tid % Plan::kThreads == 0;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // lane field of this warp's tensor memory
        const uint32_t shift = p.group2_log + 2, o_at = tm + lanes + kO + rs * 16;
        const uint8_t *ks = p.ks + hk * p.scale_pitch + (warp & 3), *vs = p.vs + hk * p.scale_pitch + (warp & 3);
        const S::Row *rows = ctl->row + rs * 4;
        uint8_t *const p_at = smem + S::kP + w * S::kWeights + l * 32 + ((rs ^ (l >> 2 & 1)) << 4);
        float sum[4], rest[4], m[4], scale[4];                        // sums of the weights times 2^(kCachedUp - m)
        uint32_t table_at[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            sum[r] = rest[r] = 0.0f, m[r] = -INFINITY, scale[r] = rows[r].scale;
            table_at[r] = sm + S::kLut + rows[r].head;
        }
        uint32_t version = 0, mine = 0;
        bool ok = true;
        int kb = 0, vb = 0;                                           // the next tile's scale bytes
        auto ahead = [&](uint32_t i) {
            if (i < tiles) kb = __ldg(ks + tile_at(i) * 4), vb = __ldg(vs + tile_at(i) * 4);
        };
        uint32_t hop_at[4];                                           // its hops, or none
#pragma unroll
        for (int r = 0; r < 4; ++r) hop_at[r] = rows[r].col < 0 ? 0 : S::hops_at(p) + (rows[r].query * kTcTile + l) * 4;
        bool shifted = false;                                         // a row's origin is not 0: the path of a raise, with every tile
        // weights of the scores x, which are against the origins, against m, as terms into the group's part of P; sums in `part`
        auto release = [&](const float (&x)[4], int ev, float (&part)[4]) {
            uint32_t words[4] = {0, 0, 0, 0};
            float y[4];
            const float back = power_of_two(-ev), up = (float)ev + kCachedUp;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                y[r] = ex2(x[r] - (m[r] == -INFINITY ? 0.0f : m[r] - up));
                part[r] = y[r] * back;
            }
            const float2 minus = make_float2(-1.0f, -1.0f), more = make_float2(kTermUp, kTermUp), zero = make_float2(0.0f, 0.0f);
            float2 u = make_float2(y[0], y[1]), v = make_float2(y[2], y[3]);
#pragma unroll
            for (int term = 0; term < kTerms; ++term) {
                const uint32_t a = to_e5m2(u.x, u.y), b = to_e5m2(v.x, v.y);
                words[term] = a | b << 16;
                if (term + 1 == kTerms) break;
                u = fma2(fma2(from_e5m2(a), minus, u), more, zero), v = fma2(fma2(from_e5m2(b), minus, v), more, zero);
            }
            *reinterpret_cast<uint4 *>(p_at) = make_uint4(words[0], words[1], words[2], words[3]);
            tc::fence_async();
        };
        // a version's m and origins (to) in the place of this thread's, whose sums follow; f: by what
        auto adopt = [&](const float *next, const float *from, const float *to, float (&f)[4]) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                f[r] = m[r] == -INFINITY ? 0.0f : ex2(m[r] + (from[r] - to[r]) - next[r]);
                m[r] = next[r];
                sum[r] *= f[r], rest[r] *= f[r];
            }
        };
        // the group's largest of each row, after a vote of the group
        auto largest = [&](const float (&y)[4], float (&top)[4]) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float a = y[r];
#pragma unroll
                for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
                if (lane == 0) ctl->tops[warp & 3][rs * 4 + r] = a;
            }
            group_any<Plan::kThreads>(w, false);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float *t = &ctl->tops[0][rs * 4 + r];
                top[r] = fmaxf(fmaxf(t[0], t[8]), fmaxf(t[16], t[24]));
            }
        };
        ahead(w);
        for (uint32_t i = w; i < tiles; i += G, ++mine) {
            const int ek = kb - kScaleBias, ev = vb - kScaleBias;
            float x[4], part[4];
            const float pk = power_of_two(ek), fe = (float)ev;
            ahead(i + G);
            // after a wait that ran out the warp goes on to the group's next vote, where all leave together
            // even lanes wait for the scores (and the hops, which landed before the keys), odd ones for this part of P to be free
            ok = lane & 1 ? mine == 0 || tc::bar_wait(&ctl->p_done[w], (mine - 1) & 1, gave_up) : tc::bar_wait(&ctl->s_full[w], mine & 1, gave_up);
            ok = __all_sync(~0u, ok);
            __syncwarp();
            tc::fence_after();
            const uint32_t hop_tile = i % S::kHopTiles * p.T * kTcTile * 4;
            const bool in = tile_at(i) * kTcTile + l < p.n;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                uint32_t at = in ? kFewHops - 1 : 0;                  // no hop information, or masked
                if (in && hop_at[r]) at = __viaddmax_s32(min(*reinterpret_cast<const int32_t *>(smem + hop_at[r] + hop_tile), 255), 1, 0);
                x[r] = table(table_at[r] + (at << shift));
            }
            uint32_t s[3][4];
#pragma unroll
            for (int term = 0; term < 3; ++term) tc::ld4(s[term], tm + lanes + w * kSN + term * kFewRows + rs * 4);
            tc::wait_ld();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(&ctl->s_empty[w]);
            bool grow = shifted;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] = fmaf(__uint_as_float(s[0][r]) + (__uint_as_float(s[1][r]) + __uint_as_float(s[2][r])), scale[r] * pk, x[r]);
            }
            const float low = fe - kTcLag;
#pragma unroll
            for (int r = 0; r < 4; ++r) grow |= x[r] > m[r] - low;        // m = -inf: of a score that is seen
            release(x, ev, part);
            ok = ok && (i == 0 || tc::bar_wait(&ctl->token[w], (w ? mine : mine - 1) & 1, gave_up));
            if (group_any<Plan::kThreads>(w, !ok || grow || *(volatile uint32_t *)&ctl->version != version)) {
                ok = !group_any<Plan::kThreads>(w, !ok);
                if (!ok) break;
                float f[4], next[4], to[4], top[4], near[4];
                const float *from = ctl->origin[version & 3] + rs * 4;
                version = *(volatile uint32_t *)&ctl->version;
#pragma unroll
                for (int r = 0; r < 4; ++r) to[r] = ctl->origin[version & 3][rs * 4 + r];
                adopt(ctl->m[version & 3] + rs * 4, from, to, f);
#pragma unroll
                for (int r = 0; r < 4; ++r) near[r] = x[r] - to[r] + fe;
                largest(near, top);
                bool raise = false, far = false;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool up = top[r] > m[r] + kTcLag || (m[r] == -INFINITY && top[r] > -INFINITY);
                    next[r] = up ? ceilf(top[r]) : m[r];
                    raise |= up, far |= up && fabsf(top[r]) >= kCachedFar;
                }
                if (group_any<Plan::kThreads>(w, raise)) {
                    if (i > 0) {
                        ok = tc::bar_wait(&ctl->p_done[(i - 1) % G], ((i - 1) / G) & 1, gave_up);     // O is at rest
                        tc::fence_after();
                    }
                    ok = !group_any<Plan::kThreads>(w, !ok);
                    if (!ok) break;
                    if (group_any<Plan::kThreads>(w, far)) {          // other origins, near the largest scores
                        bool moved[4];
                        largest(x, top);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            moved[r] = next[r] != m[r] && fabsf(next[r]) >= kCachedFar;
                            if (moved[r]) to[r] = origin_near(top[r]);
                            near[r] = x[r] - to[r] + fe;
                        }
                        group_any<Plan::kThreads>(w, false);
                        largest(near, top);
#pragma unroll
                        for (int r = 0; r < 4; ++r) next[r] = moved[r] ? ceilf(top[r]) : next[r];
                    }
                    adopt(next, ctl->origin[version & 3] + rs * 4, to, f);
                    if (i > 0) {
                        uint32_t o[16];
                        tc::ld16(o, o_at);
                        tc::wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c & 3]);
                        tc::st16(o_at, o);
                        tc::wait_st();
                    }
                    ++version;
                    if (l < 4) {
                        ctl->m[version & 3][rs * 4 + l] = l == 0 ? next[0] : l == 1 ? next[1] : l == 2 ? next[2] : next[3];
                        ctl->origin[version & 3][rs * 4 + l] = l == 0 ? to[0] : l == 1 ? to[1] : l == 2 ? to[2] : to[3];
                    }
                    if (first_thread) ctl->version = version;
                }
                shifted = false;
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = x[r] - to[r], shifted |= to[r] != 0.0f;
                release(x, ev, part);
                tc::fence_before();
                group_any<Plan::kThreads>(w, false);
            }
            if (first_thread) {
                tc::bar_arrive(&ctl->p_full[w]);
                if (i + 1 < tiles) tc::bar_arrive(&ctl->token[w + 1 == (int)G ? 0 : w + 1]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {       // what an addition cuts off is kept: very many small terms count beside a large one
                const float y = part[r] + rest[r], a = sum[r] + y, back = a - sum[r];
                rest[r] = (sum[r] - (a - back)) + (y - back);
                sum[r] = a;
            }
        }
        // ---- the block's sums and O, which all groups' tiles are in ----
        for (uint32_t k = 0; k < G && ok; ++k) {
            const uint32_t of = (tiles + G - 1 - k) / G;              // tiles of group k
            if (of) ok = tc::bar_wait(&ctl->p_done[k], (of - 1) & 1, gave_up);
        }
        tc::fence_after();
        asm volatile("bar.sync 4, %0;" ::"n"(Plan::kSoft * 32) : "memory");
        ok = !*gave_up;
        float f[4];
        const float *origin = ctl->origin[ctl->version & 3] + rs * 4;
        adopt(ctl->m[ctl->version & 3] + rs * 4, ctl->origin[version & 3] + rs * 4, origin, f);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float a = sum[r] + rest[r];
#pragma unroll
            for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(~0u, a, o);
            if (lane == 0) ctl->sums[warp][r] = a;
        }
        asm volatile("bar.sync 4, %0;" ::"n"(Plan::kSoft * 32) : "memory");
        if (ok && w == 0) {
            uint32_t o[16];
            tc::ld16(o, o_at);
            tc::wait_ld();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t row = rs * 4 + r;
                if (row >= p.rows) break;
                float acc = 0.0f, ls = 0.0f;
                if (tiles) {
#pragma unroll
                    for (int term = kTerms - 1; term >= 0; --term) acc = fmaf(acc, 1.0f / kTermUp, __uint_as_float(o[term * 4 + r]));
                }
                for (int k = rs * 4; k < Plan::kSoft; k += 4 * RS) ls += (ctl->sums[k][r] + ctl->sums[k + 1][r]) + (ctl->sums[k + 2][r] + ctl->sums[k + 3][r]);
                const uint32_t t = row / p.group, hd = hk * p.group + row - t * p.group;
                float mr = m[r] - kCachedUp;
                const float whole = without_origin(mr, origin[r], ls);
                acc *= whole, ls *= whole;
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
    if (warp == Plan::kSoft + 4) tc::dealloc(tm, 256);
    if (tid == 0 && *gave_up) atomicOr(p.status, K2T_STATUS_WAIT_TIMEOUT);
}

}  // namespace k2t
