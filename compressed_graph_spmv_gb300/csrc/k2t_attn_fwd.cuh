// k2t_attn_fwd.cuh -- forward pass of the hop-biased attention on tcgen05.
//
// One pass over the nodes with the running maximum and sum of the softmax:
// for a tile with scores s, w = exp2(s - m), l += sum w, O += w V.  Few rows
// meet many nodes, so the nodes of a head are split over blocks (tile i goes
// to block i mod splits, which also spreads the unreached nodes that
// power-law graphs keep side by side) and attn_join_kernel joins them.
//
// One block an SM.  Tiles of 128 nodes stream through a ring of slots (keys
// and values alternate); scores S = Q K^T (128 rows x 128 nodes) and outputs
// O = P V accumulate in tensor memory, the weights P go back to it over S and
// are the A operand of the second product.  Warps:
//   0-15  two softmax groups of 256 threads, with a running maximum, sum and
//         O of their own; a row of S (lane of tensor memory) has two threads,
//         one for each half of its nodes, which agree on the maximum
//   16-19 hops of a tile -> bucket bytes, and which nodes are seen
//   20-23 states of a tile's seen nodes -> slots
//   24    issues every product
// Rows.  With more than 128 rows (TWO) the groups take two row tiles and
// share each tile of nodes; else they take alternate tiles.  With 64 or 32
// rows or fewer the rows are repeated 2 or 4 times down the 128 lanes, and
// each copy takes its own part (KW = 64 or 32 nodes) of every tile: its P is
// zero elsewhere, so its O is the sum over its part, and all threads have
// scores to work on.  The copies, the groups and the splits are joined as
// separate softmaxes at the end.
//
// The maximum a group subtracts trails the true one by at most 2^8 in the
// weights: O is rescaled (a pass over tensor memory) only when a score
// exceeds it by more than 8 in units of log2; exact in fp32, and a weight of
// 256 is no less precise in 16 bits than one of 1.  In fp16, whose least
// number is 2^-24, weights are 2^7 times larger (at most 2^15): many nodes of
// small weight beside one of 1 make up much of a row.
//
// What bounds it: memory with few rows (4 rows a head over 2^20 nodes, bf16:
// 300 us, the copy rate).  With 128 rows a head or more nothing is at its limit
// (32 queries over 2^17 nodes: DRAM 46%, issue slots 59%, tensor pipe 25%
// busy; 1024 over 16384: 8, 57 and 25%): the softmax threads wait most for
// scores on their way out of tensor memory, and a score is about 15
// instructions with its table lookup.  32 queries over 2^20 nodes 363 us,
// where the bytes take 241.
#pragma once

#include <type_traits>

#include "k2t_attn.cuh"
#include "k2t_tc.cuh"

namespace k2t {

constexpr int kTcThreads = 800;
constexpr int kTcLutAlign = 8192;   // the bias table's alignment, above its size: its address joins an index by OR
constexpr float kTcLag = 8.0f;
template <typename T> constexpr float kTcUp = std::is_same<T, __half>::value ? 7.0f : 0.0f;   // weights are 2^(s - m + kTcUp)

template <int DP, bool TWO> struct TcSmem {
    static constexpr int kPanel = kTcTile * 128;              // 64 values of 128 rows
    static constexpr int kSlot = kPanel * (DP / 64);
    static constexpr int kSlots = DP == 64 ? 8 : TWO ? 4 : 5;
    static constexpr int kBufs = DP == 64 ? 6 : 3;            // bucket tiles
    static constexpr int kQ = kSlots * kSlot;
    static constexpr int kBuckets = kQ + kSlot * (TWO ? 2 : 1);
    static constexpr int kCtl = kBuckets + kBufs * 33 * kTcPitch;
    struct Ctl {
        uint64_t full[kSlots], empty[kSlots], hop_full[kBufs], hop_empty[kBufs], pair[8], s_full[2], p_full[2], o_full[2], drained;
        uint32_t tmem, gave_up, columns, all;
        uint32_t seen[kBufs][4];
        float tops[2][2][2][128];         // [turn][group][half][lane]
        uint8_t byte_of[257 + 15];        // bucket byte of hops + 1
    };
    static constexpr int kLut = kCtl + (int)((sizeof(Ctl) + 15) / 16 * 16);
    static size_t bytes(const AttnParams &p) { return kLut + kTcLutAlign + (size_t)(p.buckets + 2) * p.group2 * 4; }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)),
          "l"(*reinterpret_cast<unsigned long long *>(&c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return d;
}
// The bias table does not change once the block has set it up, so that its reads may move freely.
__device__ __forceinline__ float table(uint32_t at)
{
    float v;
    asm("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Scores of N nodes in units of log2, biased and masked, and their maximum
// with `top`.  bt: their bucket bytes; a byte b's bias lies at shared-memory
// address lg | b << shift (floats of 2^k query heads, k = shift - 2).
template <int N>
__device__ __forceinline__ float bias_scores(uint32_t (&s)[N], float scale, bool plain, const uint8_t *bt, uint32_t lg, uint32_t shift, float top)
{
    const float2 sc = make_float2(scale, scale);
    if (plain) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 x = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc, make_float2(0.0f, 0.0f));
            s[e] = __float_as_uint(x.x);
            s[e + 1] = __float_as_uint(x.y);
            top = max3(top, x.x, x.y);
        }
        return top;
    }
    const uint32_t mask = 255u << shift;
#pragma unroll
    for (int e = 0; e < N; e += 16) {
        const uint4 b16 = *reinterpret_cast<const uint4 *>(bt + e);
        const uint32_t w[4] = {b16.x, b16.y, b16.z, b16.w};
#pragma unroll
        for (int y = 0; y < 16; y += 2) {
            const uint32_t v = w[y >> 2];
            const uint32_t i0 = (y & 3) ? v >> (16 - shift) : v << shift, i1 = (y & 3) ? v >> (24 - shift) : v >> (8 - shift);
            const float2 x = fma2(make_float2(__uint_as_float(s[e + y]), __uint_as_float(s[e + y + 1])), sc,
                                  make_float2(table((i0 & mask) | lg), table((i1 & mask) | lg)));
            s[e + y] = __float_as_uint(x.x);
            s[e + y + 1] = __float_as_uint(x.y);
            top = max3(top, x.x, x.y);
        }
    }
    return top;
}

// Weights of N scores, two a word in the element type, and their sum onto `sum`.
template <typename T, int N>
__device__ __forceinline__ void weights(uint32_t (&out)[N / 2], const uint32_t (&s)[N], float m, float2 (&sum)[2])
{
    const float2 nm = make_float2(-m, -m);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
        const float2 x = add2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), nm);
        const float2 y = make_float2(ex2(x.x), ex2(x.y));
        sum[e & 1] = add2(sum[e & 1], y);
        out[e] = Elem<T>::pack(y.x, y.y);
    }
}

// A running sum over very many tiles: a tile's terms are added up first, and what the addition to the sum cuts off is kept
// beside it.  (2^20 nodes of 1.4 2^-24 each after one of 1, one by one to one fp32 sum: 1.1e-3 off in lse.)
struct LongSum {
    float sum = 0.0f, rest = 0.0f;
    __device__ __forceinline__ void add(float x)
    {
        const float y = x + rest, s = sum + y, back = s - sum;
        rest = (sum - (s - back)) + (y - back);
        sum = s;
    }
    __device__ __forceinline__ float total() const { return sum + rest; }
};

template <typename T, int DP, int KW, bool TWO>
__global__ void __launch_bounds__(kTcThreads, 1) attn_fwd_kernel(const __grid_constant__ AttnParams p)
{
    using S = TcSmem<DP, TWO>;
    using Ctl = typename S::Ctl;
    constexpr int kRows = KW;                      // distinct rows per 128 lanes: 128, 64 or 32
    constexpr int HW = KW / 2, CH = HW < 32 ? HW : 32;   // nodes of a thread's part of a tile, of them at a time
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + S::kCtl);
    const uint32_t sm = tc::saddr(smem);
    const uint32_t lut_at = (sm + S::kLut + kTcLutAlign - 1) & ~(uint32_t)(kTcLutAlign - 1);
    float *lut = reinterpret_cast<float *>(smem + (lut_at - sm));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t hk = blockIdx.y, split = blockIdx.x % p.splits;
    const uint32_t row0 = blockIdx.x / p.splits * (TWO ? 256 : kRows);
    const uint32_t tiles = (uint32_t)(split < p.tiles ? (p.tiles - split + p.splits - 1) / p.splits : 0);
    const uint32_t units = TWO ? tiles * 2 : tiles;      // unit u: group u & 1, tile TWO ? u / 2 : u
    auto tile_at = [&](uint32_t i) { return split + (uint64_t)i * p.splits; };

    // ---- set-up ----
    if (warp == 24) tc::alloc(&ctl->tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) tc::bar_init(&ctl->full[i], 128), tc::bar_init(&ctl->empty[i], 1);
        for (int i = 0; i < S::kBufs; ++i) tc::bar_init(&ctl->hop_full[i], 4), tc::bar_init(&ctl->hop_empty[i], TWO ? 16 : 8);
        for (int i = 0; i < 8; ++i) tc::bar_init(&ctl->pair[i], 2);
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(&ctl->s_full[i], 1);
            tc::bar_init(&ctl->p_full[i], 256);
            tc::bar_init(&ctl->o_full[i], 1);
        }
        tc::bar_init(&ctl->drained, 1);
        ctl->gave_up = ctl->columns = ctl->all = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (p.sources)
        for (int i = tid; i < 257; i += kTcThreads) ctl->byte_of[i] = i ? p.bucket_of[i - 1] + 1 : 0;
    tc::grid_wait();
    fill_bias<T>(lut, p, hk, tid, p.group2);
    {   // queries: lane l of tile w holds row row0 + w * 128 + l % kRows
        constexpr int C = DP / 8;
        const char *src = static_cast<const char *>(p.q);
        for (int i = tid; i < (TWO ? 256 : 128) * C; i += kTcThreads) {
            const uint32_t l = i / C, c = i % C, w = l >> 7, r = l & 127;
            const uint32_t row = row0 + w * 128 + r % kRows;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < p.rows && c < p.d / 8) {
                const uint32_t t = row / p.group, g = row - t * p.group;
                v = __ldg(reinterpret_cast<const uint4 *>(src + ((int64_t)t * p.q_row + (int64_t)(hk * p.group + g) * p.q_head + c * 8) * 2));
            }
            *reinterpret_cast<uint4 *>(smem + S::kQ + w * S::kSlot + tc::chunk(r, c, S::kPanel)) = v;
        }
    }
    tc::fence_async();
    __syncthreads();
    if (p.sources)
        for (int i = tid; i < (TWO ? 256 : kRows); i += kTcThreads)
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

    if (warp >= 16 && warp < 20) {
        hop_warps<S::kBufs>(p, ctl, smem + S::kBuckets, warp - 16, lane, tiles, split, gave_up);
    } else if (warp >= 20 && warp < 24) {
        node_warps<DP, S::kSlots, S::kBufs>(p, ctl, sm, warp - 20, lane, hk, tiles, split, gave_up);
    } else if (warp == 24) {
        {
            const bool lead = tc::elect();
            // ---- products ----
            const uint32_t id_s = tc::idesc(kBf16, kTcTile, false, false);
            const uint32_t dn = (p.d + 15) & ~15u, id_o = tc::idesc(kBf16, dn, false, true);
            const uint32_t base = sm;
            // Scores run up to two units ahead of the outputs; whichever has its operands goes first.
            uint32_t next = 0, done = 0;
            tc::Patience wait(gave_up);
            while (done < units) {
                if (next < units && next < done + 2) {
                    const uint32_t w = next & 1, item = 2 * (TWO ? next >> 1 : next), slot = item % S::kSlots;
                    if (__all_sync(~0u, tc::bar_peek(&ctl->full[slot], (item / S::kSlots) & 1))) {
                        tc::fence_async();       // the copies were made by threads, the product reads through the async proxy
                        tc::fence_after();
                        const uint64_t q = tc::desc(base + S::kQ + (TWO ? w * S::kSlot : 0), S::kPanel), k = tc::desc(base + slot * S::kSlot, S::kPanel);
#pragma unroll
                        for (uint32_t kk = 0; kk < DP / 16; ++kk)
                            if (kk * 16 < dn) {
                                const uint32_t off = (kk >> 2) * S::kPanel + (kk & 3) * 32;
                                tc::mma_ss(lead, tm + w * 128, q, off, k, off, id_s, kk > 0);
                            }
                        tc::commit(lead, &ctl->s_full[w]);
                        if (!TWO || w == 1) tc::commit(lead, &ctl->empty[slot]);
                        ++next;
                        wait.restart();
                        continue;
                    }
                }
                const uint32_t w = done & 1, item = 2 * (TWO ? done >> 1 : done) + 1, slot = item % S::kSlots;
                if (done < next && __all_sync(~0u, tc::bar_peek(&ctl->full[slot], (item / S::kSlots) & 1) && tc::bar_peek(&ctl->p_full[w], (done >> 1) & 1))) {
                    tc::fence_async();
                    tc::fence_after();
                    const uint64_t v = tc::desc(base + slot * S::kSlot, S::kPanel);
#pragma unroll
                    for (uint32_t kk = 0; kk < kTcTile / 16; ++kk)
                        tc::mma_ts(lead, tm + 256 + w * DP, tm + w * 128 + kk * 8 + (kk < 4 ? 0 : 32), v, kk * 2048, id_o, done > 1 || kk > 0);
                    if (!TWO || w == 1) tc::commit(lead, &ctl->empty[slot]);
                    if (done + 2 >= units) tc::commit(lead, &ctl->o_full[w]);
                    ++done;
                    wait.restart();
                    continue;
                }
                if (!__all_sync(~0u, wait.more())) break;
            }
            const bool ok = done == units;
            if (!ok) tc::drain(lead, &ctl->drained, 0);
        }
        __syncwarp();
    } else {
        // ---- softmax: thread = (lane of tensor memory, half of its copy's nodes) ----
        const int w = warp >> 3, half = (warp >> 2) & 1, l = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // lane field of this warp's tensor memory
        const uint32_t row = row0 + (TWO ? w * 128 : 0) + l % kRows;
        const int copy = l / kRows, key0 = copy * KW + half * HW;     // this thread's part of a tile
        const uint32_t col = row < p.rows ? row_column(p, row) : 0;
        const uint32_t G = p.group, shift = p.group2_log + 2;
        const uint32_t lg = lut_at | (row < p.rows ? row % G : 0) * 4;
        const uint32_t s_at = tm + lanes + w * 128, o_at = tm + lanes + 256 + w * DP;
        const uint8_t *bt0 = smem + S::kBuckets + col * kTcPitch + key0;
        float *tops = ctl->tops[0][w][0] + l;                         // [turn][group][half][lane]
        uint64_t *pair = &ctl->pair[w * 4 + (warp & 3)];
        float m = -INFINITY;
        LongSum sum;
        bool ok = true;
        uint32_t mine = 0;                                            // units of this group done
        for (uint32_t u = w; u < units; u += 2, ++mine) {
            const uint32_t i = TWO ? u >> 1 : u, buf = i % S::kBufs;
            ok = tc::bar_wait(&ctl->hop_full[buf], (i / S::kBufs) & 1, gave_up) && tc::bar_wait(&ctl->s_full[w], mine & 1, gave_up);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc::fence_after();
            const bool plain = !p.sources && (tile_at(i) + 1) * kTcTile <= p.n;   // no table, no node past the end
            const uint8_t *bt = bt0 + buf * 33 * kTcPitch;
            float top = -INFINITY;
            uint32_t s[CH];
            // With two chunks, biased scores go back to tensor memory between the passes: rolled loops, since the
            // whole row in registers makes code that the instruction caches do not hold.
#pragma unroll 1
            for (int b = 0; b < HW; b += CH) {
                tc::load(s, s_at + key0 + b);
                tc::wait_ld();
                top = bias_scores(s, p.scale_log2, plain, bt + b, lg, shift, top);
                if (HW > CH) tc::store(s_at + key0 + b, s);
            }
            if (HW > CH) tc::wait_st();
            // the two halves of a row agree on its maximum, and have both read their scores, before weights replace them
            const int turn = (mine & 1) * 512;
            tops[turn + half * 128] = top;
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(&ctl->hop_empty[buf]), tc::bar_arrive(pair);
            ok = __all_sync(~0u, tc::bar_wait(pair, mine & 1, gave_up));
            if (!ok) break;
            tc::fence_after();
            top = fmaxf(top, tops[turn + (half ^ 1) * 128]);
            const bool grow = top > m + kTcLag || (m == -INFINITY && top > -INFINITY);
            if (__any_sync(~0u, grow)) {
                const float next = grow ? top : m;
                const float f = m == -INFINITY ? 0.0f : ex2(m - next);      // m = -inf: nothing was summed yet
                m = next;
                sum.sum *= f, sum.rest *= f;
                if (mine > 0) {
                    // the products issued before these scores are done, so O is at rest; each half takes half of it
#pragma unroll 1
                    for (int c = half * (DP / 2); c < (half + 1) * (DP / 2); c += 16) {
                        uint32_t o[16];
                        tc::load(o, o_at + c);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::store(o_at + c, o);
                    }
                }
            }
            const float u0 = m == -INFINITY ? 0.0f : m - kTcUp<T>;
            // Weights in the element type, two a word, over S: nodes [0, 64) from its column 0 on, [64, 128) from 64 on,
            // so that a half of 64 overwrites its own scores.  Nodes of the other copies' parts weigh nothing.
            float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            if (KW == 128) {
#pragma unroll 1
                for (int b = 0; b < HW; b += CH) {
                    uint32_t out[CH / 2];
                    tc::load(s, s_at + key0 + b);
                    tc::wait_ld();
                    weights<T, CH>(out, s, u0, part);
                    tc::store(s_at + key0 + b / 2, out);
                }
            } else {
                uint32_t out[CH / 2];
                weights<T, CH>(out, s, u0, part);
#pragma unroll
                for (int j = 0; j < 128 / KW; ++j) {
                    const uint32_t at = s_at + (j * KW < 64 ? j * KW / 2 : 64 + (j * KW - 64) / 2) + half * (HW / 2);
                    if (j == copy) {
                        tc::store(at, out);
                    } else {
                        const uint32_t zero[CH / 2] = {};
                        tc::store(at, zero);
                    }
                }
            }
            tc::wait_st();
            tc::fence_before();
            tc::bar_arrive(&ctl->p_full[w]);
            sum.add((part[0].x + part[0].y) + (part[1].x + part[1].y));
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
            for (int c = half * (DP / 2); c < (half + 1) * (DP / 2); c += 16) {
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
            if (half == 0) at[DP] = m - kTcUp<T>;
            at[DP + 1 + half] = sum.total();
        }
        asm volatile("bar.sync 1, 512;" ::: "memory");
        constexpr int kSets = TWO ? 1 : 2 * (128 / kRows), kOut = TWO ? 256 : kRows, Q4 = DP / 4;
        if (ok)
            for (int i = tid; i < kOut * Q4; i += 512) {
                const int r = i / Q4, c = (i % Q4) * 4;
                const uint32_t rw = row0 + r;
                if (rw >= p.rows || c >= (int)p.d) continue;
                const float *e0 = ex + (size_t)r * P;
                float mx = -INFINITY;
#pragma unroll
                for (int k = 0; k < kSets; ++k) mx = fmaxf(mx, e0[(size_t)k * kRows * P + DP]);
                const float ux = mx == -INFINITY ? 0.0f : mx;
                float ls = 0.0f;
                float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kSets; ++k) {
                    const float *e = e0 + (size_t)k * kRows * P;
                    const float f = ex2(e[DP] - ux);
                    const float4 x = *reinterpret_cast<const float4 *>(e + c);
                    ls += f * (e[DP + 1] + e[DP + 2]);
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
    if (warp == 24) tc::dealloc(tm, 512);
    if (tid == 0 && *gave_up) atomicOr(p.status, K2T_STATUS_WAIT_TIMEOUT);
}

// Joins the splits of each row: M = max m_i, out = sum O_i 2^(m_i - M) / sum l_i 2^(m_i - M).
// One block a row, 4 values a thread, the splits over the thread groups.
template <typename T>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ float red[8];
    __shared__ float4 sum[256];
    const uint64_t row = blockIdx.x;             // t * hq + h
    const uint64_t stride = (uint64_t)p.T * p.hq;
    const int tid = threadIdx.x;
    tc::grid_wait();
    float m = -INFINITY;
    for (uint32_t s = tid; s < p.splits; s += 256) m = fmaxf(m, p.part_ml[(s * stride + row) * 2]);
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = red[0];
    for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
    const float u = m == -INFINITY ? 0.0f : m;
    const uint32_t q4 = p.d / 4, groups = 256 / q4, c = tid % q4, g = tid / q4;
    float4 acc = make_float4(0, 0, 0, 0);
    float l = 0.0f;
    if (g < groups)
        for (uint32_t s = g; s < p.splits; s += groups) {
            const uint64_t at = s * stride + row;
            const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + at * 2);
            const float f = ex2(ml.x - u);
            const float4 x = *reinterpret_cast<const float4 *>(p.part + at * p.d + c * 4);
            l += f * ml.y;
            acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
        }
    sum[tid] = acc;
    __shared__ float lsum[256];
    lsum[tid] = l;
    __syncthreads();
    if (g == 0) {
        for (uint32_t i = 1; i < groups; ++i) {
            const float4 x = sum[i * q4 + c];
            acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
            l += lsum[i * q4 + c];
        }
        const uint32_t t = (uint32_t)(row / p.hq), hd = (uint32_t)(row - (uint64_t)t * p.hq);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint2 w;
        w.x = Elem<T>::pack(acc.x * inv, acc.y * inv);
        w.y = Elem<T>::pack(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (int64_t)t * p.out_row + (int64_t)hd * p.out_head + c * 4) = w;
        if (c == 0) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

}  // namespace k2t
