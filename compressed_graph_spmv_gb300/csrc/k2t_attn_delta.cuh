// k2t_attn_delta.cuh -- what every score gradient of a row has taken off:
//   delta = sum_j p_j dp_j / sum_j p_j,  p = exp(s - lse),  dp = dout . v_j.
//
// delta equals dout . out, but out was rounded to 16 bits, and where a few
// nodes hold most of a row's weight, ds = p (dp - delta) is a small difference
// whose error is then as large as itself (one source's own node with 0.99 of
// the weight, bf16: its bucket's gradient was 20 to 48% off).  Gradients of
// the bias table sum ds over many nodes, so that the error adds up in each
// bucket in proportion to its weight.  Calls with a table therefore form delta
// from the nodes, in 32 bits; so do those in fp16, which need the largest
// p |dp| as well (ds_scale); others take dout . out, which needs no pass.
//
// The forward pass's layout (see there), with a row's lse known: no running
// maximum, no weights written back, and dP = dO V^T beside S = Q K^T in place
// of O = P V.  128 rows at most a block; repeated rows and groups as there.
// Each block writes its part of the two sums of a row, which the kernels that
// follow join in a fixed order.
//
// What bounds it: what bounds the forward pass.  32 queries over 2^18 nodes,
// forward and backward, take 467 us with it and 351 without, 257 over 8191 157
// and 137 (25 us for itself: tensor pipe 16% busy, issue slots 48%), 8 over
// 1000 without a table in fp16 28 and 25.
#pragma once

#include "k2t_attn_fwd.cuh"

namespace k2t {

template <int DP> struct DeltaSmem {
    static constexpr int kPanel = kTcTile * 128;
    static constexpr int kSlot = kPanel * (DP / 64);
    static constexpr int kSlots = DP == 64 ? 8 : 4;
    static constexpr int kBufs = DP == 64 ? 6 : 3;            // bucket tiles
    static constexpr int kQ = kSlots * kSlot;                 // queries, then dout
    static constexpr int kBuckets = kQ + 2 * kSlot;
    static constexpr int kCtl = kBuckets + kBufs * 33 * kTcPitch;
    struct Ctl {
        uint64_t full[kSlots], empty[kSlots], hop_full[kBufs], hop_empty[kBufs], s_full[2], s_read[2], drained;
        uint32_t tmem, gave_up, columns, all;
        uint32_t seen[kBufs][4];
        float2 sum[2][2][128];            // [group][half][lane]: sum of p dp, sum of p
        float tops[2][2][128];            // largest p |dp|
        uint8_t byte_of[257 + 15];
    };
    static constexpr int kLut = kCtl + (int)((sizeof(Ctl) + 15) / 16 * 16);
    static size_t bytes(const AttnParams &p) { return kLut + kTcLutAlign + (size_t)(p.buckets + 2) * p.group2 * 4; }
};

// p.splits, p.row_tiles: of this kernel (KW rows a tile).
template <typename T, int DP, int KW>
__global__ void __launch_bounds__(kTcThreads, 1) attn_delta_kernel(const __grid_constant__ AttnParams p)
{
    using S = DeltaSmem<DP>;
    using Ctl = typename S::Ctl;
    constexpr int kRows = KW, HW = KW / 2;         // distinct rows per 128 lanes; nodes of a thread's part of a tile
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + S::kCtl);
    const uint32_t sm = tc::saddr(smem);
    const uint32_t lut_at = (sm + S::kLut + kTcLutAlign - 1) & ~(uint32_t)(kTcLutAlign - 1);
    float *lut = reinterpret_cast<float *>(smem + (lut_at - sm));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t hk = blockIdx.y, split = blockIdx.x % p.splits, row0 = blockIdx.x / p.splits * kRows;
    const uint32_t units = (uint32_t)(split < p.tiles ? (p.tiles - split + p.splits - 1) / p.splits : 0);   // unit u: tile u, group u & 1

    // ---- set-up ----
    if (warp == 24) tc::alloc(&ctl->tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) tc::bar_init(&ctl->full[i], 128), tc::bar_init(&ctl->empty[i], 1);
        for (int i = 0; i < S::kBufs; ++i) tc::bar_init(&ctl->hop_full[i], 4), tc::bar_init(&ctl->hop_empty[i], 8);
        for (int i = 0; i < 2; ++i) tc::bar_init(&ctl->s_full[i], 1), tc::bar_init(&ctl->s_read[i], 256);
        tc::bar_init(&ctl->drained, 1);
        ctl->gave_up = ctl->columns = ctl->all = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (p.sources)
        for (int i = tid; i < 257; i += kTcThreads) ctl->byte_of[i] = i ? p.bucket_of[i - 1] + 1 : 0;
    tc::grid_wait();
    fill_bias<T>(lut, p, hk, tid, p.group2);
    {   // queries and dout: lane l holds row row0 + l % kRows
        constexpr int C = DP / 8;
        for (int i = tid; i < 256 * C; i += kTcThreads) {
            const uint32_t l = i / C, c = i % C, x = l >> 7, r = l & 127, row = row0 + r % kRows;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < p.rows && c < p.d / 8) {
                const uint32_t t = row / p.group, g = row - t * p.group;
                const int64_t at = (int64_t)t * (x ? p.dout_row : p.q_row) + (int64_t)(hk * p.group + g) * (x ? p.dout_head : p.q_head) + c * 8;
                v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const char *>(x ? p.dout : p.q) + at * 2));
            }
            *reinterpret_cast<uint4 *>(smem + S::kQ + x * S::kSlot + tc::chunk(r, c, S::kPanel)) = v;
        }
    }
    tc::fence_async();
    __syncthreads();
    if (p.sources && tid < kRows && row0 + tid < p.rows) {
        const uint32_t c = row_column(p, row0 + tid);
        if (c < p.sources) atomicOr(&ctl->columns, 1u << c);
        else ctl->all = 1;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    tc::grid_next();
    const uint32_t tm = ctl->tmem;                       // S of group w at w * 128, dP at 256 + w * 128
    volatile uint32_t *gave_up = &ctl->gave_up;

    if (warp >= 16 && warp < 20) {
        hop_warps<S::kBufs>(p, ctl, smem + S::kBuckets, warp - 16, lane, units, split, gave_up);
    } else if (warp >= 20 && warp < 24) {
        node_warps<DP, S::kSlots, S::kBufs>(p, ctl, sm, warp - 20, lane, hk, units, split, gave_up);
    } else if (warp == 24) {
        // ---- products ----
        const bool lead = tc::elect();
        const uint32_t id = tc::idesc(kBf16, kTcTile, false, false), dn = (p.d + 15) & ~15u;
        bool ok = true;
        for (uint32_t u = 0; u < units && ok; ++u) {
            const uint32_t w = u & 1;
            // the scores that these replace have been read
            if (u > 1) ok = __all_sync(~0u, tc::bar_wait(&ctl->s_read[w], ((u >> 1) - 1) & 1, gave_up));
#pragma unroll 1
            for (uint32_t x = 0; x < 2 && ok; ++x) {     // S of the keys, dP of the values
                const uint32_t item = 2 * u + x, slot = item % S::kSlots;
                ok = __all_sync(~0u, tc::bar_wait(&ctl->full[slot], (item / S::kSlots) & 1, gave_up));
                if (!ok) break;
                tc::fence_async();       // the copies were made by threads, the product reads through the async proxy
                tc::fence_after();
                const uint64_t rows = tc::desc(sm + S::kQ + x * S::kSlot, S::kPanel), nodes = tc::desc(sm + slot * S::kSlot, S::kPanel);
#pragma unroll
                for (uint32_t kk = 0; kk < DP / 16; ++kk)
                    if (kk * 16 < dn) {
                        const uint32_t off = (kk >> 2) * S::kPanel + (kk & 3) * 32;
                        tc::mma_ss(lead, tm + x * 256 + w * 128, rows, off, nodes, off, id, kk > 0);
                    }
                // the barrier that threads wait for last, so that no arrival is under way when the block ends
                tc::commit(lead, &ctl->empty[slot]);
                if (x) tc::commit(lead, &ctl->s_full[w]);
            }
        }
        if (!ok) tc::drain(lead, &ctl->drained, 0);
        __syncwarp();
    } else {
        // ---- sums: thread = (lane of tensor memory, half of its copy's nodes) ----
        const int w = warp >> 3, half = (warp >> 2) & 1, l = (warp & 3) * 32 + lane;
        const uint32_t row = row0 + l % kRows, t = row / p.group, g = row - t * p.group;
        const int key0 = l / kRows * KW + half * HW;                  // this thread's part of a tile
        const uint32_t col = row < p.rows ? row_column(p, row) : 0, shift = p.group2_log + 2;
        const uint32_t lg = lut_at | (row < p.rows ? g : 0) * 4;
        const uint32_t s_at = tm + ((uint32_t)(warp & 3) << 21) + w * 128 + key0;
        const uint8_t *bt0 = smem + S::kBuckets + col * kTcPitch + key0;
        const float lse = row < p.rows ? p.lse[(uint64_t)t * p.hq + hk * p.group + g] : -INFINITY;
        const float nl = lse == -INFINITY ? -INFINITY : -lse * kLog2e;              // weights of a row that saw nothing are 0
        LongSum all_dots, all_mass;
        float top = 0.0f;                                             // largest p |dp|
        uint32_t mine = 0;                                            // units of this group done
        for (uint32_t u = w; u < units; u += 2, ++mine) {
            const uint32_t buf = u % S::kBufs;
            bool ok = tc::bar_wait(&ctl->hop_full[buf], (u / S::kBufs) & 1, gave_up) && tc::bar_wait(&ctl->s_full[w], mine & 1, gave_up);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc::fence_after();
            const bool plain = !p.sources && (split + (uint64_t)u * p.splits + 1) * kTcTile <= p.n;     // no table, no node past the end
            float2 dots = make_float2(0.0f, 0.0f), mass = dots;
#pragma unroll 1
            for (int b = 0; b < HW; b += 16) {
                uint32_t s[16], d[16];
                tc::load(s, s_at + b);
                tc::load(d, s_at + 256 + b);
                tc::wait_ld();
                bias_scores(s, p.scale_log2, plain, bt0 + buf * 33 * kTcPitch + b, lg, shift, -INFINITY);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 x = add2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(nl, nl));
                    const float2 y = make_float2(ex2(x.x), ex2(x.y));
                    mass = add2(mass, y);
                    const float2 dp = make_float2(__uint_as_float(d[e]), __uint_as_float(d[e + 1]));
                    dots = fma2(y, dp, dots);
                    if (Elem<T>::kUp) top = max3(top, fabsf(y.x * dp.x), fabsf(y.y * dp.y));
                }
            }
            tc::fence_before();
            tc::bar_arrive(&ctl->s_read[w]);
            __syncwarp();
            if (lane == 0) tc::bar_arrive(&ctl->hop_empty[buf]);
            all_dots.add(dots.x + dots.y);
            all_mass.add(mass.x + mass.y);
        }
        // ---- the copies' and groups' sums of a row, one after another ----
        ctl->sum[w][half][l] = make_float2(all_dots.total(), all_mass.total());
        if (Elem<T>::kUp) ctl->tops[w][half][l] = top;
        asm volatile("bar.sync 1, 512;" ::: "memory");
        if (tid < kRows && row0 + tid < p.rows) {                     // warps 0-3 hold lane tid of group 0 as their own row
            float a = 0.0f, m = 0.0f, most = 0.0f;
            for (int c = tid; c < 128; c += kRows)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 v = ctl->sum[x >> 1][x & 1][c];
                    a += v.x, m += v.y;
                    if (Elem<T>::kUp) most = fmaxf(most, ctl->tops[x >> 1][x & 1][c]);
                }
            const uint64_t at = ((uint64_t)split * p.T + t) * p.hq + hk * p.group + g;
            p.delta_part[at] = make_float2(a, m);
            if (Elem<T>::kUp) p.pdp_top[at] = most;
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 24) tc::dealloc(tm, 512);
    if (tid == 0 && *gave_up) atomicOr(p.status, K2T_STATUS_WAIT_TIMEOUT);
}

}  // namespace k2t
