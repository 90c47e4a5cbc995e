// k2t_attn_fwd.cuh -- forward pass of the hop-biased attention.
//
// One pass over the nodes with the running maximum and sum of the softmax:
// for a tile of nodes with scores s, m' = max(m, max s), w = exp2(s - m'),
// l = l exp2(m - m') + sum w, O = O exp2(m - m') + w V.  Few rows meet many
// nodes, so the nodes of a head are split over `splits` blocks (tile i goes
// to block i mod splits, which also spreads the unreached nodes that power-law
// graphs keep side by side), and attn_join_kernel joins their (O, m, l).
#pragma once

#include "k2t_attn.cuh"

namespace k2t {

template <int DP, int BM> struct FwdSmem {
    static constexpr int kStages = 3;
    static constexpr int kTileBytes = kAttnTile * DP * 2;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kQ = kStages * kStageBytes;             // Q, then the hop part
    static constexpr int kHop = kQ + BM * DP * 2;
    static constexpr int kCol = kHop + (int)((sizeof(HopSmem) + 15) / 16 * 16);
    static constexpr int kLut = kCol + BM * 4;
    static size_t bytes(const AttnParams &p) { return kLut + (size_t)(p.buckets + 2) * p.group * 4; }
};

// 4 warps: BM / 16 of them side by side over the rows, the others over the
// nodes of a tile, each with a softmax of its own, joined at the end.
template <typename T, int DP, int BM>
__global__ void __launch_bounds__(kAttnThreads) attn_fwd_kernel(const __grid_constant__ AttnParams p)
{
    using S = FwdSmem<DP, BM>;
    constexpr int WM = BM / 16, WK = 4 / WM, KEYS = kAttnTile / WK, N8 = KEYS / 8, D16 = DP / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t hk = blockIdx.y, split = blockIdx.x % p.splits, row0 = blockIdx.x / p.splits * BM;
    HopSmem *hs = reinterpret_cast<HopSmem *>(smem + S::kHop);
    uint32_t *col_of = reinterpret_cast<uint32_t *>(smem + S::kCol);
    float *lut = reinterpret_cast<float *>(smem + S::kLut);
    const uint32_t sm = smem_u32(smem);

    copy_rows<DP, BM>(sm + S::kQ, p.q, p.q_row, p.q_head, hk * p.group, row0, p, tid);
    cp_commit();
    if (tid == 0) hs->columns = 0, hs->all = 0;
    if (p.sources)
        for (int i = tid; i < 256; i += kAttnThreads) hs->bucket_of[i] = p.bucket_of[i];
    fill_bias<T>(lut, p, hk, tid);
    for (int i = tid; i < 4 * kAttnTile; i += kAttnThreads) hs->seen[0][i] = 0;
    __syncthreads();
    for (int i = tid; i < BM; i += kAttnThreads) {
        const uint32_t c = row0 + i < p.rows ? row_column(p, row0 + i) : 0;
        col_of[i] = c * kHopPitch;
        if (row0 + i < p.rows && p.sources) {
            if (c < p.sources) atomicOr(&hs->columns, 1u << c);
            else hs->all = 1;
        }
    }
    __syncthreads();

    const uint64_t tiles = split < p.tiles ? (p.tiles - split + p.splits - 1) / p.splits : 0;
    auto tile_at = [&](uint64_t i) { return split + i * p.splits; };
    const char *kbase = static_cast<const char *>(p.k) + hk * p.k_head * 2;
    const char *vbase = static_cast<const char *>(p.v) + hk * p.v_head * 2;
    int32_t h[kHopRegs];
    auto hops_in = [&](uint64_t i) { if (p.sources && i < tiles) hops_load(h, p, tile_at(i), tid); };
    auto hops_out = [&](uint64_t i, int buf) {
        if (i >= tiles) return;
        if (p.sources) hops_store(h, hs, p, tile_at(i), buf, tid);
        else hops_none(hs, p, tile_at(i), buf, tid);
    };
    auto copy = [&](uint64_t i) {
        if (i < tiles) {
            const uint32_t st = sm + (uint32_t)(i % S::kStages) * S::kStageBytes;
            const uint8_t *seen = hs->seen[i & 3];
            const int64_t node0 = (int64_t)tile_at(i) * kAttnTile;
            copy_nodes<DP>(st, kbase, p.k_row * 2, node0, p.n, p.d / 8, seen, tid);
            copy_nodes<DP>(st + S::kTileBytes, vbase, p.v_row * 2, node0, p.n, p.d / 8, seen, tid);
        }
        cp_commit();
    };
    hops_in(0); hops_out(0, 0);
    hops_in(1); hops_out(1, 1);
    hops_in(2);
    __syncthreads();
    copy(0);
    copy(1);
    cp_wait<2>();
    __syncthreads();

    const int wm = warp % WM, wk = warp / WM;
    uint32_t q[D16][4];
#pragma unroll
    for (int i = 0; i < D16; ++i) load_a<DP>(q[i], sm + S::kQ, wm * 16, i, lane);
    const int ra = wm * 16 + (lane >> 2), rb = ra + 8;                  // this thread's two rows
    const uint32_t ca = col_of[ra], cb = col_of[rb];
    const float *lut_a = lut + (row0 + ra) % p.group, *lut_b = lut + (row0 + rb) % p.group;
    const uint32_t G = p.group;

    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float ma = -INFINITY, mb = -INFINITY, la = 0.0f, lb = 0.0f;

    for (uint64_t i = 0; i < tiles; ++i) {
        hops_out(i + 2, (i + 2) & 3);
        if (tid < kAttnTile) hs->seen[(i + 3) & 3][tid] = 0;
        cp_wait<1>();
        __syncthreads();
        copy(i + 2);
        hops_in(i + 3);

        const uint32_t ks = sm + (uint32_t)(i % S::kStages) * S::kStageBytes, vs = ks + S::kTileBytes;
        const uint8_t *bt = hs->tile[i & 3] + wk * KEYS + (lane & 3) * 2;
        float s[N8][4];
#pragma unroll
        for (int j = 0; j < N8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < D16; ++kk)
#pragma unroll
            for (int j = 0; j < N8; j += 2) {
                uint32_t b[4];
                load_b<DP>(b, ks, wk * KEYS + j * 8, kk, lane);
                Elem<T>::mma(s[j], q[kk], b[0], b[1]);
                Elem<T>::mma(s[j + 1], q[kk], b[2], b[3]);
            }
        float xa = -INFINITY, xb = -INFINITY;
#pragma unroll
        for (int j = 0; j < N8; ++j) {
            const uint32_t ba = *reinterpret_cast<const uint16_t *>(bt + ca + j * 8);
            const uint32_t bb = *reinterpret_cast<const uint16_t *>(bt + cb + j * 8);
            s[j][0] = fmaf(s[j][0], p.scale_log2, lut_a[(ba & 255) * G]);
            s[j][1] = fmaf(s[j][1], p.scale_log2, lut_a[(ba >> 8) * G]);
            s[j][2] = fmaf(s[j][2], p.scale_log2, lut_b[(bb & 255) * G]);
            s[j][3] = fmaf(s[j][3], p.scale_log2, lut_b[(bb >> 8) * G]);
            xa = fmaxf(xa, fmaxf(s[j][0], s[j][1]));
            xb = fmaxf(xb, fmaxf(s[j][2], s[j][3]));
        }
        xa = fmaxf(xa, __shfl_xor_sync(~0u, xa, 1));
        xb = fmaxf(xb, __shfl_xor_sync(~0u, xb, 1));
        xa = fmaxf(xa, __shfl_xor_sync(~0u, xa, 2));
        xb = fmaxf(xb, __shfl_xor_sync(~0u, xb, 2));
        // a row that has seen nothing yet keeps m = -inf; 0 stands in for it, so that no inf - inf arises
        const float na = fmaxf(ma, xa), nb = fmaxf(mb, xb);
        const float ua = na == -INFINITY ? 0.0f : na, ub = nb == -INFINITY ? 0.0f : nb;
        const float fa = ex2(ma - ua), fb = ex2(mb - ub);
        ma = na;
        mb = nb;
        la *= fa;
        lb *= fb;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) o[j][0] *= fa, o[j][1] *= fa, o[j][2] *= fb, o[j][3] *= fb;
#pragma unroll
        for (int j = 0; j < N8; ++j) {
            s[j][0] = ex2(s[j][0] - ua);
            s[j][1] = ex2(s[j][1] - ua);
            s[j][2] = ex2(s[j][2] - ub);
            s[j][3] = ex2(s[j][3] - ub);
            la += s[j][0] + s[j][1];
            lb += s[j][2] + s[j][3];
        }
#pragma unroll
        for (int j = 0; j < N8; j += 2) {
            // weights rounded to the element type: they are at most 1, so fp16 holds them too, and their
            // errors are independent and average out over the nodes
            const uint32_t a[4] = {Elem<T>::pack(s[j][0], s[j][1]), Elem<T>::pack(s[j][2], s[j][3]),
                                   Elem<T>::pack(s[j + 1][0], s[j + 1][1]), Elem<T>::pack(s[j + 1][2], s[j + 1][3])};
#pragma unroll
            for (int c = 0; c < D16; ++c) {
                uint32_t b[4];
                load_bt<DP>(b, vs, wk * KEYS + j * 8, c, lane);
                Elem<T>::mma(o[2 * c], a, b[0], b[1]);
                Elem<T>::mma(o[2 * c + 1], a, b[2], b[3]);
            }
        }
    }
    cp_wait<0>();
    la += __shfl_xor_sync(~0u, la, 1);
    lb += __shfl_xor_sync(~0u, lb, 1);
    la += __shfl_xor_sync(~0u, la, 2);
    lb += __shfl_xor_sync(~0u, lb, 2);

    // join the WK warps that share rows, through the freed stages: [wk][row][DP + 2] floats
    constexpr int P = DP + 4;
    float *ex = reinterpret_cast<float *>(smem);
    static_assert(WK * BM * P * 4 <= S::kQ, "exchange fits the stages");
    __syncthreads();
    {
        float *ea = ex + (size_t)(wk * BM + ra) * P, *eb = ex + (size_t)(wk * BM + rb) * P;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
            *reinterpret_cast<float2 *>(ea + j * 8 + (lane & 3) * 2) = make_float2(o[j][0], o[j][1]);
            *reinterpret_cast<float2 *>(eb + j * 8 + (lane & 3) * 2) = make_float2(o[j][2], o[j][3]);
        }
        if ((lane & 3) == 0) ea[DP] = ma, ea[DP + 1] = la, eb[DP] = mb, eb[DP + 1] = lb;
    }
    __syncthreads();
    constexpr int Q4 = DP / 4;
    for (int i = tid; i < BM * Q4; i += kAttnThreads) {
        const int r = i / Q4, c = (i % Q4) * 4;
        const uint32_t row = row0 + r;
        if (row >= p.rows || c >= (int)p.d) continue;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < WK; ++w) m = fmaxf(m, ex[(size_t)(w * BM + r) * P + DP]);
        const float u = m == -INFINITY ? 0.0f : m;
        float l = 0.0f;
        float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const float *e = ex + (size_t)(w * BM + r) * P;
            const float f = ex2(e[DP] - u);
            const float4 x = *reinterpret_cast<const float4 *>(e + c);
            l += f * e[DP + 1];
            acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
        }
        const uint32_t t = row / p.group, hd = hk * p.group + row % p.group;
        if (p.splits > 1) {
            const uint64_t at = ((uint64_t)split * p.T + t) * p.hq + hd;
            *reinterpret_cast<float4 *>(p.part + at * p.d + c) = acc;
            if (c == 0) *reinterpret_cast<float2 *>(p.part_ml + at * 2) = make_float2(m, l);
        } else {
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            uint2 w;
            w.x = Elem<T>::pack(acc.x * inv, acc.y * inv);
            w.y = Elem<T>::pack(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (int64_t)t * p.out_row + (int64_t)hd * p.out_head + c) = w;
            if (c == 0) p.lse[(uint64_t)t * p.hq + hd] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
    }
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
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        uint2 w;
        w.x = Elem<T>::pack(acc.x * inv, acc.y * inv);
        w.y = Elem<T>::pack(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (int64_t)t * p.out_row + (int64_t)hd * p.out_head + c * 4) = w;
        if (c == 0) p.lse[row] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
}

}  // namespace k2t
