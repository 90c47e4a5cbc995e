// k2t_attn_bwd.cuh -- backward pass of the hop-biased attention.
//
// With p = exp(s - lse), delta = dout . out and dp = dout . v:
//   ds = p (dp - delta),  dv = sum p dout,  dk = scale sum ds q,
//   dq = scale sum ds k,  dbias[bucket] = sum ds.
// Scores are computed transposed, nodes x rows: a warp owns 16 nodes, its
// weights p^T and ds^T come out of the accumulators in the layout of an A
// operand, so dv and dk (nodes x head_dim, summed over rows) need no exchange
// between warps.  dq sums over nodes: ds^T passes through shared memory once.
// Where all rows of a head fit one tile (32), one pass makes everything: dk
// and dv of a tile are final, dq stays in registers over the block's nodes
// (MODE 0).  With more rows, one kernel loops rows for fixed nodes (MODE 1:
// dk, dv) and one loops nodes for fixed rows (MODE 2: dq, dbias): scores are
// computed twice, and nothing is summed by atomics, so results do not depend
// on the order of blocks.
#pragma once

#include "k2t_attn.cuh"

namespace k2t {

constexpr int kBwdRows = 32;   // rows per tile

template <int DP, int MODE> struct BwdSmem {
    static constexpr int kTileBytes = kAttnTile * DP * 2;
    static constexpr int kRowBytes = kBwdRows * DP * 2;
    static constexpr int kKvStages = MODE == 1 ? 1 : 2;
    static constexpr int kRowStages = MODE == 1 ? 2 : 1;
    static constexpr int kRow = kKvStages * 2 * kTileBytes;                      // q, dout
    static constexpr int kDsPitch = kBwdRows + 8;                                // values; 80 bytes, 5 x 16: no bank conflicts
    static constexpr int kDs = kRow + kRowStages * 2 * kRowBytes;                // ds^T [node][row]
    static constexpr int kHop = kDs + (MODE == 1 ? 0 : kAttnTile * kDsPitch * 2);
    static constexpr int kStat = kHop + (int)((sizeof(HopSmem) + 15) / 16 * 16);  // lse (log2), delta, column, per row
    static constexpr int kLut = kStat + 2 * 3 * kBwdRows * 4;
    static size_t bytes(const AttnParams &p)
    {
        const size_t lut = (size_t)(p.buckets + 2) * p.group * 4;
        return kLut + lut + (MODE == 1 ? 0 : (size_t)(p.buckets + 2) * kAttnThreads * 4);
    }
};

// delta[t, h] = dout . out in fp32, a warp per row.
template <typename T>
__global__ void __launch_bounds__(256) attn_delta_kernel(const __grid_constant__ AttnParams p)
{
    const uint64_t row = (uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (uint64_t)p.T * p.hq) return;
    const int lane = threadIdx.x & 31;
    const uint32_t t = (uint32_t)(row / p.hq), hd = (uint32_t)(row - (uint64_t)t * p.hq);
    const T *o = static_cast<const T *>(p.out) + (int64_t)t * p.out_row + (int64_t)hd * p.out_head;
    const T *g = static_cast<const T *>(p.dout) + (int64_t)t * p.dout_row + (int64_t)hd * p.dout_head;
    float s = 0.0f;
    for (uint32_t c = lane * 2; c < p.d; c += 64) {
        const float2 a = Elem<T>::unpack(*reinterpret_cast<const uint32_t *>(o + c));
        const float2 b = Elem<T>::unpack(*reinterpret_cast<const uint32_t *>(g + c));
        s = fmaf(a.x, b.x, fmaf(a.y, b.y, s));
    }
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    if (lane == 0) p.delta[row] = s;
}

template <typename T, int DP, int MODE>
__global__ void __launch_bounds__(kAttnThreads) attn_bwd_kernel(const __grid_constant__ AttnParams p)
{
    using S = BwdSmem<DP, MODE>;
    constexpr int D16 = DP / 16, R8 = kBwdRows / 8;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t hk = blockIdx.y;
    // MODE 0, 2: x = split + splits * row tile; MODE 1: x = tile of nodes
    const uint32_t split = MODE == 1 ? 0 : blockIdx.x % p.splits, fixed_row0 = MODE == 1 ? 0 : blockIdx.x / p.splits * kBwdRows;
    HopSmem *hs = reinterpret_cast<HopSmem *>(smem + S::kHop);
    float *stat = reinterpret_cast<float *>(smem + S::kStat);   // [buffer][lse | delta | column][row]
    float *lut = reinterpret_cast<float *>(smem + S::kLut);
    float *hist = lut + (p.buckets + 2) * p.group;              // [bucket byte][thread]
    T *ds_s = reinterpret_cast<T *>(smem + S::kDs);
    const uint32_t sm = smem_u32(smem);
    const uint32_t G = p.group;

    auto stats_in = [&](uint32_t row0, int buf) {   // per row: lse in log2 units, delta, column
        if (tid < kBwdRows) {
            const uint32_t row = row0 + tid;
            float lse = INFINITY, dl = 0.0f;
            uint32_t c = 0;
            if (row < p.rows) {
                const uint32_t t = row / G, hd = hk * G + row - t * G;
                lse = p.lse[(uint64_t)t * p.hq + hd] * kLog2e;
                if (lse == -INFINITY) lse = INFINITY;       // nothing left for this row: its weights become 0
                dl = p.delta[(uint64_t)t * p.hq + hd];
                c = row_column(p, row);
            }
            float *s = stat + buf * 3 * kBwdRows;
            s[tid] = lse;
            s[kBwdRows + tid] = dl;
            reinterpret_cast<uint32_t *>(s)[2 * kBwdRows + tid] = c * kHopPitch;
        }
    };
    auto rows_in = [&](uint32_t row0, int buf) {
        const uint32_t at = sm + S::kRow + buf * 2 * S::kRowBytes;
        copy_rows<DP, kBwdRows>(at, p.q, p.q_row, p.q_head, hk * G, row0, p, tid);
        copy_rows<DP, kBwdRows>(at + S::kRowBytes, p.dout, p.dout_row, p.dout_head, hk * G, row0, p, tid);
    };

    if (tid == 0) hs->columns = 0, hs->all = 0;
    if (p.sources)
        for (int i = tid; i < 256; i += kAttnThreads) hs->bucket_of[i] = p.bucket_of[i];
    fill_bias<T>(lut, p, hk, tid, p.group);
    for (int i = tid; i < 4 * kAttnTile; i += kAttnThreads) hs->seen[0][i] = 0;
    if (MODE != 1)
        for (uint32_t i = tid; i < (p.buckets + 2) * kAttnThreads; i += kAttnThreads) hist[i] = 0.0f;
    __syncthreads();
    if (p.sources) {   // columns in use: of the block's rows, or of all queries
        const uint32_t r0 = MODE == 1 ? 0 : fixed_row0, r1 = MODE == 1 ? p.rows : min(p.rows, fixed_row0 + kBwdRows);
        uint32_t cols = 0;
        bool all = false;
        for (uint32_t r = r0 + tid * (MODE == 1 ? G : 1); r < r1; r += kAttnThreads * (MODE == 1 ? G : 1)) {
            const uint32_t c = row_column(p, r);
            if (c < p.sources) cols |= 1u << c;
            else all = true;
        }
        if (cols) atomicOr(&hs->columns, cols);
        if (all) hs->all = 1;
    }
    __syncthreads();

    const char *kbase = static_cast<const char *>(p.k) + hk * p.k_head * 2;
    const char *vbase = static_cast<const char *>(p.v) + hk * p.v_head * 2;
    const uint64_t tiles = MODE == 1 ? 1 : (split < p.tiles ? (p.tiles - split + p.splits - 1) / p.splits : 0);
    auto tile_at = [&](uint64_t i) { return MODE == 1 ? (uint64_t)blockIdx.x : split + i * p.splits; };
    int32_t h[kHopRegs];
    auto hops_in = [&](uint64_t i) { if (p.sources && i < tiles) hops_load(h, p, tile_at(i), tid); };
    auto hops_out = [&](uint64_t i, int buf) {
        if (i >= tiles) return;
        if (p.sources) hops_store(h, hs, p, tile_at(i), buf, tid);
        else hops_none(hs, p, tile_at(i), buf, tid);
    };
    auto copy = [&](uint64_t i) {
        if (i < tiles) {
            const uint32_t st = sm + (uint32_t)(i % S::kKvStages) * 2 * S::kTileBytes;
            const int64_t node0 = (int64_t)tile_at(i) * kAttnTile;
            copy_nodes<DP>(st, kbase, p.k_row * 2, node0, p.n, p.d / 8, hs->seen[i & 3], tid);
            copy_nodes<DP>(st + S::kTileBytes, vbase, p.v_row * 2, node0, p.n, p.d / 8, hs->seen[i & 3], tid);
        }
        cp_commit();
    };

    // p^T and ds^T of this warp's 16 nodes against the 32 rows in buffer rb
    float pt[R8][4], dt[R8][4];
    auto scores = [&](uint32_t kst, uint32_t vst, uint32_t rst, int rb, uint32_t row0, const uint8_t *bt) {
#pragma unroll
        for (int j = 0; j < R8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) pt[j][x] = dt[j][x] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < D16; ++kk) {
            uint32_t a[4], b[4];
            load_a<DP>(a, kst, warp * 16, kk, lane);
#pragma unroll
            for (int j = 0; j < R8; j += 2) {
                load_b<DP>(b, rst, j * 8, kk, lane);
                Elem<T>::mma(pt[j], a, b[0], b[1]);
                Elem<T>::mma(pt[j + 1], a, b[2], b[3]);
            }
            load_a<DP>(a, vst, warp * 16, kk, lane);
#pragma unroll
            for (int j = 0; j < R8; j += 2) {
                load_b<DP>(b, rst + S::kRowBytes, j * 8, kk, lane);
                Elem<T>::mma(dt[j], a, b[0], b[1]);
                Elem<T>::mma(dt[j + 1], a, b[2], b[3]);
            }
        }
        const float *st = stat + rb * 3 * kBwdRows;
        const uint32_t *cs = reinterpret_cast<const uint32_t *>(st) + 2 * kBwdRows;
        const int na = warp * 16 + (lane >> 2), nb = na + 8;
#pragma unroll
        for (int j = 0; j < R8; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = j * 8 + (lane & 3) * 2 + x;
                const float lse = st[r], dl = st[kBwdRows + r];
                const uint32_t c = cs[r], g = (row0 + r) % G;
                const float ba = lut[bt[c + na] * G + g], bb = lut[bt[c + nb] * G + g];
                const float wa = ex2(fmaf(pt[j][x], p.scale_log2, ba) - lse);
                const float wb = ex2(fmaf(pt[j][x + 2], p.scale_log2, bb) - lse);
                pt[j][x] = wa;
                pt[j][x + 2] = wb;
                dt[j][x] = wa * (dt[j][x] - dl);
                dt[j][x + 2] = wb * (dt[j][x + 2] - dl);
            }
    };
    // acc[16 nodes x DP] += w^T (nodes x rows) times the row tile at rst (rows x DP)
    auto node_product = [&](float (&acc)[DP / 8][4], const float (&w)[R8][4], uint32_t rst) {
#pragma unroll
        for (int j = 0; j < R8; j += 2) {
            const uint32_t a[4] = {Elem<T>::pack(w[j][0], w[j][1]), Elem<T>::pack(w[j][2], w[j][3]),
                                   Elem<T>::pack(w[j + 1][0], w[j + 1][1]), Elem<T>::pack(w[j + 1][2], w[j + 1][3])};
#pragma unroll
            for (int c = 0; c < D16; ++c) {
                uint32_t b[4];
                load_bt<DP>(b, rst, j * 8, c, lane);
                Elem<T>::mma(acc[2 * c], a, b[0], b[1]);
                Elem<T>::mma(acc[2 * c + 1], a, b[2], b[3]);
            }
        }
    };
    // the warp's 16 x DP accumulators to its rows of a tile in shared memory, then out in 16-byte pieces
    auto store_nodes = [&](const float (&acc)[DP / 8][4], float f, uint32_t stage, void *out, int64_t s_row, int64_t s_head,
                           int64_t node0) {
        const int na = warp * 16 + (lane >> 2);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
            const uint32_t a = tile_addr<DP>(stage, na, j) + (lane & 3) * 4, b = tile_addr<DP>(stage, na + 8, j) + (lane & 3) * 4;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(Elem<T>::pack(acc[j][0] * f, acc[j][1] * f)) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(b), "r"(Elem<T>::pack(acc[j][2] * f, acc[j][3] * f)) : "memory");
        }
        __syncwarp();
        constexpr int C = DP / 8;
        T *dst = static_cast<T *>(out) + (int64_t)hk * s_head;
#pragma unroll
        for (int i = lane; i < 16 * C; i += 32) {
            const int r = warp * 16 + i / C, c = i % C;
            if ((uint64_t)(node0 + r) < p.n && c < (int)(p.d / 8)) {
                uint4 v;
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(tile_addr<DP>(stage, r, c)) : "memory");
                __stcs(reinterpret_cast<uint4 *>(dst + (node0 + r) * s_row + c * 8), v);
            }
        }
        __syncwarp();
    };

    if constexpr (MODE == 1) {
        hops_in(0);
        hops_out(0, 0);
        __syncthreads();
        copy(0);
        const uint32_t nt = p.row_tiles;
        if (nt) rows_in(0, 0), stats_in(0, 0);
        cp_commit();
        float dk[DP / 8][4], dv[DP / 8][4];
#pragma unroll
        for (int j = 0; j < DP / 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) dk[j][x] = dv[j][x] = 0.0f;
        const uint32_t ks = sm, vs = sm + S::kTileBytes;
        for (uint32_t i = 0; i < nt; ++i) {
            cp_wait<0>();
            __syncthreads();
            if (i + 1 < nt) rows_in((i + 1) * kBwdRows, (i + 1) & 1), stats_in((i + 1) * kBwdRows, (i + 1) & 1);
            cp_commit();
            const uint32_t rs = sm + S::kRow + (i & 1) * 2 * S::kRowBytes;
            scores(ks, vs, rs, i & 1, i * kBwdRows, hs->tile[0]);
            node_product(dv, pt, rs + S::kRowBytes);
            node_product(dk, dt, rs);
        }
        cp_wait<0>();
        __syncthreads();
        const int64_t node0 = (int64_t)blockIdx.x * kAttnTile;
        store_nodes(dv, 1.0f, vs, p.dv, p.dv_row, p.dv_head, node0);
        store_nodes(dk, p.scale, vs, p.dk, p.dk_row, p.dk_head, node0);
    } else {
        rows_in(fixed_row0, 0);
        stats_in(fixed_row0, 0);
        hops_in(0);
        hops_out(0, 0);
        hops_in(1);
        __syncthreads();
        copy(0);
        float dq[kBwdRows / 16][DP / 32][4];     // all rows x this warp's quarter of head_dim
#pragma unroll
        for (int m = 0; m < kBwdRows / 16; ++m)
#pragma unroll
            for (int j = 0; j < DP / 32; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) dq[m][j][x] = 0.0f;
        const uint32_t rs = sm + S::kRow;
        const int hr = tid % kBwdRows, hp = tid / kBwdRows;    // the sum by bucket: this thread's row and quarter of the nodes
        for (uint64_t i = 0; i < tiles; ++i) {
            hops_out(i + 1, (i + 1) & 3);
            if (tid < kAttnTile) hs->seen[(i + 2) & 3][tid] = 0;
            cp_wait<0>();
            __syncthreads();
            copy(i + 1);
            hops_in(i + 2);
            const uint32_t ks = sm + (uint32_t)(i & 1) * 2 * S::kTileBytes, vs = ks + S::kTileBytes;
            const uint8_t *bt = hs->tile[i & 3];
            scores(ks, vs, rs, 0, fixed_row0, bt);
            {   // ds^T to shared memory in the element type: operand of dq, and terms of dbias (summed in fp32)
                const int na = warp * 16 + (lane >> 2);
#pragma unroll
                for (int j = 0; j < R8; ++j) {
                    T *at = ds_s + na * S::kDsPitch + j * 8 + (lane & 3) * 2;
                    *reinterpret_cast<uint32_t *>(at) = Elem<T>::pack(dt[j][0], dt[j][1]);
                    *reinterpret_cast<uint32_t *>(at + 8 * S::kDsPitch) = Elem<T>::pack(dt[j][2], dt[j][3]);
                }
            }
            if (MODE == 0) {
                const int64_t node0 = (int64_t)tile_at(i) * kAttnTile;
                float acc[DP / 8][4];
#pragma unroll
                for (int j = 0; j < DP / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
                node_product(acc, pt, rs + S::kRowBytes);
                store_nodes(acc, 1.0f, vs, p.dv, p.dv_row, p.dv_head, node0);
#pragma unroll
                for (int j = 0; j < DP / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
                node_product(acc, dt, rs);
                store_nodes(acc, p.scale, vs, p.dk, p.dk_row, p.dk_head, node0);
            }
            __syncthreads();
            const uint32_t dss = sm + S::kDs;
#pragma unroll
            for (int kk = 0; kk < kAttnTile / 16; ++kk) {
                uint32_t a[kBwdRows / 16][4];
#pragma unroll
                for (int m = 0; m < kBwdRows / 16; ++m) {
                    // A (rows x nodes) from ds^T [node][row]: transposed loads; matrices (nodes 0-7, rows 0-7),
                    // (nodes 0-7, rows 8-15), (nodes 8-15, rows 0-7), (nodes 8-15, rows 8-15)
                    const int nd = kk * 16 + (lane & 7) + ((lane >> 4) << 3), rw = m * 16 + ((lane >> 3) & 1) * 8;
                    ldsm4t(a[m], dss + (nd * S::kDsPitch + rw) * 2);
                }
#pragma unroll
                for (int c = 0; c < DP / 64; ++c) {
                    uint32_t b[4];
                    load_bt<DP>(b, ks, kk * 16, warp * (DP / 64) + c, lane);
#pragma unroll
                    for (int m = 0; m < kBwdRows / 16; ++m) {
                        Elem<T>::mma(dq[m][2 * c], a[m], b[0], b[1]);
                        Elem<T>::mma(dq[m][2 * c + 1], a[m], b[2], b[3]);
                    }
                }
            }
            if (p.buckets) {
                constexpr int N = kAttnTile / (kAttnThreads / kBwdRows);
                const uint8_t *bc = bt + reinterpret_cast<const uint32_t *>(stat)[2 * kBwdRows + hr] + hp * N;
                const T *d = ds_s + hp * N * S::kDsPitch + hr;
#pragma unroll
                for (int k = 0; k < N; k += 4) {
                    const uint32_t b4 = *reinterpret_cast<const uint32_t *>(bc + k);
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        hist[((b4 >> (8 * y)) & 255) * kAttnThreads + tid] += Elem<T>::to_float(d[(k + y) * S::kDsPitch]);
                }
            }
        }
        cp_wait<0>();
        // partial dq of this block: part[split][t][h][d]
        const uint32_t T_ = p.T;
#pragma unroll
        for (int m = 0; m < kBwdRows / 16; ++m)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint32_t row = fixed_row0 + m * 16 + (lane >> 2) + y * 8;
                if (row >= p.rows) continue;
                const uint32_t t = row / G, hd = hk * G + row - t * G;
                float *at = p.part + (((uint64_t)split * T_ + t) * p.hq + hd) * p.d;
#pragma unroll
                for (int j = 0; j < DP / 32; ++j) {
                    const uint32_t c = warp * (DP / 4) + j * 8 + (lane & 3) * 2;
                    if (c < p.d) *reinterpret_cast<float2 *>(at + c) = make_float2(dq[m][j][2 * y], dq[m][j][2 * y + 1]);
                }
            }
        __syncthreads();
        // partial dbias: part_ml[split][t][h][bucket]
        for (uint32_t i = tid; i < p.buckets * kBwdRows; i += kAttnThreads) {
            const uint32_t b = i % p.buckets, r = i / p.buckets, row = fixed_row0 + r;
            if (row >= p.rows) continue;
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < kAttnThreads / kBwdRows; ++k) s += hist[(b + 1) * kAttnThreads + k * kBwdRows + r];
            const uint32_t t = row / G, hd = hk * G + row - t * G;
            p.part_ml[(((uint64_t)split * T_ + t) * p.hq + hd) * p.buckets + b] = s;
        }
    }
}

// dq = scale * sum over splits; dbias = sum over splits and queries, in a fixed order.
// Blocks [0, T * hq): a row of dq each; then one block per head for dbias.
template <typename T>
__global__ void __launch_bounds__(256) attn_bwd_join_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ float red[256];
    const int tid = threadIdx.x;
    const uint64_t rows = (uint64_t)p.T * p.hq;
    if (blockIdx.x < rows) {
        const uint64_t row = blockIdx.x;
        __shared__ float4 sum[256];
        const uint32_t q4 = p.d / 4, groups = 256 / q4, c = tid % q4, g = tid / q4;
        float4 acc = make_float4(0, 0, 0, 0);
        if (g < groups)
            for (uint32_t s = g; s < p.splits; s += groups) {
                const float4 x = *reinterpret_cast<const float4 *>(p.part + (s * rows + row) * p.d + c * 4);
                acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
            }
        sum[tid] = acc;
        __syncthreads();
        if (g == 0) {
            for (uint32_t i = 1; i < groups; ++i) {
                const float4 x = sum[i * q4 + c];
                acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
            }
            const uint32_t t = (uint32_t)(row / p.hq), hd = (uint32_t)(row - (uint64_t)t * p.hq);
            uint2 w;
            w.x = Elem<T>::pack(acc.x * p.scale, acc.y * p.scale);
            w.y = Elem<T>::pack(acc.z * p.scale, acc.w * p.scale);
            *reinterpret_cast<uint2 *>(static_cast<T *>(p.dq) + (int64_t)t * p.dq_row + (int64_t)hd * p.dq_head + c * 4) = w;
        }
        return;
    }
    // block: (head, bucket)
    const uint64_t at = blockIdx.x - rows;
    const uint32_t hd = (uint32_t)(at / p.buckets), b = (uint32_t)(at - (uint64_t)hd * p.buckets);
    float s = 0.0f;
    const uint64_t total = (uint64_t)p.splits * p.T;
    for (uint64_t i = tid; i < total; i += 256) s += p.part_ml[(i * p.hq + hd) * p.buckets + b];
    red[tid] = s;
    __syncthreads();
    for (int x = 128; x; x >>= 1) {
        if (tid < x) red[tid] += red[tid + x];
        __syncthreads();
    }
    if (tid == 0) {
        // a masked bucket has weights of 0 and so a gradient of 0
        static_cast<T *>(p.dbias)[(uint64_t)hd * p.buckets + b] = Elem<T>::from_float(red[0]);
    }
}

}  // namespace k2t
