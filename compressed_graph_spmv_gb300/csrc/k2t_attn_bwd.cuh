// k2t_attn_bwd.cuh -- backward pass of the hop-biased attention on tcgen05.
//
// With p = exp(s - lse), dp = dout . v and delta = sum p dp = dout . out:
//   ds = p (dp - delta),  dv = sum p dout,  dk = scale sum ds q,
//   dq = scale sum ds k,  dbias[bucket] = sum ds.
// delta comes from attn_delta_kernel where there is a bias table.
// Everything is computed transposed, 128 nodes x 32 rows a unit: S^T = K Q^T
// and dP^T = V dO^T come out of tensor memory one node a thread; P^T and dS^T
// go back over them as A operands of dV += P^T dO and dK += dS^T Q (nodes x
// head_dim), and dS^T goes to shared memory as B operand of
// dQ^T += K^T dS (head_dim x rows) and for the sums by bucket.  As an operand it
// is rounded to the element type; the sums by bucket add what that took off,
// itself rounded, so that they sum 16 bits or more of each term.
//
// attn_bwd_nodes_kernel streams nodes past up to RT row tiles that stay: dQ^T
// accumulates in tensor memory over all nodes of the block, and (DKV) dV and
// dK of a tile are final after its row tiles: one pass makes every gradient.
// With more rows than that, attn_bwd_rows_kernel streams rows past a tile of
// nodes for dV and dK, and the first kernel runs without them: the scores are
// computed twice, and nothing is summed by atomics, so that results do not
// depend on the order of blocks.
//
// A row tile holds whole queries: (32 / G) queries x G heads, so that a row's
// head is the same in every tile, and the sums by bucket need one table a row
// of the tile.
//
// What bounds it: 32 queries over 2^18 nodes take 467 us forward and backward,
// 115 of them for delta, where the bytes take 147 (284 with keys and values
// read a second and third time): the latency of a tile's chain of scores,
// softmax, products, sums and stores, with two units in flight.  With 257
// queries over 8191 nodes the kernel that streams rows takes 40 us (tensor pipe
// busy 18% of it) and the one that streams nodes 63 (9%): there the sums by
// bucket, reads, adds and writes of shared memory for each score gradient, are
// the longest stage.
#pragma once

#include <type_traits>

#include "k2t_attn.cuh"
#include "k2t_tc.cuh"

namespace k2t {

constexpr int kBwdThreads = 800;
constexpr int kBwdRowThreads = 544;
constexpr int kBwdRows = 32;
constexpr float kWhole = 0x1p-10f;   // how far from 1 the sum of a row's weights may be: no more than this is lost in delta, less than out's rounding
using Rest = __nv_bfloat16;      // what rounding took off a score gradient, in either type: where fp16 keeps nothing, this is all of it

// What the kernels need of a row, made once by attn_rows_kernel: lse in units
// of log2 (+inf for a row that saw nothing or does not exist: its weights
// become 0), less Elem::kUp, delta, ds_scale, byte offset of its column in a bucket tile, its head's
// offset in the bias table; a row tile's together.
struct RowInfo {
    float lse[kBwdRows], delta[kBwdRows], up[kBwdRows];
    uint32_t place[kBwdRows];              // column | head << 16
};

// dout . out of query t, head hd, by L neighbour lanes (x: this one of them).
template <typename T, int L>
__device__ __forceinline__ float dout_out(const AttnParams &p, uint32_t t, uint32_t hd, int x, uint32_t lanes)
{
    float s = 0.0f;
    const T *o = static_cast<const T *>(p.out) + (int64_t)t * p.out_row + (int64_t)hd * p.out_head;
    const T *d = static_cast<const T *>(p.dout) + (int64_t)t * p.dout_row + (int64_t)hd * p.dout_head;
    for (uint32_t k = x * 8; k < p.d; k += L * 8) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(o + k)), b = __ldg(reinterpret_cast<const uint4 *>(d + k));
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 u = Elem<T>::unpack(aw[e]), v = Elem<T>::unpack(bw[e]);
            s = fmaf(u.x, v.x, fmaf(u.y, v.y, s));
        }
    }
    for (int y = L / 2; y; y >>= 1) s += __shfl_xor_sync(lanes, s, y);
    return s;
}

// delta of query t, head hd, by L neighbour lanes (x: this one of them): from the sums over nodes that attn_delta_kernel left,
// or dout . out without them; 0 for a query that does not exist or saw nothing.  up: ds_scale of the row.
// The weights of a row sum to 1, but for the rounding of lse, unless its lse and out are of more nodes than this call's (nodes
// taken in parts): what these nodes' sums lack is then in out.
template <typename T, int L>
__device__ __forceinline__ float row_delta(const AttnParams &p, uint32_t t, uint32_t hd, int x, uint32_t lanes, float &up)
{
    float top = 0.0f, delta = 0.0f;
    if (t < p.T) {
        if (p.delta_splits) {
            float s = 0.0f, m = 0.0f;
            for (uint32_t i = x; i < p.delta_splits; i += L) {
                const uint64_t at = ((uint64_t)i * p.T + t) * p.hq + hd;
                const float2 v = p.delta_part[at];
                s += v.x, m += v.y;
                if (Elem<T>::kUp) top = fmaxf(top, p.pdp_top[at]);
            }
            for (int y = L / 2; y; y >>= 1) {
                s += __shfl_xor_sync(lanes, s, y);
                m += __shfl_xor_sync(lanes, m, y);
                if (Elem<T>::kUp) top = fmaxf(top, __shfl_xor_sync(lanes, top, y));
            }
            delta = m == 0.0f ? 0.0f : fabsf(m - 1.0f) > kWhole ? dout_out<T, L>(p, t, hd, x, lanes) : s / m;
        } else {
            delta = dout_out<T, L>(p, t, hd, x, lanes);
        }
    }
    up = ds_scale<T>(top + fabsf(delta));
    return delta;
}

template <typename T>
__global__ void __launch_bounds__(256) attn_rows_kernel(const __grid_constant__ AttnParams p)
{
    const uint32_t at = blockIdx.x * 8 + (threadIdx.x >> 5), hk = blockIdx.y;     // row of a tile, padded: a warp each
    if (at >= p.row_tiles * kBwdRows) return;
    tc::grid_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t G = p.group, per = kBwdRows / G, c = at % kBwdRows, t = at / kBwdRows * per + c / G, g = c % G;
    float lse = INFINITY, s = 0.0f, up = ds_scale<T>(0.0f);
    uint32_t place = 0;
    if (c < per * G && t < p.T) {
        const uint32_t hd = hk * G + g;
        s = row_delta<T, 32>(p, t, hd, lane, ~0u, up);
        const float l = p.lse[(uint64_t)t * p.hq + hd];
        if (l != -INFINITY) lse = l * kLog2e - Elem<T>::kUp;
        place = row_column(p, t * G) * kTcPitch | (g * 4) << 16;
    }
    RowInfo *to = static_cast<RowInfo *>(p.row_info) + (uint64_t)hk * p.row_tiles + at / kBwdRows;
    if (lane == 0) to->lse[c] = lse, to->delta[c] = s, to->up[c] = up, to->place[c] = place;
}

// The least ds_scale of some row tiles' rows, by a warp.
__device__ __forceinline__ float least_up(const RowInfo *info, uint32_t row_tiles, int lane)
{
    float up = info[0].up[lane];
    for (uint32_t i = 1; i < row_tiles; ++i) up = fminf(up, info[i].up[lane]);
    return __uint_as_float(__reduce_min_sync(~0u, __float_as_uint(up)));        // of numbers that are not negative: as their bits
}

// Copies ROWS (a multiple of 32) rows of tile `tile` on of a [T, heads, d] tensor into row tiles of 32 rows:
// panels of 64 values, 4096 bytes each, swizzled.  Rows that do not exist are zeros.
template <int DP>
__device__ __forceinline__ void copy_row_tile(uint32_t dst, const void *base, int64_t s_row, int64_t s_head, uint32_t head0,
                                              uint32_t tile, const AttnParams &p, int first, int step)
{
    constexpr int C = DP / 8;
    const uint32_t G = p.group, per = kBwdRows / G, fill = (p.d / 8 + 1) & ~1u;
    for (int i = first; i < kBwdRows * C; i += step) {
        const uint32_t r = i / C, c = i % C, q = r / G, t = tile * per + q, g = r - q * G;
        const bool on = q < per && t < p.T && c < p.d / 8;
        const char *src = static_cast<const char *>(base) + (on ? ((int64_t)t * s_row + (int64_t)(head0 + g) * s_head + c * 8) * 2 : 0);
        if (c < fill) cp16(dst + tc::chunk(r, c, 4096), src, on ? 16 : 0);
    }
}

// up: the least ds_scale of the head's rows.
// A unit's softmax step for one node: S^T and dP^T at `at` (32 columns each, a row of the tile a column) become P^T
// and dS^T in the element type, two rows a column; ds: this node's row of dS^T in shared memory, from chunk `chunk` on
// (null: not wanted), and `rest` bytes on what the rounding took off, itself rounded (rest 0: not wanted); bt: the node's bytes in the bucket tile (column 0); lut: bias table, bytes.
// Eight rows at a time in a rolled loop: the warps of an SM run half a dozen different loops, and the instruction
// caches hold them only while each is small.
template <typename T>
__device__ __forceinline__ void unit32(uint32_t at, const RowInfo *info, bool plain, float scale, float up, const uint8_t *bt,
                                       const uint8_t *lut, uint32_t shift, uint8_t *ds, uint32_t rest, uint32_t chunk, uint32_t node)
{
#pragma unroll 1
    for (int r0 = 0; r0 < kBwdRows; r0 += 8) {
        uint32_t s[8], d[8], pw[4], dw[4], rw[4], kw[4];
        tc::ld8(s, at + r0);
        tc::ld8(d, at + 32 + r0);
        float b[8] = {};
        if (!plain) {
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const uint4 c4 = *reinterpret_cast<const uint4 *>(&info->place[r0 + e]);
                const uint32_t place[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint32_t k = bt[place[y] & 0xffff];
                    b[e + y] = *reinterpret_cast<const float *>(lut + (k << shift) + (place[y] >> 16));
                }
            }
        }
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const float4 lse4 = *reinterpret_cast<const float4 *>(&info->lse[r0 + e]), dl4 = *reinterpret_cast<const float4 *>(&info->delta[r0 + e]);
            const float lse[4] = {lse4.x, lse4.y, lse4.z, lse4.w}, delta[4] = {dl4.x, dl4.y, dl4.z, dl4.w};
            float pv[4], dv[4], own[4];
            if (Elem<T>::kUp && ds) *reinterpret_cast<float4 *>(own) = *reinterpret_cast<const float4 *>(&info->up[r0 + e]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                pv[y] = ex2(fmaf(__uint_as_float(s[e + y]), scale, b[e + y]) - lse[y]);
                const float x = __uint_as_float(d[e + y]) - delta[y];
                dv[y] = pv[y] * (Elem<T>::kUp ? x * (ds ? own[y] : up) : x);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                pw[e / 2 + y] = Elem<T>::pack(pv[2 * y], pv[2 * y + 1]);
                dw[e / 2 + y] = Elem<T>::pack(dv[2 * y], dv[2 * y + 1]);
                const float2 kept = Elem<T>::unpack(dw[e / 2 + y]);
                rw[e / 2 + y] = Elem<Rest>::pack(dv[2 * y] - kept.x, dv[2 * y + 1] - kept.y);
                kw[e / 2 + y] = Elem<T>::kUp && ds ? Elem<T>::pack(dv[2 * y] * (up * inverse_power(own[2 * y])),
                                                                   dv[2 * y + 1] * (up * inverse_power(own[2 * y + 1]))) : dw[e / 2 + y];
            }
        }
        tc::st4(at + r0 / 2, pw);
        tc::st4(at + 32 + r0 / 2, kw);
        if (ds) {
            uint8_t *to = ds + (((chunk + r0 / 8) ^ (node & 7)) << 4);
            *reinterpret_cast<uint4 *>(to) = make_uint4(dw[0], dw[1], dw[2], dw[3]);
            if (rest) *reinterpret_cast<uint4 *>(to + rest) = make_uint4(rw[0], rw[1], rw[2], rw[3]);
        }
    }
}

// One node's (lane's) head_dim of fp32 accumulators, rounded, to row `row` of a tile in shared memory.
template <typename T, int DP>
__device__ __forceinline__ void load_nodes(uint32_t tm_at, float f, uint32_t stage, int row)
{
#pragma unroll 1
    for (int c = 0; c < DP; c += 32) {
        uint32_t v[32];
        tc::ld32(v, tm_at + c);
        tc::wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = Elem<T>::pack(__uint_as_float(v[j * 8 + 2 * e]) * f, __uint_as_float(v[j * 8 + 2 * e + 1]) * f);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(stage + tc::chunk(row, c / 8 + j, kTcTile * 128)), "r"(w[0]),
                         "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
        }
    }
}
// S^T = K Q^T at `at`, dP^T = V dO^T 32 columns on.
template <int DP, int PANEL>
__device__ __forceinline__ void score_products(bool lead, uint32_t at, uint64_t k, uint64_t q, uint64_t v, uint64_t g, uint32_t id, uint32_t dn)
{
#pragma unroll
    for (uint32_t kk = 0; kk < DP / 16; ++kk)
        if (kk * 16 < dn) tc::mma_ss(lead, at, k, (kk >> 2) * PANEL + (kk & 3) * 32, q, (kk >> 2) * 4096 + (kk & 3) * 32, id, kk > 0);
#pragma unroll
    for (uint32_t kk = 0; kk < DP / 16; ++kk)
        if (kk * 16 < dn) tc::mma_ss(lead, at + 32, v, (kk >> 2) * PANEL + (kk & 3) * 32, g, (kk >> 2) * 4096 + (kk & 3) * 32, id, kk > 0);
}
// dV (+)= P^T dO, dK (+)= dS^T Q with P^T at `at` and dS^T 32 columns on.
__device__ __forceinline__ void node_products(bool lead, uint32_t at, uint32_t dv, uint32_t dk, uint64_t q, uint64_t g, uint32_t id, bool add)
{
#pragma unroll
    for (uint32_t kk = 0; kk < 2; ++kk) tc::mma_ts(lead, dv, at + kk * 8, g, kk * 2048, id, add || kk > 0);
#pragma unroll
    for (uint32_t kk = 0; kk < 2; ++kk) tc::mma_ts(lead, dk, at + 32 + kk * 8, q, kk * 2048, id, add || kk > 0);
}

template <int DP, int RT, bool DKV> struct BwdSmem {
    static constexpr int kPanel = kTcTile * 128;
    static constexpr int kSlot = kPanel * (DP / 64);
    static constexpr int kSlots = DP == 64 ? (RT == 1 ? 8 : 6) : DKV ? 4 : 3;
    static constexpr int kBufs = DP == 64 ? 6 : 2;                            // bucket tiles
    static constexpr int kRowTile = kBwdRows * DP * 2;                        // q or dout of a row tile
    static constexpr int kRow = kSlots * kSlot;                               // [RT][q | dout]
    static constexpr int kDs = kRow + RT * 2 * kRowTile;                      // dS^T [node][unit parity][32 rows]
    static constexpr int kBuckets = kDs + 2 * kPanel;                         // after what rounding took off dS^T
    static constexpr int kInfo = kBuckets + kBufs * 33 * kTcPitch;
    static constexpr int kCtl = kInfo + RT * (int)sizeof(RowInfo);
    struct Ctl {
        uint64_t full[kSlots], empty[kSlots], hop_full[kBufs], hop_empty[kBufs], sp_full[2], ds_full[2], hist_done[2];
        uint64_t tile_full, tile_empty, staged, dq_full, drained;
        uint32_t tmem, gave_up, columns, all;
        uint32_t seen[kBufs][4];
        uint8_t byte_of[257 + 15];
    };
    static constexpr int kLut = kCtl + (int)((sizeof(Ctl) + 15) / 16 * 16);
    // threads: those that sum by bucket, a table each
    static size_t bytes(const AttnParams &p, uint32_t threads)
    {
        return kLut + ((size_t)(p.buckets + 2) * p.group2 + (p.buckets ? (size_t)(p.buckets + 2) * threads : 0)) * 4;
    }
};

template <typename T, int DP, int RT, bool DKV>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_bwd_nodes_kernel(const __grid_constant__ AttnParams p)
{
    using S = BwdSmem<DP, RT, DKV>;
    using Ctl = typename S::Ctl;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kDv = 128, kDk = 128 + DP, kDq = DKV ? 128 + 2 * DP : 128;    // columns of tensor memory
    static_assert(kDq + RT * 32 <= 512, "tensor memory");
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + S::kCtl);
    const uint32_t sm = tc::saddr(smem);
    float *lut = reinterpret_cast<float *>(smem + S::kLut), *hist = lut + (p.buckets + 2) * p.group2;   // [bucket byte][thread]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t hk = blockIdx.y, split = blockIdx.x % p.splits, rows_of = blockIdx.x / p.splits;
    const uint32_t rt0 = rows_of * RT, rts = min((uint32_t)RT, p.row_tiles - rt0);      // row tiles of this block
    const uint32_t tiles = (uint32_t)(split < p.tiles ? (p.tiles - split + p.splits - 1) / p.splits : 0);
    const uint32_t units = tiles * rts;                                                 // unit u: tile u / rts, row tile u % rts
    auto tile_at = [&](uint32_t i) { return split + (uint64_t)i * p.splits; };

    // ---- set-up ----
    if (warp == 24) tc::alloc(&ctl->tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) tc::bar_init(&ctl->full[i], 128), tc::bar_init(&ctl->empty[i], 1);
        for (int i = 0; i < S::kBufs; ++i) {
            tc::bar_init(&ctl->hop_full[i], 4);
            tc::bar_init(&ctl->hop_empty[i], rts * (4 + (p.buckets ? p.hist_threads / 32 : 0)));
        }
        for (int i = 0; i < 2; ++i) tc::bar_init(&ctl->sp_full[i], 1), tc::bar_init(&ctl->ds_full[i], 128), tc::bar_init(&ctl->hist_done[i], p.hist_threads / 32);
        tc::bar_init(&ctl->tile_full, 1);
        tc::bar_init(&ctl->tile_empty, 128);
        tc::bar_init(&ctl->staged, 128);
        tc::bar_init(&ctl->dq_full, 1);
        tc::bar_init(&ctl->drained, 1);
        ctl->gave_up = ctl->columns = ctl->all = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc::grid_wait();
    for (uint32_t r = 0; r < rts; ++r) {
        const uint32_t at = sm + S::kRow + r * 2 * S::kRowTile;
        copy_row_tile<DP>(at, p.q, p.q_row, p.q_head, hk * p.group, rt0 + r, p, tid, kBwdThreads);
        copy_row_tile<DP>(at + S::kRowTile, p.dout, p.dout_row, p.dout_head, hk * p.group, rt0 + r, p, tid, kBwdThreads);
    }
    cp_commit();
    if (p.sources)
        for (int i = tid; i < 257; i += kBwdThreads) ctl->byte_of[i] = i ? p.bucket_of[i - 1] + 1 : 0;
    fill_bias<T>(lut, p, hk, tid, p.group2);
    if (p.buckets)
        for (uint32_t i = tid; i < (p.buckets + 2) * p.hist_threads; i += kBwdThreads) hist[i] = 0.0f;
    RowInfo *info = reinterpret_cast<RowInfo *>(smem + S::kInfo);
    __syncthreads();
    auto seen_by = [&](uint32_t place) {
        const uint32_t col = (place & 0xffff) / kTcPitch;
        if (col < p.sources) atomicOr(&ctl->columns, 1u << col);
        else ctl->all = 1;
    };
    if (DKV) {
        // what attn_rows_kernel does, for the rows that this block holds: eight threads a row
        for (int at = tid >> 3; at < (int)rts * kBwdRows; at += kBwdThreads / 8) {
            const uint32_t c = at % kBwdRows, per = kBwdRows / p.group, t = (rt0 + at / kBwdRows) * per + c / p.group, g = c % p.group;
            const bool on = c < per * p.group && t < p.T;
            const uint32_t hd = hk * p.group + g;
            float row_up;
            const float s = row_delta<T, 8>(p, on ? t : p.T, hd, tid & 7, 0xffu << (lane & 24), row_up);
            if ((tid & 7) == 0) {
                RowInfo *to = info + at / kBwdRows;
                float lse = INFINITY;
                uint32_t place = 0;
                if (on) {
                    const float l = p.lse[(uint64_t)t * p.hq + hd];
                    if (l != -INFINITY) lse = l * kLog2e - Elem<T>::kUp;
                    place = row_column(p, t * p.group) * kTcPitch | (g * 4) << 16;
                    if (p.sources) seen_by(place);
                }
                to->lse[c] = lse, to->delta[c] = s, to->up[c] = row_up, to->place[c] = place;
            }
        }
    } else if (tid < (int)rts * kBwdRows) {
        const RowInfo *from = static_cast<const RowInfo *>(p.row_info) + (uint64_t)hk * p.row_tiles + rt0 + tid / kBwdRows;
        RowInfo *to = info + tid / kBwdRows;
        const uint32_t c = tid % kBwdRows, place = from->place[c], per = kBwdRows / p.group, t = (rt0 + tid / kBwdRows) * per + c / p.group;
        to->lse[c] = from->lse[c], to->delta[c] = from->delta[c], to->up[c] = from->up[c], to->place[c] = place;
        if (p.sources && c < per * p.group && t < p.T) seen_by(place);
    }
    cp_wait<0>();
    tc::fence_async();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    tc::grid_next();
    const uint32_t tm = ctl->tmem;
    volatile uint32_t *gave_up = &ctl->gave_up;
    const float up = Elem<T>::kUp ? least_up(info, rts, lane) : 1.0f;      // and what takes the powers of two out of the results:
    const float p_down = 1.0f / (1u << Elem<T>::kUp), ds_down = p_down / up;
    auto row_down = [&](uint32_t r, uint32_t c) { return Elem<T>::kUp ? p_down * inverse_power(info[r].up[c]) : 1.0f; };

    if (warp < 8) {
        // ---- softmax: thread = node of a tile; group w takes the units of parity w ----
        const int w = warp >> 2, l = tid & 127;
        const uint32_t at = tm + ((uint32_t)(warp & 3) << 21) + w * 64, shift = p.group2_log + 2;
        uint8_t *ds = smem + S::kDs + l * 128;
        uint32_t i = 0, r = w;
        while (r >= rts) r -= rts, ++i;
        for (uint32_t u = w, k = 0; u < units; u += 2, ++k) {
            const uint32_t buf = i % S::kBufs;
            bool ok = tc::bar_wait(&ctl->hop_full[buf], (i / S::kBufs) & 1, gave_up) && tc::bar_wait(&ctl->sp_full[w], k & 1, gave_up);
            if (ok && k > 0 && p.buckets) ok = tc::bar_wait(&ctl->hist_done[w], (k - 1) & 1, gave_up);
            if (!__all_sync(~0u, ok)) break;
            tc::fence_after();
            const bool plain = !p.sources && (tile_at(i) + 1) * kTcTile <= p.n;
            unit32<T>(at, info + r, plain, p.scale_log2, up, smem + S::kBuckets + buf * 33 * kTcPitch + l,
                      reinterpret_cast<const uint8_t *>(lut), shift, ds, p.buckets ? S::kPanel : 0, w * 4, l);
            tc::wait_st();
            tc::fence_async();
            tc::fence_before();
            tc::bar_arrive(&ctl->ds_full[w]);
            __syncwarp();
            if (lane == 0) tc::bar_arrive(&ctl->hop_empty[buf]);
            r += 2;
            while (r >= rts) r -= rts, ++i;
        }
    } else if (warp < 12) {
        hop_warps<S::kBufs>(p, ctl, smem + S::kBuckets, warp - 8, lane, tiles, split, gave_up);
    } else if (warp < 16) {
        node_warps<DP, S::kSlots, S::kBufs>(p, ctl, sm, warp - 12, lane, hk, tiles, split, gave_up);
    } else if (warp < 20) {
        // ---- results: dv and dk of each tile, then dq ----
        const int ew = warp - 16, l = ew * 32 + lane;
        const uint32_t lanes = (uint32_t)ew << 21;
        bool ok = true;
        if (DKV)
            for (uint32_t i = 0; i < tiles; ++i) {
                ok = __all_sync(~0u, tc::bar_wait(&ctl->tile_full, i & 1, gave_up));
                if (!ok) break;
                tc::fence_after();
                // the tile's own slots are free to hold its results: every product that read them is done
                const uint32_t ks = slot_of<S::kSlots>(2 * i), vs = slot_of<S::kSlots>(2 * i + 1);
#pragma unroll 1
                for (int x = 0; x < 2; ++x) load_nodes<T, DP>(tm + lanes + (x ? kDk : kDv), x ? p.scale * ds_down : p_down, sm + (x ? ks : vs) * S::kSlot, l);
                tc::fence_before();
                tc::bar_arrive(&ctl->tile_empty);
                tc::fence_async();
                tc::bar_arrive(&ctl->staged);
                if (l == 0) {
                    ok = tc::bar_wait(&ctl->staged, i & 1, gave_up);
                    if (!ok) break;
                    const int32_t node0 = (int32_t)(tile_at(i) * kTcTile);
                    for (int c = 0; c < (int)p.d; c += 64) {
                        tc::store_box(&p.dk_map, sm + ks * S::kSlot + c / 64 * S::kPanel, c, hk, node0);
                        tc::store_box(&p.dv_map, sm + vs * S::kSlot + c / 64 * S::kPanel, c, hk, node0);
                    }
                    tc::stores_commit();
                    tc::stores_read();
                    tc::bar_arrive(&ctl->empty[ks]);
                    tc::bar_arrive(&ctl->empty[vs]);
                }
            }
        if (l == 0) tc::stores_done();
        ok = __all_sync(~0u, ok);
        if (ok && units > 0) ok = __all_sync(~0u, tc::bar_wait(&ctl->dq_full, 0, gave_up));
        if (ok) {
            tc::fence_after();
            const uint32_t G = p.group, per = kBwdRows / G;
            for (uint32_t r = 0; r < rts; ++r) {
                uint32_t v[32];
                if (units > 0) {
                    tc::ld32(v, tm + lanes + kDq + r * 32);
                    tc::wait_ld();
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const uint32_t q = c / G, t = (rt0 + r) * per + q, hd = hk * G + c - q * G;
                    if (l < (int)p.d && q < per && t < p.T) {
                        const float x = units > 0 ? __uint_as_float(v[c]) * row_down(r, c) : 0.0f;
                        if (p.splits > 1) p.part[(((uint64_t)split * p.T + t) * p.hq + hd) * p.d + l] = x;
                        else static_cast<T *>(p.dq)[(int64_t)t * p.dq_row + (int64_t)hd * p.dq_head + l] = Elem<T>::from_float(x * p.scale);
                    }
                }
            }
        }
    } else if (warp < 24) {
        // ---- sums of ds by bucket: thread = (row of the tile, quarter or half of the nodes), with a table of its own ----
        if (p.buckets) {
            const int t = tid - 640, c = t & 31, part = t >> 5, parts = p.hist_threads / 32, span = kTcTile / parts;
            const uint32_t pitch = p.hist_threads * 4;                          // bytes a bucket
            uint8_t *mine = reinterpret_cast<uint8_t *>(hist + t);
            uint32_t i = 0, r = 0;
            for (uint32_t u = 0; u < units && part < parts; ++u) {
                const uint32_t w = u & 1, buf = i % S::kBufs;
                bool ok = tc::bar_wait(&ctl->hop_full[buf], (i / S::kBufs) & 1, gave_up) && tc::bar_wait(&ctl->ds_full[w], (u >> 1) & 1, gave_up);
                if (!__all_sync(~0u, ok)) break;
                const uint8_t *bt = smem + S::kBuckets + buf * 33 * kTcPitch + (info[r].place[c] & 0xffff) + part * span;
                const uint8_t *ds = smem + S::kDs + part * span * 128 + (c & 7) * 2;
                const uint32_t chunk = w * 4 + (c >> 3);
                // ds in full: its rounded value and what that took off
                const float down = row_down(r, c);
                auto term = [&](int node) {
                    const uint8_t *at = ds + node * 128 + ((chunk ^ (node & 7)) << 4);
                    const float x = Elem<T>::to_float(*reinterpret_cast<const T *>(at)) + Elem<Rest>::to_float(*reinterpret_cast<const Rest *>(at + S::kPanel));
                    return Elem<T>::kUp ? x * down : x;
                };
                // A node is a read, an add and a write of its bucket.  Four nodes go on at once: the reads before the first
                // write, a node that shares the bucket of one before it continues from that one's sum, and the writes in the
                // nodes' order, so that the last of a bucket stands.  The next four nodes' terms are read meanwhile.  (257 queries
                // over 8191 nodes, forward and backward, 157 us, one node after another 163; 32 over 2^18 467 and 474.)
                uint32_t bw = *reinterpret_cast<const uint32_t *>(bt);
                float x0 = term(0), x1 = term(1), x2 = term(2), x3 = term(3);
#pragma unroll 1
                for (int k = 0; k < span; k += 4) {
                    float *a0 = reinterpret_cast<float *>(mine + (bw & 255) * pitch), *a1 = reinterpret_cast<float *>(mine + (bw >> 8 & 255) * pitch);
                    float *a2 = reinterpret_cast<float *>(mine + (bw >> 16 & 255) * pitch), *a3 = reinterpret_cast<float *>(mine + (bw >> 24) * pitch);
                    const float s0 = *a0, s1 = *a1, s2 = *a2, s3 = *a3;
                    const int next = k + 4 < span ? k + 4 : k;
                    bw = *reinterpret_cast<const uint32_t *>(bt + next);
                    const float n0 = term(next), n1 = term(next + 1), n2 = term(next + 2), n3 = term(next + 3);
                    const float v0 = s0 + x0;
                    const float v1 = (a1 == a0 ? v0 : s1) + x1;
                    const float v2 = (a2 == a1 ? v1 : a2 == a0 ? v0 : s2) + x2;
                    const float v3 = (a3 == a2 ? v2 : a3 == a1 ? v1 : a3 == a0 ? v0 : s3) + x3;
                    *a0 = v0;
                    *a1 = v1;
                    *a2 = v2;
                    *a3 = v3;
                    x0 = n0, x1 = n1, x2 = n2, x3 = n3;
                }
                __syncwarp();
                if (lane == 0) tc::bar_arrive(&ctl->hist_done[w]), tc::bar_arrive(&ctl->hop_empty[buf]);
                if (++r == rts) r = 0, ++i;
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            // part_ml[split][row group][head][bucket]
            const uint32_t G = p.group, per = kBwdRows / G;
            float *out = p.part_ml + (((uint64_t)blockIdx.x * p.hkv + hk) * G) * p.buckets;
            for (uint32_t k = t; k < G * p.buckets; k += 128) {
                const uint32_t g = k / p.buckets, b = k - g * p.buckets;
                float s = 0.0f;
                for (uint32_t q = 0; q < per; ++q)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (x < parts) s += hist[(b + 1) * p.hist_threads + x * 32 + q * G + g];
                out[k] = s;
            }
        }
    } else {
        // ---- products ----
        const bool lead = tc::elect();
        const uint32_t dn = (p.d + 15) & ~15u;
        const uint32_t id_s = tc::idesc(kBf16, 32, false, false), id_n = tc::idesc(kBf16, dn, false, true), id_q = tc::idesc(kBf16, 32, true, true);
        // Scores run up to two units ahead of the gradients' products; whichever has its operands goes first.
        uint32_t next = 0, si = 0, sr = 0, done = 0, i = 0, r = 0;      // (tile, row tile) of the next scores, of the next gradients
        tc::Patience wait(gave_up);
        while (done < units) {
            if (next < units && next < done + 2) {
                const uint32_t w = next & 1, ks = slot_of<S::kSlots>(2 * si), vs = slot_of<S::kSlots>(2 * si + 1);
                if (sr > 0 || __all_sync(~0u, tc::bar_peek(&ctl->full[ks], slot_use<S::kSlots>(2 * si) & 1) &&
                                                  tc::bar_peek(&ctl->full[vs], slot_use<S::kSlots>(2 * si + 1) & 1))) {
                    tc::fence_async();
                    tc::fence_after();
                    const uint32_t qa = sm + S::kRow + sr * 2 * S::kRowTile;
                    const uint64_t q = tc::desc(qa, 4096), g = tc::desc(qa + S::kRowTile, 4096);
                    const uint64_t k = tc::desc(sm + ks * S::kSlot, S::kPanel), v = tc::desc(sm + vs * S::kSlot, S::kPanel);
                    score_products<DP, S::kPanel>(lead, tm + w * 64, k, q, v, g, id_s, dn);
                    tc::commit(lead, &ctl->sp_full[w]);
                    if (!DKV && sr + 1 == rts) tc::commit(lead, &ctl->empty[vs]);      // values are read by the scores alone
                    if (++sr == rts) sr = 0, ++si;
                    ++next;
                    wait.restart();
                    continue;
                }
            }
            const uint32_t w = done & 1;
            if (done < next && __all_sync(~0u, tc::bar_peek(&ctl->ds_full[w], (done >> 1) & 1) &&
                                                   (!DKV || r > 0 || i == 0 || tc::bar_peek(&ctl->tile_empty, (i - 1) & 1)))) {
                tc::fence_async();
                tc::fence_after();
                const uint32_t ks = slot_of<S::kSlots>(2 * i), qa = sm + S::kRow + r * 2 * S::kRowTile;
                if (DKV) node_products(lead, tm + w * 64, tm + kDv, tm + kDk, tc::desc(qa, 4096), tc::desc(qa + S::kRowTile, 4096), id_n, r > 0);
                const uint64_t k = tc::desc(sm + ks * S::kSlot, S::kPanel), ds = tc::desc(sm + S::kDs + w * 64, 4096);
#pragma unroll
                for (uint32_t kk = 0; kk < kTcTile / 16; ++kk)
                    tc::mma_ss(lead, tm + kDq + r * 32, k, kk * 2048, ds, kk * 2048, id_q, i > 0 || kk > 0);
                if (r + 1 == rts) {
                    if (DKV) tc::commit(lead, &ctl->tile_full);
                    else tc::commit(lead, &ctl->empty[ks]);
                }
                if (++done == units) tc::commit(lead, &ctl->dq_full);
                if (++r == rts) r = 0, ++i;
                wait.restart();
                continue;
            }
            if (!__all_sync(~0u, wait.more())) break;
        }
        const bool ok = done == units;
        if (!ok) tc::drain(lead, &ctl->drained, 0);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 24) tc::dealloc(tm, 512);
    if (tid == 0 && *gave_up) atomicOr(p.status, K2T_STATUS_WAIT_TIMEOUT);
}

template <int DP> struct BwdRowSmem {
    static constexpr int kPanel = kTcTile * 128;
    static constexpr int kSlot = kPanel * (DP / 64);
    static constexpr int kRowTile = kBwdRows * DP * 2;
    static constexpr int kRing = 5;                                         // row tiles in flight
    static constexpr int kRow = 2 * kSlot;                                  // keys, values; then [ring][q | dout]
    static constexpr int kBuckets = kRow + kRing * 2 * kRowTile;
    static constexpr int kInfo = kBuckets + 33 * kTcPitch;
    static constexpr int kCtl = kInfo + kRing * (int)sizeof(RowInfo);
    struct Ctl {
        uint64_t full[2], empty[2], hop_full[1], hop_empty[1], row_full[kRing], row_empty[kRing], sp_full[2], ds_full[2], tile_full, drained;
        uint32_t tmem, gave_up, columns, all, up;
        uint32_t seen[1][4];
        uint8_t byte_of[257 + 15];
    };
    static constexpr int kLut = kCtl + (int)((sizeof(Ctl) + 15) / 16 * 16);
    static size_t bytes(const AttnParams &p) { return kLut + (size_t)(p.buckets + 2) * p.group2 * 4; }
};

// dv and dk of one tile of nodes: the rows stream past it.
template <typename T, int DP>
__global__ void __launch_bounds__(kBwdRowThreads, 1) attn_bwd_rows_kernel(const __grid_constant__ AttnParams p)
{
    using S = BwdRowSmem<DP>;
    using Ctl = typename S::Ctl;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kDv = 128, kDk = 128 + DP, kCols = DP == 64 ? 256 : 512;     // columns of tensor memory
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + S::kCtl);
    const uint32_t sm = tc::saddr(smem);
    float *lut = reinterpret_cast<float *>(smem + S::kLut);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t hk = blockIdx.y, units = p.row_tiles;
    const uint64_t tile = blockIdx.x;

    if (warp == 16) tc::alloc(&ctl->tmem, kCols);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) tc::bar_init(&ctl->full[i], 128), tc::bar_init(&ctl->empty[i], 1), tc::bar_init(&ctl->sp_full[i], 1), tc::bar_init(&ctl->ds_full[i], 128);
        tc::bar_init(&ctl->hop_full[0], 4);
        tc::bar_init(&ctl->hop_empty[0], 1);
        for (int i = 0; i < S::kRing; ++i) tc::bar_init(&ctl->row_full[i], 128), tc::bar_init(&ctl->row_empty[i], 1);
        tc::bar_init(&ctl->tile_full, 1);
        tc::bar_init(&ctl->drained, 1);
        ctl->gave_up = ctl->columns = ctl->all = 0;
        ctl->up = __float_as_uint(INFINITY);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (p.sources)
        for (int i = tid; i < 257; i += kBwdRowThreads) ctl->byte_of[i] = i ? p.bucket_of[i - 1] + 1 : 0;
    tc::grid_wait();
    fill_bias<T>(lut, p, hk, tid, p.group2);
    __syncthreads();
    if (Elem<T>::kUp) {
        const RowInfo *rows = static_cast<const RowInfo *>(p.row_info) + (uint64_t)hk * p.row_tiles;
        const uint32_t each = (p.row_tiles + kBwdRowThreads / 32 - 1) / (kBwdRowThreads / 32), from = warp * each;
        if (from < p.row_tiles) {
            const float up = least_up(rows + from, min(each, p.row_tiles - from), lane);
            if (lane == 0) atomicMin(&ctl->up, __float_as_uint(up));
        }
    }
    if (p.sources) {
        uint32_t cols = 0;
        bool all = false;
        for (uint32_t t = tid; t < p.T; t += kBwdRowThreads) {
            const uint32_t c = row_column(p, t * p.group);
            if (c < p.sources) cols |= 1u << c;
            else all = true;
        }
        if (cols) atomicOr(&ctl->columns, cols);
        if (all) ctl->all = 1;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    tc::grid_next();
    const uint32_t tm = ctl->tmem;
    volatile uint32_t *gave_up = &ctl->gave_up;
    const float up = Elem<T>::kUp ? __uint_as_float(ctl->up) : 1.0f;       // and what takes the powers of two out of the results:
    const float p_down = 1.0f / (1u << Elem<T>::kUp), ds_down = p_down / up;

    if (warp < 8) {
        const int w = warp >> 2, l = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21, shift = p.group2_log + 2;
        const bool plain = !p.sources && (tile + 1) * kTcTile <= p.n;
        bool ok = __all_sync(~0u, tc::bar_wait(&ctl->hop_full[0], 0, gave_up));
        for (uint32_t u = w, k = 0; u < units && ok; u += 2, ++k) {
            const uint32_t slot = u % S::kRing;
            // row_full: this thread reads the row facts that came with the row tile
            ok = tc::bar_wait(&ctl->row_full[slot], (u / S::kRing) & 1, gave_up) && tc::bar_wait(&ctl->sp_full[w], k & 1, gave_up);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc::fence_after();
            unit32<T>(tm + lanes + w * 64, reinterpret_cast<const RowInfo *>(smem + S::kInfo) + slot, plain, p.scale_log2, up,
                      smem + S::kBuckets + l, reinterpret_cast<const uint8_t *>(lut), shift, nullptr, 0, 0, 0);
            tc::wait_st();
            tc::fence_before();
            tc::bar_arrive(&ctl->ds_full[w]);
        }
        // results: group 0 dv, group 1 dk, through the slots of values and keys
        if (ok) ok = __all_sync(~0u, tc::bar_wait(&ctl->tile_full, 0, gave_up));
        const uint32_t stage = sm + (w ? 0 : S::kSlot);
        if (ok) {
            tc::fence_after();
            load_nodes<T, DP>(tm + lanes + (w ? kDk : kDv), w ? p.scale * ds_down : p_down, stage, l);
            tc::fence_async();
        }
        asm volatile("bar.sync %0, 128;" ::"r"(w + 1) : "memory");
        if (l == 0 && ok) {
            for (int c = 0; c < (int)p.d; c += 64)
                tc::store_box(w ? &p.dk_map : &p.dv_map, stage + c / 64 * S::kPanel, c, hk, (int32_t)(tile * kTcTile));
            tc::stores_commit();
            tc::stores_done();
        }
    } else if (warp < 12) {
        hop_warps<1>(p, ctl, smem + S::kBuckets, warp - 8, lane, 1, tile, gave_up);
    } else if (warp < 16) {
        node_warps<DP, 2, 1>(p, ctl, sm, warp - 12, lane, hk, 1, tile, gave_up);
        // Row tiles: this thread's chunks are the same of every tile, so that their places are worked out once.
        const int t = tid - 384;
        constexpr int C = DP / 8, RP = 128 / C, kPasses = kBwdRows / RP;
        const uint32_t G = p.group, per = kBwdRows / G, c = t % C, fill = (p.d / 8 + 1) & ~1u;
        const char *qsrc[kPasses], *gsrc[kPasses];
        uint32_t first[kPasses];                         // query of the pass's row in tile 0; past every T for none
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            const uint32_t r = t / C + k * RP, q = r / G, g = r - q * G;
            const bool on = q < per && c < p.d / 8;
            first[k] = on ? q : 0x80000000u;
            qsrc[k] = static_cast<const char *>(p.q) + (on ? ((int64_t)q * p.q_row + (int64_t)(hk * G + g) * p.q_head + c * 8) * 2 : 0);
            gsrc[k] = static_cast<const char *>(p.dout) + (on ? ((int64_t)q * p.dout_row + (int64_t)(hk * G + g) * p.dout_head + c * 8) * 2 : 0);
        }
        const int64_t qstep = (int64_t)per * p.q_row * 2, gstep = (int64_t)per * p.dout_row * 2;
        const uint32_t to = sm + S::kRow + tc::chunk(t / C, c, 4096);          // passes are whole swizzle periods apart
        static_assert(RP % 8 == 0, "whole swizzle periods");
        const char *info = reinterpret_cast<const char *>(static_cast<const RowInfo *>(p.row_info) + (uint64_t)hk * p.row_tiles) + t * 16;
        bool ok = true;
        for (uint32_t u = 0; u < units; ++u) {
            const uint32_t slot = u % S::kRing;
            if (u >= (uint32_t)S::kRing) ok = __all_sync(~0u, tc::bar_wait(&ctl->row_empty[slot], (u / S::kRing - 1) & 1, gave_up));
            if (!ok) break;
            if (c < fill) {
#pragma unroll
                for (int k = 0; k < kPasses; ++k) {
                    const uint32_t n = first[k] + u * per < p.T ? 16 : 0;
                    cp16(to + slot * 2 * S::kRowTile + k * RP * 128, n ? qsrc[k] : static_cast<const char *>(p.q), n);
                    cp16(to + slot * 2 * S::kRowTile + S::kRowTile + k * RP * 128, n ? gsrc[k] : static_cast<const char *>(p.dout), n);
                    qsrc[k] += qstep;
                    gsrc[k] += gstep;
                }
            }
            if (t < (int)sizeof(RowInfo) / 16) cp16(sm + S::kInfo + slot * (int)sizeof(RowInfo) + t * 16, info + (uint64_t)u * sizeof(RowInfo), 16);
            tc::cp_arrive(&ctl->row_full[slot]);
        }
        cp_commit();
        cp_wait<0>();
    } else {
        const bool lead = tc::elect();
        const uint32_t dn = (p.d + 15) & ~15u, id_s = tc::idesc(kBf16, 32, false, false), id_n = tc::idesc(kBf16, dn, false, true);
        bool ok = tc::bar_wait(&ctl->full[0], 0, gave_up) && tc::bar_wait(&ctl->full[1], 0, gave_up);
        auto scores = [&](uint32_t u) {
            const uint32_t w = u & 1, slot = u % S::kRing;
            ok = tc::bar_wait(&ctl->row_full[slot], (u / S::kRing) & 1, gave_up);
            if (!ok) return;
            tc::fence_async();
            tc::fence_after();
            const uint32_t qa = sm + S::kRow + slot * 2 * S::kRowTile;
            score_products<DP, S::kPanel>(lead, tm + w * 64, tc::desc(sm, S::kPanel), tc::desc(qa, 4096), tc::desc(sm + S::kSlot, S::kPanel),
                                          tc::desc(qa + S::kRowTile, 4096), id_s, dn);
            tc::commit(lead, &ctl->sp_full[w]);
        };
        if (ok && units > 0) scores(0);
        if (ok && units > 1) scores(1);
        for (uint32_t u = 0; u < units && ok; ++u) {
            const uint32_t w = u & 1, slot = u % S::kRing;
            ok = tc::bar_wait(&ctl->ds_full[w], (u >> 1) & 1, gave_up);
            if (!ok) break;
            tc::fence_after();
            const uint32_t qa = sm + S::kRow + slot * 2 * S::kRowTile;
            node_products(lead, tm + w * 64, tm + kDv, tm + kDk, tc::desc(qa, 4096), tc::desc(qa + S::kRowTile, 4096), id_n, u > 0);
            tc::commit(lead, &ctl->row_empty[slot]);
            if (u + 1 == units) tc::commit(lead, &ctl->tile_full);
            if (u + 2 < units) scores(u + 2);
        }
        if (!ok) tc::drain(lead, &ctl->drained, 0);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 16) tc::dealloc(tm, kCols);
    if (tid == 0 && *gave_up) atomicOr(p.status, K2T_STATUS_WAIT_TIMEOUT);
}

constexpr uint32_t kJoinThreads = 1024;
// dq = scale * sum over splits; dbias = sum over splits and row groups, in a fixed order.
// One block per head of dbias, which take longest, then one per four rows of dq (with one split, dq is written already).
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) attn_bwd_join_kernel(const __grid_constant__ AttnParams p)
{
    const int tid = threadIdx.x;
    const uint32_t heads = p.buckets ? p.hq : 0;
    tc::grid_wait();
    if (blockIdx.x >= heads) {
        const uint64_t rows = (uint64_t)p.T * p.hq, row = (uint64_t)(blockIdx.x - heads) * 4 + (tid >> 8);
        const uint32_t in = tid & 255;
        __shared__ float4 sum[kJoinThreads];
        const uint32_t q4 = p.d / 4, groups = 256 / q4, c = in % q4, g = in / q4;
        float4 acc = make_float4(0, 0, 0, 0);
        if (g < groups && row < rows)
#pragma unroll 4
            for (uint32_t s = g; s < p.splits; s += groups) {
                const float4 x = *reinterpret_cast<const float4 *>(p.part + (s * rows + row) * p.d + c * 4);
                acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
            }
        sum[tid] = acc;
        __syncthreads();
        if (g == 0 && row < rows) {
            for (uint32_t i = 1; i < groups; ++i) {
                const float4 x = sum[(tid & ~255) + i * q4 + c];
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
    const uint32_t hd = blockIdx.x;
    // W neighbour threads of a warp a bucket
    uint32_t W = 32;
    while (W * p.buckets > kJoinThreads) W >>= 1;
    const uint32_t b = tid / W, x = tid % W;
    float s = 0.0f;
    if (b < p.buckets) {
#pragma unroll 4
        for (uint32_t i = x; i < p.hist_parts; i += W) s += p.part_ml[((uint64_t)i * p.hq + hd) * p.buckets + b];
    }
    for (uint32_t y = W >> 1; y; y >>= 1) s += __shfl_xor_sync(~0u, s, y);
    if (b < p.buckets && x == 0) static_cast<T *>(p.dbias)[(uint64_t)hd * p.buckets + b] = Elem<T>::from_float(s);
}

}  // namespace k2t
