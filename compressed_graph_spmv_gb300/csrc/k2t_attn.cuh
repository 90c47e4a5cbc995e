// k2t_attn.cuh -- attention of queries to node states with a hop-bucket bias:
// what its forward and backward kernels share.
//
// Rows of one key/value head hk are r = t * G + g (query t, head hk * G + g,
// G query heads share hk), so the states of hk are read once for all of them.
// Scores are kept in units of log2: s2 = (q.k) * scale * log2(e) + bias *
// log2(e), so that a weight is one exp2.
//
// Hop tables.  A tile of 128 nodes brings its 128 x n_sources hops; each is
// turned into a byte once: 0 masked, 1 + bucket, and in one more column
// n_buckets + 1 for queries without hop information.  The bytes are stored
// [column][node], so that the lanes of a score tile read neighbouring ones,
// and select the bias from a table of (n_buckets + 2) x G floats in shared
// memory, -inf at 0.  The bytes of a tile also say which of its nodes no row
// sees: their states are not read (the copy fills zeros), which saves their
// bytes and keeps what they hold away from the products.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "k2t_internal.h"
#include "k2t_tc.cuh"

namespace k2t {

extern thread_local int g_last_cuda;

constexpr int kTcTile = 128;           // nodes per tile
constexpr int kTcPitch = 144;          // bytes per column of a bucket tile: 16-byte loads of 8 columns meet no bank twice
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What the kernels need of k2t_attn, by value.
struct AttnParams {
    uint32_t T, hq, hkv, group, d, sources, buckets;
    uint64_t n;
    uint32_t rows;            // T * group
    uint32_t group2, group2_log;  // group rounded up to a power of two
    uint32_t row_tiles;
    uint32_t splits;          // blocks that share the nodes of one head
    uint64_t tiles;           // ceil(n / kTcTile)
    float scale, scale_log2;
    const void *q, *k, *v, *dout;
    const int32_t *hops, *qsrc;
    const void *bias;
    void *out, *dq, *dk, *dv, *dbias;
    float *lse;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head, dout_row, dout_head;
    int64_t dq_row, dq_head, dk_row, dk_head, dv_row, dv_head;
    float *part;              // partial sums: see the kernels
    float *part_ml;
    void *row_info;           // RowInfo[hkv][row_tiles * 32] (backward)
    float2 *delta_part;       // [delta_splits][T][hq]: sums of p dp and of p
    float *pdp_top;           // fp16: [delta_splits][T][hq]: largest p |dp|
    uint32_t delta_splits, delta_tiles;   // of attn_delta_kernel; 0: delta is dout . out
    uint32_t hist_parts;      // partial dbias tables
    uint32_t hist_threads;    // threads that sum by bucket, 128 or 64
    CUtensorMap dk_map, dv_map;   // (head_dim, kv heads, nodes), boxes of 64 x 1 x 128 (backward)
    uint32_t *status;         // device status word, at the start of the work buffer
    uint8_t bucket_of[256];   // bucket of each hop count; larger hops share the last
};

// ---- element types -------------------------------------------------------
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u)
    {
        return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&u));
    }
    static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
    static constexpr float kMasked = -1e38f;      // table entries not above this mask
    static constexpr int kUp = 0;                 // see fp16's
};
template <> struct Elem<__half> {
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) { return __half22float2(*reinterpret_cast<__half2 *>(&u)); }
    static __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
    static constexpr float kMasked = -65504.0f;
    // Weights of a row over n nodes are about 1/n, below fp16's least normal number from 2^14 nodes on and 0 from 2^25 on.
    // Backward, weights (at most 1) are multiplied by 2^15 before they are rounded, which leaves 29 bits of normal numbers
    // below 1, and score gradients by 2^15 and a power of two that brings the largest to 1 at most (ds_scale): of the row for
    // dq and the sums by bucket, of the head for dk, which sums over rows.  The powers are taken out of the fp32 results
    // again.
    static constexpr int kUp = 15;
};

// Factor of score gradients of which none exceeds `top`: |ds| <= max p |dp| + |delta|.  Where top is no number the factor
// undoes kUp; where it is 0 it is the largest factor, since the least one of the rows is the head's.
template <typename T> __device__ __forceinline__ float ds_scale(float top)
{
    if (Elem<T>::kUp == 0) return 1.0f;
    if (!(top <= 3.4e38f)) return __uint_as_float((127u - Elem<T>::kUp) << 23);
    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127 + 1, -100), 100);
    return __uint_as_float((uint32_t)(127 - e) << 23);
}
// 1 / a power of two.
__device__ __forceinline__ float inverse_power(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

// ---- small PTX wrappers ---------------------------------------------------
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Column of a row in the bucket tile: `sources` (the last) without hop information.
__device__ __forceinline__ uint32_t row_column(const AttnParams &p, uint32_t row)
{
    if (!p.sources) return 0;
    const uint32_t t = row / p.group;
    const int32_t c = p.qsrc ? __ldg(p.qsrc + t) : (int32_t)t;
    return (uint32_t)c < p.sources ? (uint32_t)c : p.sources;
}

// Bias table in units of log2, [bucket byte][pitch]: -inf at 0 (masked), 0 at buckets + 1.
template <typename T>
__device__ __forceinline__ void fill_bias(float *lut, const AttnParams &p, uint32_t hk, int tid, uint32_t pitch)
{
    const T *bias = static_cast<const T *>(p.bias);
    const uint32_t total = (p.buckets + 2) * pitch;
    for (uint32_t i = tid; i < total; i += blockDim.x) {
        const uint32_t b = i / pitch, g = i - b * pitch;
        float v = 0.0f;
        if (b == 0) v = -INFINITY;
        else if (b <= p.buckets && bias && g < p.group) {
            v = Elem<T>::to_float(bias[(uint64_t)(hk * p.group + g) * p.buckets + b - 1]);
            v = v <= Elem<T>::kMasked ? -INFINITY : v * kLog2e;
        }
        lut[i] = v;
    }
}

// ---- warps that the forward and backward kernels share -------------------------
// ctl: the kernel's control block in shared memory (barriers hop_full,
// hop_empty, full, empty; columns in use; seen nodes).  Tile i of the block is
// tile tile0 + i * p.splits of the nodes.

// Items 2 i (keys of tile i) and 2 i + 1 (values) go round the slots; three
// slots are two for keys and one for values, which are read first.  use: how
// often the slot was filled before.
template <int SLOTS> __device__ __forceinline__ uint32_t slot_of(uint32_t item)
{
    return SLOTS == 3 ? (item & 1 ? 2 : (item >> 1) & 1) : item % SLOTS;
}
template <int SLOTS> __device__ __forceinline__ uint32_t slot_use(uint32_t item)
{
    return SLOTS == 3 ? (item & 1 ? item >> 1 : item >> 2) : item / SLOTS;
}

// Hops of nodes [32 hw, 32 hw + 32) of a tile -> bucket bytes, and which of those nodes a column in use sees.  W lanes
// side by side (a power of two, at least n_sources; a quarter of that where four columns come in one load) read a node's
// columns, and the other lanes the nodes after those that the first ones take one after another.  The loads of a tile
// are in flight while the tile before is turned into bytes.  Four columns a load halve the instructions: of few rows and
// many columns these warps set the pace (32 queries over 2^18 nodes, head_dim 64: 2400 clocks a tile before).  Other
// numbers of columns go 16 nodes at a time in a rolled loop: code that is not fetched is what a short call waits least for.
template <int BUFS, typename Ctl>
__device__ __forceinline__ void hop_warps(const AttnParams &p, Ctl *ctl, uint8_t *buckets, int hw, int lane, uint32_t tiles,
                                          uint64_t tile0, volatile uint32_t *gave_up)
{
    const uint32_t cols = ctl->columns, B = p.sources;
    const bool all = ctl->all || !B, four = B && (B & 3) == 0 && ((uintptr_t)p.hops & 15) == 0;
    uint32_t W = 1;
    while (W < B) W *= 2;
    const uint32_t Q = four ? W / 4 : W;                                // lanes of a node, and nodes of a lane
    const uint32_t col = (lane & (Q - 1)) * (four ? 4 : 1), first = lane & ~(Q - 1);
    const bool on = col < B;
    uint32_t unused[4];                                                // all ones where a column does not count
#pragma unroll
    for (int j = 0; j < 4; ++j) unused[j] = col + j < 32 && ((cols >> (col + j)) & 1) ? 0u : ~0u;
    int32_t h[32];       // four columns of 8 nodes, or one column of 16; those past a lane's part stay masked
#pragma unroll
    for (int e = 0; e < 32; ++e) h[e] = -1;
    auto place = [&](uint32_t t, uint32_t k, uint32_t &left) {         // the lane's node k of tile t on, and how many follow
        const uint64_t node = (tile0 + (uint64_t)t * p.splits) * kTcTile + hw * 32 + first + k;
        left = t < tiles && on && node < p.n ? (uint32_t)min((uint64_t)(Q - k), p.n - node) : 0;
        return p.hops + node * B + col;
    };
    auto four_in = [&](uint32_t t) {
        uint32_t left;
        const int32_t *at = place(t, 0, left);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            int4 x = make_int4(-1, -1, -1, -1);
            if (e < (int)left) asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(at));
            h[4 * e] = x.x, h[4 * e + 1] = x.y, h[4 * e + 2] = x.z, h[4 * e + 3] = x.w;
            at += B;
        }
    };
    auto one_in = [&](uint32_t t, uint32_t k) {
        uint32_t left;
        const int32_t *at = place(t, k, left);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            h[e] = -1;
            if (e < (int)left) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(h[e]) : "l"(at));
            at += B;
        }
    };
    auto byte = [&](int32_t x) -> uint32_t { return ctl->byte_of[__viaddmax_s32(min(x, 255), 1, 0)]; };
    auto put = [&](uint8_t *to, uint32_t nodes, uint32_t b) {           // the bytes of up to 4 nodes of a column
        if (nodes >= 4) *reinterpret_cast<uint32_t *>(to) = b;
        else if (nodes == 2) *reinterpret_cast<uint16_t *>(to) = (uint16_t)b;
        else *to = (uint8_t)b;
    };
    if (four) four_in(0);
    else if (B) one_in(0, 0);
    for (uint32_t t = 0; t < tiles; ++t) {
        const uint32_t buf = t % BUFS;
        if (t >= BUFS && !__all_sync(~0u, tc::bar_wait(&ctl->hop_empty[buf], (t / BUFS - 1) & 1, gave_up))) break;
        uint8_t *bt = buckets + buf * 33 * kTcPitch + hw * 32, *to = bt + col * kTcPitch + first;
        const uint64_t node0 = (tile0 + (uint64_t)t * p.splits) * kTcTile + hw * 32;
        uint32_t unseen = 0;                                           // bit e: this lane's columns do not see its node e
        if (four) {
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                if (e && Q <= 4) break;
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = (byte(h[4 * e + 12 + j]) * 256 + byte(h[4 * e + 8 + j])) * 65536 + byte(h[4 * e + 4 + j]) * 256 + byte(h[4 * e + j]);
                if (on) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) put(to + j * kTcPitch + e, Q, w[j]);
                }
            }
#pragma unroll
            for (int e = 7; e >= 0; --e) {
                const int32_t m = max(max(h[4 * e] | (int)unused[0], h[4 * e + 1] | (int)unused[1]), max(h[4 * e + 2] | (int)unused[2], h[4 * e + 3] | (int)unused[3]));
                unseen = __funnelshift_l(m, unseen, 1);                // a negative hop count's sign
            }
            four_in(t + 1);
        } else if (B) {
#pragma unroll 1
            for (uint32_t k = 0; k < Q; k += 16) {
                uint32_t part = 0;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    if (e >= (int)Q) break;
                    const uint32_t w = (byte(h[e + 3]) * 256 + byte(h[e + 2])) * 65536 + byte(h[e + 1]) * 256 + byte(h[e]);
                    if (on) put(to + k + e, Q, w);
                }
#pragma unroll
                for (int e = 15; e >= 0; --e) part = __funnelshift_l(h[e] | (int)unused[0], part, 1);
                unseen |= part << k;
                const bool more = k + 16 < Q;
                one_in(more ? t : t + 1, more ? k + 16 : 0);
            }
        }
        const uint32_t mine = Q >= 32 ? ~0u : (1u << Q) - 1, sees = on ? (~unseen & mine) << first : 0;
        const bool in = node0 + lane < p.n;
        bt[B * kTcPitch + lane] = in ? p.buckets + 1 : 0;
        const uint32_t inside = __ballot_sync(~0u, in), seen = (all ? ~0u : __reduce_or_sync(~0u, sees)) & inside;
        __syncwarp();
        if (lane == 0) {
            ctl->seen[buf][hw] = seen;
            tc::bar_arrive(&ctl->hop_full[buf]);
        }
    }
}

// States of a tile's seen nodes -> slots, keys then values; this warp brings nodes [32 cw, 32 cw + 32).
template <int DP, int SLOTS, int BUFS, typename Ctl>
__device__ __forceinline__ void node_warps(const AttnParams &p, Ctl *ctl, uint32_t sm, int cw, int lane, uint32_t hk,
                                           uint32_t tiles, uint64_t tile0, volatile uint32_t *gave_up)
{
    constexpr int kPanel = kTcTile * 128, kSlot = kPanel * (DP / 64);
    constexpr int C = DP / 8, RP = 32 / C, kTurn = 8 / RP;     // chunks a row, rows a pass, passes until the swizzle repeats
    const uint32_t c = lane % C, r0 = lane / C;
    const uint32_t fill = (p.d / 8 + 1) & ~1u;                 // chunks the products read: whole steps of 16 values
    uint32_t at[kTurn];
#pragma unroll
    for (int k = 0; k < kTurn; ++k) at[k] = sm + tc::chunk(cw * 32 + k * RP + r0, c, kPanel) - k * RP * 128;
    uint32_t item = 0;
    bool ok = true;
    auto bring = [&](const char *src, int64_t step, uint32_t seen) {
        const uint32_t slot = slot_of<SLOTS>(item), use = slot_use<SLOTS>(item);
        if (use) ok = __all_sync(~0u, tc::bar_wait(&ctl->empty[slot], (use - 1) & 1, gave_up));
        if (!ok) return;
        if (c < fill) {
#pragma unroll
            for (int k = 0; k < 32 / RP; ++k) {
                // a node that no query sees, or past n, or a chunk past head_dim: zeros, and nothing is read
                cp16(at[k % kTurn] + slot * kSlot + k * RP * 128, src, (seen >> (k * RP)) & 1 ? 16 : 0);
                src += step;
            }
        }
        tc::cp_arrive(&ctl->full[slot]);      // counts this thread's copies once they have landed
        ++item;
    };
    const int64_t kstep = RP * p.k_row * 2, vstep = RP * p.v_row * 2;
    const char *k0 = static_cast<const char *>(p.k) + ((int64_t)hk * p.k_head + c * 8) * 2;
    const char *v0 = static_cast<const char *>(p.v) + ((int64_t)hk * p.v_head + c * 8) * 2;
    for (uint32_t i = 0; i < tiles && ok; ++i) {
        const uint32_t buf = i % BUFS;
        ok = __all_sync(~0u, tc::bar_wait(&ctl->hop_full[buf], (i / BUFS) & 1, gave_up));
        if (!ok) break;
        const uint32_t seen = c < p.d / 8 ? ctl->seen[buf][cw] >> r0 : 0;
        const int64_t node = (int64_t)((tile0 + (uint64_t)i * p.splits) * kTcTile) + cw * 32 + r0;
        bring(k0 + node * p.k_row * 2, kstep, seen);
        if (ok) bring(v0 + node * p.v_row * 2, vstep, seen);
    }
    cp_commit();
    cp_wait<0>();
}

}  // namespace k2t
