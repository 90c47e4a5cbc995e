// k2t_attn.cuh -- attention of queries to node states with a hop-bucket bias:
// kernels on warp-level matrix instructions (m16n8k16, fp32 accumulators).
//
// Rows of one key/value head hk are r = t * G + g (query t, head hk * G + g,
// G query heads share hk), so the states of hk are read once for all of them.
// Scores are kept in units of log2: s2 = (q.k) * scale * log2(e) + bias *
// log2(e), so that a weight is one exp2.
//
// Hop tables.  A tile of 64 nodes brings its 64 x n_sources hops; each is
// turned into a byte once: 0 masked, 1 + bucket, and in one more column
// n_buckets + 1 for queries without hop information.  The bytes are stored
// [column][node], so that the lanes of a score tile read neighbouring ones,
// and select the bias from a table of (n_buckets + 2) x G floats in shared
// memory, -inf at 0.  The bytes of a tile also say which of its nodes no row
// sees: their states are not read (the copy fills zeros), which saves their
// bytes and keeps what they hold away from the products.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "k2t_internal.h"

namespace k2t {

extern thread_local int g_last_cuda;

constexpr int kAttnTile = 64;          // nodes per tile
constexpr int kAttnThreads = 128;
constexpr int kHopPitch = 68;          // bytes per column of a bucket tile: 17 words, odd, so that 8 columns differ in bank
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
    uint64_t tiles;           // ceil(n / kAttnTile)
    uint32_t hop_magic;       // ceil(2^16 / sources): i / sources for i < 64 * 32
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
    float *delta;
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
    static __device__ __forceinline__ void mma(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
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
    static __device__ __forceinline__ void mma(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// ---- small PTX wrappers ---------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldsm4(uint32_t r[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t r[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Byte address of 16-byte chunk c of row r in a tile of DP 2-byte values a
// row: the chunk index is xored with the row, so that the 8 rows of one
// matrix load lie in 8 different bank groups (the row pitch is a multiple of
// 128 bytes).
template <int DP> __device__ __forceinline__ uint32_t tile_addr(uint32_t base, int r, int c)
{
    return base + r * (DP * 2) + ((c ^ (r & 7)) << 4);
}

// Fragment loads from such a tile.  lane-dependent row/chunk of an x4 load:
// matrices 0..3 = (rows 0-7, k 0-7), (rows 8-15, k 0-7), (rows 0-7, k 8-15),
// (rows 8-15, k 8-15): an A operand of 16 rows x 16 k.
template <int DP> __device__ __forceinline__ void load_a(uint32_t a[4], uint32_t base, int row0, int k16, int lane)
{
    ldsm4(a, tile_addr<DP>(base, row0 + (lane & 15), k16 * 2 + (lane >> 4)));
}
// B operand for k = 16 along the row, n = 16 rows (two n8 blocks): b[0], b[1]
// of the first block, b[2], b[3] of the second.
template <int DP> __device__ __forceinline__ void load_b(uint32_t b[4], uint32_t base, int row0, int k16, int lane)
{
    ldsm4(b, tile_addr<DP>(base, row0 + (lane & 7) + ((lane >> 4) << 3), k16 * 2 + ((lane >> 3) & 1)));
}
// B operand for k = 16 rows, n = 16 values along the row (two n8 blocks).
template <int DP> __device__ __forceinline__ void load_bt(uint32_t b[4], uint32_t base, int row0, int n16, int lane)
{
    ldsm4t(b, tile_addr<DP>(base, row0 + (lane & 15), n16 * 2 + (lane >> 4)));
}

// Where a block copies the states of tile nodes from: rows that no query
// sees, rows past n and chunks past head_dim are filled with zeros.
template <int DP>
__device__ __forceinline__ void copy_nodes(uint32_t dst, const char *src, int64_t row_bytes, int64_t node0, uint64_t n,
                                           uint32_t chunks, const uint8_t *seen, int tid)
{
    constexpr int C = DP / 8;
    const int c = tid % C;
#pragma unroll
    for (int r = tid / C; r < kAttnTile; r += kAttnThreads / C) {
        const bool on = c < (int)chunks && (uint64_t)(node0 + r) < n && seen[r];
        cp16(tile_addr<DP>(dst, r, c), on ? src + (node0 + r) * row_bytes + c * 16 : src, on ? 16 : 0);
    }
}

// Rows [row0, row0 + ROWS) of a [T, heads, d] tensor, as rows t * G + g.
template <int DP, int ROWS>
__device__ __forceinline__ void copy_rows(uint32_t dst, const void *base, int64_t s_row, int64_t s_head, uint32_t head0,
                                          uint32_t row0, const AttnParams &p, int tid)
{
    constexpr int C = DP / 8;
    const char *src = static_cast<const char *>(base);
    for (int i = tid; i < ROWS * C; i += kAttnThreads) {
        const int r = i / C, c = i % C;
        const uint32_t row = row0 + r;
        const bool on = row < p.rows && c < (int)(p.d / 8);
        const uint32_t t = row / p.group, g = row - t * p.group;
        cp16(tile_addr<DP>(dst, r, c), on ? src + ((int64_t)t * s_row + (int64_t)(head0 + g) * s_head + c * 8) * 2 : src,
             on ? 16 : 0);
    }
}

// Column of a row in the bucket tile: `sources` (the last) without hop information.
__device__ __forceinline__ uint32_t row_column(const AttnParams &p, uint32_t row)
{
    if (!p.sources) return 0;
    const uint32_t t = row / p.group;
    const int32_t c = p.qsrc ? __ldg(p.qsrc + t) : (int32_t)t;
    return (uint32_t)c < p.sources ? (uint32_t)c : p.sources;
}

// The part of shared memory that turns hops into biases.
struct HopSmem {
    uint8_t bucket_of[256];
    uint32_t columns;                       // bit c: some row of the block uses column c
    uint32_t all;                           // some row sees every node
    uint8_t seen[4][kAttnTile];
    uint8_t tile[4][33 * kHopPitch];        // [buffer][column][node]
};

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

// Hops of a tile: each thread holds up to 16 of the 64 x sources, flat in
// their order in memory (neighbouring threads read neighbouring words).
constexpr int kHopRegs = kAttnTile * 32 / kAttnThreads;

__device__ __forceinline__ void hops_load(int32_t h[kHopRegs], const AttnParams &p, uint64_t tile, int tid)
{
    const uint64_t at = tile * (uint64_t)kAttnTile * p.sources, end = p.n * (uint64_t)p.sources;
    const uint32_t count = kAttnTile * p.sources;
#pragma unroll
    for (int i = 0; i < kHopRegs; ++i) {
        const uint32_t k = tid + i * kAttnThreads;
        h[i] = -1;
        if (k < count && at + k < end) h[i] = __ldg(p.hops + at + k);
    }
}

// ... stored as bytes into buffer `buf`; the caller has zeroed seen[buf] a barrier earlier.
__device__ __forceinline__ void hops_store(const int32_t h[kHopRegs], HopSmem *s, const AttnParams &p, uint64_t tile,
                                           int buf, int tid)
{
    const uint32_t count = kAttnTile * p.sources, columns = s->columns;
#pragma unroll
    for (int i = 0; i < kHopRegs; ++i) {
        const uint32_t k = tid + i * kAttnThreads;
        if (k >= count) break;
        const uint32_t node = (k * p.hop_magic) >> 16, col = k - node * p.sources;
        const int32_t x = h[i];
        s->tile[buf][col * kHopPitch + node] = x < 0 ? 0 : s->bucket_of[min(x, 255)] + 1;
        if (x >= 0 && ((columns >> col) & 1)) s->seen[buf][node] = 1;
    }
    if (tid < kAttnTile) {
        const bool in = tile * kAttnTile + tid < p.n;
        s->tile[buf][p.sources * kHopPitch + tid] = in ? p.buckets + 1 : 0;
        if (in && s->all) s->seen[buf][tid] = 1;
    }
}

// Without a hop table every node is seen; one column says which lie past n.
__device__ __forceinline__ void hops_none(HopSmem *s, const AttnParams &p, uint64_t tile, int buf, int tid)
{
    if (tid < kAttnTile) {
        const bool in = tile * kAttnTile + tid < p.n;
        s->tile[buf][tid] = in ? p.buckets + 1 : 0;
        s->seen[buf][tid] = in;
    }
}

}  // namespace k2t
