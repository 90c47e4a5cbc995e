// k2t_attn_cached.cu -- launches of the attention over the 8-bit cache.
#include <algorithm>

#include "k2t_attn_cached.cuh"
#include "k2t_attn_few.cuh"
#include "k2t_attn_launch.cuh"

namespace k2t {

// Hops -> bucket bytes and seen nodes of every tile, once for all heads and row tiles of the call (the main kernel's blocks
// each turned their tiles' hops into bytes themselves before: 32 queries over 2^20 nodes, 4 key/value heads, 425 us, then
// 388, of which this kernel 30; 400 since rows may have origins).  Bound by memory: 32 columns of 2^20 hops at 4.4 TB/s.  As many blocks as fit at once: with
// more than fit and 48 registers a thread it took 43 us, columns that are no multiple of 4 by a value a thread 13 us of 100003
// nodes and 13 columns (a node a pair of threads: 7).
constexpr int kHopThreads = 256, kHopBlocks = 6;      // of an SM
static __global__ void __launch_bounds__(kHopThreads, kHopBlocks) attn_hops_kernel(const __grid_constant__ CachedParams p)
{
    __shared__ __align__(16) uint8_t bytes[33 * kTcPitch];
    __shared__ __align__(16) uint32_t seen[4];
    __shared__ uint32_t columns, all;
    __shared__ uint8_t byte_of[257];
    const uint32_t tid = threadIdx.x, B = p.sources;
    if (tid == 0) columns = all = 0;
    for (uint32_t i = tid; i < 257; i += kHopThreads) byte_of[i] = i ? p.bucket_of[i - 1] + 1 : 0;
    tc::grid_wait();
    tc::grid_next();
    __syncthreads();
    for (uint32_t t = tid; t < p.T; t += kHopThreads) {
        const int32_t c = p.qsrc ? __ldg(p.qsrc + t) : (int32_t)t;
        if ((uint32_t)c < B) atomicOr(&columns, 1u << c);
        else all = 1;
    }
    __syncthreads();
    const uint32_t used = columns;
    const bool four = (B & 3) == 0 && kHopThreads % (B / 4) == 0 && ((uintptr_t)p.hops & 15) == 0;
    auto byte = [&](int32_t x) -> uint32_t { return byte_of[__viaddmax_s32(min(x, 255), 1, 0)]; };
    for (uint64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        if (tid < 4) seen[tid] = 0;
        __syncthreads();
        const uint64_t node0 = tile * kTcTile;
        const uint32_t in = (uint32_t)min((uint64_t)kTcTile, p.n - node0);          // nodes of the tile
        const int32_t *hops = p.hops + node0 * B;
        if (four) {
            // four columns of four nodes a thread: a word of bytes for each column
            const uint32_t Q = B / 4, q = tid % Q, m = tid / Q;
            for (uint32_t j = m; j < kTcTile / 4; j += kHopThreads / Q) {
                int4 h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    h[k] = make_int4(-1, -1, -1, -1);
                    if (j * 4 + k < in) h[k] = __ldg(reinterpret_cast<const int4 *>(hops) + (j * 4 + k) * Q + q);
                }
                const uint32_t mine = used >> (q * 4);
                uint32_t sees = 0;
                uint32_t *to = reinterpret_cast<uint32_t *>(bytes + q * 4 * kTcPitch + j * 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if ((h[k].x >= 0 && mine & 1) || (h[k].y >= 0 && mine & 2) || (h[k].z >= 0 && mine & 4) || (h[k].w >= 0 && mine & 8)) sees |= 1u << k;
                to[0] = byte(h[0].x) | byte(h[1].x) << 8 | byte(h[2].x) << 16 | byte(h[3].x) << 24;
                to[kTcPitch / 4] = byte(h[0].y) | byte(h[1].y) << 8 | byte(h[2].y) << 16 | byte(h[3].y) << 24;
                to[kTcPitch / 2] = byte(h[0].z) | byte(h[1].z) << 8 | byte(h[2].z) << 16 | byte(h[3].z) << 24;
                to[kTcPitch / 4 * 3] = byte(h[0].w) | byte(h[1].w) << 8 | byte(h[2].w) << 16 | byte(h[3].w) << 24;
                if (Q == 8) {                          // a warp's nodes are in one word
                    sees = __reduce_or_sync(~0u, sees << ((j & 7) * 4));
                    if ((tid & 31) == 0) atomicOr(&seen[j >> 3], sees);
                } else if (sees) {
                    atomicOr(&seen[j >> 3], sees << ((j & 7) * 4));
                }
            }
        } else {
            static_assert(kHopThreads == 2 * kTcTile);
            // every second column of a node a thread; neighbouring loads share their lines
            const uint32_t node = tid % kTcTile, half = tid / kTcTile;
            bool sees = false;
            for (uint32_t c0 = half; c0 < B; c0 += 16) {
                int32_t h[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) h[k] = c0 + 2 * k < B && node < in ? __ldg(hops + node * B + c0 + 2 * k) : -1;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t c = c0 + 2 * k;
                    if (c >= B) break;
                    bytes[c * kTcPitch + node] = (uint8_t)byte(h[k]);
                    sees |= h[k] >= 0 && used >> c & 1;
                }
            }
            const uint32_t some = __ballot_sync(~0u, sees);
            if ((tid & 31) == 0) atomicOr(&seen[node >> 5], some);
        }
        if (tid < kTcTile) bytes[B * kTcPitch + tid] = tid < in ? (uint8_t)(p.buckets + 1) : 0;
        __syncthreads();
        uint4 *to = reinterpret_cast<uint4 *>(p.hop_tiles + tile * p.hop_tile);
        const uint32_t pieces = (B + 1) * (kTcPitch / 16);
        for (uint32_t i = tid; i < pieces; i += kHopThreads) to[i] = reinterpret_cast<const uint4 *>(bytes)[i];
        if (tid < 4) {
            const uint32_t inside = in >= tid * 32 + 32 ? ~0u : in > tid * 32 ? (1u << (in - tid * 32)) - 1 : 0;
            reinterpret_cast<uint32_t *>(to + pieces)[tid] = all ? inside : seen[tid];
        }
        __syncthreads();
    }
}

// bm: rows a block takes, 32, 64 or 128.
template <typename T, int DP> static int cached_dim(const CachedParams &p, int bm, cudaStream_t st)
{
    const dim3 grid(p.splits * p.row_tiles, p.hkv);
    const size_t smem = CachedSmem<DP>::bytes(p);
    switch (bm) {
    case 32: return attn_launch<attn_cached_kernel<T, DP, 32>>(grid, CachedSmem<DP>::kThreads, smem, p, st);
    case 64: return attn_launch<attn_cached_kernel<T, DP, 64>>(grid, CachedSmem<DP>::kThreads, smem, p, st);
    default: return attn_launch<attn_cached_kernel<T, DP, 128>>(grid, CachedSmem<DP>::kThreads, smem, p, st);
    }
}

template <typename T> static int few_rows(const CachedParams &p, cudaStream_t st)
{
    const dim3 grid(p.splits, p.hkv);
    const size_t smem = FewSmem::bytes(p);
    if (p.rows <= 4) return attn_launch<attn_few_kernel<T, 1>>(grid, FewPlan<1>::kAll, smem, p, st);
    return attn_launch<attn_few_kernel<T, 2>>(grid, FewPlan<2>::kAll, smem, p, st);
}

template <typename T> static int launch_cached(const CachedParams &p, int bm, cudaStream_t st)
{
    if (p.hop_tiles && p.tiles) {
        const unsigned blocks = (unsigned)std::min<uint64_t>(p.tiles, 152 * kHopBlocks);
        if (int rc = next_launch(attn_hops_kernel, dim3(blocks), kHopThreads, 0, p, st)) return rc;
    }
    const int rc = p.rows <= kFewMost ? few_rows<T>(p, st) : p.d <= 64 ? cached_dim<T, 64>(p, bm, st) : cached_dim<T, 128>(p, bm, st);
    if (rc || p.splits == 1) return rc;
    return next_launch(attn_join_kernel<T>, dim3((unsigned)((uint64_t)p.T * p.hq)), 256, 0, static_cast<const AttnParams &>(p), st);
}

int attn_cached(const CachedParams &p, uint32_t dtype, int bm, cudaStream_t st)
{
    return dtype == K2T_BF16 ? launch_cached<__nv_bfloat16>(p, bm, st) : launch_cached<__half>(p, bm, st);
}

}  // namespace k2t
