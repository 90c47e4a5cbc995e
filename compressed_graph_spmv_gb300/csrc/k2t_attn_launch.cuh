// k2t_attn_launch.cuh -- launches of the attention kernels.
#pragma once

#include <atomic>

#include "k2t_attn_bwd.cuh"
#include "k2t_attn_delta.cuh"
#include "k2t_attn_fwd.cuh"

namespace k2t {

constexpr int kAttnMaxSmem = 232448;   // 227 KB

#define K2T_ATTN_CUDA(call)                              \
    do {                                                 \
        cudaError_t e_ = (call);                         \
        if (e_ != cudaSuccess) {                         \
            g_last_cuda = (int)e_;                       \
            return K2T_ECUDA;                            \
        }                                                \
    } while (0)

// Programmatic launch: a kernel's blocks may be set up while the kernel before it on the stream (whichever that is) still
// runs; they wait for its end (griddepcontrol.wait) before they touch global memory.
template <typename K> int next_launch(K kernel, dim3 grid, int threads, size_t smem, const AttnParams &p, cudaStream_t st)
{
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &a;
    c.numAttrs = 1;
    K2T_ATTN_CUDA(cudaLaunchKernelEx(&c, kernel, p));
    return K2T_OK;
}

// The shared memory a kernel may have is a setting of the kernel on a device: raised once, to what any call can need.
template <auto kernel> int attn_launch(dim3 grid, int threads, size_t smem, const AttnParams &p, cudaStream_t st)
{
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    K2T_ATTN_CUDA(cudaGetDevice(&dev));
    if (dev >= 64 || !(set.load() >> dev & 1)) {
        K2T_ATTN_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnMaxSmem));
        if (dev < 64) set.fetch_or(1ull << dev);
    }
    if (smem > (size_t)kAttnMaxSmem) return K2T_ERANGE;
    return next_launch(kernel, grid, threads, smem, p, st);
}

// bm: rows a block takes, 32, 64, 128 or 256.
template <typename T, int DP, int KW, bool TWO> int forward_tile(const AttnParams &p, cudaStream_t st)
{
    return attn_launch<attn_fwd_kernel<T, DP, KW, TWO>>(dim3(p.splits * p.row_tiles, p.hkv), kTcThreads, TcSmem<DP, TWO>::bytes(p), p, st);
}

template <typename T, int DP> int forward_dim(const AttnParams &p, int bm, cudaStream_t st)
{
    switch (bm) {
    case 32: return forward_tile<T, DP, 32, false>(p, st);
    case 64: return forward_tile<T, DP, 64, false>(p, st);
    case 128: return forward_tile<T, DP, 128, false>(p, st);
    default: return forward_tile<T, DP, 128, true>(p, st);
    }
}

template <typename T> int launch_forward(const AttnParams &p, int bm, cudaStream_t st)
{
    int rc = p.d <= 64 ? forward_dim<T, 64>(p, bm, st) : forward_dim<T, 128>(p, bm, st);
    if (rc || p.splits == 1) return rc;
    return next_launch(attn_join_kernel<T>, dim3((unsigned)((uint64_t)p.T * p.hq)), 256, 0, p, st);
}

// Rows a block of attn_delta_kernel takes: the fewest lanes that hold them all, as in the forward pass (32 rows a head over
// 2^18 nodes, forward and backward, 467 us, in 128 lanes 501).
inline uint32_t delta_rows(const AttnParams &p) { return p.rows <= 32 ? 32 : p.rows <= 64 ? 64 : 128; }

template <typename T, int DP> int delta_dim(const AttnParams &from, cudaStream_t st)
{
    AttnParams p = from;
    p.splits = p.delta_splits, p.row_tiles = p.delta_tiles;
    const dim3 grid(p.splits * p.row_tiles, p.hkv);
    switch (delta_rows(p)) {
    case 32: return attn_launch<attn_delta_kernel<T, DP, 32>>(grid, kTcThreads, DeltaSmem<DP>::bytes(p), p, st);
    case 64: return attn_launch<attn_delta_kernel<T, DP, 64>>(grid, kTcThreads, DeltaSmem<DP>::bytes(p), p, st);
    default: return attn_launch<attn_delta_kernel<T, DP, 128>>(grid, kTcThreads, DeltaSmem<DP>::bytes(p), p, st);
    }
}

// Row tiles that the one-pass kernel holds: 4 of head_dim 64 or less, 2 of more (shared and tensor memory).  One pass reads
// states and computes scores once: 32 queries over 2^18 nodes, forward and backward, 467 us; with two kernels 1225 us.
inline uint32_t bwd_fused_tiles(uint32_t d) { return d <= 64 ? 4 : 2; }

template <typename T, int DP, int RT, bool DKV> int backward_nodes(const AttnParams &from, cudaStream_t st)
{
    using S = BwdSmem<DP, RT, DKV>;
    AttnParams p = from;
    const uint32_t groups = (p.row_tiles + RT - 1) / RT;
    // 128 threads sum by bucket, 64 where their tables do not fit beside the tiles (32 queries over 2^18 nodes, forward and
    // backward, 467 us, with 64 threads 515)
    p.hist_threads = S::bytes(p, 128) <= (size_t)kAttnMaxSmem ? 128 : 64;
    return attn_launch<attn_bwd_nodes_kernel<T, DP, RT, DKV>>(dim3(p.splits * groups, p.hkv), kBwdThreads, S::bytes(p, p.hist_threads), p, st);
}

template <typename T, int DP> int backward_dim(const AttnParams &p, cudaStream_t st)
{
    if (p.row_tiles == 1) return backward_nodes<T, DP, 1, true>(p, st);
    if (p.row_tiles == 2) return backward_nodes<T, DP, 2, true>(p, st);
    if constexpr (DP == 64) {
        if (p.row_tiles <= 4) return backward_nodes<T, DP, 4, true>(p, st);
    }
    if (p.tiles) {
        int rc = attn_launch<attn_bwd_rows_kernel<T, DP>>(dim3((unsigned)p.tiles, p.hkv), kBwdRowThreads, BwdRowSmem<DP>::bytes(p), p, st);
        if (rc) return rc;
    }
    return backward_nodes<T, DP, 4, false>(p, st);
}

template <typename T> int launch_backward(const AttnParams &p, cudaStream_t st)
{
    if (p.delta_splits) {
        int rc = p.d <= 64 ? delta_dim<T, 64>(p, st) : delta_dim<T, 128>(p, st);
        if (rc) return rc;
    }
    if (p.row_tiles > bwd_fused_tiles(p.d)) {
        int rc = next_launch(attn_rows_kernel<T>, dim3(p.row_tiles * (kBwdRows / 8), p.hkv), 256, 0, p, st);
        if (rc) return rc;
    }
    int rc = p.d <= 64 ? backward_dim<T, 64>(p, st) : backward_dim<T, 128>(p, st);
    if (rc) return rc;
    const uint64_t rows = p.splits > 1 ? (uint64_t)p.T * p.hq : 0, blocks = (rows + 3) / 4 + (p.buckets ? p.hq : 0);
    return blocks ? next_launch(attn_bwd_join_kernel<T>, dim3((unsigned)blocks), kJoinThreads, 0, p, st) : K2T_OK;
}

}  // namespace k2t
