// k2t_attn_launch.cuh -- launches of the attention kernels.
#pragma once

#include "k2t_attn_bwd.cuh"
#include "k2t_attn_fwd.cuh"

namespace k2t {

#define K2T_ATTN_CUDA(call)                              \
    do {                                                 \
        cudaError_t e_ = (call);                         \
        if (e_ != cudaSuccess) {                         \
            g_last_cuda = (int)e_;                       \
            return K2T_ECUDA;                            \
        }                                                \
    } while (0)

template <typename K>
int attn_launch(K kernel, dim3 grid, int threads, size_t smem, const AttnParams &p, cudaStream_t st)
{
    K2T_ATTN_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    kernel<<<grid, threads, smem, st>>>(p);
    K2T_ATTN_CUDA(cudaGetLastError());
    return K2T_OK;
}

// bm: rows a block takes, 32, 64, 128 or 256.
template <typename T, int DP, int KW, bool TWO> int forward_tile(const AttnParams &p, cudaStream_t st)
{
    return attn_launch(attn_fwd_kernel<T, DP, KW, TWO>, dim3(p.splits * p.row_tiles, p.hkv), kTcThreads, TcSmem<DP, TWO>::bytes(p), p, st);
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
    attn_join_kernel<T><<<(unsigned)((uint64_t)p.T * p.hq), 256, 0, st>>>(p);
    K2T_ATTN_CUDA(cudaGetLastError());
    return K2T_OK;
}

template <typename T, int DP> int backward_dim(const AttnParams &p, cudaStream_t st)
{
    const dim3 by_rows(p.splits * p.row_tiles, p.hkv), by_nodes((unsigned)p.tiles, p.hkv);
    if (p.row_tiles == 1) return attn_launch(attn_bwd_kernel<T, DP, 0>, by_rows, kAttnThreads, BwdSmem<DP, 0>::bytes(p), p, st);
    int rc = K2T_OK;
    if (p.tiles) rc = attn_launch(attn_bwd_kernel<T, DP, 1>, by_nodes, kAttnThreads, BwdSmem<DP, 1>::bytes(p), p, st);
    if (!rc && p.rows) rc = attn_launch(attn_bwd_kernel<T, DP, 2>, by_rows, kAttnThreads, BwdSmem<DP, 2>::bytes(p), p, st);
    return rc;
}

template <typename T> int launch_backward(const AttnParams &p, cudaStream_t st)
{
    const uint64_t rows = (uint64_t)p.T * p.hq;
    if (rows) {
        attn_delta_kernel<T><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p);
        K2T_ATTN_CUDA(cudaGetLastError());
    }
    int rc = p.d <= 64 ? backward_dim<T, 64>(p, st) : backward_dim<T, 128>(p, st);
    if (rc) return rc;
    const uint64_t blocks = rows + (uint64_t)p.hq * p.buckets;
    if (blocks) {
        attn_bwd_join_kernel<T><<<(unsigned)blocks, 256, 0, st>>>(p);
        K2T_ATTN_CUDA(cudaGetLastError());
    }
    return K2T_OK;
}

}  // namespace k2t
