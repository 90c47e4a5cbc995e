// k2t_attn_cached.cu -- launches of the attention over the 8-bit cache.
#include "k2t_attn_cached.cuh"
#include "k2t_attn_few.cuh"
#include "k2t_attn_launch.cuh"

namespace k2t {

// bm: rows a block takes, 32, 64 or 128.
template <typename T, int DP> static int cached_dim(const CachedParams &p, int bm, cudaStream_t st)
{
    const dim3 grid(p.splits * p.row_tiles, p.hkv);
    const size_t smem = CachedSmem<DP>::bytes(p);
    switch (bm) {
    case 32: return attn_launch<attn_cached_kernel<T, DP, 32>>(grid, kCachedThreads, smem, p, st);
    case 64: return attn_launch<attn_cached_kernel<T, DP, 64>>(grid, kCachedThreads, smem, p, st);
    default: return attn_launch<attn_cached_kernel<T, DP, 128>>(grid, kCachedThreads, smem, p, st);
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
    const int rc = p.rows <= 8 ? few_rows<T>(p, st) : p.d <= 64 ? cached_dim<T, 64>(p, bm, st) : cached_dim<T, 128>(p, bm, st);
    if (rc || p.splits == 1) return rc;
    return next_launch(attn_join_kernel<T>, dim3((unsigned)((uint64_t)p.T * p.hq)), 256, 0, static_cast<const AttnParams &>(p), st);
}

int attn_cached(const CachedParams &p, uint32_t dtype, int bm, cudaStream_t st)
{
    return dtype == K2T_BF16 ? launch_cached<__nv_bfloat16>(p, bm, st) : launch_cached<__half>(p, bm, st);
}

}  // namespace k2t
