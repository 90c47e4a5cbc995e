// k2t_attn_cached.cu -- launches of the attention over the 8-bit cache.
#include "k2t_attn_cached.cuh"
#include "k2t_attn_launch.cuh"

namespace k2t {

template <typename T> static int launch_cached(const CachedParams &p, cudaStream_t st)
{
    if (int rc = next_launch(attn_cached_kernel<T>, dim3((unsigned)((uint64_t)p.T * p.hq), p.splits), 128, 0, p, st)) return rc;
    if (p.splits == 1) return K2T_OK;
    return next_launch(attn_join_kernel<T>, dim3((unsigned)((uint64_t)p.T * p.hq)), 256, 0, static_cast<const AttnParams &>(p), st);
}

int attn_cached(const CachedParams &p, uint32_t dtype, cudaStream_t st)
{
    return dtype == K2T_BF16 ? launch_cached<__nv_bfloat16>(p, st) : launch_cached<__half>(p, st);
}

}  // namespace k2t
