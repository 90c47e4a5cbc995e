// k2t_attn_cached.cuh -- hop-biased attention over the 8-bit cache of node
// states (k2t_cache.cuh): the simplest form, a block for a query head and a
// share of the nodes.
//
// One pass with the running maximum and sum of the softmax, everything in
// fp32.  A lane scores a node of its warp's 32 (one scale for each), then the
// warp adds up the weighted values, four columns a lane.
#pragma once

#include "k2t_attn.cuh"
#include "k2t_cache.cuh"

namespace k2t {

struct CachedParams : AttnParams {
    uint32_t pitch;                       // bytes of a cached row
    uint64_t scale_pitch, cached;         // of a head's scales; nodes of the cache
    const uint8_t *kc, *vc, *ks, *vs;
};

template <typename T>
__global__ void __launch_bounds__(128) attn_cached_kernel(const __grid_constant__ CachedParams p)
{
    __shared__ __align__(16) float q[K2T_ATTN_MAX_HEAD_DIM];
    __shared__ float part[4][K2T_ATTN_MAX_HEAD_DIM], ml[4][2];
    const uint32_t row = blockIdx.x, t = row / p.hq, hd = row - t * p.hq, hk = hd / p.group, split = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    tc::grid_wait();
    tc::grid_next();
    for (uint32_t i = tid; i < p.pitch; i += 128)
        q[i] = i < p.d ? Elem<T>::to_float(static_cast<const T *>(p.q)[(int64_t)t * p.q_row + (int64_t)hd * p.q_head + i]) * p.scale_log2 : 0.0f;
    __syncthreads();
    const uint32_t col = row_column(p, t * p.group);
    const uint8_t *kc = p.kc + (uint64_t)hk * p.cached * p.pitch, *vc = p.vc + (uint64_t)hk * p.cached * p.pitch;
    const uint8_t *ks = p.ks + hk * p.scale_pitch, *vs = p.vs + hk * p.scale_pitch;
    float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
    const uint64_t blocks = (p.n + 31) / 32;
    for (uint64_t b = split * 4 + warp; b < blocks; b += p.splits * 4) {
        const uint64_t node = b * 32 + lane;
        float s = -INFINITY;
        bool seen = node < p.n;
        float bias = 0.0f;
        if (seen && col < p.sources) {
            const int32_t h = p.hops[node * p.sources + col];
            seen = h >= 0;
            if (seen && p.buckets) {
                bias = Elem<T>::to_float(static_cast<const T *>(p.bias)[(uint64_t)hd * p.buckets + p.bucket_of[min(h, 255)]]);
                if (bias <= Elem<T>::kMasked) seen = false;
            }
        }
        if (seen) {
            float dot = 0.0f;
            for (uint32_t c = 0; c < p.pitch; c += 16) {
                const uint4 u = *reinterpret_cast<const uint4 *>(kc + node * p.pitch + c);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = from_e4m3(w[e] & 0xffffu), hi = from_e4m3(w[e] >> 16);
                    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), z = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                    const float4 k = *reinterpret_cast<const float4 *>(q + c + 4 * e);
                    dot += y.x * k.x + y.y * k.y + z.x * k.z + z.y * k.w;
                }
            }
            s = dot * power_of_two(ks[b] - kScaleBias) + bias * kLog2e;
        }
        float top = s;
        for (int x = 16; x; x >>= 1) {
            const float y = __shfl_xor_sync(~0u, top, x);
            top = top != top || y != y ? NAN : fmaxf(top, y);
        }
        if (top == -INFINITY) continue;
        const float next = m != m || top != top ? NAN : fmaxf(m, top), f = m == -INFINITY ? 0.0f : ex2(m - next);
        float w = seen ? ex2(s - next) : 0.0f, sum = w;
        for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(~0u, sum, x);
        l = l * f + sum;
        m = next;
        w *= power_of_two(vs[b] - kScaleBias);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= f;
        const uint32_t any = __ballot_sync(~0u, seen);
        for (int j = 0; j < 32; ++j) {
            const float wj = __shfl_sync(~0u, w, j);
            if (!(any >> j & 1) || lane * 4 >= (int)p.pitch) continue;
            const uint32_t u = *reinterpret_cast<const uint32_t *>(vc + (b * 32 + j) * p.pitch + lane * 4);
            const uint32_t lo = from_e4m3(u & 0xffffu), hi = from_e4m3(u >> 16);
            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), z = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            o[0] = fmaf(wj, y.x, o[0]), o[1] = fmaf(wj, y.y, o[1]), o[2] = fmaf(wj, z.x, o[2]), o[3] = fmaf(wj, z.y, o[3]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][lane * 4 + e] = o[e];
    if (lane == 0) ml[warp][0] = m, ml[warp][1] = l;
    __syncthreads();
    float mx = -INFINITY, ls = 0.0f, acc = 0.0f;
    for (int w = 0; w < 4; ++w) mx = mx != mx || ml[w][0] != ml[w][0] ? NAN : fmaxf(mx, ml[w][0]);
    for (int w = 0; w < 4; ++w) {
        const float f = mx == -INFINITY ? 0.0f : ex2(ml[w][0] - mx);
        ls += f * ml[w][1];
        if (tid < (int)p.d) acc += f * part[w][tid];
    }
    if (p.splits > 1) {
        const uint64_t at = ((uint64_t)split * p.T + t) * p.hq + hd;
        if (tid < (int)p.d) p.part[at * p.d + tid] = acc;
        if (tid == 0) p.part_ml[at * 2] = mx, p.part_ml[at * 2 + 1] = ls;
    } else {
        const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
        if (tid < (int)p.d) static_cast<T *>(p.out)[(int64_t)t * p.out_row + (int64_t)hd * p.out_head + tid] = Elem<T>::from_float(acc * inv);
        if (tid == 0) p.lse[(uint64_t)t * p.hq + hd] = ls == 0.0f ? -INFINITY : (mx + log2f(ls)) * kLn2;
    }
}

}  // namespace k2t
