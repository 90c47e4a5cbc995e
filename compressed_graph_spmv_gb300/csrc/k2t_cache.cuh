// k2t_cache.cuh -- the 8-bit cache of node states: what its kernels share.
//
// Keys and values are e4m3 (a sign, 4 bits of exponent, 3 of fraction; largest
// 448, least 2^-9) times a power of two for each block of 32 nodes and head,
// kept as a byte s: 2^(s - 64).  A power of two costs e4m3 no precision, makes
// division and multiplication exact (what is read back is exactly what the
// byte stands for, and bf16 holds it), and lets a block that is written a few
// nodes at a time change its scale with no second rounding of what stays,
// except of the values that the new scale makes subnormal.
// Layout [head][node][pitch], pitch = head_dim rounded up to 16: a tile of
// nodes of one head is one piece of memory.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "k2t_internal.h"

namespace k2t {

constexpr uint32_t kCacheBlock = K2T_CACHE_BLOCK;
constexpr int kScaleBias = 64;                        // scale byte s stands for 2^(s - 64), s = 0..127

// The least scale byte that holds finite magnitudes up to `top`: top <= 448 2^(s - 64).
__device__ __forceinline__ int scale_for(float top)
{
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);      // 448 = 1.75 2^8
    return min(max(e + kScaleBias, 0), 127);
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two values as e4m3, to nearest even, a in the low byte.  Magnitudes over 448 become 448; what is no number NaN.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// The two e4m3 values of a half word, exactly, as fp16.
__device__ __forceinline__ uint32_t from_e4m3(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

__device__ __forceinline__ float2 e4m3_pair(uint32_t two)
{
    const uint32_t h = from_e4m3(two);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 8 values of a row.
template <typename T> struct Eight;
template <> struct Eight<float> {
    float v[8];
    __device__ __forceinline__ void load(const float *p)
    {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void store(float *p) const
    {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <> struct Eight<__half> {
    float v[8];
    __device__ __forceinline__ void load(const __half *p) { set(*reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void set(uint4 u)
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ void store(__half *p) const
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Eight<__nv_bfloat16> {
    float v[8];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { set(*reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void set(uint4 u)
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The same as they lie in memory, to be held in fewer registers.
template <typename T> struct RawEight {
    uint4 u;
    __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ Eight<T> values() const
    {
        Eight<T> e;
        e.set(u);
        return e;
    }
};
template <> struct RawEight<float> : Eight<float> {
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    }
    __device__ __forceinline__ const Eight<float> &values() const { return *this; }
};

// What the kernels need of k2t_cache, by value.
struct CacheParams {
    uint32_t heads, d, pitch, scale_pitch;
    uint64_t n, first, count;
    uint8_t *codes[2], *scales[2];               // keys, values
    void *x[2];                                  // a write's inputs, a read's outputs
    int64_t x_row[2], x_head[2];
    const int32_t *nodes;
};

inline uint32_t cache_pitch(uint32_t d) { return (d + 15) / 16 * 16; }
inline uint64_t cache_scale_pitch(uint64_t n) { return ((n + kCacheBlock - 1) / kCacheBlock + 15) / 16 * 16; }

// Sizes and the cache's own tensors, for every call that takes one.
int check_cache(const k2t_cache *c);

}  // namespace k2t
