// k2t_cache.cu -- node states written into the 8-bit cache and read back.
//
// Both calls are one pass over their tensors and bound by memory.
#include <algorithm>
#include <atomic>

#include "k2t_cache.cuh"
#include "k2t_norm.cuh"
#include "k2t_rows.h"

namespace k2t {

namespace {

constexpr int kWriteThreads = 128;

// The largest magnitude of 8 values onto `top`, as bits: of 16-bit types two a word, of which those of numbers are in order and
// below those of what is not.
template <typename T> struct Magnitude {
    static constexpr uint32_t kInfinite = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    static __device__ __forceinline__ void add(uint32_t &top, const RawEight<T> &x)
    {
        top = __vimax3_u16x2(top, x.u.x & 0x7fff7fffu, x.u.y & 0x7fff7fffu);
        top = __vimax3_u16x2(top, x.u.z & 0x7fff7fffu, x.u.w & 0x7fff7fffu);
    }
    static __device__ __forceinline__ uint32_t one(uint32_t top) { return max(top & 0xffffu, top >> 16); }
    static __device__ __forceinline__ float value(uint32_t bits)
    {
        return std::is_same<T, __half>::value ? __half2float(__ushort_as_half((unsigned short)bits)) : __uint_as_float(bits << 16);
    }
};
template <> struct Magnitude<float> {
    static constexpr uint32_t kInfinite = 0x7f800000u;
    static __device__ __forceinline__ void add(uint32_t &top, const RawEight<float> &x)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x.v[e]) & 0x7fffffffu);
    }
    static __device__ __forceinline__ uint32_t one(uint32_t top) { return top; }
    static __device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits); }
};

// A block of nodes of U heads, keys and values: all in registers, the largest magnitudes, then the bytes.  A thread has PPH
// pieces of 8 values of a head; of narrow heads U are taken together.  Rows of the block that the call does not write stay;
// where the block's scale grows, they are rounded again.  What is not finite does not count, and becomes NaN: a block that has
// such values is looked through again, so that the others spend two instructions less a value.
template <typename T, int PPH>
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const __grid_constant__ CacheParams p)
{
    using M = Magnitude<T>;
    constexpr int U = PPH == 1 ? 4 : PPH == 2 ? 2 : 1;
    __shared__ uint32_t tops[2][U][kWriteThreads / 32];
    const uint32_t tid = threadIdx.x, h0 = blockIdx.y * U;
    const uint32_t P = p.d / 8, over = 65536 / P + 1;      // a piece's row, at / P = at * over >> 16 of at < 512
    const uint64_t block = p.first / kCacheBlock + blockIdx.x, node0 = block * kCacheBlock;
    const uint64_t begin = max(p.first, node0), end = min(p.first + p.count, node0 + kCacheBlock);
    const uint32_t r0 = (uint32_t)(begin - node0), r1 = (uint32_t)(end - node0);          // rows that the call writes
    const uint32_t rows = (uint32_t)min((uint64_t)kCacheBlock, p.n - node0);             // and that the cache has
    const bool whole = r1 - r0 == rows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint32_t row[PPH], col[PPH];
    bool mine[PPH];
#pragma unroll
    for (int i = 0; i < PPH; ++i) {
        const uint32_t at = i * kWriteThreads + tid;
        row[i] = at * over >> 16, col[i] = (at - row[i] * P) * 8;
        mine[i] = row[i] >= r0 && row[i] < r1;
    }
    RawEight<T> a[2][U][PPH];
    uint32_t top[2][U];
    int old[2][U];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = h0 + u < p.heads;
            const T *x = static_cast<const T *>(p.x[w]) + (int64_t)(h0 + u) * p.x_head[w] - (int64_t)p.x_row[w] * (int64_t)(p.first - node0);
            old[w][u] = in && !whole ? p.scales[w][(uint64_t)(h0 + u) * p.scale_pitch + block] : 0;
#pragma unroll
            for (int i = 0; i < PPH; ++i) {
                a[w][u][i].clear();
                if (in && mine[i]) a[w][u][i].load(x + (int64_t)row[i] * p.x_row[w] + col[i]);
            }
        }
    auto join = [&] {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                top[w][u] = __reduce_max_sync(~0u, M::one(top[w][u]));
                if ((tid & 31) == 0) tops[w][u][tid >> 5] = top[w][u];
            }
        __syncthreads();                                   // the scales of before have been read, too
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < kWriteThreads / 32; ++i) top[w][u] = max(top[w][u], tops[w][u][i]);
    };
    bool finite = true;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            top[w][u] = 0;
#pragma unroll
            for (int i = 0; i < PPH; ++i) M::add(top[w][u], a[w][u][i]);
        }
    join();
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int u = 0; u < U; ++u) finite &= top[w][u] < M::kInfinite;
    if (!finite) {                                         // the same in all threads
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float most = 0.0f;
#pragma unroll
                for (int i = 0; i < PPH; ++i) {
                    const Eight<T> x8 = a[w][u][i].values();
#pragma unroll
                    for (int e = 0; e < 8; ++e) most = fabsf(x8.v[e]) < INFINITY ? fmaxf(most, fabsf(x8.v[e])) : most;
                }
                top[w][u] = __reduce_max_sync(~0u, __float_as_uint(most));
                if ((tid & 31) == 0) tops[w][u][tid >> 5] = top[w][u];
            }
        __syncthreads();
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h0 + u >= p.heads) break;
            if (!finite)
                for (int i = 0; i < kWriteThreads / 32; ++i) top[w][u] = max(top[w][u], tops[w][u][i]);
            int s = scale_for(finite ? M::value(top[w][u]) : __uint_as_float(top[w][u]));
            if (!whole) s = max(s, old[w][u]);
            const float f = power_of_two(kScaleBias - s);
            uint8_t *codes = p.codes[w] + ((uint64_t)(h0 + u) * p.n + node0) * p.pitch;
#pragma unroll
            for (int i = 0; i < PPH; ++i) {
                uint2 *to = reinterpret_cast<uint2 *>(codes + row[i] * p.pitch + col[i]);
                uint32_t y[2];
                if (mine[i]) {
                    Eight<T> x8 = a[w][u][i].values();
                    if (!finite)
#pragma unroll
                        for (int e = 0; e < 8; ++e) x8.v[e] += x8.v[e] * 0.0f;     // an infinite value becomes NaN, not the largest
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        y[e] = to_e4m3(x8.v[4 * e] * f, x8.v[4 * e + 1] * f) | to_e4m3(x8.v[4 * e + 2] * f, x8.v[4 * e + 3] * f) << 16;
                    // to the row's end, with what fills its last 16 bytes: part of a sector written costs it read first
                    if (col[i] + 8 == p.d && p.pitch != p.d) *reinterpret_cast<uint4 *>(to) = make_uint4(y[0], y[1], 0, 0);
                    else *to = make_uint2(y[0], y[1]);
                } else if (row[i] < rows && s != old[w][u]) {
                    const float again = power_of_two(max(old[w][u] - s, -126));
                    const uint2 held = *to;
                    const uint32_t v[2] = {held.x, held.y};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 c = e4m3_pair(v[e] & 0xffffu), g = e4m3_pair(v[e] >> 16);
                        y[e] = to_e4m3(c.x * again, c.y * again) | to_e4m3(g.x * again, g.y * again) << 16;
                    }
                    *to = make_uint2(y[0], y[1]);
                }
            }
            if (tid == 0) p.scales[w][(uint64_t)(h0 + u) * p.scale_pitch + block] = (uint8_t)s;
        }
}

constexpr int kReadThreads = 256;
constexpr int kReadAhead = 4;                              // rows of a thread in flight

// A thread takes 16 bytes of results at the same place of kReadAhead neighbouring rows at a time.
template <typename T>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ CacheParams p, uint32_t per, uint32_t at_once)
{
    constexpr uint32_t V = 16 / sizeof(T);
    using Codes = std::conditional_t<V == 8, uint2, uint32_t>;
    const uint32_t i = blockIdx.x * kReadThreads + threadIdx.x, first = i / per, rest = i - first * per;
    if (first >= at_once) return;
    const uint32_t P = p.d / V, wh = rest / P, c = rest - wh * P, which = wh / p.heads, h = wh - which * p.heads;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint8_t *codes = p.codes[which] + (uint64_t)h * p.n * p.pitch + c * V, *scales = p.scales[which] + (uint64_t)h * p.scale_pitch;
    T *out = static_cast<T *>(p.x[which]) + (int64_t)h * p.x_head[which] + c * V;
    for (uint64_t row = (uint64_t)first * kReadAhead; row < p.count; row += (uint64_t)at_once * kReadAhead) {
        Codes u[kReadAhead];
        float f[kReadAhead];
#pragma unroll
        for (int k = 0; k < kReadAhead; ++k) {
            const uint64_t at = row + k;
            u[k] = Codes{}, f[k] = 0.0f;
            if (at >= p.count) continue;
            const uint64_t node = p.nodes ? (uint64_t)(int64_t)p.nodes[at] : p.first + at;     // a negative one is past the end
            if (node >= p.n) continue;
            u[k] = *reinterpret_cast<const Codes *>(codes + node * p.pitch);
            f[k] = power_of_two(scales[node / kCacheBlock] - kScaleBias);
        }
#pragma unroll
        for (int k = 0; k < kReadAhead; ++k) {
            const uint64_t at = row + k;
            if (at >= p.count) break;
            T *to = out + (int64_t)at * p.x_row[which];
            if constexpr (V == 8) {
                const uint32_t w[2] = {u[k].x, u[k].y};
                Eight<T> a;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 y = e4m3_pair(w[e] & 0xffffu), z = e4m3_pair(w[e] >> 16);
                    a.v[4 * e] = y.x * f[k], a.v[4 * e + 1] = y.y * f[k], a.v[4 * e + 2] = z.x * f[k], a.v[4 * e + 3] = z.y * f[k];
                }
                a.store(to);
            } else {
                const float2 y = e4m3_pair(u[k] & 0xffffu), z = e4m3_pair(u[k] >> 16);
                *reinterpret_cast<float4 *>(to) = make_float4(y.x * f[k], y.y * f[k], z.x * f[k], z.y * f[k]);
            }
        }
    }
}

int check_call(const k2t_cache *c, bool read)
{
    if (int rc = check_cache(c)) return rc;
    if (c->dtype > K2T_FP32) return K2T_EINVAL;
    if (c->count && (!c->x_k || !c->x_v)) return K2T_EINVAL;
    if (!rows_aligned(c->x_k, c->xk_row, c->xk_head) || !rows_aligned(c->x_v, c->xv_row, c->xv_head) || ((uintptr_t)c->nodes & 3u))
        return K2T_EINVAL;
    if (!read && c->nodes) return K2T_EINVAL;
    if (c->nodes ? c->first != 0 : c->first > c->n_nodes || c->count > c->n_nodes - c->first) return K2T_ERANGE;
    if (c->count > K2T_ATTN_MAX_NODES) return K2T_ERANGE;
    if (read && c->count &&
        (rows_overlap(c->xk_row, c->xk_head, c->count, c->n_kv_heads, c->head_dim) || rows_overlap(c->xv_row, c->xv_head, c->count, c->n_kv_heads, c->head_dim)))
        return K2T_EINVAL;
    return K2T_OK;
}

CacheParams params(const k2t_cache *c)
{
    CacheParams p{};
    p.heads = c->n_kv_heads, p.d = c->head_dim, p.pitch = cache_pitch(c->head_dim), p.scale_pitch = (uint32_t)cache_scale_pitch(c->n_nodes);
    p.n = c->n_nodes, p.first = c->first, p.count = c->count, p.nodes = c->nodes;
    p.codes[0] = static_cast<uint8_t *>(c->k), p.codes[1] = static_cast<uint8_t *>(c->v);
    p.scales[0] = c->k_scale, p.scales[1] = c->v_scale;
    p.x[0] = c->x_k, p.x[1] = c->x_v;
    p.x_row[0] = c->xk_row, p.x_row[1] = c->xv_row, p.x_head[0] = c->xk_head, p.x_head[1] = c->xv_head;
    return p;
}

template <typename T, int PPH> int write_pieces(const CacheParams &p, cudaStream_t st)
{
    constexpr uint32_t U = PPH == 1 ? 4 : PPH == 2 ? 2 : 1;
    const uint64_t blocks = (p.first + p.count - 1) / kCacheBlock - p.first / kCacheBlock + 1;
    return norm_launch(cache_write_kernel<T, PPH>, dim3((unsigned)blocks, (p.heads + U - 1) / U), kWriteThreads, 0, st, p);
}

template <typename T> int write(const CacheParams &p, cudaStream_t st)
{
    const uint32_t pieces = p.d / 8;
    if (pieces <= 4) return write_pieces<T, 1>(p, st);
    if (pieces <= 8) return write_pieces<T, 2>(p, st);
    if (pieces <= 12) return write_pieces<T, 3>(p, st);
    return write_pieces<T, 4>(p, st);
}

template <typename T> int read(const CacheParams &p, cudaStream_t st)
{
    const uint64_t per = (uint64_t)2 * p.heads * (p.d * sizeof(T) / 16);              // threads a row: at most 2^22
    const uint64_t runs = (p.count + kReadAhead - 1) / kReadAhead, at_once = std::min(runs, std::max<uint64_t>(152 * 2048 * 16, per) / per);
    const unsigned blocks = (unsigned)((at_once * per + kReadThreads - 1) / kReadThreads);
    return norm_launch(cache_read_kernel<T>, dim3(blocks), kReadThreads, 0, st, p, (uint32_t)per, (uint32_t)at_once);
}

}  // namespace

int check_cache(const k2t_cache *c)
{
    if (!c || c->reserved || c->n_kv_heads == 0 || c->head_dim == 0 || c->head_dim % 8) return K2T_EINVAL;
    if (c->head_dim > K2T_ATTN_MAX_HEAD_DIM || c->n_kv_heads > 65535 || c->n_nodes > K2T_ATTN_MAX_NODES) return K2T_ERANGE;
    if (c->n_nodes && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return K2T_EINVAL;
    if (((uintptr_t)c->k | (uintptr_t)c->v | (uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 15u) return K2T_EINVAL;
    return K2T_OK;
}

}  // namespace k2t

using namespace k2t;

extern "C" {

int k2t_cache_write(const k2t_cache *c, void *stream)
{
    if (int rc = check_call(c, false)) return rc;
    if (!c->count) return K2T_OK;
    const CacheParams p = params(c);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return c->dtype == K2T_BF16 ? write<__nv_bfloat16>(p, st) : c->dtype == K2T_FP16 ? write<__half>(p, st) : write<float>(p, st);
}

int k2t_cache_read(const k2t_cache *c, void *stream)
{
    if (int rc = check_call(c, true)) return rc;
    if (!c->count) return K2T_OK;
    const CacheParams p = params(c);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return c->dtype == K2T_BF16 ? read<__nv_bfloat16>(p, st) : c->dtype == K2T_FP16 ? read<__half>(p, st) : read<float>(p, st);
}

}  // extern "C"
