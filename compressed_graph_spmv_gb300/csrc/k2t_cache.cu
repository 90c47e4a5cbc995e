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
constexpr int kRowChunks = K2T_ATTN_MAX_HEAD_DIM / 16;
constexpr int kPieces = kCacheBlock * kRowChunks / kWriteThreads;      // chunks of 16 values a thread, at most

// One block of nodes of one head, keys or values: largest magnitude first, then the bytes.  Rows of the block that the call
// does not write stay; where the block's scale grows, they are rounded again.
template <typename T>
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const __grid_constant__ CacheParams p)
{
    __shared__ uint32_t tops[kWriteThreads / 32];
    const uint32_t which = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
    const uint64_t block = p.first / kCacheBlock + blockIdx.x, node0 = block * kCacheBlock;
    const uint32_t C = p.pitch / 16;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint8_t *codes = p.codes[which] + ((uint64_t)h * p.n + node0) * p.pitch, *scale = p.scales[which] + (uint64_t)h * p.scale_pitch + block;
    const T *x = static_cast<const T *>(p.x[which]) + (int64_t)h * p.x_head[which];
    const int old = *scale;
    Eight<T> a[kPieces], b[kPieces];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const uint32_t at = tid + i * kWriteThreads, r = at / C, c = at - r * C;
        const uint64_t node = node0 + r;
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i].v[e] = b[i].v[e] = 0.0f;
        if (r < kCacheBlock && node >= p.first && node < p.first + p.count) {
            const T *src = x + (int64_t)(node - p.first) * p.x_row[which] + c * 16;
            a[i].load(src);
            if (c * 16 + 8 < p.d) b[i].load(src + 8);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t u = __float_as_uint(a[i].v[e]) & 0x7fffffffu, w = __float_as_uint(b[i].v[e]) & 0x7fffffffu;
            top = max(top, max(u < 0x7f800000u ? u : 0, w < 0x7f800000u ? w : 0));
        }
    }
    top = __reduce_max_sync(~0u, top);
    if ((tid & 31) == 0) tops[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWriteThreads / 32; ++i) top = max(top, tops[i]);
    const uint64_t begin = max(p.first, node0), end = min(p.first + p.count, node0 + kCacheBlock);
    const bool whole = end - begin == min((uint64_t)kCacheBlock, p.n - node0);
    int s = scale_for(__uint_as_float(top));
    if (!whole) s = max(s, old);
    const float f = power_of_two(kScaleBias - s), again = power_of_two(max(old - s, -126));
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const uint32_t at = tid + i * kWriteThreads, r = at / C, c = at - r * C;
        const uint64_t node = node0 + r;
        if (r >= kCacheBlock || node >= p.n) continue;
        uint4 *to = reinterpret_cast<uint4 *>(codes + (uint64_t)r * p.pitch + c * 16);
        uint32_t w[4];
        if (node >= p.first && node < p.first + p.count) {
            // x 0 + x f: an infinite value becomes NaN, not the largest
            auto two = [&](float v0, float v1) { return to_e4m3(fmaf(v0, f, v0 * 0.0f), fmaf(v1, f, v1 * 0.0f)); };
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[e] = two(a[i].v[4 * e], a[i].v[4 * e + 1]) | two(a[i].v[4 * e + 2], a[i].v[4 * e + 3]) << 16;
                w[2 + e] = two(b[i].v[4 * e], b[i].v[4 * e + 1]) | two(b[i].v[4 * e + 2], b[i].v[4 * e + 3]) << 16;
            }
        } else {
            if (s == old) continue;
            const uint4 was = *to;
            const uint32_t u[4] = {was.x, was.y, was.z, was.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = from_e4m3(u[e] & 0xffffu), hi = from_e4m3(u[e] >> 16);
                const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), z = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                w[e] = to_e4m3(y.x * again, y.y * again) | to_e4m3(z.x * again, z.y * again) << 16;
            }
        }
        *to = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (tid == 0) *scale = (uint8_t)s;
}

constexpr int kReadThreads = 256;

// A thread takes 16 values of a row.
template <typename T>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ CacheParams p)
{
    const uint32_t C = p.pitch / 16, per = C * p.heads * 2;
    const uint64_t total = p.count * per;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (uint64_t i = (uint64_t)blockIdx.x * kReadThreads + threadIdx.x; i < total; i += (uint64_t)gridDim.x * kReadThreads) {
        const uint64_t row = i / per;
        const uint32_t rest = (uint32_t)(i - row * per), c = rest % C, h = rest / C % p.heads, which = rest / C / p.heads;
        const uint64_t node = p.nodes ? (uint64_t)(int64_t)p.nodes[row] : p.first + row;      // a negative one is past the end
        Eight<T> a, b;
#pragma unroll
        for (int e = 0; e < 8; ++e) a.v[e] = b.v[e] = 0.0f;
        if (node < p.n) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p.codes[which] + ((uint64_t)h * p.n + node) * p.pitch + c * 16);
            const float f = power_of_two(p.scales[which][(uint64_t)h * p.scale_pitch + node / kCacheBlock] - kScaleBias);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = from_e4m3(w[e] & 0xffffu), hi = from_e4m3(w[e] >> 16);
                const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), z = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                float *to = e < 2 ? a.v + 4 * e : b.v + 4 * (e - 2);
                to[0] = y.x * f, to[1] = y.y * f, to[2] = z.x * f, to[3] = z.y * f;
            }
        }
        T *out = static_cast<T *>(p.x[which]) + (int64_t)row * p.x_row[which] + (int64_t)h * p.x_head[which] + c * 16;
        a.store(out);
        if (c * 16 + 8 < p.d) b.store(out + 8);
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

template <typename T> int write(const CacheParams &p, cudaStream_t st)
{
    const uint64_t blocks = (p.first + p.count - 1) / kCacheBlock - p.first / kCacheBlock + 1;
    return norm_launch(cache_write_kernel<T>, dim3((unsigned)blocks, p.heads, 2), kWriteThreads, 0, st, p);
}

template <typename T> int read(const CacheParams &p, cudaStream_t st)
{
    const uint64_t total = p.count * (p.pitch / 16) * p.heads * 2;
    const unsigned blocks = (unsigned)std::min<uint64_t>((total + kReadThreads - 1) / kReadThreads, 152 * 64);
    return norm_launch(cache_read_kernel<T>, dim3(blocks), kReadThreads, 0, st, p);
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
