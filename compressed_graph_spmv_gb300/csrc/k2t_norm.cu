// k2t_norm.cu -- layer norm of node states with the residual sum before it,
// forward and backward.
//
// Both passes read each tensor once: a row lies in the registers of TPR
// threads (VEC values a load, PER loads a thread) while its statistics are
// formed, the mean first and then the squares around it, so that no
// cancellation of large sums arises.  Bound by memory: the passes are loads,
// two reductions of a few shuffles, and stores.  Blocks stay for many rows,
// keep the weight in registers, and in the backward pass sum their rows'
// terms of dweight and dbias there; each block writes one partial row, and
// norm_join_kernel adds those in a fixed order.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "k2t_internal.h"

namespace k2t {

extern thread_local int g_last_cuda;

namespace {

struct NormParams {
    uint32_t dim;
    uint64_t n;
    float eps, inv_dim;
    const void *x, *residual, *weight, *bias, *z_in, *dy, *dz;
    void *y, *z, *dx, *dweight, *dbias;
    float *mean, *rstd, *part;
    uint32_t parts;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC values, moved as one word where VEC fills 16 bytes.
template <typename T, int VEC> struct alignas(VEC * sizeof(T)) Pack { T v[VEC]; };

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load_once(const T *p)
{
    Pack<T, VEC> r;
    if constexpr (VEC * sizeof(T) == 16) {
        *reinterpret_cast<uint4 *>(&r) = __ldcs(reinterpret_cast<const uint4 *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.v[i] = p[i];
    }
    return r;
}
template <typename T, int VEC> __device__ __forceinline__ void store(T *p, const Pack<T, VEC> &r)
{
    if constexpr (VEC * sizeof(T) == 16) {
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&r);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = r.v[i];
    }
}

// Threads of a block: groups of TPR, each with a row of its own.
template <int TPR> struct Group {
    static constexpr int kThreads = TPR < 256 ? 256 : TPR;
    static constexpr int kGroups = kThreads / TPR;
    static constexpr int kWarps = TPR / 32;
};

// Sums of a and b over the TPR threads of a group.  buf: two alternating
// buffers, so that one barrier a call is enough.
template <int TPR>
__device__ __forceinline__ void group_sum(float &a, float &b, float2 *buf, int group, int &turn)
{
#pragma unroll
    for (int x = 16; x; x >>= 1) {
        a += __shfl_xor_sync(~0u, a, x);
        b += __shfl_xor_sync(~0u, b, x);
    }
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        float2 *at = buf + (turn * Group<TPR>::kGroups + group) * W;
        const int tid = threadIdx.x % TPR;
        if ((tid & 31) == 0) at[tid >> 5] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) a += at[i].x, b += at[i].y;
        turn ^= 1;
    }
}

template <typename T, int VEC, int TPR, int PER>
__global__ void __launch_bounds__(Group<TPR>::kThreads) norm_fwd_kernel(const __grid_constant__ NormParams p)
{
    using P = Pack<T, VEC>;
    using Gr = Group<TPR>;
    __shared__ float2 buf[2 * Gr::kGroups * Gr::kWarps];
    const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
    int turn = 0;
    P w[PER], bi[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t c = (tid + i * TPR) * VEC;
        if (c < p.dim) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                w[i].v[e] = static_cast<const T *>(p.weight)[c + e];
                bi[i].v[e] = p.bias ? static_cast<const T *>(p.bias)[c + e] : from_f<T>(0.0f);
            }
        }
    }
    for (uint64_t row = (uint64_t)blockIdx.x * Gr::kGroups + group; row < p.n; row += (uint64_t)gridDim.x * Gr::kGroups) {
        const uint64_t at = row * p.dim;
        P z[PER], r[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = (tid + i * TPR) * VEC;
            if (c < p.dim) z[i] = load_once<T, VEC>(static_cast<const T *>(p.x) + at + c);
        }
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t c = (tid + i * TPR) * VEC;
                if (c < p.dim) r[i] = load_once<T, VEC>(static_cast<const T *>(p.residual) + at + c);
            }
        }
        float s = 0.0f, none = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = (tid + i * TPR) * VEC;
            if (c < p.dim) {
                if (p.residual) {
                    // the sum is what the next layer reads: rounded first, then normalised as it stands
#pragma unroll
                    for (int e = 0; e < VEC; ++e) z[i].v[e] = from_f<T>(to_f(z[i].v[e]) + to_f(r[i].v[e]));
                    store<T, VEC>(static_cast<T *>(p.z) + at + c, z[i]);
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += to_f(z[i].v[e]);
            }
        }
        group_sum<TPR>(s, none, buf, group, turn);
        const float mean = s * p.inv_dim;
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = (tid + i * TPR) * VEC;
            if (c < p.dim) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = to_f(z[i].v[e]) - mean;
                    q = fmaf(d, d, q);
                }
            }
        }
        none = 0.0f;
        group_sum<TPR>(q, none, buf, group, turn);
        const float rstd = rsqrtf(q * p.inv_dim + p.eps);
        if (tid == 0) p.mean[row] = mean, p.rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = (tid + i * TPR) * VEC;
            if (c < p.dim) {
                P y;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    y.v[e] = from_f<T>(fmaf((to_f(z[i].v[e]) - mean) * rstd, to_f(w[i].v[e]), to_f(bi[i].v[e])));
                store<T, VEC>(static_cast<T *>(p.y) + at + c, y);
            }
        }
    }
}

// dx = rstd (w dy - c1 - xh c2) + dz with c1 = mean(w dy), c2 = mean(w dy xh);
// part[block][0 | 1][dim]: the block's sums of dy xh and dy.
template <typename T, int VEC, int TPR, int PER>
__global__ void __launch_bounds__(Group<TPR>::kThreads) norm_bwd_kernel(const __grid_constant__ NormParams p)
{
    using P = Pack<T, VEC>;
    using Gr = Group<TPR>;
    __shared__ float2 buf[2 * Gr::kGroups * Gr::kWarps];
    const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
    int turn = 0;
    P w[PER];
    float dw[PER][VEC], db[PER][VEC];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t c = (tid + i * TPR) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            dw[i][e] = db[i][e] = 0.0f;
            if (c < p.dim) w[i].v[e] = static_cast<const T *>(p.weight)[c + e];
        }
    }
    for (uint64_t row = (uint64_t)blockIdx.x * Gr::kGroups + group; row < p.n; row += (uint64_t)gridDim.x * Gr::kGroups) {
        const uint64_t at = row * p.dim;
        P z[PER], g[PER], extra[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = (tid + i * TPR) * VEC;
            if (c < p.dim) {
                z[i] = load_once<T, VEC>(static_cast<const T *>(p.z_in) + at + c);
                g[i] = load_once<T, VEC>(static_cast<const T *>(p.dy) + at + c);
                if (p.dz) extra[i] = load_once<T, VEC>(static_cast<const T *>(p.dz) + at + c);
            }
        }
        const float mean = p.mean[row], rstd = p.rstd[row];
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = (tid + i * TPR) * VEC;
            if (c < p.dim) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (to_f(z[i].v[e]) - mean) * rstd, dy = to_f(g[i].v[e]), a = dy * to_f(w[i].v[e]);
                    c1 += a;
                    c2 = fmaf(a, xh, c2);
                    dw[i][e] = fmaf(dy, xh, dw[i][e]);
                    db[i][e] += dy;
                }
            }
        }
        group_sum<TPR>(c1, c2, buf, group, turn);
        c1 *= p.inv_dim;
        c2 *= p.inv_dim;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = (tid + i * TPR) * VEC;
            if (c < p.dim) {
                P o;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (to_f(z[i].v[e]) - mean) * rstd, a = to_f(g[i].v[e]) * to_f(w[i].v[e]);
                    float dx = (a - c1 - xh * c2) * rstd;
                    if (p.dz) dx += to_f(extra[i].v[e]);
                    o.v[e] = from_f<T>(dx);
                }
                store<T, VEC>(static_cast<T *>(p.dx) + at + c, o);
            }
        }
    }
    // the groups of a block add up one after another through shared memory
    extern __shared__ float sums[];    // [2][dim], with more than one group
    float *out = p.part + (uint64_t)blockIdx.x * 2 * p.dim;
    for (int turn_of = 0; turn_of < Gr::kGroups; ++turn_of) {
        if (Gr::kGroups > 1) __syncthreads();
        if (group != turn_of) continue;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = (tid + i * TPR) * VEC;
            if (c < p.dim) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float a = dw[i][e], b = db[i][e];
                    if (turn_of > 0) a += sums[c + e], b += sums[p.dim + c + e];
                    if (turn_of + 1 < Gr::kGroups) sums[c + e] = a, sums[p.dim + c + e] = b;
                    else out[c + e] = a, out[p.dim + c + e] = b;
                }
            }
        }
    }
}

// dweight, dbias: 32 columns a block, 32 threads a column over the partial rows.
template <typename T>
__global__ void __launch_bounds__(1024) norm_join_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const uint32_t which = blockIdx.y, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < p.dim)
        for (uint32_t i = g; i < p.parts; i += 32) s += p.part[((uint64_t)i * 2 + which) * p.dim + c];
    red[g][lane] = s;
    __syncthreads();
    s = red[lane][g];
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    const uint32_t col = blockIdx.x * 32 + g;
    T *out = static_cast<T *>(which ? p.dbias : p.dweight);
    if (lane == 0 && col < p.dim && out) out[col] = from_f<T>(s);
}

#define K2T_NORM_CUDA(call)                              \
    do {                                                 \
        cudaError_t e_ = (call);                         \
        if (e_ != cudaSuccess) {                         \
            g_last_cuda = (int)e_;                       \
            return K2T_ECUDA;                            \
        }                                                \
    } while (0)

constexpr uint32_t kNormBlocks = 152 * 8;   // blocks of a full GPU: eight of 256 threads an SM

uint32_t norm_parts(uint64_t n, int groups)
{
    return (uint32_t)std::min<uint64_t>((n + groups - 1) / groups, kNormBlocks);
}

template <typename T, int VEC, int TPR, int PER> int run_norm(NormParams &p, bool backward, cudaStream_t st)
{
    using Gr = Group<TPR>;
    const uint32_t blocks = norm_parts(p.n, Gr::kGroups);
    if (!backward) {
        if (!blocks) return K2T_OK;
        norm_fwd_kernel<T, VEC, TPR, PER><<<blocks, Gr::kThreads, 0, st>>>(p);
        K2T_NORM_CUDA(cudaGetLastError());
        return K2T_OK;
    }
    p.parts = blocks;
    if (blocks) {
        norm_bwd_kernel<T, VEC, TPR, PER><<<blocks, Gr::kThreads, Gr::kGroups > 1 ? 2 * p.dim * sizeof(float) : 0, st>>>(p);
        K2T_NORM_CUDA(cudaGetLastError());
    }
    norm_join_kernel<T><<<dim3((p.dim + 31) / 32, p.dbias ? 2 : 1), 1024, 0, st>>>(p);
    K2T_NORM_CUDA(cudaGetLastError());
    return K2T_OK;
}

// Threads a row: as few as hold it with one load each, up to a block, then
// more loads a thread.  Rows whose pitch is no multiple of 16 bytes (or whose
// tensors are not 16-byte aligned) move value by value.
template <typename T> int norm_dispatch(NormParams &p, bool vec, bool backward, cudaStream_t st)
{
    if (vec) {
        constexpr int V = 16 / sizeof(T);
        const uint32_t c = p.dim / V;
        if (c <= 32) return run_norm<T, V, 32, 1>(p, backward, st);
        if (c <= 64) return run_norm<T, V, 64, 1>(p, backward, st);
        if (c <= 128) return run_norm<T, V, 128, 1>(p, backward, st);
        if (c <= 256) return run_norm<T, V, 256, 1>(p, backward, st);
        if (c <= 512) return run_norm<T, V, 256, 2>(p, backward, st);
        if (c <= 1024) return run_norm<T, V, 512, 2>(p, backward, st);
        return run_norm<T, V, 512, 8>(p, backward, st);
    }
    if (p.dim <= 128) return run_norm<T, 1, 32, 4>(p, backward, st);
    if (p.dim <= 512) return run_norm<T, 1, 128, 4>(p, backward, st);
    if (p.dim <= 2048) return run_norm<T, 1, 256, 8>(p, backward, st);
    return run_norm<T, 1, 512, 32>(p, backward, st);
}

int check_norm(const k2t_norm *a)
{
    if (!a) return K2T_EINVAL;
    if (a->dtype > K2T_FP32) return K2T_EINVAL;
    if (a->dim == 0 || a->dim > K2T_NORM_MAX_DIM || a->n_rows > (1ull << 32)) return K2T_ERANGE;
    if (!(a->eps > 0.0f)) return K2T_EINVAL;
    return K2T_OK;
}

int dispatch(const k2t_norm *a, NormParams &p, bool backward, cudaStream_t st)
{
    uintptr_t all = 0;
    for (const void *q : {p.x, p.residual, p.z_in, p.dy, p.dz, (const void *)p.y, (const void *)p.z, (const void *)p.dx})
        all |= (uintptr_t)q;
    const uint32_t size = a->dtype == K2T_FP32 ? 4 : 2;
    if ((all | (uintptr_t)a->weight | (uintptr_t)a->bias | (uintptr_t)a->dweight | (uintptr_t)a->dbias) & (size - 1)) return K2T_EINVAL;
    const bool vec = !(all & 15) && (a->dim * size) % 16 == 0;
    p.dim = a->dim;
    p.n = a->n_rows;
    p.eps = a->eps;
    p.inv_dim = 1.0f / (float)a->dim;
    p.weight = a->weight;
    p.mean = a->mean;
    p.rstd = a->rstd;
    if (a->dtype == K2T_BF16) return norm_dispatch<__nv_bfloat16>(p, vec, backward, st);
    if (a->dtype == K2T_FP16) return norm_dispatch<__half>(p, vec, backward, st);
    return norm_dispatch<float>(p, vec, backward, st);
}

}  // namespace
}  // namespace k2t

using namespace k2t;

extern "C" {

uint64_t k2t_norm_work_bytes(const k2t_norm *a)
{
    if (check_norm(a)) return 0;
    return align_up((uint64_t)norm_parts(a->n_rows, 1) * 2 * a->dim * sizeof(float), 256);
}

int k2t_norm_forward(const k2t_norm *a, void *stream)
{
    int rc = check_norm(a);
    if (rc) return rc;
    if (!a->weight || (a->n_rows && (!a->x || !a->y || !a->mean || !a->rstd || (a->residual && !a->z)))) return K2T_EINVAL;
    if (a->residual && a->n_rows && a->y == a->z) return K2T_EINVAL;
    NormParams p{};
    p.x = a->x, p.residual = a->residual, p.bias = a->bias, p.y = a->y, p.z = a->residual ? a->z : nullptr;
    return dispatch(a, p, false, static_cast<cudaStream_t>(stream));
}

int k2t_norm_backward(const k2t_norm *a, void *work, uint64_t work_bytes, void *stream)
{
    int rc = check_norm(a);
    if (rc) return rc;
    if (!a->weight || !a->dweight || (a->n_rows && (!a->z || !a->dy || !a->dx || !a->mean || !a->rstd))) return K2T_EINVAL;
    if (a->n_rows && (!work || ((uintptr_t)work & 15u))) return K2T_EINVAL;
    if (work_bytes < k2t_norm_work_bytes(a)) return K2T_ENOMEM;
    NormParams p{};
    p.z_in = a->z, p.dy = a->dy, p.dz = a->dz, p.dx = a->dx, p.dweight = a->dweight, p.dbias = a->dbias;
    p.part = static_cast<float *>(work);
    return dispatch(a, p, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
