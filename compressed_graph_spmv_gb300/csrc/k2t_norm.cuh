// k2t_norm.cuh -- what the layer norm's two ways of moving rows share.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "k2t_internal.h"

namespace k2t {

extern thread_local int g_last_cuda;

struct NormParams {
    uint32_t dim;
    uint64_t n;
    float eps, inv_dim;
    const void *x, *residual, *weight, *bias, *z_in, *dy, *dz;
    void *y, *z, *dx, *dweight, *dbias;
    float *mean, *rstd, *part;    // backward: no mean and rstd, form them
    uint32_t parts;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Threads of a block: groups of TPR, each with a row of its own.
template <int TPR> struct Group {
    static constexpr int kThreads = TPR < 256 ? 256 : TPR;
    static constexpr int kGroups = kThreads / TPR;
    static constexpr int kWarps = TPR < 32 ? 1 : TPR / 32;
};

// The lanes of this thread's group (several groups share a warp and may end at different rows).
template <int TPR> __device__ __forceinline__ uint32_t group_lanes()
{
    return TPR >= 32 ? ~0u : ((1u << (TPR & 31)) - 1) << (threadIdx.x & 31 & ~(TPR - 1));
}

// Sums of a and b over the TPR threads of a group.  buf: two alternating
// buffers, so that one barrier a call is enough.
template <int TPR>
__device__ __forceinline__ void group_sum(float &a, float &b, float2 *buf, int group, int &turn)
{
    const uint32_t lanes = group_lanes<TPR>();
#pragma unroll
    for (int x = TPR < 32 ? TPR / 2 : 16; x; x >>= 1) {
        a += __shfl_xor_sync(lanes, a, x);
        b += __shfl_xor_sync(lanes, b, x);
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

// Statistics of a row of values z formed beside the sums of a = w dy, with one barrier a row: each warp (or group, if that
// is no more) takes its own values' mean m_w first, sums squares and products around it, and the warps' sums are joined.
// With n_w values of a warp, sum (z - m)^2 = sum_w (squares_w + n_w (m_w - m)^2) and sum a (z - m) = sum_w (az_w +
// (m_w - m) a_w): every difference is small against what it is taken of.
struct RowSums { float mean, squares, a, az; };
template <int TPR> struct WarpJoin {
    static constexpr bool kMoves = true;      // join changes the mean
    static constexpr int W = Group<TPR>::kWarps;
    struct Shared { float4 sums[2][Group<TPR>::kGroups][W]; float count[Group<TPR>::kGroups][W]; };
    Shared *sh;
    int group, turn;
    float inv;                          // 1 / this warp's values
    // count: values of this thread; the same of every row
    __device__ __forceinline__ WarpJoin(Shared *shared, int group_, float count, uint32_t dim) : sh(shared), group(group_), turn(0)
    {
        float none = 0.0f;
        if (TPR > 32) add(count, none);
        else count = (float)dim;
        inv = count > 0.0f ? 1.0f / count : 0.0f;
        if (TPR > 32 && (threadIdx.x & 31) == 0) sh->count[group][threadIdx.x % TPR >> 5] = count;   // read behind a row's barrier
    }
    __device__ __forceinline__ static void add(float &a, float &b)
    {
        const uint32_t lanes = group_lanes<TPR>();
#pragma unroll
        for (int x = TPR < 32 ? TPR / 2 : 16; x; x >>= 1) {
            a += __shfl_xor_sync(lanes, a, x);
            b += __shfl_xor_sync(lanes, b, x);
        }
    }
    __device__ __forceinline__ RowSums join(RowSums r, float inv_dim)
    {
        if constexpr (TPR > 32) {
            float4 *at = sh->sums[turn][group];
            if ((threadIdx.x & 31) == 0) at[threadIdx.x % TPR >> 5] = make_float4(r.mean, r.squares, r.a, r.az);
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
            // lane i has warp i mod W's sums
            const int i = threadIdx.x & (W - 1);
            const float4 v = at[i];
            const float n = sh->count[group][i];
            r.mean = v.x * (n * inv_dim);
            r.a = v.z;
#pragma unroll
            for (int x = W / 2; x; x >>= 1) {
                r.mean += __shfl_xor_sync(~0u, r.mean, x);
                r.a += __shfl_xor_sync(~0u, r.a, x);
            }
            const float d = v.x - r.mean;
            r.squares = fmaf(n * d, d, v.y);
            r.az = fmaf(d, v.z, v.w);
#pragma unroll
            for (int x = W / 2; x; x >>= 1) {
                r.squares += __shfl_xor_sync(~0u, r.squares, x);
                r.az += __shfl_xor_sync(~0u, r.az, x);
            }
            turn ^= 1;
        }
        return r;
    }
};

// One value's sum.
template <int TPR> __device__ __forceinline__ float group_sum1(float a, float2 *buf, int group, int &turn)
{
    if constexpr (TPR <= 32) {
        const uint32_t lanes = group_lanes<TPR>();
#pragma unroll
        for (int x = TPR / 2; x; x >>= 1) a += __shfl_xor_sync(lanes, a, x);
        return a;
    } else {
        float b = 0.0f;
        group_sum<TPR>(a, b, buf, group, turn);
        return a;
    }
}

// The same with the whole group's sums at once: two barriers a row, fewer instructions.
template <int TPR> struct GroupJoin {
    static constexpr bool kMoves = false;
    using Shared = float2[2 * Group<TPR>::kGroups * Group<TPR>::kWarps];
    float2 *buf;
    int group, turn;
    float inv;
    __device__ __forceinline__ GroupJoin(Shared *shared, int group_, float, uint32_t dim) : buf(*shared), group(group_), turn(0), inv(1.0f / (float)dim) {}
    __device__ __forceinline__ void add(float &a, float &b) { group_sum<TPR>(a, b, buf, group, turn); }
    __device__ __forceinline__ RowSums join(RowSums r, float) { return r; }
};
// A kernel that reads its statistics.
template <int TPR> struct NoJoin {
    using Shared = float2[2 * Group<TPR>::kGroups * Group<TPR>::kWarps];
    template <typename... A> __device__ __forceinline__ NoJoin(const A &...) {}
};

// dweight, dbias: 8 columns (one 32-byte sector) a block, 128 threads a column over the partial rows, so that few loads
// follow one another.
template <typename T>
__global__ void __launch_bounds__(1024) norm_join_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float red[32][9];
    const int col = threadIdx.x & 7, g = threadIdx.x >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t which = blockIdx.y, c = blockIdx.x * 8 + col;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.0f;
    if (c < p.dim) {
#pragma unroll 4
        for (uint32_t i = g; i < p.parts; i += 128) s += p.part[((uint64_t)i * 2 + which) * p.dim + c];
    }
    s += __shfl_xor_sync(~0u, s, 8);
    s += __shfl_xor_sync(~0u, s, 16);
    if (lane < 8) red[warp][lane] = s;
    __syncthreads();
    if (warp < 8) {
        s = red[lane][warp];
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
        const uint32_t at = blockIdx.x * 8 + warp;
        T *out = static_cast<T *>(which ? p.dbias : p.dweight);
        if (lane == 0 && at < p.dim && out) out[at] = from_f<T>(s);
    }
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

inline uint32_t norm_parts(uint64_t n, int groups)
{
    return (uint32_t)std::min<uint64_t>((n + groups - 1) / groups, kNormBlocks);
}

// The dynamic shared memory a kernel may have is a setting of the kernel on a device, which calls of every width and every
// host thread share: raised once, to all that its static shared memory leaves of the 227 KB.
template <auto kernel> int norm_shared()
{
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    K2T_NORM_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && set.load() >> dev & 1) return K2T_OK;
    cudaFuncAttributes a{};
    K2T_NORM_CUDA(cudaFuncGetAttributes(&a, kernel));
    K2T_NORM_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448 - (int)a.sharedSizeBytes));
    if (dev < 64) set.fetch_or(1ull << dev);
    return K2T_OK;
}

// Backward blocks: as many as the GPU runs at once, and no more than `blocks`; each writes a partial row of the
// weight's gradient, so that more of them cost more than they even out (445 us against 458 us with twice as many).
template <typename K> int norm_resident(K kernel, uint32_t &blocks, int threads, size_t smem)
{
    int per_sm = 0;
    K2T_NORM_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem));
    blocks = std::min<uint32_t>(blocks, 152u * std::max(per_sm, 1));
    return K2T_OK;
}

template <typename K, typename... A> int norm_launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args)
{
    // programmatic launch: blocks may be set up while the kernel before them on the stream still runs, and wait for its
    // end before they touch global memory
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
    K2T_NORM_CUDA(cudaLaunchKernelEx(&c, kernel, args...));
    return K2T_OK;
}

// rows that are not whole 16-byte pieces (k2t_norm_ragged.cu)
int norm_ragged(NormParams &p, uint32_t dtype, bool backward, cudaStream_t st);

}  // namespace k2t
