// k2t_head_norm.cuh -- RMS norm of each head of queries or keys with the
// rotation by position in the same pass, forward and backward.
//
// A head's values are taken as d / 2 pairs: first those that turn together
// (value i with i + rotary / 2, or neighbours), then the others, which turn by
// nothing.  A thread holds V pairs as two vectors, so that the rotation stays
// inside it and only the sums over the head (of squares; backward also of
// w g x) cross its group of lanes.
//
//   y = R(p) (w x r),  r = 1 / sqrt(mean x^2 + eps)
//   g = R(-p) dy,  dx = r (w g - x r^2 mean(w g x)),  dw = sum over rows and heads of g x r
//
// An angle is position x rate in turns, and rates are 64-bit fractions of a
// turn: the product modulo 2^64 is the fraction of a turn exactly, however far
// the position (an fp32 product of position 2^20 and rate 1 is 0.06 off).
// In 16 bits sine and cosine are the special function unit's (2^-20 off in one
// turn, where results round to 2^-9 or 2^-12), in fp32 the library's.
//
// What bounds it: memory.  Squares, sums and rotations are fp32; each value is rounded once.
#pragma once

#include <type_traits>

#include "k2t_norm.cuh"

namespace k2t {

struct HeadParams {
    uint32_t heads, d, rotary, slots, lanes;     // slots: V pairs each; lanes (a power of two) share a head
    uint32_t chunks;                             // of the heads of a row
    uint64_t n, units;                           // unit: a chunk of a row's heads
    float eps, inv_d;
    const void *x, *weight, *dy;
    const int32_t *positions;
    void *y, *dx;
    int64_t x_row, x_head, y_row, y_head, dy_row, dy_head, dx_row, dx_head;
    float *part;                                 // backward: [blocks][2][d], of which [0] is used
    uint64_t rate[K2T_HEAD_MAX_DIM / 2];
};

template <typename T, int V> struct HeadVec {
    static constexpr int kBytes = V * (int)sizeof(T);
    using Raw = std::conditional_t<kBytes == 16, uint4, std::conditional_t<kBytes == 8, uint2, std::conditional_t<kBytes == 4, uint32_t, uint16_t>>>;
    union { Raw raw; T v[V]; };
    __device__ __forceinline__ HeadVec() {}
    __device__ __forceinline__ void load(const T *p) { raw = *reinterpret_cast<const Raw *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Raw *>(p) = raw; }
};

// The V pairs of a thread: where its two vectors lie in a head, and which value of a pair an element is.
template <typename T, int V, bool PAIRED> struct HeadPairs {
    uint32_t lo, hi, angle;          // first values of both vectors; first rate
    bool on, turns;
    __device__ __forceinline__ HeadPairs(const HeadParams &p, uint32_t slot)
    {
        const uint32_t half = p.rotary / 2, j = slot * V;
        on = slot < p.slots;
        turns = j < half;
        angle = j;
        if (PAIRED) {
            lo = 2 * j, hi = lo + V;
        } else if (turns) {
            lo = j, hi = half + j;
        } else {
            lo = p.rotary + j - half, hi = lo + (p.d - p.rotary) / 2;
        }
    }
    // element i of the pairs' first and second values
    template <typename A> static __device__ __forceinline__ void split(float (&a)[V], float (&b)[V], const A &x, const A &y)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (PAIRED && V == 1) {
                a[i] = to_f(x.v[0]), b[i] = to_f(y.v[0]);
            } else if constexpr (PAIRED) {
                a[i] = to_f(2 * i < V ? x.v[2 * i % V] : y.v[2 * i % V]);
                b[i] = to_f(2 * i < V ? x.v[(2 * i + 1) % V] : y.v[(2 * i + 1) % V]);
            } else {
                a[i] = to_f(x.v[i]), b[i] = to_f(y.v[i]);
            }
        }
    }
    template <typename A> static __device__ __forceinline__ void join(A &x, A &y, const float (&a)[V], const float (&b)[V])
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (PAIRED && V > 1) {
                (2 * i < V ? x : y).v[2 * i % V] = from_f<T>(a[i]);
                (2 * i < V ? x : y).v[(2 * i + 1) % V] = from_f<T>(b[i]);
            } else {
                x.v[i] = from_f<T>(a[i]), y.v[i] = from_f<T>(b[i]);
            }
        }
    }
};

template <typename T> __device__ __forceinline__ void turn_by(float &c, float &s, uint64_t position, uint64_t rate)
{
    const float turn = (float)(int32_t)(uint32_t)((position * rate) >> 32) * 0x1p-32f;     // -1/2 .. 1/2
    if constexpr (std::is_same<T, float>::value) sincospif(2.0f * turn, &s, &c);
    else __sincosf(turn * 6.283185307179586f, &s, &c);
}

__device__ __forceinline__ float head_sum(float a, uint32_t lanes, uint32_t mask)
{
    for (uint32_t x = lanes / 2; x; x >>= 1) a += __shfl_xor_sync(mask, a, x);
    return a;
}

constexpr int kHeadThreads = 256;

// S slots a lane, HC heads a unit.
template <typename T, int V, int S, int HC, bool PAIRED>
__global__ void __launch_bounds__(kHeadThreads) head_norm_fwd_kernel(const __grid_constant__ HeadParams p)
{
    using Pairs = HeadPairs<T, V, PAIRED>;
    const uint32_t L = p.lanes, lane = threadIdx.x & (L - 1), group = threadIdx.x / L, groups = kHeadThreads / L;
    const uint32_t mask = L == 32 ? ~0u : ((1u << L) - 1) << (threadIdx.x & 31 & ~(L - 1));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float wa[S][V], wb[S][V];
    uint64_t rate[S][V];
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const Pairs at(p, lane + k * L);
        HeadVec<T, V> x, y;
#pragma unroll
        for (int i = 0; i < V; ++i) wa[k][i] = wb[k][i] = 1.0f, rate[k][i] = at.on && at.turns ? p.rate[at.angle + i] : 0;
        if (p.weight && at.on) {
            x.load(static_cast<const T *>(p.weight) + at.lo);
            y.load(static_cast<const T *>(p.weight) + at.hi);
            Pairs::split(wa[k], wb[k], x, y);
        }
    }
    for (uint64_t u = (uint64_t)blockIdx.x * groups + group; u < p.units; u += (uint64_t)gridDim.x * groups) {
        const uint64_t row = u / p.chunks;
        const uint32_t h0 = (uint32_t)(u - row * p.chunks) * HC, hn = min((uint32_t)HC, p.heads - h0);
        const T *x = static_cast<const T *>(p.x) + (int64_t)row * p.x_row + (int64_t)h0 * p.x_head;
        T *y = static_cast<T *>(p.y) + (int64_t)row * p.y_row + (int64_t)h0 * p.y_head;
        HeadVec<T, V> lo[HC][S], hi[HC][S];
#pragma unroll
        for (int h = 0; h < HC; ++h)
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const Pairs at(p, lane + k * L);
                if (h < hn && at.on) {
                    lo[h][k].load(x + h * p.x_head + at.lo);
                    hi[h][k].load(x + h * p.x_head + at.hi);
                }
            }
        float c[S][V], s[S][V];
        if (p.rotary) {
            const uint64_t pos = p.positions ? (uint64_t)(int64_t)__ldg(p.positions + row) : row;
#pragma unroll
            for (int k = 0; k < S; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) turn_by<T>(c[k][i], s[k][i], pos, rate[k][i]);
        }
#pragma unroll
        for (int h = 0; h < HC; ++h) {
            if (h >= hn) break;
            float a[S][V], b[S][V], sum = 0.0f;
#pragma unroll
            for (int k = 0; k < S; ++k) {
                if (lane + k * L < p.slots) {
                    Pairs::split(a[k], b[k], lo[h][k], hi[h][k]);
#pragma unroll
                    for (int i = 0; i < V; ++i) sum = fmaf(a[k][i], a[k][i], fmaf(b[k][i], b[k][i], sum));
                }
            }
            const float r = rsqrtf(head_sum(sum, L, mask) * p.inv_d + p.eps);
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const Pairs at(p, lane + k * L);
                if (!at.on) continue;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float u0 = a[k][i] * r * wa[k][i], v0 = b[k][i] * r * wb[k][i];
                    a[k][i] = u0, b[k][i] = v0;
                    if (p.rotary) a[k][i] = u0 * c[k][i] - v0 * s[k][i], b[k][i] = v0 * c[k][i] + u0 * s[k][i];
                }
                HeadVec<T, V> o, q;
                Pairs::join(o, q, a[k], b[k]);
                o.store(y + h * p.y_head + at.lo);
                q.store(y + h * p.y_head + at.hi);
            }
        }
    }
}

template <typename T, int V, int S, int HC, bool PAIRED>
__global__ void __launch_bounds__(kHeadThreads) head_norm_bwd_kernel(const __grid_constant__ HeadParams p)
{
    using Pairs = HeadPairs<T, V, PAIRED>;
    extern __shared__ float sums[];              // [groups][d]
    const uint32_t L = p.lanes, lane = threadIdx.x & (L - 1), group = threadIdx.x / L, groups = kHeadThreads / L;
    const uint32_t mask = L == 32 ? ~0u : ((1u << L) - 1) << (threadIdx.x & 31 & ~(L - 1));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float wa[S][V], wb[S][V], da[S][V], db[S][V];
    uint64_t rate[S][V];
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const Pairs at(p, lane + k * L);
        HeadVec<T, V> x, y;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            wa[k][i] = wb[k][i] = 1.0f, rate[k][i] = at.on && at.turns ? p.rate[at.angle + i] : 0;
            da[k][i] = db[k][i] = 0.0f;
        }
        if (p.weight && at.on) {
            x.load(static_cast<const T *>(p.weight) + at.lo);
            y.load(static_cast<const T *>(p.weight) + at.hi);
            Pairs::split(wa[k], wb[k], x, y);
        }
    }
    for (uint64_t u = (uint64_t)blockIdx.x * groups + group; u < p.units; u += (uint64_t)gridDim.x * groups) {
        const uint64_t row = u / p.chunks;
        const uint32_t h0 = (uint32_t)(u - row * p.chunks) * HC, hn = min((uint32_t)HC, p.heads - h0);
        const T *x = static_cast<const T *>(p.x) + (int64_t)row * p.x_row + (int64_t)h0 * p.x_head;
        const T *dy = static_cast<const T *>(p.dy) + (int64_t)row * p.dy_row + (int64_t)h0 * p.dy_head;
        T *dx = static_cast<T *>(p.dx) + (int64_t)row * p.dx_row + (int64_t)h0 * p.dx_head;
        HeadVec<T, V> lo[HC][S], hi[HC][S], glo[HC][S], ghi[HC][S];
#pragma unroll
        for (int h = 0; h < HC; ++h)
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const Pairs at(p, lane + k * L);
                if (h < hn && at.on) {
                    lo[h][k].load(x + h * p.x_head + at.lo);
                    hi[h][k].load(x + h * p.x_head + at.hi);
                    glo[h][k].load(dy + h * p.dy_head + at.lo);
                    ghi[h][k].load(dy + h * p.dy_head + at.hi);
                }
            }
        float c[S][V], s[S][V];
        if (p.rotary) {
            const uint64_t pos = p.positions ? (uint64_t)(int64_t)__ldg(p.positions + row) : row;
#pragma unroll
            for (int k = 0; k < S; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) turn_by<T>(c[k][i], s[k][i], pos, rate[k][i]);
        }
#pragma unroll
        for (int h = 0; h < HC; ++h) {
            if (h >= hn) break;
            float a[S][V], b[S][V], ga[S][V], gb[S][V], sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int k = 0; k < S; ++k) {
                if (lane + k * L < p.slots) {
                    Pairs::split(a[k], b[k], lo[h][k], hi[h][k]);
                    Pairs::split(ga[k], gb[k], glo[h][k], ghi[h][k]);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float g = ga[k][i], f = gb[k][i];
                        if (p.rotary) ga[k][i] = g * c[k][i] + f * s[k][i], gb[k][i] = f * c[k][i] - g * s[k][i];
                        sum = fmaf(a[k][i], a[k][i], fmaf(b[k][i], b[k][i], sum));
                        dot = fmaf(ga[k][i] * wa[k][i], a[k][i], fmaf(gb[k][i] * wb[k][i], b[k][i], dot));
                    }
                }
            }
            for (uint32_t o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(mask, sum, o), dot += __shfl_xor_sync(mask, dot, o);
            const float r = rsqrtf(sum * p.inv_d + p.eps), m = dot * p.inv_d * r * r;
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const Pairs at(p, lane + k * L);
                if (!at.on) continue;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    da[k][i] = fmaf(ga[k][i], a[k][i] * r, da[k][i]);
                    db[k][i] = fmaf(gb[k][i], b[k][i] * r, db[k][i]);
                    a[k][i] = r * (ga[k][i] * wa[k][i] - a[k][i] * m);
                    b[k][i] = r * (gb[k][i] * wb[k][i] - b[k][i] * m);
                }
                HeadVec<T, V> o, q;
                Pairs::join(o, q, a[k], b[k]);
                o.store(dx + h * p.dx_head + at.lo);
                q.store(dx + h * p.dx_head + at.hi);
            }
        }
    }
    if (!p.part) return;
    // the groups' sums, in the order of the groups
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const Pairs at(p, lane + k * L);
        if (!at.on) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sums[group * p.d + (PAIRED ? at.lo + 2 * i : at.lo + i)] = da[k][i];
            sums[group * p.d + (PAIRED ? at.lo + 2 * i + 1 : at.hi + i)] = db[k][i];
        }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < p.d; i += kHeadThreads) {
        float sum = 0.0f;
        for (uint32_t g = 0; g < groups; ++g) sum += sums[g * p.d + i];
        p.part[(uint64_t)blockIdx.x * 2 * p.d + i] = sum;
    }
}

}  // namespace k2t
