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
// the position (an fp32 product of position 2^20 and rate 1 is 0.06 off); fp32
// then holds it to 2^-26.
// In 16 bits sine and cosine are the special function unit's (2^-20 off in one
// turn, where results round to 2^-9 or 2^-12), in fp32 the library's.
//
// What bounds it: memory.  Squares, sums and rotations are fp32; each value is rounded once.
#pragma once

#include <type_traits>

#include "k2t_norm.cuh"

namespace k2t {

struct HeadParams {
    uint32_t heads, d, rotary, slots, lanes;     // slots: V pairs each; lanes share a head
    uint32_t reach;                              // the largest power of two below lanes, 0 for one lane
    uint32_t per, chunks;                        // heads of a unit; units of a row
    uint32_t blocks;                             // of a backward pass
    uint64_t n, units;                           // unit: `per` heads of a row
    float eps, inv_d;
    const void *x, *weight, *dy;
    const int32_t *positions;
    void *y, *dx;
    int64_t x_row, x_head, y_row, y_head, dy_row, dy_head, dx_row, dx_head;
    float *part;                                 // backward: [blocks][2][d], of which [0] is used
    uint64_t rate[K2T_HEAD_MAX_DIM / 2];
};

// V values at once, two an instruction: a b, a b + c.
__device__ __forceinline__ float2 two_fma(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)),
          "l"(*reinterpret_cast<unsigned long long *>(&c)));
    return d;
}
__device__ __forceinline__ float2 two_mul(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return d;
}
template <int V> struct Many {
    float2 v[(V + 1) / 2];           // V odd: the last one's second value stays 0
    __device__ __forceinline__ Many() {}
    __device__ __forceinline__ explicit Many(float x)
    {
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) v[i] = make_float2(x, 2 * i + 1 < V ? x : 0.0f);
    }
    __device__ __forceinline__ float get(int i) const { return i & 1 ? v[i / 2].y : v[i / 2].x; }
    __device__ __forceinline__ void set(int i, float x) { (i & 1 ? v[i / 2].y : v[i / 2].x) = x; }
    __device__ __forceinline__ Many operator*(const Many &o) const
    {
        Many r;
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) r.v[i] = two_mul(v[i], o.v[i]);
        return r;
    }
    __device__ __forceinline__ Many operator*(float o) const
    {
        Many r;
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) r.v[i] = two_mul(v[i], make_float2(o, o));
        return r;
    }
    __device__ __forceinline__ static Many fma(const Many &a, const Many &b, const Many &c)
    {
        Many r;
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) r.v[i] = two_fma(a.v[i], b.v[i], c.v[i]);
        return r;
    }
    // onto a sum of two
    __device__ __forceinline__ static void add_products(float2 &sum, const Many &a, const Many &b)
    {
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) sum = two_fma(a.v[i], b.v[i], sum);
    }
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
    // The pairs' first and second values.
    template <typename A> static __device__ __forceinline__ void split(Many<V> &a, Many<V> &b, const A &x, const A &y)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (PAIRED && V > 1) {
                a.set(i, to_f(2 * i < V ? x.v[2 * i % V] : y.v[2 * i % V]));
                b.set(i, to_f(2 * i < V ? x.v[(2 * i + 1) % V] : y.v[(2 * i + 1) % V]));
            } else {
                a.set(i, to_f(x.v[i])), b.set(i, to_f(y.v[i]));
            }
        }
        if (V & 1) a.v[V / 2].y = b.v[V / 2].y = 0.0f;
    }
    template <typename A> static __device__ __forceinline__ void join(A &x, A &y, const Many<V> &a, const Many<V> &b)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (PAIRED && V > 1) {
                (2 * i < V ? x : y).v[2 * i % V] = from_f<T>(a.get(i));
                (2 * i < V ? x : y).v[(2 * i + 1) % V] = from_f<T>(b.get(i));
            } else {
                x.v[i] = from_f<T>(a.get(i)), y.v[i] = from_f<T>(b.get(i));
            }
        }
    }
};

template <typename T> __device__ __forceinline__ void turn_by(float &c, float &s, uint64_t position, uint64_t rate)
{
    // -1/2 .. 1/2: the upper 32 bits of the 64 of the product
    const uint32_t at = (uint32_t)position * (uint32_t)(rate >> 32) + __umulhi((uint32_t)position, (uint32_t)rate) + (uint32_t)(position >> 32) * (uint32_t)rate;
    const float turn = (float)(int32_t)at * 0x1p-32f;
    if constexpr (std::is_same<T, float>::value) sincospif(2.0f * turn, &s, &c);
    else __sincosf(turn * 6.283185307179586f, &s, &c);
}

constexpr int kHeadThreads = 128;

// A thread's place: `lanes` neighbours of a warp share a head, as many heads as fit a warp; its last lanes may have none.
struct HeadLane {
    uint32_t lane, first, group, groups, mask;
    bool on;
    __device__ __forceinline__ explicit HeadLane(const HeadParams &p)
    {
        const uint32_t l = threadIdx.x & 31, per = 32 / p.lanes, g = l / p.lanes;
        first = g * p.lanes, lane = l - first, on = g < per;
        group = (threadIdx.x >> 5) * per + g, groups = kHeadThreads / 32 * per;
        mask = p.lanes == 32 ? ~0u : ((1u << p.lanes) - 1) << first;
    }
    // Sums of N values over the lanes of a head: with a power of two of them each ends with the sum, else the first, which
    // shares it.
    template <int N> __device__ __forceinline__ void sum(const HeadParams &p, float (&a)[N]) const
    {
        const bool even = (p.lanes & (p.lanes - 1)) == 0;
#pragma unroll
        for (uint32_t o = 16; o; o >>= 1) {
            if (o > p.reach) continue;
            if (even) {
#pragma unroll
                for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(mask, a[i], o);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float x = __shfl_down_sync(mask, a[i], o);
                    if (lane < o && lane + o < p.lanes) a[i] += x;
                }
            }
        }
        if (!even) {
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] = __shfl_sync(mask, a[i], first);
        }
    }
};

// The vectors of a thread's heads, one after another.  A unit is `per` heads of a row; a group of lanes takes units `stride`
// apart.  AHEAD: the thread's vectors of so many heads to come are on their way to places of its own in shared memory, which
// holds more loads in flight than registers do; 0: a head's own loads.
template <typename T, int V, int S, int N, int AHEAD> struct HeadStream {
    using Vec = HeadVec<T, V>;
    static constexpr int kPlace = Vec::kBytes * kHeadThreads, kSlot = N * kPlace, kBytes = AHEAD ? (AHEAD + 1) * kSlot : 0;
    const HeadParams &p;
    const T *from[N], *at[N];        // first values of the thread's two vectors of each tensor, of head 0 and of the next one
    int64_t row_step[N / 2], head_step[N / 2];
    uint64_t unit, stride;           // of the head that is asked for next
    uint32_t head, end, left;        // left: heads to ask for
    uint32_t place, to, take;        // this thread's places: where the next loads go, and where the next head's are
    bool on;
    __device__ __forceinline__ HeadStream(const HeadParams &p_, uint32_t base, uint64_t first, uint64_t stride_, bool on_)
        : p(p_), unit(first), stride(stride_), place(base + threadIdx.x * Vec::kBytes), on(on_)
    {
        to = place, take = threadIdx.x * Vec::kBytes;
    }
    // The heads of unit `unit`.  Loads run ahead only where a unit is a row: no division then.
    __device__ __forceinline__ static void heads(const HeadParams &p, uint64_t unit, uint64_t &row, uint32_t &head, uint32_t &end)
    {
        row = AHEAD ? unit : unit / p.chunks;
        head = AHEAD ? 0 : (uint32_t)(unit - row * p.chunks) * p.per;
        end = AHEAD ? p.heads : min(head + p.per, p.heads);
    }
    __device__ __forceinline__ void move()
    {
        uint64_t row;
        heads(p, unit, row, head, end);
#pragma unroll
        for (int i = 0; i < N; ++i) at[i] = from[i] + (int64_t)row * row_step[i / 2] + (int64_t)head * head_step[i / 2];
    }
    __device__ __forceinline__ void start()
    {
        if (unit < p.units) move();
        if constexpr (AHEAD > 0) {
            left = unit < p.units ? (uint32_t)((p.units - unit + stride - 1) / stride) * p.heads : 0;
#pragma unroll 1
            for (int i = 0; i < AHEAD; ++i) ask();
        }
    }
    __device__ __forceinline__ void next()
    {
        if (++head == end) {
            unit += stride;
            if (unit < p.units) move();
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) at[i] += head_step[i / 2];
        }
    }
    __device__ __forceinline__ void ask()
    {
        if (left) {
            --left;
            if (on) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if constexpr (Vec::kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * kPlace), "l"(at[i]) : "memory");
                    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + i * kPlace), "l"(at[i]), "n"(Vec::kBytes) : "memory");
                }
            }
            next();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        to = to == place + AHEAD * kSlot ? place : to + kSlot;
    }
    // The next head's vectors.
    __device__ __forceinline__ void get(Vec (&x)[N], const uint8_t *smem)
    {
        if constexpr (AHEAD > 0) {
            asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
#pragma unroll
            for (int i = 0; i < N; ++i) x[i].load(reinterpret_cast<const T *>(smem + take + i * kPlace));
            take = take == threadIdx.x * Vec::kBytes + AHEAD * kSlot ? threadIdx.x * Vec::kBytes : take + kSlot;
            ask();
        } else {
            if (on) {
#pragma unroll
                for (int i = 0; i < N; ++i) x[i].load(at[i]);
            }
            next();
        }
    }
};

// Shared memory of a kernel: the streams' places, then rates, then (backward) the groups' sums.
template <typename T, int V, int S, bool PAIRED> struct HeadThread {
    using Pairs = HeadPairs<T, V, PAIRED>;
    Many<V> wa[S], wb[S], c[S], s[S], ns[S];     // weights, cosines, sines and what is subtracted
    const uint64_t *rates;
    __device__ __forceinline__ void weights(const HeadParams &p, uint32_t lane)
    {
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const Pairs at(p, lane + k * p.lanes);
            HeadVec<T, V> x, y;
            wa[k] = wb[k] = c[k] = Many<V>(1.0f), s[k] = ns[k] = Many<V>(0.0f);
            if (p.weight && at.on) {
                x.load(static_cast<const T *>(p.weight) + at.lo);
                y.load(static_cast<const T *>(p.weight) + at.hi);
                Pairs::split(wa[k], wb[k], x, y);
            }
        }
    }
    __device__ __forceinline__ void angles(const HeadParams &p, uint32_t lane, uint64_t row)
    {
        if (!p.rotary) return;
        const uint64_t pos = p.positions ? (uint64_t)(int64_t)__ldg(p.positions + row) : row;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const Pairs at(p, lane + k * p.lanes);
            if (!at.on || !at.turns) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float x, y;
                turn_by<T>(x, y, pos, rates[at.angle + i]);
                c[k].set(i, x), s[k].set(i, y), ns[k].set(i, -y);
            }
        }
    }
};

__device__ __forceinline__ const uint64_t *head_rates(const HeadParams &p, uint8_t *at)
{
    uint64_t *r = reinterpret_cast<uint64_t *>(at);
    for (uint32_t i = threadIdx.x; i < p.rotary / 2; i += kHeadThreads) r[i] = p.rate[i];
    __syncthreads();
    return r;
}

template <typename T, int V, int S, int AHEAD, bool PAIRED>
__global__ void __launch_bounds__(kHeadThreads, V * S <= 4 ? 6 : 5) head_norm_fwd_kernel(const __grid_constant__ HeadParams p)
{
    using Thread = HeadThread<T, V, S, PAIRED>;
    using Pairs = typename Thread::Pairs;
    using Stream = HeadStream<T, V, S, 2 * S, AHEAD>;
    extern __shared__ __align__(16) uint8_t head_smem[];
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(head_smem);
    const HeadLane me(p);
    Thread t;
    t.rates = head_rates(p, head_smem + Stream::kBytes);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!me.on) return;
    t.weights(p, me.lane);
    const uint64_t stride = (uint64_t)gridDim.x * me.groups;
    uint64_t unit = (uint64_t)blockIdx.x * me.groups + me.group;
    Stream in(p, base, unit, stride, S > 1 || me.lane < p.slots);
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const Pairs at(p, me.lane + k * p.lanes);
        in.from[2 * k] = static_cast<const T *>(p.x) + (at.on ? at.lo : 0), in.from[2 * k + 1] = static_cast<const T *>(p.x) + (at.on ? at.hi : 0);
        in.row_step[k] = p.x_row, in.head_step[k] = p.x_head;
    }
    in.start();
    for (; unit < p.units; unit += stride) {
        uint64_t row;
        uint32_t h0, h1;
        Stream::heads(p, unit, row, h0, h1);
        t.angles(p, me.lane, row);
        T *y = static_cast<T *>(p.y) + (int64_t)row * p.y_row + (int64_t)h0 * p.y_head;
        for (uint32_t h = h0; h < h1; ++h) {
            HeadVec<T, V> x[2 * S];
            in.get(x, head_smem);
            Many<V> a[S], b[S];
            float2 squares = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < S; ++k) {
                if (me.lane + k * p.lanes < p.slots) {
                    Pairs::split(a[k], b[k], x[2 * k], x[2 * k + 1]);
                    Many<V>::add_products(squares, a[k], a[k]);
                    Many<V>::add_products(squares, b[k], b[k]);
                }
            }
            float sum[1] = {squares.x + squares.y};
            me.sum(p, sum);
            const float r = rsqrtf(sum[0] * p.inv_d + p.eps);
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const Pairs at(p, me.lane + k * p.lanes);
                if (!at.on) continue;
                const Many<V> u = a[k] * r * t.wa[k], v = b[k] * r * t.wb[k];
                if (p.rotary) {
                    a[k] = Many<V>::fma(u, t.c[k], v * t.ns[k]);
                    b[k] = Many<V>::fma(v, t.c[k], u * t.s[k]);
                } else {
                    a[k] = u, b[k] = v;
                }
                Pairs::join(x[2 * k], x[2 * k + 1], a[k], b[k]);
                x[2 * k].store(y + at.lo);
                x[2 * k + 1].store(y + at.hi);
            }
            y += p.y_head;
        }
    }
}

template <typename T, int V, int S, int AHEAD, bool PAIRED>
__global__ void __launch_bounds__(kHeadThreads, V * S <= 4 ? 4 : 3) head_norm_bwd_kernel(const __grid_constant__ HeadParams p)
{
    using Thread = HeadThread<T, V, S, PAIRED>;
    using Pairs = typename Thread::Pairs;
    using Stream = HeadStream<T, V, S, 4 * S, AHEAD>;
    extern __shared__ __align__(16) uint8_t head_smem[];
    float *sums = reinterpret_cast<float *>(head_smem + Stream::kBytes + sizeof(p.rate));       // [groups][d]
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(head_smem);
    const HeadLane me(p);
    Thread t;
    t.rates = head_rates(p, head_smem + Stream::kBytes);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Many<V> da[S], db[S];
#pragma unroll
    for (int k = 0; k < S; ++k) da[k] = db[k] = Many<V>(0.0f);
    if (me.on) {
        t.weights(p, me.lane);
        const uint64_t stride = (uint64_t)gridDim.x * me.groups;
        uint64_t unit = (uint64_t)blockIdx.x * me.groups + me.group;
        Stream in(p, base, unit, stride, S > 1 || me.lane < p.slots);
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const Pairs at(p, me.lane + k * p.lanes);
            const uint32_t lo = at.on ? at.lo : 0, hi = at.on ? at.hi : 0;
            in.from[4 * k] = static_cast<const T *>(p.x) + lo, in.from[4 * k + 1] = static_cast<const T *>(p.x) + hi;
            in.from[4 * k + 2] = static_cast<const T *>(p.dy) + lo, in.from[4 * k + 3] = static_cast<const T *>(p.dy) + hi;
            in.row_step[2 * k] = p.x_row, in.head_step[2 * k] = p.x_head, in.row_step[2 * k + 1] = p.dy_row, in.head_step[2 * k + 1] = p.dy_head;
        }
        in.start();
        for (; unit < p.units; unit += stride) {
            uint64_t row;
            uint32_t h0, h1;
            Stream::heads(p, unit, row, h0, h1);
            t.angles(p, me.lane, row);
            T *dx = static_cast<T *>(p.dx) + (int64_t)row * p.dx_row + (int64_t)h0 * p.dx_head;
            for (uint32_t h = h0; h < h1; ++h) {
                HeadVec<T, V> x[4 * S];
                in.get(x, head_smem);
                Many<V> a[S], b[S], ga[S], gb[S], pa[S], pb[S];
                float2 squares = make_float2(0.0f, 0.0f), dots = squares;
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    if (me.lane + k * p.lanes < p.slots) {
                        Pairs::split(a[k], b[k], x[4 * k], x[4 * k + 1]);
                        Pairs::split(ga[k], gb[k], x[4 * k + 2], x[4 * k + 3]);
                        if (p.rotary) {
                            const Many<V> g = ga[k];
                            ga[k] = Many<V>::fma(g, t.c[k], gb[k] * t.s[k]);
                            gb[k] = Many<V>::fma(gb[k], t.c[k], g * t.ns[k]);
                        }
                        Many<V>::add_products(squares, a[k], a[k]);
                        Many<V>::add_products(squares, b[k], b[k]);
                        pa[k] = ga[k] * a[k], pb[k] = gb[k] * b[k];
                        Many<V>::add_products(dots, pa[k], t.wa[k]);
                        Many<V>::add_products(dots, pb[k], t.wb[k]);
                    }
                }
                float sum[2] = {squares.x + squares.y, dots.x + dots.y};
                me.sum(p, sum);
                const float r = rsqrtf(sum[0] * p.inv_d + p.eps), m = sum[1] * p.inv_d * r * r;
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    const Pairs at(p, me.lane + k * p.lanes);
                    if (!at.on) continue;
                    da[k] = Many<V>::fma(pa[k], Many<V>(r), da[k]);
                    db[k] = Many<V>::fma(pb[k], Many<V>(r), db[k]);
                    a[k] = Many<V>::fma(ga[k], t.wa[k] * r, a[k] * (-m * r));
                    b[k] = Many<V>::fma(gb[k], t.wb[k] * r, b[k] * (-m * r));
                    Pairs::join(x[4 * k], x[4 * k + 1], a[k], b[k]);
                    x[4 * k].store(dx + at.lo);
                    x[4 * k + 1].store(dx + at.hi);
                }
                dx += p.dx_head;
            }
        }
    }
    if (!p.part) return;
    // the groups' sums, in the order of the groups
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const Pairs at(p, me.lane + k * p.lanes);
        if (!at.on || !me.on) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sums[me.group * p.d + (PAIRED ? at.lo + 2 * i : at.lo + i)] = da[k].get(i);
            sums[me.group * p.d + (PAIRED ? at.lo + 2 * i + 1 : at.hi + i)] = db[k].get(i);
        }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < p.d; i += kHeadThreads) {
        float sum = 0.0f;
        for (uint32_t g = 0; g < me.groups; ++g) sum += sums[g * p.d + i];
        p.part[(uint64_t)blockIdx.x * 2 * p.d + i] = sum;
    }
}

}  // namespace k2t
