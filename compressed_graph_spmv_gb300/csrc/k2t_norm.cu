// k2t_norm.cu -- layer norm of node states with the residual sum before it,
// forward and backward.
//
// Both passes read each tensor once: a row lies in the registers of TPR
// threads (VEC values a load, PER loads a thread) while its statistics are
// formed, the mean first and then the squares around it, so that no
// cancellation of large sums arises.  Bound by memory: the passes are loads,
// two reductions of a few shuffles, and stores (2^18 x 1024 bf16 with the
// residual: 314 us forward and 327 backward, 101 and 97% of the copy rate;
// 2^17 x 2048 without it 177 and 294, 90 and 81%, where a row's reductions
// are not hidden by a third and fourth tensor).  Blocks stay for many rows,
// keep the weight in registers, and in the backward pass sum their rows'
// terms of dweight and dbias there; each block writes one partial row, and
// norm_join_kernel adds those in a fixed order.
#include "k2t_norm.cuh"

#include <type_traits>

namespace k2t {
namespace {

// VEC values, which fill 16 bytes, or a single one.
template <typename T, int VEC> struct alignas(VEC * sizeof(T)) Pack { T v[VEC]; };

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load_once(const T *p)
{
    Pack<T, VEC> r;
    if constexpr (VEC == 1) r.v[0] = *p;
    else *reinterpret_cast<uint4 *>(&r) = __ldcs(reinterpret_cast<const uint4 *>(p));
    return r;
}
template <typename T, int VEC> __device__ __forceinline__ void store(T *p, const Pack<T, VEC> &r)
{
    if constexpr (VEC == 1) *p = r.v[0];
    else *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&r);
}

// Value e of an array of pairs (e is known when compiling), and operations on pairs.
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> zero_pack()
{
    Pack<T, VEC> r;
#pragma unroll
    for (int e = 0; e < VEC; ++e) r.v[e] = from_f<T>(0.0f);
    return r;
}
template <typename T, int VEC> __device__ __forceinline__ float2 pair_of(const Pack<T, VEC> *p, int e)
{
    if constexpr (sizeof(T) == 2 && VEC > 1) {
        const uint32_t word = reinterpret_cast<const uint32_t *>(p[2 * e / VEC].v)[e % (VEC / 2)];
        if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2 *>(&word));
        else return make_float2(__uint_as_float(word << 16), __uint_as_float(word & 0xffff0000u));
    } else {
        return make_float2(to_f(p[2 * e / VEC].v[2 * e % VEC]), to_f(p[(2 * e + 1) / VEC].v[(2 * e + 1) % VEC]));
    }
}
template <typename T, int VEC> __device__ __forceinline__ void set_pair(Pack<T, VEC> *p, int e, float2 v)
{
    if constexpr (sizeof(T) == 2 && VEC > 1) {
        uint32_t &word = reinterpret_cast<uint32_t *>(p[2 * e / VEC].v)[e % (VEC / 2)];
        if constexpr (std::is_same_v<T, __half>) *reinterpret_cast<__half2 *>(&word) = __float22half2_rn(v);
        else *reinterpret_cast<__nv_bfloat162 *>(&word) = __float22bfloat162_rn(v);
    } else {
        p[2 * e / VEC].v[2 * e % VEC] = from_f<T>(v.x);
        p[(2 * e + 1) / VEC].v[(2 * e + 1) % VEC] = from_f<T>(v.y);
    }
}
__device__ __forceinline__ float &half_of(float2 *v, int e) { return e & 1 ? v[e >> 1].y : v[e >> 1].x; }
__device__ __forceinline__ unsigned long long bits(const float2 &v) { return *reinterpret_cast<const unsigned long long *>(&v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(*reinterpret_cast<unsigned long long *>(&d)) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(*reinterpret_cast<unsigned long long *>(&d)) : "l"(bits(a)), "l"(bits(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(*reinterpret_cast<unsigned long long *>(&d)) : "l"(bits(a)), "l"(bits(b)));
    return d;
}

// The loads of a row, either when the row's turn comes (AHEAD 0) or AHEAD rows earlier into shared memory, each thread
// its own pieces: nothing waits on another thread, and the loads in flight (AHEAD rows of every thread) are not bounded
// by registers.  Rows of one thread are `step` apart.
//
// SHIFT: rows whose pitch is no multiple of 16 bytes, of tensors that start on one.  Pieces are still the 16 aligned
// bytes: a row that starts `shift` values into one has its pieces that much to the left, the first and the last of them
// shared with the neighbour rows.  Rows of a thread are a multiple of VEC apart, so that its shift stays, and with it
// the columns of its registers (weights, sums of the weight's gradient).  A shared piece's other values count as 0 and
// are not written; past the end of the tensor nothing is read.
template <typename T, int VEC, int TPR, int PER, int TENSORS, int AHEAD, bool SHIFT> struct RowStream {
    static constexpr int kBytes = AHEAD * TENSORS * PER * 16;            // shared memory a thread
    uint32_t base;                                                       // this thread's first piece
    uint32_t dim;
    uint64_t n, step, next;                                              // next row to ask for
    const T *src[TENSORS];
    int tid, slot_in, slot_out, shift;

    __device__ __forceinline__ RowStream(uint8_t *smem, uint64_t first, uint64_t n_, uint64_t step_, uint32_t dim_, int tid_, int shift_)
    {
        base = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
        dim = dim_, n = n_, step = step_, next = first, tid = tid_, shift = shift_;
        slot_in = slot_out = 0;
    }
    __device__ __forceinline__ uint32_t at(int slot, int t, int i) const { return base + ((slot * TENSORS + t) * PER + i) * (blockDim.x * 16); }
    __device__ __forceinline__ void ask()
    {
        if (next < n) {
#pragma unroll
            for (int t = 0; t < TENSORS; ++t)
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int c = (tid + i * TPR) * VEC - shift;
                    if (c < (int)dim && src[t]) {
                        const int64_t from = (int64_t)(next * dim) + c;
                        if constexpr (SHIFT) {
                            const uint32_t bytes = (uint32_t)min((int64_t)VEC, (int64_t)(n * dim) - from) * (uint32_t)sizeof(T);
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(slot_in, t, i)), "l"(src[t] + from), "r"(bytes) : "memory");
                        } else {
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(slot_in, t, i)), "l"(src[t] + from) : "memory");
                        }
                    }
                }
            next += step;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++slot_in == AHEAD) slot_in = 0;
    }
    __device__ __forceinline__ void start()
    {
        if constexpr (AHEAD > 0) {
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) ask();
        }
    }
    __device__ __forceinline__ void ready()
    {
        if constexpr (AHEAD > 0) asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD > 0 ? AHEAD - 1 : 0) : "memory");
    }
    __device__ __forceinline__ Pack<T, VEC> get(uint64_t row, int t, int i) const
    {
        if constexpr (AHEAD > 0) {
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at(slot_out, t, i)) : "memory");
            Pack<T, VEC> r;
            static_assert(sizeof(r) == 16, "whole pieces");
            *reinterpret_cast<uint4 *>(&r) = v;
            return r;
        } else {
            return load_once<T, VEC>(src[t] + row * dim + (tid + i * TPR) * VEC);
        }
    }
    __device__ __forceinline__ void taken()                              // the row's pieces are in registers
    {
        if constexpr (AHEAD > 0) {
            if (++slot_out == AHEAD) slot_out = 0;
            ask();
        }
    }
};

// A thread's piece of a row: columns c .. c + VEC - 1.  Of a shifted row's first piece only the last values are its own,
// of its last only the first ones; rows this long have none that is both.
template <typename T, int VEC, bool SHIFT> struct Piece {
    int c, dim;
    __device__ __forceinline__ Piece(int first, uint32_t d) : c(first), dim((int)d) {}
    __device__ __forceinline__ bool on() const { return c < dim; }
    __device__ __forceinline__ bool has(int e) const { return !SHIFT || (c + e >= 0 && c + e < dim); }
    __device__ __forceinline__ bool whole() const { return SHIFT ? c >= 0 && c + VEC <= dim : c < dim; }
    __device__ __forceinline__ Pack<T, VEC> own(Pack<T, VEC> v) const           // others' values as 0
    {
        if constexpr (SHIFT) {
            if (!whole()) {
                int at = c;
                asm volatile("" : "+r"(at));                                    // worked out here, not kept in registers from row to row
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (at + e < 0 || at + e >= dim) v.v[e] = from_f<T>(0.0f);
            }
        }
        return v;
    }
    // An edge is written in stores of 8, 4 and 2 bytes, one for each bit of its length, the widest to the side of the row.
    __device__ __forceinline__ void put(T *row, const Pack<T, VEC> &v) const
    {
        if constexpr (SHIFT) {
            if (!whole()) {
                int first = c;
                asm volatile("" : "+r"(first));
                const bool left = first < 0;
                const int len = left ? VEC + first : dim - first;
                const uint4 u = *reinterpret_cast<const uint4 *>(&v);
                char *to = reinterpret_cast<char *>(row + c);
                const int bytes = len * (int)sizeof(T);
                if (bytes & 8) *reinterpret_cast<uint2 *>(to + (left ? 8 : 0)) = left ? make_uint2(u.z, u.w) : make_uint2(u.x, u.y);
                const uint2 half = ((bytes & 8) != 0) == left ? make_uint2(u.x, u.y) : make_uint2(u.z, u.w);
                const int at = ((bytes & 8) != 0) == left ? 0 : 8;
                if (bytes & 4) *reinterpret_cast<uint32_t *>(to + at + (left ? 4 : 0)) = left ? half.y : half.x;
                if constexpr (sizeof(T) == 2) {
                    const bool second = ((bytes & 4) != 0) != left;
                    const uint32_t word = second ? half.y : half.x;
                    if (bytes & 2) *reinterpret_cast<uint16_t *>(to + at + (second ? 4 : 0) + (left ? 2 : 0)) = (uint16_t)(left ? word >> 16 : word);
                }
                return;
            }
        }
        store<T, VEC>(row + c, v);
    }
};

template <typename T, int VEC, int TPR, int PER, int AHEAD, bool SHIFT>
__global__ void __launch_bounds__(Group<TPR>::kThreads) norm_fwd_kernel(const __grid_constant__ NormParams p)
{
    using P = Pack<T, VEC>;
    using Gr = Group<TPR>;
    __shared__ float2 buf[2 * Gr::kGroups * Gr::kWarps];
    const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
    int turn = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint64_t first = (uint64_t)blockIdx.x * Gr::kGroups + group, step = (uint64_t)gridDim.x * Gr::kGroups;
    const int shift = SHIFT ? (int)(first * p.dim % VEC) : 0;
    using Pc = Piece<T, VEC, SHIFT>;
    auto piece = [&](int i) { return Pc((tid + i * TPR) * VEC - shift, p.dim); };
    constexpr int N2 = PER * VEC / 2;
    P w[PER], bi[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const auto c = piece(i);
        w[i] = bi[i] = zero_pack<T, VEC>();
        if (c.on()) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (c.has(e) && p.y) {
                    w[i].v[e] = static_cast<const T *>(p.weight)[c.c + e];
                    if (p.bias) bi[i].v[e] = static_cast<const T *>(p.bias)[c.c + e];
                }
        }
    }
    extern __shared__ __align__(16) uint8_t ring[];
    RowStream<T, VEC, TPR, PER, 2, AHEAD, SHIFT> in(ring, first, p.n, step, p.dim, tid, shift);
    in.src[0] = static_cast<const T *>(p.x);
    in.src[1] = static_cast<const T *>(p.residual);
    in.start();
    for (uint64_t row = first; row < p.n; row += step) {
        const uint64_t at = row * p.dim;
        P z[PER], r[PER];
        in.ready();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const auto c = piece(i);
            z[i] = r[i] = zero_pack<T, VEC>();
            if (c.on()) {
                z[i] = c.own(in.get(row, 0, i));
                if (p.residual) r[i] = c.own(in.get(row, 1, i));
            }
        }
        in.taken();
        if (p.residual) {
            // the sum is what the next layer reads: rounded first, then normalised as it stands
#pragma unroll
            for (int e = 0; e < N2; ++e) set_pair<T, VEC>(z, e, add2(pair_of<T, VEC>(z, e), pair_of<T, VEC>(r, e)));
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const auto c = piece(i);
                if (c.on()) c.put(static_cast<T *>(p.z) + at, z[i]);
            }
        }
        float2 d[N2], s = make_float2(0.0f, 0.0f), q = s;
#pragma unroll
        for (int e = 0; e < N2; ++e) d[e] = pair_of<T, VEC>(z, e), s = add2(s, d[e]);
        const float mean = group_sum1<TPR>(s.x + s.y, buf, group, turn) * p.inv_dim;
        const float2 nm = make_float2(-mean, -mean);
#pragma unroll
        for (int e = 0; e < N2; ++e) d[e] = add2(d[e], nm);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const auto c = piece(i);
            if (!c.whole()) {
                int first_c = c.c;
                if constexpr (SHIFT) asm volatile("" : "+r"(first_c));
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (first_c + e < 0 || first_c + e >= c.dim) half_of(d, i * VEC + e) = 0.0f;
            }
        }
#pragma unroll
        for (int e = 0; e < N2; ++e) q = fma2(d[e], d[e], q);
        const float rstd = rsqrtf(group_sum1<TPR>(q.x + q.y, buf, group, turn) * p.inv_dim + p.eps);
        const float2 r2 = make_float2(rstd, rstd);
        if (tid == 0) p.mean[row] = mean, p.rstd[row] = rstd;
        if (!p.y) continue;                              // only the statistics
#pragma unroll
        for (int e = 0; e < N2; ++e) set_pair<T, VEC>(z, e, fma2(mul2(d[e], r2), pair_of<T, VEC>(w, e), pair_of<T, VEC>(bi, e)));
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const auto c = piece(i);
            if (c.on()) c.put(static_cast<T *>(p.y) + at, z[i]);
        }
    }
}

// dx = rstd (w dy - c1 - xh c2) + dz with c1 = mean(w dy), c2 = mean(w dy xh);
// part[block][0 | 1][dim]: the block's sums of dy xh and dy.
// FORM: mean and rstd are formed from z, which lies in registers (see WarpJoin), else read.
template <typename T, int VEC, int TPR, int PER, int AHEAD, bool SHIFT, bool FORM>
__global__ void __launch_bounds__(Group<TPR>::kThreads, TPR == 512 ? 1 : PER > 1 ? 2 : 3) norm_bwd_kernel(const __grid_constant__ NormParams p)
{
    using P = Pack<T, VEC>;
    using Gr = Group<TPR>;
    // Two barriers a row in up to 128 threads, one in more or where edges are masked: measured with the other, 2^18 x 1024
    // bf16 (64 threads) 328 us, one barrier 369; 65536 x 4096 (256 threads) 289, two 323; 200000 x 777 (shifted) 399, two 416.
    using Join = std::conditional_t<!FORM, NoJoin<TPR>, std::conditional_t<SHIFT || (TPR > 128), WarpJoin<TPR>, GroupJoin<TPR>>>;
    __shared__ typename Join::Shared buf;
    const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
    int turn = 0;
    // a thread's values go in pairs, one instruction for two; those past the row count as 0
    constexpr int N2 = PER * VEC / 2;
    static_assert(PER * VEC % 2 == 0, "pairs");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint64_t first = (uint64_t)blockIdx.x * Gr::kGroups + group, step = (uint64_t)gridDim.x * Gr::kGroups;
    const int shift = SHIFT ? (int)(first * p.dim % VEC) : 0;
    using Pc = Piece<T, VEC, SHIFT>;
    auto piece = [&](int i) { return Pc((tid + i * TPR) * VEC - shift, p.dim); };
    float2 w[N2], dw[N2], db[N2];
#pragma unroll
    for (int e = 0; e < PER * VEC; ++e) {
        const auto c = piece(e / VEC);
        half_of(w, e) = c.on() && c.has(e % VEC) ? to_f(static_cast<const T *>(p.weight)[c.c + e % VEC]) : 0.0f;
        half_of(dw, e) = half_of(db, e) = 0.0f;
    }
    extern __shared__ __align__(16) uint8_t ring[];
    RowStream<T, VEC, TPR, PER, 3, AHEAD, SHIFT> in(ring, first, p.n, step, p.dim, tid, shift);
    in.src[0] = static_cast<const T *>(p.z_in);
    in.src[1] = static_cast<const T *>(p.dy);
    in.src[2] = static_cast<const T *>(p.dz);
    in.start();
    float count = 0.0f;
    if (FORM) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const auto c = piece(i);
            if (c.on()) count += SHIFT ? (float)(min(c.c + VEC, c.dim) - max(c.c, 0)) : (float)VEC;
        }
    }
    Join joins(&buf, group, count, p.dim);
    for (uint64_t row = first; row < p.n; row += step) {
        const uint64_t at = row * p.dim;
        float mean = 0.0f, rstd = 0.0f;
        if (!FORM) mean = p.mean[row], rstd = p.rstd[row];
        P z[PER], g[PER], x[PER];
        in.ready();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const auto c = piece(i);
            if (c.on()) {
                z[i] = c.own(in.get(row, 0, i)), g[i] = c.own(in.get(row, 1, i));
                if (p.dz) x[i] = in.get(row, 2, i);
            } else {
                z[i] = g[i] = x[i] = zero_pack<T, VEC>();
            }
        }
        float2 xh[N2], a[N2], s0 = make_float2(0.0f, 0.0f), s1 = s0, s2 = s0;
        float c1, c2;
        if constexpr (FORM) {
            in.taken();
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                const float2 dy = pair_of<T, VEC>(g, e);
                xh[e] = pair_of<T, VEC>(z, e);
                a[e] = mul2(dy, w[e]);
                s0 = add2(s0, xh[e]);
                s1 = add2(s1, a[e]);
                db[e] = add2(db[e], dy);
            }
            float c0 = s0.x + s0.y;
            c1 = s1.x + s1.y;
            joins.add(c0, c1);
            const float own = c0 * joins.inv;
            const float2 nm = make_float2(-own, -own);
            s0 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < N2; ++e) xh[e] = add2(xh[e], nm);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const auto c = piece(i);
                if (!c.whole()) {
                    int first_c = c.c;
                    if constexpr (SHIFT) asm volatile("" : "+r"(first_c));
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (first_c + e < 0 || first_c + e >= c.dim) half_of(xh, i * VEC + e) = 0.0f;
                }
            }
#pragma unroll
            for (int e = 0; e < N2; ++e) s0 = fma2(xh[e], xh[e], s0), s2 = fma2(a[e], xh[e], s2);
            c0 = s0.x + s0.y;
            c2 = s2.x + s2.y;
            joins.add(c0, c2);
            const RowSums sums = joins.join(RowSums{own, c0, c1, c2}, p.inv_dim);
            mean = sums.mean;
            rstd = rsqrtf(sums.squares * p.inv_dim + p.eps);
            c1 = sums.a;
            c2 = sums.az * rstd;
            const float2 off = make_float2(own - mean, own - mean), r2 = make_float2(rstd, rstd);
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                xh[e] = mul2(Join::kMoves ? add2(xh[e], off) : xh[e], r2);
                dw[e] = fma2(pair_of<T, VEC>(g, e), xh[e], dw[e]);
            }
        } else {
            const float2 nm = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                const float2 dy = pair_of<T, VEC>(g, e);
                xh[e] = mul2(add2(pair_of<T, VEC>(z, e), nm), r2);
                a[e] = mul2(dy, w[e]);
                s1 = add2(s1, a[e]);
                s2 = fma2(a[e], xh[e], s2);
                dw[e] = fma2(dy, xh[e], dw[e]);
                db[e] = add2(db[e], dy);
            }
            in.taken();
            c1 = s1.x + s1.y, c2 = s2.x + s2.y;
            group_sum<TPR>(c1, c2, buf, group, turn);
        }
        const float2 r2 = make_float2(rstd, rstd);
        const float2 n1 = make_float2(-c1 * p.inv_dim, -c1 * p.inv_dim), n2 = make_float2(-c2 * p.inv_dim, -c2 * p.inv_dim);
#pragma unroll
        for (int e = 0; e < N2; ++e) {
            a[e] = fma2(xh[e], n2, add2(a[e], n1));
            set_pair<T, VEC>(z, e, p.dz ? fma2(a[e], r2, pair_of<T, VEC>(x, e)) : mul2(a[e], r2));
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const auto c = piece(i);
            if (c.on()) {
                c.put(static_cast<T *>(p.dx) + at, z[i]);
            }
        }
    }
    // the groups of a block add up one after another through shared memory
    float *sums = reinterpret_cast<float *>(ring);    // [2][dim], with more than one group
    if (AHEAD > 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    float *out = p.part + (uint64_t)blockIdx.x * 2 * p.dim;
    for (int turn_of = 0; turn_of < Gr::kGroups; ++turn_of) {
        if (Gr::kGroups > 1) __syncthreads();
        if (group != turn_of) continue;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const auto c = piece(i);
            if (c.on()) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    if (!c.has(e)) continue;
                    const uint32_t k = c.c + e;
                    float a = half_of(dw, i * VEC + e), b = half_of(db, i * VEC + e);
                    if (turn_of > 0) a += sums[k], b += sums[p.dim + k];
                    if (turn_of + 1 < Gr::kGroups) sums[k] = a, sums[p.dim + k] = b;
                    else out[k] = a, out[p.dim + k] = b;
                }
            }
        }
    }
}

// AHEAD: rows asked for ahead where blocks stay for several (0: a row's loads wait for its turn, less to set up).
template <typename T, int VEC, int TPR, int PER, int AHEAD, bool SHIFT, bool BACK, bool FORM = false> int run_norm(NormParams &p, uint32_t blocks, cudaStream_t st)
{
    using Gr = Group<TPR>;
    if constexpr (!BACK) {
        if (!blocks) return K2T_OK;
        constexpr auto kernel = norm_fwd_kernel<T, VEC, TPR, PER, AHEAD, SHIFT>;
        const size_t ring = (size_t)Gr::kThreads * RowStream<T, VEC, TPR, PER, 2, AHEAD, SHIFT>::kBytes;
        if (int rc = norm_shared<kernel>()) return rc;
        // short blocks even out the SMs: 16 rounds of them 322 us, 2 rounds 357 us on 2^18 x 1024 bf16
        if (AHEAD > 0) blocks = (uint32_t)std::min<uint64_t>((p.n + Gr::kGroups * 4 - 1) / (Gr::kGroups * 4), kNormBlocks * 4);
        if (SHIFT) blocks = (blocks + 7) / 8 * 8;      // a thread's rows a multiple of VEC apart
        return norm_launch(kernel, dim3(blocks), Gr::kThreads, ring, st, p);
    } else {
        // rows of more than 1024 pieces spill registers as it is: their statistics come from a pass of their own (dispatch)
        if constexpr (!FORM && (VEC == 1 || PER <= 2))
            if (!p.mean) return run_norm<T, VEC, TPR, PER, AHEAD, SHIFT, BACK, true>(p, blocks, st);
        if (blocks) {
            const size_t ring = (size_t)Gr::kThreads * RowStream<T, VEC, TPR, PER, 3, AHEAD, SHIFT>::kBytes;
            const size_t sums = Gr::kGroups > 1 ? 2 * p.dim * sizeof(float) : 0;
            constexpr auto kernel = norm_bwd_kernel<T, VEC, TPR, PER, AHEAD, SHIFT, FORM>;
            int rc = norm_shared<kernel>();
            if (!rc && AHEAD > 0) rc = norm_resident(kernel, blocks, Gr::kThreads, std::max(ring, sums));
            if (rc) return rc;
            if (SHIFT) blocks = blocks < 8 ? 8 : blocks / 8 * 8;
            rc = norm_launch(kernel, dim3(blocks), Gr::kThreads, std::max(ring, sums), st, p);
            if (rc) return rc;
        }
        p.parts = blocks;
        return norm_launch(norm_join_kernel<T>, dim3((p.dim + 7) / 8, p.dbias ? 2 : 1), 1024, 0, st, p);
    }
}

// Blocks: every SM full of them at most (kNormBlocks).  With more than four rows a group the loads run ahead: measured
// on 2^20 x 512 and 2^18 x 1024 bf16 against a row's own loads; below that there is little to run ahead of.
template <typename T, int VEC, int TPR, int PER, int AHEAD, bool BACK> int plan_norm(NormParams &p, cudaStream_t st)
{
    constexpr int G = Group<TPR>::kGroups;
    const uint32_t blocks = norm_parts(p.n, G);
    if constexpr (AHEAD > 0) {
        if (p.n > (uint64_t)4 * G * kNormBlocks) return run_norm<T, VEC, TPR, PER, AHEAD, false, BACK>(p, blocks, st);
    }
    return run_norm<T, VEC, TPR, PER, 0, false, BACK>(p, blocks, st);
}

// Threads a row: as few as hold it with two pieces each, up to a block, then more loads a thread.  Two pieces spread the
// work of a row that does not grow with it, in registers of which every thread has 128 backward (2^18 x 1024 bf16: 325 us,
// one piece 365; 2^20 x 256: 326 and 354); rows of 8 pieces only lose threads (2^20 x 64: 131 us, one piece 108).
template <typename T, bool BACK> int norm_pieces(NormParams &p, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const uint32_t c = p.dim / V;
    constexpr int A = BACK ? 2 : 4;                        // rows ahead
    if constexpr (BACK)
        if (c <= 8) return plan_norm<T, V, 8, 1, 4, BACK>(p, st);
    if (c <= 16) return plan_norm<T, V, 8, 2, A, BACK>(p, st);
    if (c <= 32) return plan_norm<T, V, 16, 2, A, BACK>(p, st);
    if (c <= 64) return plan_norm<T, V, 32, 2, A, BACK>(p, st);
    if (c <= 128) return plan_norm<T, V, 64, 2, A, BACK>(p, st);
    if (c <= 256) return plan_norm<T, V, 128, 2, A, BACK>(p, st);
    if (c <= 512) return plan_norm<T, V, 256, 2, 2, BACK>(p, st);
    if (c <= 1024) return plan_norm<T, V, 512, 2, 2, BACK>(p, st);
    return plan_norm<T, V, 512, 8, 0, BACK>(p, st);
}

// Shifted rows, forward of more than 512 values and backward of 97 pieces, up to 1024 pieces: 200000 x 513 fp16 229 us
// forward, value by value 438; 200000 x 777 bf16 321 and 318, value by value 541 and in stretches 502; 65536 x 3999 bf16
// 338 and 432, in stretches 611 and 1117.  In shorter rows the two edges cost more than the wide loads give (200000 x 513
// fp16 backward 315 us, in stretches 275; 200000 x 333 fp32 172 and 207, in stretches 148 and 187).  One piece a thread
// up to 256 (100000 x 1465 fp16: 259 and 283 us, two pieces 284 and 332): an edge holds up fewer others.
inline bool shift_pays(uint32_t dim, uint32_t pieces, bool backward) { return (backward ? pieces > 96 : dim > 512) && pieces <= 1024; }
inline uint32_t shifted_pieces(uint32_t dim, uint32_t v) { return (dim + 2 * v - 2) / v; }   // at the largest shift

template <typename T, bool BACK> int norm_shifted(NormParams &p, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const uint32_t c = shifted_pieces(p.dim, V), blocks = norm_parts(p.n, 1);
    if (c <= 128) return run_norm<T, V, 128, 1, 4, true, BACK>(p, norm_parts(p.n, Group<128>::kGroups), st);
    if (c <= 256) return run_norm<T, V, 256, 1, 4, true, BACK>(p, blocks, st);
    if (c <= 512) return run_norm<T, V, 256, 2, 2, true, BACK>(p, blocks, st);
    return run_norm<T, V, 512, 2, 2, true, BACK>(p, blocks, st);
}

template <typename T, bool BACK> int norm_dispatch(NormParams &p, bool vec, bool shift, cudaStream_t st)
{
    if (vec) return norm_pieces<T, BACK>(p, st);
    if (shift) return norm_shifted<T, BACK>(p, st);
    if (p.dim <= 128) return plan_norm<T, 1, 32, 4, 0, BACK>(p, st);
    if (p.dim <= 512) return plan_norm<T, 1, 128, 4, 0, BACK>(p, st);
    return plan_norm<T, 1, 256, 8, 0, BACK>(p, st);
}

int check_norm(const k2t_norm *a)
{
    if (!a) return K2T_EINVAL;
    if (a->dtype > K2T_FP32) return K2T_EINVAL;
    if (a->dim == 0 || a->dim > K2T_NORM_MAX_DIM || a->n_rows > (1ull << 32)) return K2T_ERANGE;
    if (!(a->eps > 0.0f) || (a->flags & ~(uint32_t)K2T_NORM_FORM_STATS)) return K2T_EINVAL;
    return K2T_OK;
}

// Partial sums of the weight's gradient: whole 256 bytes of them.
uint64_t norm_part_floats(const k2t_norm *a)
{
    return align_up(((uint64_t)norm_parts(a->n_rows, 1) + 7) / 8 * 8 * 2 * a->dim * sizeof(float), 256) / sizeof(float);
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
    const bool form = backward && (a->flags & K2T_NORM_FORM_STATS);
    p.mean = form ? nullptr : a->mean;
    p.rstd = form ? nullptr : a->rstd;
    // Rows that are not whole pieces: shifted where that pays; else value by value while there are few of them, when a call
    // is its latency (4999 x 333 fp32, training: 18 us against 20), else in stretches (200000 x 333 bf16, forward: 170 us
    // against 220; 65536 x 3999: 610 us against 2335).  Forward rows of 1025 to 2048 values fill a block with single values
    // and stay with them (100000 x 1465 fp16: 308 us against 417; backward 422 against 393).
    const bool few = a->n_rows <= 16384 && a->dim <= 2048, fill = !backward && a->dim > 1024 && a->dim <= 2048;
    const uint32_t c = shifted_pieces(a->dim, 16 / size);
    const bool shift = !vec && !few && !(all & 15) && shift_pays(a->dim, c, backward);
    const bool ragged = !vec && !shift && !few && !fill;
    if (form && (ragged ? a->dim > 4096 : vec && a->dim * size / 16 > 1024)) {
        // statistics in a forward pass that writes nothing else, behind the partial sums
        NormParams f{};
        f.x = p.z_in;
        k2t_norm b = *a;
        b.mean = p.part + norm_part_floats(a);
        b.rstd = b.mean + a->n_rows;
        if (int rc = dispatch(&b, f, false, st)) return rc;
        p.mean = b.mean, p.rstd = b.rstd;
    }
    if (ragged) return norm_ragged(p, a->dtype, backward, st);
    const auto run = [&](auto zero) {
        using T = decltype(zero);
        return backward ? norm_dispatch<T, true>(p, vec, shift, st) : norm_dispatch<T, false>(p, vec, shift, st);
    };
    if (a->dtype == K2T_BF16) return run(__nv_bfloat16());
    if (a->dtype == K2T_FP16) return run(__half());
    return run(0.0f);
}

}  // namespace
}  // namespace k2t

using namespace k2t;

extern "C" {

uint64_t k2t_norm_work_bytes(const k2t_norm *a)
{
    if (check_norm(a)) return 0;
    return norm_part_floats(a) * sizeof(float) + (a->flags & K2T_NORM_FORM_STATS ? align_up(a->n_rows * 2 * sizeof(float), 256) : 0);
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
    if (!a->weight || !a->dweight || (a->n_rows && (!a->z || !a->dy || !a->dx))) return K2T_EINVAL;
    if (a->n_rows && !(a->flags & K2T_NORM_FORM_STATS) && (!a->mean || !a->rstd)) return K2T_EINVAL;
    if (a->n_rows && (!work || ((uintptr_t)work & 15u))) return K2T_EINVAL;
    if (work_bytes < k2t_norm_work_bytes(a)) return K2T_ENOMEM;
    NormParams p{};
    p.z_in = a->z, p.dy = a->dy, p.dz = a->dz, p.dx = a->dx, p.dweight = a->dweight, p.dbias = a->dbias;
    p.part = static_cast<float *>(work);
    return dispatch(a, p, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
