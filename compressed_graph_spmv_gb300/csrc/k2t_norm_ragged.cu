// k2t_norm_ragged.cu -- layer norm of rows that are not whole 16-byte pieces
// (a pitch that is no multiple of 16 bytes, or tensors that do not start on one).
//
// Bound by memory like the other rows, if they can be moved in wide pieces:
// a block takes a batch of consecutive rows, which is one stretch of memory,
// and copies the 16-byte pieces that cover it into shared memory (two batches
// in turn, the next one's copies in flight while this one is worked on).
// There its rows are read value by value, lane c of a group of TPR threads
// the columns c, c + TPR, ..., and the results written over what they came
// from; the stretch leaves in 16-byte pieces again, its two ragged ends value
// by value, since the pieces there belong to the neighbours too.
// Measured: 200000 x 333 bf16 with the residual 164 us forward and 173
// backward (208 with the statistics formed), 46% of the copy rate: what bounds it is the shared memory's
// accesses and the address arithmetic of single values.  Long rows of tensors
// that start on a piece go another way (see shift_pays).
#include "k2t_norm.cuh"

namespace k2t {
namespace {

constexpr uint32_t kBlockBytes = 73728;      // two batches of every tensor, about: three blocks an SM

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A stretch of `bytes` bytes at `at` in global memory and its image: the image starts at the 16-byte piece that holds
// the first byte, so that the two agree modulo 16.
struct Stretch {
    const char *at;
    uint32_t bytes, skew;
    __device__ __forceinline__ Stretch(const void *base, uint64_t first, uint32_t n) : bytes(n)
    {
        at = static_cast<const char *>(base) + first;
        skew = (uint32_t)((uintptr_t)at & 15);
    }
    // whole pieces come from inside the tensor or share their 16 bytes with its first or last value: the ends are
    // copied value by value instead, so that nothing outside the tensor is read
    template <typename T, int kRaggedThreads> __device__ __forceinline__ void bring(uint8_t *image, int tid) const
    {
        const uint32_t s = (uint32_t)__cvta_generic_to_shared(image);
        const uint32_t lo = (skew + 15) / 16, hi = (skew + bytes) / 16;
        for (uint32_t k = lo + tid; k < hi; k += kRaggedThreads) copy16(s + k * 16, at - skew + k * 16);
        const uint32_t head = min(lo * 16, skew + bytes) - skew, tail = max(hi * 16, skew + head) - skew;
        for (uint32_t b = tid * sizeof(T); b < head; b += kRaggedThreads * sizeof(T))
            *reinterpret_cast<T *>(image + skew + b) = *reinterpret_cast<const T *>(at + b);
        for (uint32_t b = tail + tid * sizeof(T); b < bytes; b += kRaggedThreads * sizeof(T))
            *reinterpret_cast<T *>(image + skew + b) = *reinterpret_cast<const T *>(at + b);
    }
    template <typename T, int kRaggedThreads> __device__ __forceinline__ void leave(const uint8_t *image, int tid) const
    {
        char *to = const_cast<char *>(at);
        const uint32_t lo = (skew + 15) / 16, hi = (skew + bytes) / 16;
        for (uint32_t k = lo + tid; k < hi; k += kRaggedThreads)
            *reinterpret_cast<uint4 *>(to - skew + k * 16) = *reinterpret_cast<const uint4 *>(image + k * 16);
        const uint32_t head = min(lo * 16, skew + bytes) - skew, tail = max(hi * 16, skew + head) - skew;
        for (uint32_t b = tid * sizeof(T); b < head; b += kRaggedThreads * sizeof(T))
            *reinterpret_cast<T *>(to + b) = *reinterpret_cast<const T *>(image + skew + b);
        for (uint32_t b = tail + tid * sizeof(T); b < bytes; b += kRaggedThreads * sizeof(T))
            *reinterpret_cast<T *>(to + b) = *reinterpret_cast<const T *>(image + skew + b);
    }
};

// Rows of a batch (as many for every group, where that is not too much), and bytes of an image.
struct Batch { uint32_t rows, image; };
inline Batch batch_of(uint64_t n, uint32_t dim, size_t size, uint32_t groups, uint32_t tensors)
{
    const uint32_t target = std::min<uint32_t>(16384, kBlockBytes / 2 / tensors);
    const uint32_t row = dim * (uint32_t)size, turn = groups * row;
    uint32_t rows = turn <= target * 3 / 2 ? groups * std::max<uint32_t>(1, target / turn) : std::max<uint32_t>(1, target / row);
    // few rows: a batch for every block before a block has two
    const uint64_t each = (n + (uint64_t)groups * kNormBlocks - 1) / ((uint64_t)groups * kNormBlocks) * groups;
    if (each && each < rows) rows = (uint32_t)each;
    return {rows, (rows * row + 31 + 15) / 16 * 16};
}

// Where a result goes: over the image of the tensor it came from, if the two agree modulo 16, else straight to memory.
__device__ __forceinline__ bool same_skew(const void *a, const void *b) { return (((uintptr_t)a ^ (uintptr_t)b) & 15) == 0; }

template <typename T, int TPR, int PER>
__global__ void __launch_bounds__(Group<TPR>::kThreads) ragged_fwd_kernel(const __grid_constant__ NormParams p, uint32_t rows, uint32_t image, int images)
{
    using Gr = Group<TPR>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 buf[2 * Gr::kGroups * Gr::kWarps];
    const int tid = threadIdx.x, c0 = tid % TPR, group = tid / TPR;
    const uint32_t tensors = p.residual ? 2 : 1;
    int turn = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float w[PER], b[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t c = c0 + i * TPR;
        w[i] = c < p.dim && p.y ? to_f(static_cast<const T *>(p.weight)[c]) : 0.0f;
        b[i] = c < p.dim && p.bias ? to_f(static_cast<const T *>(p.bias)[c]) : 0.0f;
    }
    const uint32_t row_bytes = p.dim * (uint32_t)sizeof(T);
    const uint64_t step = (uint64_t)gridDim.x * rows, step_bytes = step * row_bytes;
    uint64_t row0 = (uint64_t)blockIdx.x * rows, off = row0 * row_bytes;     // the batch's first row, and its byte
    auto stretch = [&](const void *base) { return Stretch(base, off, (uint32_t)min((uint64_t)rows, p.n - row0) * row_bytes); };
    auto skew = [&](const void *base) { return (uint32_t)((uintptr_t)base + off) & 15; };
    auto at = [&](int slot, int t) { return smem + (size_t)(slot * tensors + t) * image; };
    auto bring = [&](int slot, bool next) {              // this batch, or the block's next one
        const uint64_t r = row0 + (next ? step : 0), o = off + (next ? step_bytes : 0);
        if (r < p.n) {
            const uint32_t bytes = (uint32_t)min((uint64_t)rows, p.n - r) * row_bytes;
            Stretch(p.x, o, bytes).template bring<T, Gr::kThreads>(at(slot, 0), tid);
            if (p.residual) Stretch(p.residual, o, bytes).template bring<T, Gr::kThreads>(at(slot, 1), tid);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const bool y_over = p.y && same_skew(p.x, p.y), z_over = p.residual && same_skew(p.residual, p.z);
    int slot = 0;
    bring(0, false);
    for (; row0 < p.n; row0 += step, off += step_bytes) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();                                    // this batch is here; the other image has left
        if (images > 1) bring(slot ^ 1, true);
        const uint32_t here = (uint32_t)min((uint64_t)rows, p.n - row0);
        T *xs = reinterpret_cast<T *>(at(slot, 0) + skew(p.x));
        T *rs = p.residual ? reinterpret_cast<T *>(at(slot, 1) + skew(p.residual)) : nullptr;
        for (uint32_t r = group; r < here; r += Gr::kGroups) {
            const uint64_t row = row0 + r;
            T *xr = xs + (size_t)r * p.dim, *rr = p.residual ? rs + (size_t)r * p.dim : nullptr;
            float v[PER], s = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t c = c0 + i * TPR;
                v[i] = 0.0f;
                if (c < p.dim) {
                    T z = xr[c];
                    if (p.residual) {
                        z = from_f<T>(to_f(z) + to_f(rr[c]));       // rounded first, then normalised as it stands
                        if (z_over) rr[c] = z;
                        else static_cast<T *>(p.z)[row * p.dim + c] = z;
                    }
                    v[i] = to_f(z);
                    s += v[i];
                }
            }
            s = group_sum1<TPR>(s, buf, group, turn);
            const float mean = s * p.inv_dim;
            float q = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const float d = c0 + i * TPR < p.dim ? v[i] - mean : 0.0f;
                v[i] = d;
                q = fmaf(d, d, q);
            }
            q = group_sum1<TPR>(q, buf, group, turn);
            const float rstd = rsqrtf(q * p.inv_dim + p.eps);
            if (c0 == 0) p.mean[row] = mean, p.rstd[row] = rstd;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t c = c0 + i * TPR;
                if (c < p.dim) {
                    const T y = from_f<T>(fmaf(v[i] * rstd, w[i], b[i]));
                    if (y_over) xr[c] = y;
                    else if (p.y) static_cast<T *>(p.y)[row * p.dim + c] = y;
                }
            }
        }
        __syncthreads();
        if (y_over) stretch(p.y).template leave<T, Gr::kThreads>(at(slot, 0), tid);
        if (z_over) stretch(p.z).template leave<T, Gr::kThreads>(at(slot, 1), tid);
        if (images > 1) slot ^= 1;
        else {
            __syncthreads();
            bring(0, true);
        }
    }
}

// FORM: mean and rstd are formed from z (see WarpJoin), else read.
template <typename T, int TPR, int PER, bool FORM>
__global__ void __launch_bounds__(Group<TPR>::kThreads) ragged_bwd_kernel(const __grid_constant__ NormParams p, uint32_t rows, uint32_t image, int images)
{
    using Gr = Group<TPR>;
    extern __shared__ __align__(16) uint8_t smem[];
    using Join = std::conditional_t<FORM, WarpJoin<TPR>, NoJoin<TPR>>;
    __shared__ typename Join::Shared buf;
    const int tid = threadIdx.x, c0 = tid % TPR, group = tid / TPR;
    const uint32_t tensors = p.dz ? 3 : 2;
    int turn = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float w[PER], dw[PER], db[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t c = c0 + i * TPR;
        w[i] = c < p.dim ? to_f(static_cast<const T *>(p.weight)[c]) : 0.0f;
        dw[i] = db[i] = 0.0f;
    }
    const uint32_t row_bytes = p.dim * (uint32_t)sizeof(T);
    const uint64_t step = (uint64_t)gridDim.x * rows, step_bytes = step * row_bytes;
    uint64_t row0 = (uint64_t)blockIdx.x * rows, off = row0 * row_bytes;     // the batch's first row, and its byte
    auto stretch = [&](const void *base) { return Stretch(base, off, (uint32_t)min((uint64_t)rows, p.n - row0) * row_bytes); };
    auto skew = [&](const void *base) { return (uint32_t)((uintptr_t)base + off) & 15; };
    auto at = [&](int slot, int t) { return smem + (size_t)(slot * tensors + t) * image; };
    auto bring = [&](int slot, bool next) {              // this batch, or the block's next one
        const uint64_t r = row0 + (next ? step : 0), o = off + (next ? step_bytes : 0);
        if (r < p.n) {
            const uint32_t bytes = (uint32_t)min((uint64_t)rows, p.n - r) * row_bytes;
            Stretch(p.z_in, o, bytes).template bring<T, Gr::kThreads>(at(slot, 0), tid);
            Stretch(p.dy, o, bytes).template bring<T, Gr::kThreads>(at(slot, 1), tid);
            if (p.dz) Stretch(p.dz, o, bytes).template bring<T, Gr::kThreads>(at(slot, 2), tid);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const bool over = same_skew(p.dy, p.dx);
    auto in_row = [&](int i) { return c0 + i * TPR < p.dim; };
    float count = 0.0f;
    if (FORM) {
#pragma unroll
        for (int i = 0; i < PER; ++i) count += in_row(i) ? 1.0f : 0.0f;
    }
    Join joins(&buf, group, count, p.dim);
    int slot = 0;
    bring(0, false);
    for (; row0 < p.n; row0 += step, off += step_bytes) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        if (images > 1) bring(slot ^ 1, true);
        const uint32_t here = (uint32_t)min((uint64_t)rows, p.n - row0);
        const T *zs = reinterpret_cast<const T *>(at(slot, 0) + skew(p.z_in));
        T *gs = reinterpret_cast<T *>(at(slot, 1) + skew(p.dy));
        const T *es = p.dz ? reinterpret_cast<const T *>(at(slot, 2) + skew(p.dz)) : nullptr;
        for (uint32_t r = group; r < here; r += Gr::kGroups) {
            const uint64_t row = row0 + r;
            const size_t off = (size_t)r * p.dim;
            float xh[PER], a[PER], rstd, c1 = 0.0f, c2 = 0.0f;
            if constexpr (FORM) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const uint32_t c = c0 + i * TPR;
                    xh[i] = a[i] = 0.0f;
                    if (c < p.dim) {
                        const float dy = to_f(gs[off + c]);
                        xh[i] = to_f(zs[off + c]);
                        a[i] = dy * w[i];
                        sum += xh[i];
                        c1 += a[i];
                        db[i] += dy;
                    }
                }
                joins.add(sum, c1);
                const float own = sum * joins.inv;
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    xh[i] = in_row(i) ? xh[i] - own : 0.0f;
                    sum = fmaf(xh[i], xh[i], sum);
                    c2 = fmaf(a[i], xh[i], c2);
                }
                joins.add(sum, c2);
                const RowSums sums = joins.join(RowSums{own, sum, c1, c2}, p.inv_dim);
                rstd = rsqrtf(sums.squares * p.inv_dim + p.eps);
                c1 = sums.a;
                c2 = sums.az * rstd;
                const float to = own - sums.mean;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    xh[i] = (xh[i] + to) * rstd;
                    if (in_row(i)) dw[i] = fmaf(to_f(gs[off + c0 + i * TPR]), xh[i], dw[i]);
                }
            } else {
                const float mean = p.mean[row];
                rstd = p.rstd[row];
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const uint32_t c = c0 + i * TPR;
                    xh[i] = a[i] = 0.0f;
                    if (c < p.dim) {
                        const float dy = to_f(gs[off + c]);
                        xh[i] = (to_f(zs[off + c]) - mean) * rstd;
                        a[i] = dy * w[i];
                        c1 += a[i];
                        c2 = fmaf(a[i], xh[i], c2);
                        dw[i] = fmaf(dy, xh[i], dw[i]);
                        db[i] += dy;
                    }
                }
                group_sum<TPR>(c1, c2, buf, group, turn);
            }
            c1 *= p.inv_dim;
            c2 *= p.inv_dim;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t c = c0 + i * TPR;
                if (c < p.dim) {
                    const T dx = from_f<T>(fmaf(a[i] - c1 - xh[i] * c2, rstd, p.dz ? to_f(es[off + c]) : 0.0f));
                    if (over) gs[off + c] = dx;
                    else static_cast<T *>(p.dx)[row * p.dim + c] = dx;
                }
            }
        }
        __syncthreads();
        if (over) stretch(p.dx).template leave<T, Gr::kThreads>(at(slot, 1), tid);
        if (images > 1) slot ^= 1;
        else {
            __syncthreads();
            bring(0, true);
        }
    }
    // the groups of a block add up one after another through shared memory
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float *sums = reinterpret_cast<float *>(smem), *out = p.part + (uint64_t)blockIdx.x * 2 * p.dim;
    for (int g = 0; g < Gr::kGroups; ++g) {
        if (Gr::kGroups > 1) __syncthreads();
        if (group != g) continue;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = c0 + i * TPR;
            if (c < p.dim) {
                float a = dw[i], b = db[i];
                if (g > 0) a += sums[c], b += sums[p.dim + c];
                if (g + 1 < Gr::kGroups) sums[c] = a, sums[p.dim + c] = b;
                else out[c] = a, out[p.dim + c] = b;
            }
        }
    }
}

template <auto K> struct Kernel { static constexpr auto value = K; };

constexpr size_t kRaggedSmem = 225 * 1024;     // of the 227 KB a block may have, beside the few bytes of the group sums

template <typename T, int TPR, int PER> int run_ragged(NormParams &p, bool backward, cudaStream_t st)
{
    const size_t tensors = backward ? (p.dz ? 3 : 2) : p.residual ? 2 : 1;
    const Batch b = batch_of(p.n, p.dim, sizeof(T), Group<TPR>::kGroups, (uint32_t)tensors);
    const int images = 2 * tensors * b.image <= kRaggedSmem ? 2 : 1;
    const size_t smem = std::max<size_t>(images * tensors * b.image, backward ? 2 * p.dim * sizeof(float) : 0);
    uint32_t blocks = (uint32_t)std::min<uint64_t>((p.n + b.rows - 1) / b.rows, kNormBlocks);
    auto launch = [&](auto of) -> int {
        constexpr auto kernel = decltype(of)::value;
        int rc = norm_shared<kernel>();
        // as many as run at once: blocks stay, and their copies run ahead
        if (!rc) rc = norm_resident(kernel, blocks, Group<TPR>::kThreads, smem);
        p.parts = blocks;
        if (rc || !blocks) return rc;
        return norm_launch(kernel, dim3(blocks), Group<TPR>::kThreads, smem, st, p, b.rows, b.image, images);
    };
    if (!backward) return launch(Kernel<ragged_fwd_kernel<T, TPR, PER>>());
    int rc;
    // rows of more than 4096 values come with their statistics
    if constexpr (PER <= 16) rc = p.mean ? launch(Kernel<ragged_bwd_kernel<T, TPR, PER, false>>()) : launch(Kernel<ragged_bwd_kernel<T, TPR, PER, true>>());
    else rc = launch(Kernel<ragged_bwd_kernel<T, TPR, PER, false>>());
    return rc ? rc : norm_launch(norm_join_kernel<T>, dim3((p.dim + 7) / 8, p.dbias ? 2 : 1), 1024, 0, st, p);
}

// Threads a row: eight values a thread, up to a block, then more.  (200000 x 333 bf16 forward: 8 values 148 us, 16 values
// 171 us.)
template <typename T> int ragged_dim(NormParams &p, bool backward, cudaStream_t st)
{
    if (p.dim <= 64) return run_ragged<T, 8, 8>(p, backward, st);
    if (p.dim <= 128) return run_ragged<T, 16, 8>(p, backward, st);
    if (p.dim <= 256) return run_ragged<T, 32, 8>(p, backward, st);
    if (p.dim <= 512) return run_ragged<T, 64, 8>(p, backward, st);
    if (p.dim <= 1024) return run_ragged<T, 128, 8>(p, backward, st);
    if (p.dim <= 2048) return run_ragged<T, 256, 8>(p, backward, st);
    if (p.dim <= 4096) return run_ragged<T, 256, 16>(p, backward, st);
    return run_ragged<T, 256, 64>(p, backward, st);
}

}  // namespace

int norm_ragged(NormParams &p, uint32_t dtype, bool backward, cudaStream_t st)
{
    if (dtype == K2T_BF16) return ragged_dim<__nv_bfloat16>(p, backward, st);
    if (dtype == K2T_FP16) return ragged_dim<__half>(p, backward, st);
    return ragged_dim<float>(p, backward, st);
}

}  // namespace k2t
