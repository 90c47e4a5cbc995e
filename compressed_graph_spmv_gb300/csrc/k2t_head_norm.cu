// k2t_head_norm.cu -- the head norm calls of the C ABI: checks, plan, launch.
#include <cmath>

#include "k2t_head_norm.cuh"
#include "k2t_rows.h"

namespace k2t {
namespace {

constexpr uint32_t kHeadBlocks = 152 * 8;      // of a backward pass, at most: each writes a partial row of dweight

template <typename T, int V, int S, int HC, bool PAIRED> int head_launch(HeadParams &p, bool backward, cudaStream_t st)
{
    p.chunks = (p.heads + HC - 1) / HC;
    p.units = p.n * p.chunks;
    const uint32_t groups = kHeadThreads / p.lanes;
    const uint64_t all = (p.units + groups - 1) / groups;
    if (!backward) {
        const uint32_t blocks = (uint32_t)std::min<uint64_t>(all, kHeadBlocks * 4);
        return norm_launch(head_norm_fwd_kernel<T, V, S, HC, PAIRED>, dim3(blocks), kHeadThreads, 0, st, p);
    }
    constexpr auto kernel = head_norm_bwd_kernel<T, V, S, HC, PAIRED>;
    const uint32_t blocks = (uint32_t)std::min<uint64_t>(all, kHeadBlocks);
    const size_t smem = p.part ? (size_t)groups * p.d * sizeof(float) : 0;
    return norm_launch(kernel, dim3(blocks), kHeadThreads, smem, st, p);
}

template <typename T, int V, int S, bool PAIRED> int head_chunks(HeadParams &p, bool backward, cudaStream_t st)
{
    if constexpr (V == 1) {
        return head_launch<T, V, S, 1, PAIRED>(p, backward, st);
    } else {
        constexpr int HC = 2;
        if (p.heads > 1 && p.n * p.heads * p.lanes > (uint64_t)152 * 2048) return head_launch<T, V, S, HC, PAIRED>(p, backward, st);
        return head_launch<T, V, S, 1, PAIRED>(p, backward, st);
    }
}

template <typename T, int V, int S> int head_pairs(HeadParams &p, bool paired, bool backward, cudaStream_t st)
{
    p.slots = p.d / 2 / V;
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes < p.slots) p.lanes *= 2;
    return paired ? head_chunks<T, V, S, true>(p, backward, st) : head_chunks<T, V, S, false>(p, backward, st);
}

// Pairs a thread takes: as many as fill a 16-byte load, where both halves of what turns, and of what does not, are whole
// vectors of them.
template <typename T> int head_type(HeadParams &p, bool paired, bool backward, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const uint32_t parts = (p.rotary / 2) | ((p.d - p.rotary) / 2);
    if (parts % V == 0) return head_pairs<T, V, 1>(p, paired, backward, st);
    if (V == 8 && parts % 4 == 0) return head_pairs<T, 4, 1>(p, paired, backward, st);
    return head_pairs<T, 1, 4>(p, paired, backward, st);
}

int check_head(const k2t_head_norm *a)
{
    if (!a || a->dtype > K2T_FP32 || a->n_heads == 0 || a->head_dim == 0 || a->head_dim % 8) return K2T_EINVAL;
    if (a->rotary_dim % 2 || a->rotary_dim > a->head_dim || (a->flags & ~(uint32_t)K2T_HEAD_PAIRED)) return K2T_EINVAL;
    if (!(a->eps > 0.0f)) return K2T_EINVAL;
    if (a->head_dim > K2T_HEAD_MAX_DIM || a->n_heads > K2T_HEAD_MAX_HEADS || a->n_rows > (1ull << 32)) return K2T_ERANGE;
    return K2T_OK;
}

bool overlap(const k2t_head_norm *a, int64_t row, int64_t head) { return a->n_rows && rows_overlap(row, head, a->n_rows, a->n_heads, a->head_dim); }

void fill(const k2t_head_norm *a, HeadParams &p)
{
    p.heads = a->n_heads, p.d = a->head_dim, p.rotary = a->rotary_dim, p.n = a->n_rows;
    p.eps = a->eps, p.inv_d = 1.0f / (float)a->head_dim;
    p.x = a->x, p.weight = a->weight, p.dy = a->dy, p.positions = a->positions, p.y = a->y, p.dx = a->dx;
    p.x_row = a->x_row, p.x_head = a->x_head, p.y_row = a->y_row, p.y_head = a->y_head;
    p.dy_row = a->dy_row, p.dy_head = a->dy_head, p.dx_row = a->dx_row, p.dx_head = a->dx_head;
    for (uint32_t i = 0; i < p.rotary / 2; ++i) p.rate[i] = a->rates[i];
}

int run(const k2t_head_norm *a, HeadParams &p, bool backward, cudaStream_t st)
{
    const bool paired = a->flags & K2T_HEAD_PAIRED;
    if (a->dtype == K2T_BF16) return head_type<__nv_bfloat16>(p, paired, backward, st);
    if (a->dtype == K2T_FP16) return head_type<__half>(p, paired, backward, st);
    return head_type<float>(p, paired, backward, st);
}

}  // namespace
}  // namespace k2t

using namespace k2t;

extern "C" {

int k2t_head_rates(double base, uint32_t rotary_dim, uint64_t *rates)
{
    if (!rates || rotary_dim % 2 || rotary_dim > K2T_HEAD_MAX_DIM || !(base >= 1.0) || std::isinf(base)) return K2T_EINVAL;
    for (uint32_t i = 0; i < rotary_dim / 2; ++i) {
        const long double turns = powl((long double)base, -2.0L * i / rotary_dim) * 0.159154943091895335768883763372514362L;
        rates[i] = (uint64_t)llroundl(turns * 0x1p63L) * 2;      // turns is at most 1 / (2 pi)
    }
    return K2T_OK;
}

uint64_t k2t_head_norm_work_bytes(const k2t_head_norm *a)
{
    return check_head(a) ? 0 : (uint64_t)kHeadBlocks * 2 * a->head_dim * sizeof(float);
}

int k2t_head_norm_forward(const k2t_head_norm *a, void *stream)
{
    if (int rc = check_head(a)) return rc;
    if (a->n_rows && (!a->x || !a->y)) return K2T_EINVAL;
    if (!rows_aligned(a->x, a->x_row, a->x_head) || !rows_aligned(a->y, a->y_row, a->y_head) || ((uintptr_t)a->weight & 15u) ||
        ((uintptr_t)a->positions & 3u))
        return K2T_EINVAL;
    if (overlap(a, a->y_row, a->y_head)) return K2T_EINVAL;
    if (!a->n_rows) return K2T_OK;
    HeadParams p{};
    fill(a, p);
    return run(a, p, false, static_cast<cudaStream_t>(stream));
}

int k2t_head_norm_backward(const k2t_head_norm *a, void *work, uint64_t work_bytes, void *stream)
{
    if (int rc = check_head(a)) return rc;
    if (a->n_rows && (!a->x || !a->dy || !a->dx)) return K2T_EINVAL;
    if (!rows_aligned(a->x, a->x_row, a->x_head) || !rows_aligned(a->dy, a->dy_row, a->dy_head) ||
        !rows_aligned(a->dx, a->dx_row, a->dx_head) || (((uintptr_t)a->weight | (uintptr_t)a->dweight) & 15u) || ((uintptr_t)a->positions & 3u))
        return K2T_EINVAL;
    if ((a->weight != nullptr) != (a->dweight != nullptr) || overlap(a, a->dx_row, a->dx_head)) return K2T_EINVAL;
    if (a->weight && (!work || ((uintptr_t)work & 15u))) return K2T_EINVAL;
    if (a->weight && work_bytes < k2t_head_norm_work_bytes(a)) return K2T_ENOMEM;
    if (!a->n_rows && !a->weight) return K2T_OK;
    HeadParams p{};
    fill(a, p);
    p.part = a->weight ? static_cast<float *>(work) : nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t parts = 0;
    if (a->n_rows) {
        if (int rc = run(a, p, true, st)) return rc;
        const uint32_t groups = kHeadThreads / p.lanes;
        parts = (uint32_t)std::min<uint64_t>((p.units + groups - 1) / groups, kHeadBlocks);
    }
    if (!a->weight) return K2T_OK;
    NormParams j{};
    j.dim = p.d, j.part = p.part, j.parts = parts, j.dweight = a->dweight;
    const auto sum = [&](auto zero) { return norm_launch(norm_join_kernel<decltype(zero)>, dim3((p.d + 7) / 8, 1), 1024, 0, st, j); };
    if (a->dtype == K2T_BF16) return sum(__nv_bfloat16());
    if (a->dtype == K2T_FP16) return sum(__half());
    return sum(0.0f);
}

}  // extern "C"
