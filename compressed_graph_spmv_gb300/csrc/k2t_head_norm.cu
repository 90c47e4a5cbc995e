// k2t_head_norm.cu -- the head norm calls of the C ABI: checks, plan, launch.
#include <cmath>

#include "k2t_head_norm.cuh"
#include "k2t_rows.h"

namespace k2t {
namespace {

constexpr uint32_t kHeadBlocks = 152 * 4;       // of a backward pass, at most: each writes a partial row of dweight

template <typename T, int V, int S, int AHEAD, bool PAIRED, bool BACK> int head_launch(HeadParams &p, cudaStream_t st)
{
    const uint32_t groups = kHeadThreads / 32 * (32 / p.lanes);
    p.chunks = (p.heads + p.per - 1) / p.per;
    p.units = p.n * p.chunks;
    constexpr auto kernel = [] {
        if constexpr (BACK) return head_norm_bwd_kernel<T, V, S, AHEAD, PAIRED>;
        else return head_norm_fwd_kernel<T, V, S, AHEAD, PAIRED>;
    }();
    size_t smem = HeadStream<T, V, S, (BACK ? 4 : 2) * S, AHEAD>::kBytes + sizeof(p.rate);
    if (BACK && p.part) smem += (size_t)groups * p.d * sizeof(float);
    if (int rc = norm_shared<kernel>()) return rc;
    const uint64_t all = (p.units + groups - 1) / groups;
    uint32_t blocks = (uint32_t)std::min<uint64_t>(all, BACK ? kHeadBlocks : kHeadBlocks * 8);
    if (AHEAD) {
        if (int rc = norm_resident(kernel, blocks, kHeadThreads, smem)) return rc;      // each starts its own queue of loads
    }
    p.blocks = blocks;
    return norm_launch(kernel, dim3(blocks), kHeadThreads, smem, st, p);
}

// Where there are rows enough to fill the GPU a group of lanes takes all heads of a row, whose angles it forms once, and
// its loads run ahead; else a head each: such a call is its latency.
template <typename T, int V, int S, bool PAIRED, bool BACK> int head_rows(HeadParams &p, cudaStream_t st)
{
    p.slots = p.d / 2 / V;
    p.lanes = std::min(32u, p.slots);
    p.reach = 0;
    for (uint32_t r = 1; r < p.lanes; r *= 2) p.reach = r;
    const bool many = p.n * p.lanes > (uint64_t)152 * 2048;
    p.per = many ? p.heads : 1;
    if constexpr (S == 1) {
        // heads ahead: 96 bytes of a thread, 50 to 100 KB of an SM's, in 3 to 8 heads.  More costs as less does: 2^20 rows of 4
        // heads of 128, fp32, forward, 3 heads ahead 642 us, 6 ahead 696.
        constexpr int kBytes = (BACK ? 4 : 2) * V * (int)sizeof(T), kAhead = std::min(std::max(96 / kBytes, 3), 8);
        if (many) return head_launch<T, V, S, kAhead, PAIRED, BACK>(p, st);
    }
    return head_launch<T, V, S, 0, PAIRED, BACK>(p, st);
}

// Pairs a thread takes: vectors of 16 bytes, where both halves of what turns, and of what does not, are whole vectors of them,
// else of fewer: what a head costs besides its values (its sums over the lanes, its loads) is shared by more of them (2^20 rows
// of 4 heads of 128, bf16, backward 602 us, in vectors of 8 bytes 805).
template <typename T, bool PAIRED, bool BACK> int head_type(HeadParams &p, cudaStream_t st)
{
    const uint32_t parts = (p.rotary / 2) | ((p.d - p.rotary) / 2);
    if constexpr (sizeof(T) == 2) {
        if (parts % 8 == 0) return head_rows<T, 8, 1, PAIRED, BACK>(p, st);
    }
    if (parts % 4 == 0) return head_rows<T, 4, 1, PAIRED, BACK>(p, st);
    if (parts % 2 == 0) return p.d <= 128 ? head_rows<T, 2, 1, PAIRED, BACK>(p, st) : head_rows<T, 2, 2, PAIRED, BACK>(p, st);
    return head_rows<T, 1, 4, PAIRED, BACK>(p, st);
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

template <bool BACK> int run(const k2t_head_norm *a, HeadParams &p, cudaStream_t st)
{
    const auto go = [&](auto zero) {
        using T = decltype(zero);
        return a->flags & K2T_HEAD_PAIRED ? head_type<T, true, BACK>(p, st) : head_type<T, false, BACK>(p, st);
    };
    if (a->dtype == K2T_BF16) return go(__nv_bfloat16());
    if (a->dtype == K2T_FP16) return go(__half());
    return go(0.0f);
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
    return run<false>(a, p, static_cast<cudaStream_t>(stream));
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
        if (int rc = run<true>(a, p, st)) return rc;
        parts = p.blocks;
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
