// k2t_attn.cu -- the attention calls of the C ABI: checks, plan, launch.
#include <algorithm>

#include "k2t_attn_launch.cuh"

namespace k2t {

int attn_forward_bf16(const AttnParams &p, int bm, cudaStream_t st);
int attn_forward_fp16(const AttnParams &p, int bm, cudaStream_t st);
int attn_backward_bf16(const AttnParams &p, cudaStream_t st);
int attn_backward_fp16(const AttnParams &p, cudaStream_t st);

namespace {

// Sizes: the part of the checks that k2t_attn_work_bytes shares.
int check_sizes(const k2t_attn *a)
{
    if (!a) return K2T_EINVAL;
    if (a->dtype != K2T_BF16 && a->dtype != K2T_FP16) return K2T_EINVAL;
    if (a->n_heads == 0 || a->n_kv_heads == 0 || a->n_heads % a->n_kv_heads) return K2T_EINVAL;
    if (a->head_dim == 0 || a->head_dim % 8) return K2T_EINVAL;
    if (a->head_dim > K2T_ATTN_MAX_HEAD_DIM || a->n_heads / a->n_kv_heads > K2T_ATTN_MAX_GROUP) return K2T_ERANGE;
    if (a->n_kv_heads > 65535) return K2T_ERANGE;
    if (a->n_sources > K2T_MAX_BATCH || a->n_buckets > K2T_ATTN_MAX_BUCKETS) return K2T_ERANGE;
    if (a->n_nodes > K2T_ATTN_MAX_NODES || (uint64_t)a->n_queries * a->n_heads > (1ull << 30)) return K2T_ERANGE;
    if (a->n_buckets && !a->n_sources) return K2T_EINVAL;
    if (!(a->scale == a->scale)) return K2T_EINVAL;
    for (uint32_t b = 0; b < a->n_buckets; ++b)
        if (b == 0 ? a->edges[0] != 0 : a->edges[b] <= a->edges[b - 1]) return K2T_EINVAL;
    return K2T_OK;
}

// Rows of 16-byte pieces, with pitches that a tensor map holds (40 bits of bytes).
bool aligned(const void *p, int64_t row, int64_t head)
{
    return !((uintptr_t)p & 15u) && !(row & 7) && !(head & 7) && row >= 0 && head >= 0 && row < (1ll << 38) && head < (1ll << 38);
}

// Whether two rows of an output [rows, heads, d] share values: rows i apart and heads j apart the other way, |i row - j head| < d.
bool overlaps(int64_t row, int64_t head, uint64_t rows, uint64_t heads, uint32_t d)
{
    using Wide = unsigned __int128;
    if ((rows > 1 && row < d) || (heads > 1 && head < d)) return true;
    if (rows < 2 || heads < 2) return false;
    if (row >= (Wide)(heads - 1) * head + d || head >= (Wide)(rows - 1) * row + d) return false;     // one inside the other
    for (uint64_t j = 1; j < heads; ++j) {
        const Wide at = (Wide)j * head, i = at / row, left = at - i * row;
        if ((i < rows && left < d) || (i + 1 < rows && row - left < d)) return true;
    }
    return false;
}

constexpr uint64_t kSms = 152;

// Blocks that share the nodes of one (head, row tile): as many as make the
// fewest rounds of the GPU's SMs (one block each) times tiles a block, with
// two tiles' time for a block's start and end and three (a short kernel) for
// joining them.  For a number of rounds, the most blocks
// that it holds.
uint32_t pick_splits(uint64_t blocks, uint64_t tiles)
{
    const uint64_t most = std::min<uint64_t>(std::max<uint64_t>(1, tiles), kSms);
    uint64_t best = 1, cost = ~0ull;
    for (uint64_t rounds = (blocks + kSms - 1) / kSms, last = rounds + 8; rounds <= last; ++rounds) {
        const uint64_t s = std::min(most, rounds * kSms / blocks), c = rounds * ((tiles + s - 1) / s + 2) + 3;
        if (c < cost) cost = c, best = s;
        if (s == most) break;
    }
    const uint64_t alone = (blocks + kSms - 1) / kSms * (tiles + 2);
    return alone <= cost ? 1 : (uint32_t)best;
}

struct Plan {
    AttnParams p;
    int bm;
    uint64_t part_floats, ml_floats, info_floats, delta_floats;
};

void make_plan(const k2t_attn *a, bool backward, Plan &pl)
{
    AttnParams &p = pl.p;
    p = AttnParams{};
    p.T = a->n_queries;
    p.hq = a->n_heads;
    p.hkv = a->n_kv_heads;
    p.group = p.hq / p.hkv;
    p.d = a->head_dim;
    p.sources = a->n_sources;
    p.buckets = a->n_buckets;
    p.n = a->n_nodes;
    p.rows = p.T * p.group;
    while ((1u << p.group2_log) < p.group) ++p.group2_log;
    p.group2 = 1u << p.group2_log;
    p.scale = a->scale;
    p.scale_log2 = a->scale * kLog2e;
    p.tiles = (p.n + kTcTile - 1) / kTcTile;
    const uint64_t rows = (uint64_t)p.T * p.hq;
    pl.delta_floats = 0;
    if (backward) {
        // for sums of score gradients by bucket (see k2t_attn_delta.cuh), and for the power of two that keeps fp16 ones in range
        if ((p.buckets || a->dtype == K2T_FP16) && p.T && p.n) {
            p.delta_tiles = (p.rows + delta_rows(p) - 1) / delta_rows(p);
            p.delta_splits = pick_splits((uint64_t)p.hkv * p.delta_tiles, p.tiles);
            pl.delta_floats = p.delta_splits * rows * 3;
        }
        const uint32_t per = kBwdRows / p.group;              // whole queries of a row tile
        p.row_tiles = std::max(1u, (p.T + per - 1) / per);
        const uint32_t fused = bwd_fused_tiles(p.d), held = p.row_tiles <= fused ? fused : 4;
        const uint32_t groups = (p.row_tiles + held - 1) / held;
        p.splits = pick_splits((uint64_t)p.hkv * groups, p.tiles);
        p.hist_parts = p.splits * groups;
        pl.part_floats = p.splits > 1 ? p.splits * rows * p.d : 0;
        pl.ml_floats = (uint64_t)p.hist_parts * p.hq * p.buckets;
        pl.info_floats = p.row_tiles <= fused ? 0 : (uint64_t)p.hkv * p.row_tiles * (sizeof(RowInfo) / 4);
        return;
    }
    // rows per block: the fewest lanes that hold them all, since the states are read once per row block.  Measured, bf16:
    // 4 rows a head over 2^20 nodes 297 us, in 128 lanes 339; 39 rows over 100003 nodes (fp16) 26 us, in 128 lanes 30; 1024
    // rows over 16384 nodes 123 us, with one row tile a block 8% more.
    pl.bm = p.rows <= 32 ? 32 : p.rows <= 64 ? 64 : p.rows <= 128 ? 128 : 256;
    p.row_tiles = std::max(1u, (p.rows + pl.bm - 1) / pl.bm);
    p.splits = pick_splits((uint64_t)p.hkv * p.row_tiles, p.tiles);
    pl.part_floats = p.splits > 1 ? p.splits * rows * p.d : 0;
    pl.ml_floats = p.splits > 1 ? p.splits * rows * 2 : 0;
    pl.info_floats = 0;
}

// The driver's tensor map encoder, found through the runtime (nothing links to libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encoder()
{
    static const EncodeTiled f = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<EncodeTiled>(fn);
    }();
    return f;
}

// A gradient [n, kv heads, head_dim] as boxes of 128 nodes x 64 values of one head.
bool node_map(CUtensorMap *map, void *base, int64_t row, int64_t head, const AttnParams &p, uint32_t dtype)
{
    const cuuint64_t dims[3] = {p.d, p.hkv, p.n};
    // a dimension of one value has no pitch
    const cuuint64_t strides[2] = {(cuuint64_t)(p.hkv > 1 ? head : p.d) * 2, (cuuint64_t)(p.n > 1 ? row : p.d) * 2};
    const cuuint32_t box[3] = {64, 1, kTcTile}, step[3] = {1, 1, 1};
    return encoder() && encoder()(map, dtype == K2T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base,
                                  dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr uint64_t kWorkHead = 256;   // the device status word

uint64_t plan_bytes(const Plan &pl)
{
    return kWorkHead + align_up(pl.part_floats * 4, 256) + align_up(pl.ml_floats * 4, 256) + align_up(pl.info_floats * 4, 256) +
           align_up(pl.delta_floats * 4, 256);
}

int check_call(const k2t_attn *a, const void *work, bool backward)
{
    const bool q = a->n_queries != 0, n = a->n_nodes != 0;
    if ((q && (!a->q || !a->out || !a->lse)) || (n && (!a->k || !a->v))) return K2T_EINVAL;
    if (!aligned(a->q, a->q_row, a->q_head) || !aligned(a->k, a->k_row, a->k_head) ||
        !aligned(a->v, a->v_row, a->v_head) || !aligned(a->out, a->out_row, a->out_head))
        return K2T_EINVAL;
    if (a->n_sources && n && !a->hops) return K2T_EINVAL;
    if ((a->n_buckets != 0) != (a->bias != nullptr)) return K2T_EINVAL;
    if (a->n_sources && !a->query_source && a->n_queries > a->n_sources) return K2T_ERANGE;
    if (!work || ((uintptr_t)work & 15u)) return K2T_EINVAL;
    const auto shared = [&](int64_t row, int64_t head, bool nodes) {
        return overlaps(row, head, nodes ? a->n_nodes : a->n_queries, nodes ? a->n_kv_heads : a->n_heads, a->head_dim);
    };
    if (!backward) return a->n_queries && shared(a->out_row, a->out_head, false) ? K2T_EINVAL : K2T_OK;
    if ((q && (!a->dout || !a->dq)) || (n && (!a->dk || !a->dv)) || (a->n_buckets && !a->dbias)) return K2T_EINVAL;
    if (!aligned(a->dout, a->dout_row, a->dout_head) || !aligned(a->dq, a->dq_row, a->dq_head) ||
        !aligned(a->dk, a->dk_row, a->dk_head) || !aligned(a->dv, a->dv_row, a->dv_head))
        return K2T_EINVAL;
    if ((q && shared(a->dq_row, a->dq_head, false)) || (n && (shared(a->dk_row, a->dk_head, true) || shared(a->dv_row, a->dv_head, true))))
        return K2T_EINVAL;
    return K2T_OK;
}

void fill_pointers(const k2t_attn *a, void *work, Plan &pl)
{
    AttnParams &p = pl.p;
    p.q = a->q, p.k = a->k, p.v = a->v, p.dout = a->dout;
    if (!a->n_queries) p.q = p.dout = p.k;   // a readable address for copies of no bytes
    p.hops = a->hops, p.qsrc = a->query_source, p.bias = a->bias;
    p.out = a->out, p.dq = a->dq, p.dk = a->dk, p.dv = a->dv, p.dbias = a->dbias;
    p.lse = a->lse;
    p.q_row = a->q_row, p.q_head = a->q_head, p.k_row = a->k_row, p.k_head = a->k_head;
    p.v_row = a->v_row, p.v_head = a->v_head, p.out_row = a->out_row, p.out_head = a->out_head;
    p.dout_row = a->dout_row, p.dout_head = a->dout_head, p.dq_row = a->dq_row, p.dq_head = a->dq_head;
    p.dk_row = a->dk_row, p.dk_head = a->dk_head, p.dv_row = a->dv_row, p.dv_head = a->dv_head;
    p.status = static_cast<uint32_t *>(work);
    char *w = static_cast<char *>(work) + kWorkHead;
    p.part = reinterpret_cast<float *>(w);
    p.part_ml = reinterpret_cast<float *>(w + align_up(pl.part_floats * 4, 256));
    w += align_up(pl.part_floats * 4, 256) + align_up(pl.ml_floats * 4, 256);
    p.row_info = w;
    p.delta_part = reinterpret_cast<float2 *>(w + align_up(pl.info_floats * 4, 256));
    p.pdp_top = reinterpret_cast<float *>(p.delta_part + (uint64_t)p.delta_splits * p.T * p.hq);
    uint32_t b = 0;
    for (uint32_t x = 0; x < 256; ++x) {
        while (b + 1 < a->n_buckets && a->edges[b + 1] <= x) ++b;
        p.bucket_of[x] = (uint8_t)b;
    }
}

}  // namespace
}  // namespace k2t

using namespace k2t;

extern "C" {

uint64_t k2t_attn_work_bytes(const k2t_attn *a, int32_t backward)
{
    if (check_sizes(a)) return 0;
    Plan pl;
    make_plan(a, backward != 0, pl);
    return plan_bytes(pl);
}

int k2t_attn_forward(const k2t_attn *a, void *work, uint64_t work_bytes, void *stream)
{
    int rc = check_sizes(a);
    if (rc) return rc;
    Plan pl;
    make_plan(a, false, pl);
    if ((rc = check_call(a, work, false))) return rc;
    if (work_bytes < plan_bytes(pl)) return K2T_ENOMEM;
    if (a->n_queries == 0) return K2T_OK;
    fill_pointers(a, work, pl);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a->dtype == K2T_BF16 ? attn_forward_bf16(pl.p, pl.bm, st) : attn_forward_fp16(pl.p, pl.bm, st);
}

int k2t_attn_backward(const k2t_attn *a, void *work, uint64_t work_bytes, void *stream)
{
    int rc = check_sizes(a);
    if (rc) return rc;
    Plan pl;
    make_plan(a, true, pl);
    if ((rc = check_call(a, work, true))) return rc;
    if (work_bytes < plan_bytes(pl)) return K2T_ENOMEM;
    fill_pointers(a, work, pl);
    if (a->n_nodes && (!node_map(&pl.p.dk_map, a->dk, a->dk_row, a->dk_head, pl.p, a->dtype) ||
                       !node_map(&pl.p.dv_map, a->dv, a->dv_row, a->dv_head, pl.p, a->dtype)))
        return K2T_ECUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a->dtype == K2T_BF16 ? attn_backward_bf16(pl.p, st) : attn_backward_fp16(pl.p, st);
}

}  // extern "C"
