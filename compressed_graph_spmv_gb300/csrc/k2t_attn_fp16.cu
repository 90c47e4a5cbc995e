// k2t_attn_fp16.cu -- attention kernels for one element type (compiled in
// parallel with the other).
#include "k2t_attn_launch.cuh"

namespace k2t {

int attn_forward_fp16(const AttnParams &p, int bm, cudaStream_t st) { return launch_forward<__half>(p, bm, st); }
int attn_backward_fp16(const AttnParams &p, cudaStream_t st) { return launch_backward<__half>(p, st); }

}  // namespace k2t
