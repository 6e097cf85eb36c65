// pa_rotary_axes.cu -- rotary positions of several axes: queries, keys and the slot
// writer.
#include "pa_rotate_kernel.cuh"

namespace pa {

cudaError_t launch_rotate_axes(void *out, const void *x, int64_t x_stride, const int64_t *positions,
                               int64_t num_tokens, int32_t num_heads, int32_t head_dim, const pa_rotary &rotary,
                               const AxesView &axes, cudaStream_t stream) {
    RotateParams p = rotate_params(out, x, x_stride, positions, num_heads, head_dim, rotary);
    return launch_rotate_any<false>(p, axes, rotary.rot_dim, (rotary.flags & PA_ROTARY_INTERLEAVED) != 0,
                                    num_tokens, stream);
}

cudaError_t launch_rotate_and_cache_axes(const PoolView &pool, void *q_out, const void *q, int64_t q_stride,
                                         const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                         const int64_t *positions, const int64_t *slots, int64_t num_tokens,
                                         int32_t num_q_heads, const pa_rotary &rotary, const AxesView &axes,
                                         cudaStream_t stream) {
    return launch_rotate_cache(pool, q_out, q, q_stride, k, k_stride, v, v_stride, positions, slots, num_tokens,
                               num_q_heads, rotary, axes, stream);
}

}  // namespace pa
