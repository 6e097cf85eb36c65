// pa_decode_diff_d128.cu -- differential decode attention, heads of 128 components
// (keys and values of a pair: 256).
#include "pa_decode_kernel.cuh"

namespace pa {

cudaError_t launch_decode_diff_d128(const DecodeArgs &a, cudaStream_t stream) {
    return decode::launch_diff_for_dim<256>(a, stream);
}

}  // namespace pa
