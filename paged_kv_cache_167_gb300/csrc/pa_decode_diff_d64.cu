// pa_decode_diff_d64.cu -- differential decode attention, heads of 64 components
// (keys and values of a pair: 128).
#include "pa_decode_kernel.cuh"

namespace pa {

cudaError_t launch_decode_diff_d64(const DecodeArgs &a, cudaStream_t stream) {
    return decode::launch_diff_for_dim<128>(a, stream);
}

}  // namespace pa
