// The paged decode kernel's instantiations for 64-dim keys and 64-dim values.
#include "paged_decode.cuh"

namespace saga {
cudaError_t launch_paged_decode_d64(const PagedDecodeArgs& a, int sms, cudaStream_t stream) {
    return run_shape<64, 64>(a, sms, stream);
}
}  // namespace saga
