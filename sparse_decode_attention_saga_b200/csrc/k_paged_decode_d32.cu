// The paged decode kernel's instantiations for 32-dim keys and 64-dim values.
#include "paged_decode.cuh"

namespace saga {
cudaError_t launch_paged_decode_d32(const PagedDecodeArgs& a, int sms, cudaStream_t stream) {
    return run_shape<32, 64>(a, sms, stream);
}
}  // namespace saga
