// The paged decode kernel's instantiations for 128-dim keys and 128-dim values.
#include "paged_decode.cuh"

namespace saga {
cudaError_t launch_paged_decode_d128(const PagedDecodeArgs& a, int sms, cudaStream_t stream) {
    return run_shape<128, 128>(a, sms, stream);
}
}  // namespace saga
