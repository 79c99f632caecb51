// swa_q8_decode_64.cu - the kernels of swa_q8_decode.cuh for d = 64 (a file to a head
// dimension, so that they compile side by side).
#include "swa_q8_decode.cuh"

namespace swa {
cudaError_t launch_q8_decode_64(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  return launch_d<64>(p, maps, stream);
}
}  // namespace swa
