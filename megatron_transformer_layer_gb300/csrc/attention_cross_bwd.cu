// Attention to keys of another length, backward: not in this build yet, the
// entry point refuses every call.
#include "attention_cross.cuh"

namespace mc {

size_t attention_cross_ws_bytes(const mc_cross_attention&) { return 16; }
int launch_attention_cross_bwd(const uint16_t*, const uint16_t*, const uint16_t*, const uint16_t*,
                               const float*, const uint16_t*, uint16_t*, uint16_t*, uint16_t*,
                               float*, const mc_cross_attention&, uint8_t*, size_t, int*,
                               cudaStream_t) {
  return MC_ERR_UNSUPPORTED;
}

}  // namespace mc
