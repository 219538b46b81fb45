// Host-only stand-ins for the few-token launchers, for the sanitizer build of csrc/decode_api.cpp: no path
// reaches a launch without a gfx950 device; if one did, it would report an error.
#include "decode.h"

namespace w8a8 {

hipError_t launch_w4_quantize(const uint16_t*, int64_t, int64_t, int, uint8_t*, uint16_t*, hipStream_t) {
  return hipErrorInvalidValue;
}
hipError_t launch_w4_pack(const uint8_t*, const uint16_t*, int64_t, int64_t, int, uint8_t*, uint16_t*, hipStream_t) {
  return hipErrorInvalidValue;
}
hipError_t launch_w4_linear(const uint16_t*, const uint8_t*, const uint16_t*, const uint16_t*, uint16_t*, int64_t,
                            int64_t, int64_t, int, void*, hipStream_t) {
  return hipErrorInvalidValue;
}
int w4_splits(int64_t, int64_t) { return 3; }
hipError_t launch_kv_append(const KvCache&, const uint16_t*, int64_t, const uint16_t*, int64_t, int64_t, int64_t,
                            hipStream_t) {
  return hipErrorInvalidValue;
}
hipError_t launch_kv_read(const KvCache&, int64_t, int64_t, uint16_t*, uint16_t*, hipStream_t) {
  return hipErrorInvalidValue;
}
int64_t kv_attention_splits(int64_t, int64_t, int, int, int, int, int64_t) { return 2; }
hipError_t launch_kv_attention(const KvCache&, const uint16_t*, int64_t, int64_t, int64_t, int, float, uint16_t*,
                               void*, hipStream_t) {
  return hipErrorInvalidValue;
}

}  // namespace w8a8
