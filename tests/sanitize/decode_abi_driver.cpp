// The few-token entry points at the ends of their argument ranges, under AddressSanitizer and
// UndefinedBehaviorSanitizer.  Pointers are dummies that the library must never dereference.
#include <cstdint>
#include <cstdio>

#include "w8a8.h"

static int failures = 0;
#define EXPECT(call, want)                                                              \
  do {                                                                                  \
    const long long got = (long long)(call);                                            \
    if (got != (long long)(want)) {                                                     \
      std::fprintf(stderr, "%s:%d: %s -> %lld, expected %lld\n", __FILE__, __LINE__, #call, got, (long long)(want)); \
      ++failures;                                                                       \
    }                                                                                   \
  } while (0)

int main() {
  void* a = reinterpret_cast<void*>(0x10000);
  auto u16 = static_cast<uint16_t*>(a);
  auto u8 = static_cast<uint8_t*>(a);
  auto i8 = static_cast<int8_t*>(a);
  auto f = static_cast<float*>(a);
  auto i32 = static_cast<int32_t*>(a);
  const int64_t ends[] = {INT64_MIN, -1, 0, 1, 16, 128, 1 << 20, (int64_t)1 << 31, INT64_MAX};
  const w8a8_status DEV = W8A8_ERR_UNSUPPORTED_DEVICE;

  // every combination is refused or gets as far as the device check: no overflow on the way
  int64_t seen = 0;
  for (int64_t m : ends)
    for (int64_t n : ends)
      for (int64_t k : ends) {
        seen += w8a8_w4_linear(u16, u8, u16, u16, u16, m, n, k, 32, a, SIZE_MAX, nullptr) == DEV;
        (void)w8a8_w4_workspace_bytes(m, n, k);
        (void)w8a8_w4_code_bytes(n, k);
        (void)w8a8_w4_scale_bytes(n, k, 32);
        seen += w8a8_w4_quantize(u16, n, k, 64, u8, u16, nullptr) == DEV;
        seen += w8a8_w4_pack(u8, u16, n, k, 128, u8, u16, nullptr) == DEV;
        for (int64_t w : ends) {
          seen += w8a8_kv_append(u16, 1 << 20, u16, 1 << 20, i8, f, i8, f, n, i32, w, i32, m, k, 16, 128, 16, nullptr) == DEV;
          seen += w8a8_kv_append(u16, k, u16, k, i8, f, i8, f, 1, i32, 1, i32, m, 1, n, 64, w, nullptr) == DEV;
          seen += w8a8_kv_read(i8, f, i8, f, n, i32, w, i32, m, k, 16, 128, 16, u16, u16, nullptr) == DEV;
          seen += w8a8_kv_attention(u16, 1 << 20, i8, f, i8, f, n, i32, w, i32, m, k, 16, 1, 128, 16, 1.0f, u16, a, SIZE_MAX, nullptr) == DEV;
          seen += w8a8_kv_attention(u16, k, i8, f, i8, f, 1, i32, 1, i32, 1, m, n, w, 64, 16, 1.0f, u16, a, SIZE_MAX, nullptr) == DEV;
          (void)w8a8_kv_attention_workspace_bytes(m, n, k, w, 64, 16, 9);
          (void)w8a8_kv_attention_workspace_bytes(1, 1, 8, 8, m, n, k);
        }
      }
  EXPECT(seen > 0, 1);
  EXPECT(w8a8_w4_linear(u16, u8, u16, nullptr, u16, 1, 16, 256, 64, a, 4096, nullptr), DEV);
  EXPECT(w8a8_w4_linear(u16, u8, u16, nullptr, u16, 1, 12, 256, 64, a, 4096, nullptr), W8A8_ERR_BAD_SHAPE);
  if (failures == 0) std::printf("all argument checks as expected\n");
  return failures ? 1 : 0;
}
