// Host quantizer of dense weights into 4-bit codes with a step and a minimum
// per group, by the library's quantizer rule at width 4: in IEEE float32
// without fused operations, s = fp16_rne((max - min) / 15), s = 1 if that is
// 0, m = fp16_rne(min), q = clamp(nearbyint((w - m) / s), 0, 15).
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "bitsmoe.h"
#include "common.h"

namespace bitsmoe {
namespace {

// float32 to float16 bits, to nearest with ties to even, for |v| < 65520.
uint16_t half_bits(float v) {
  uint32_t u;
  memcpy(&u, &v, 4);
  const uint16_t sign = (uint16_t)((u >> 16) & 0x8000u);
  const uint32_t a = u & 0x7FFFFFFFu;
  if (a < 0x38800000u) {  // below 2^-14: steps of 2^-24
    float f;
    memcpy(&f, &a, 4);
    return (uint16_t)(sign | (uint16_t)nearbyintf(f * 16777216.0f));
  }
  const uint32_t r = a + 0xFFFu + ((a >> 13) & 1u);
  return (uint16_t)(sign | ((r >> 13) - (112u << 10)));
}

float half_value(uint16_t h) {
  const int ex = (h >> 10) & 31, man = h & 1023;
  const float v = ex ? ldexpf(1.0f + (float)man / 1024.0f, ex - 15) : ldexpf((float)man, -24);
  return h & 0x8000u ? -v : v;
}

}  // namespace
}  // namespace bitsmoe

using namespace bitsmoe;

extern "C" int bitsmoe_w4_pack(const float* w, int64_t rows, int K, int G, uint8_t* codes,
                               uint16_t* scales, uint16_t* mins) {
  if (rows < 0 || K < 1) return fail(BITSMOE_ESHAPE, "rows=%lld K=%d", (long long)rows, K);
  if (G != 32 && G != 64 && G != 128) return fail(BITSMOE_ESHAPE, "G=%d (32, 64 or 128)", G);
  if (K % G) return fail(BITSMOE_ESHAPE, "K=%d is not a multiple of G=%d", K, G);
  if (rows && (!w || !codes || !scales || !mins)) return fail(BITSMOE_EINVAL, "null pointer argument");
  const int64_t groups = rows * (K / G);
  for (int64_t g = 0; g < groups; ++g) {
    const float* p = w + g * G;
    float lo = p[0], hi = p[0];
    for (int i = 0; i < G; ++i) {
      if (!(fabsf(p[i]) <= 60000.0f))
        return fail(BITSMOE_EBITS, "a weight is not finite or beyond 60000");
      lo = p[i] < lo ? p[i] : lo;
      hi = p[i] > hi ? p[i] : hi;
    }
    scales[g] = half_bits((hi - lo) / 15.0f);
    if (scales[g] == 0) scales[g] = 0x3C00;
    mins[g] = half_bits(lo);
    const float s = half_value(scales[g]), m = half_value(mins[g]);
    for (int i = 0; i < G; i += 2) {
      int q[2];
      for (int j = 0; j < 2; ++j) {
        const float v = nearbyintf((p[i + j] - m) / s);
        q[j] = v < 0.0f ? 0 : v > 15.0f ? 15 : (int)v;
      }
      codes[(g * G + i) / 2] = (uint8_t)(q[0] | q[1] << 4);
    }
  }
  return BITSMOE_OK;
}
