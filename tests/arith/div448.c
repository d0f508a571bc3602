/* The block quantizer's scale a / 448 by q = a c, c = fl(1 / 448), and one correction q + (a - 448 q) c, against the IEEE
 * quotient: every fp32 mantissa, in the smallest, some middle and the largest binades of a in [2^-96, 2^128). */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

int main(void) {
  static const int exps[] = {-96, -95, -94, -60, -1, 0, 1, 2, 3, 60, 126, 127};
  const float c = 1.0f / 448.0f;
  uint64_t bad = 0;
  for (unsigned i = 0; i < sizeof exps / sizeof *exps; ++i)
    for (uint32_t m = 0; m < (1u << 23); ++m) {
      const uint32_t u = ((uint32_t)(exps[i] + 127) << 23) | m;
      float a;
      memcpy(&a, &u, 4);
      const float q = a * c, r = fmaf(-448.0f, q, a), s = fmaf(r, c, q);
      bad += s != a / 448.0f;
    }
  printf("%llu mismatches\n", (unsigned long long)bad);
  return bad != 0;
}
