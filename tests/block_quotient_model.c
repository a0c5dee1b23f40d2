/* The quotient that the norm and activation kernels encode, beside FP8's borders.
 *
 * A block's values v are divided by its scale s without a division. With the
 * correctly rounded reciprocal rs = RN(1 / s), all signs turned so that a zero
 * keeps its own:
 *     p = RN(v * -rs);  r = RN(fma(p, s, v));  -q = RN(fma(r, -rs, p))
 * which is Markstein's correction of v * rs. The FP8 code of q can differ from
 * that of the correctly rounded v / s only where a border between two codes (a
 * value half way between FP8 neighbours) lies between the two or is one of them.
 * Both are within 2 units of FP32's last place of v / s, so only those v matter
 * that lie within 4 units of border * s.
 *
 * This program takes every mantissa of s and every mantissa that a border or an
 * FP8 value of E4M3 or E5M2 can have (m / 16, m = 16 .. 31), with the 9 values of
 * v around each product, and compares q with v / s bit for bit. Exponents only
 * scale all of it, since the kernels use the form where nothing over- or
 * underflows. It also counts where v * rs alone falls on another side of the
 * border than v / s.
 *
 * Exit status 0 means no q differs. The one argument is the step between
 * mantissas (1: all). Build with -ffp-contract=off.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static float from_bits(uint32_t u) {
  float f;
  memcpy(&f, &u, 4);
  return f;
}

static uint32_t bits_of(float f) {
  uint32_t u;
  memcpy(&u, &f, 4);
  return u;
}

static int side(float q, float border) { return (q > border) - (q < border); }

int main(int argc, char** argv) {
  const uint32_t step = argc > 1 ? (uint32_t)atoi(argv[1]) : 1;
  long long pairs = 0, bad = 0, wrong_side = 0;
#pragma omp parallel for schedule(dynamic, 4096) reduction(+ : pairs, bad, wrong_side)
  for (uint32_t m = 0; m < (1u << 23); m += step) {
    const float s = from_bits(0x3F800000u | m);
    volatile float one = 1.0f;
    const float rs = one / s;
    for (int b = 16; b < 32; ++b) {
      const float border = (float)b / 16.0f;
      const uint32_t near = bits_of(border * s);
      for (int d = -4; d <= 4; ++d) {
        const float v = from_bits(near + (uint32_t)d);
        volatile float sv = s;
        const float want = v / sv;
        const float p = v * -rs;
        const float r = fmaf(p, s, v);
        const float q = -fmaf(r, -rs, p);
        pairs++;
        bad += bits_of(q) != bits_of(want);
        wrong_side += side(v * rs, border) != side(want, border);
      }
    }
  }
  printf("%lld pairs, %lld differ; the product alone is on another side of a border %lld times\n", pairs, bad, wrong_side);
  return bad != 0 || wrong_side == 0;
}
