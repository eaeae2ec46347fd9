/* Host model of the quantizers' corrected quotient (packed FP32 on the device:
 * one product, two fused multiply-adds), for the test that compiles it.
 *   y  = the FP32 reciprocal of s, rounded to nearest, negated
 *   q0 = x y,  r = x + q0 s,  q1 = r y + q0,  result -q1
 * `y` may be moved by `nudge` ulps to show what the check on it is for.
 */
#include <math.h>
#include <stdint.h>

static float reciprocal(float s) {
  /* correctly rounded: the double quotient has 29 spare bits, and 1/s is never
   * within 2^-49 of a rounding midpoint of FP32 */
  return (float)(1.0 / (double)s);
}

/* the device's exact check that y is within half an ulp of 1/s */
int reciprocal_ok(float s, float y) {
  float e = fmaf(-s, y, 1.0f);
  int x;
  (void)frexpf(y, &x); /* y in [2^(x-1), 2^x) */
  float half_ulp = ldexpf(1.0f, x - 1 - 24);
  return fabsf(e) <= s * half_ulp;
}

void quotients(const float* x, const float* s, int64_t n, int nudge, float* out, uint8_t* ok) {
  for (int64_t i = 0; i < n; ++i) {
    float y = reciprocal(s[i]);
    for (int k = 0; k < (nudge < 0 ? -nudge : nudge); ++k) y = nextafterf(y, nudge < 0 ? 0.0f : INFINITY);
    ok[i] = (uint8_t)reciprocal_ok(s[i], y);
    float ny = -y;
    float q0 = x[i] * ny;
    float r = fmaf(q0, s[i], x[i]);
    out[i] = -fmaf(r, ny, q0);
  }
}
