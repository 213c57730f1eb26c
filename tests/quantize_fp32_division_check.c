/* The block norm forms v / s for fp32 values v as t = v * y, then
 * t' = fma(-fma(t, s, -v), y, t), y = 1 / s, s = max(amax, 1e-12) / 127 (int8)
 * or / 448 (E4M3).  Next to every boundary between two codes (the seven fp32
 * values around it), for random maxima, t' must lie on the same side of the
 * boundary as the correctly rounded v / s; and a zero must keep v's sign.
 * Arguments: maxima, seed.  Prints the pairs checked; exits 1 on a difference. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static uint64_t state;
static uint64_t next(void) {
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state;
}
static float from_bits(uint32_t b) {
    float f;
    memcpy(&f, &b, 4);
    return f;
}
static uint32_t to_bits(float f) {
    uint32_t b;
    memcpy(&b, &f, 4);
    return b;
}
static float quotient(float v, float s, float y) {
    const float t = v * y;
    volatile float r = fmaf(t, s, -v); /* gcc makes one instruction of it and its negation, which loses a zero's sign */
    return fmaf(-r, y, t);
}
static int side(float t, double at) { return (t > at) - (t < at); }

int main(int argc, char **argv) {
    if (argc != 3) return 2;
    const long maxima = atol(argv[1]);
    state = 88172645463325252ULL + (uint64_t)atol(argv[2]) * 0x9E3779B97F4A7C15ULL;
    double at[2][256];
    int n[2] = {0, 0};
    for (int k = 0; k < 127; ++k) at[0][n[0]++] = k + 0.5;
    for (int m = 0; m < 8; ++m) at[1][n[1]++] = ldexp(m + 0.5, -9);   /* subnormal codes */
    for (int e = -6; e <= 8; ++e)
        for (int m = 0; m < 8; ++m) at[1][n[1]++] = ldexp(8 + m + 0.5, e - 3);
    long pairs = 0;
    for (long i = 0; i < maxima; ++i) {
        /* every other one between 1/2 and 64, the rest of any finite size */
        const uint32_t b = i & 1 ? 0x3f000000u + (uint32_t)(next() % 0x03800000u) : (uint32_t)(next() % 0x7f800000u);
        const float amax = from_bits(b);
        for (int f = 0; f < 2; ++f) {
            const float s = fmaxf(amax, 1e-12f) / (f ? 448.0f : 127.0f), y = 1.0f / s;
            if (signbit(quotient(0.0f, s, y)) || !signbit(quotient(-0.0f, s, y))) return 1;
            for (int j = 0; j < n[f]; ++j) {
                const uint32_t x = to_bits((float)(at[f][j] * (double)s));
                for (int d = -3; d <= 3; ++d) {
                    const float v = from_bits(x + d);
                    if (!(v <= amax)) continue;
                    if (side(quotient(v, s, y), at[f][j]) != side(v / s, at[f][j])) {
                        printf("amax %a v %a: %a, not %a\n", amax, v, quotient(v, s, y), v / s);
                        return 1;
                    }
                    ++pairs;
                }
            }
        }
    }
    printf("%ld\n", pairs);
    return 0;
}
