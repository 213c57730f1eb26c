/* The int8 token quantiser forms x / s as t = x * y, t' = fma(fma(-t, s, x), y, t)
 * with y = 1 / s and s = amax / 127.  For every bf16 (argument "bf16") or fp16
 * ("fp16") maximum in the range given and every x of at most that magnitude
 * (signs are symmetric), the rounded, clamped result must be the one of the
 * correctly rounded x / s.  Prints the number of pairs checked; exits 1 on a
 * difference. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static float from_bits(int fp16, uint32_t b) {
    if (fp16) {
        const int e = (int)(b >> 10), m = (int)(b & 1023);
        return e == 0 ? ldexpf((float)m, -24) : ldexpf((float)(1024 + m), e - 25);
    }
    uint32_t w = b << 16;
    float f;
    memcpy(&f, &w, 4);
    return f;
}

int main(int argc, char **argv) {
    if (argc != 4) return 2;
    const int fp16 = strcmp(argv[1], "fp16") == 0;
    const uint32_t top = fp16 ? 0x7c00u : 0x7f80u; /* the first non-finite pattern */
    const uint32_t lo = (uint32_t)atoi(argv[2]), step = (uint32_t)atoi(argv[3]);
    long long pairs = 0;
    for (uint32_t a = lo; a < top; a += step) {
        const float amax = from_bits(fp16, a);
        const float s = fmaxf(amax, 1e-12f) / 127.0f, y = 1.0f / s;
        for (uint32_t b = 0; b <= a; ++b) {
            const float x = from_bits(fp16, b);
            const float t = x * y, u = fmaf(fmaf(-t, s, x), y, t);
            const float want = rintf(fminf(x / s, 127.0f)), got = rintf(fminf(u, 127.0f));
            if (want != got) {
                printf("amax %a x %a: %a want %a\n", amax, x, got, want);
                return 1;
            }
            ++pairs;
        }
    }
    printf("%lld\n", pairs);
    return 0;
}
