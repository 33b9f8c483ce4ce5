/*
 * Exhaustive check of the E4M3 conversion by a corrected quotient (test infrastructure;
 * the device arithmetic of quant_f32.cuh restated in C, one IEEE rounding per operation).
 *
 * For every block maximum amax among the positive finite BF16 values whose scale
 * s = fl32(amax / 448) lies in the window [2^-100, 2^100], and every BF16 x with
 * |x| <= amax:
 *   r = fl32(1 / s), z = fl32(x * -r), e = fma(z, s, x), q = fma(e, -r, z)
 * must have, but for its sign, the E4M3 code of fl32(x / s): z is the negative of the
 * quotient's first approximation, and with this order of signs a zero keeps its own.
 * Prints the number of mismatches.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

static uint8_t e4m3(float v)
{
    uint32_t u;
    memcpy(&u, &v, 4);
    uint8_t sign = (uint8_t)((u >> 31) << 7);
    uint32_t mag = u & 0x7FFFFFFFu;
    float a;
    memcpy(&a, &mag, 4);
    if (a > 448.0f) return sign | 0x7E;
    if (a < 0x1p-6f) return sign | (uint8_t)rintf(a * 512.0f);
    int32_t e = (int32_t)((mag >> 23) & 0xFF) - 127;
    uint32_t m3 = (mag >> 20) & 7u, rem = mag & 0xFFFFFu;
    if (rem > 0x80000u || (rem == 0x80000u && (m3 & 1u))) ++m3;
    if (m3 == 8u) { m3 = 0; ++e; }
    return sign | (uint8_t)(((uint32_t)(e + 7) << 3) | m3);
}

static float bf16(uint32_t h)
{
    uint32_t u = h << 16;
    float f;
    memcpy(&f, &u, 4);
    return f;
}

int main(void)
{
    long long bad = 0, pairs = 0;
#pragma omp parallel for schedule(dynamic, 64) reduction(+ : bad, pairs)
    for (uint32_t ah = 1; ah < 0x7F80u; ++ah) {
        const float s = bf16(ah) / 448.0f;
        if (!(s >= 0x1p-100f && s <= 0x1p100f)) continue;
        const float r = 1.0f / s;
        for (uint32_t xm = 0; xm <= ah; ++xm) {
            for (uint32_t sg = 0; sg < 2; ++sg) {
                const float x = bf16(xm | (sg << 15));
                const float z = x * -r;
                const float e = fmaf(z, s, x);
                const uint8_t got = e4m3(fmaf(e, -r, z)) ^ 0x80, want = e4m3(x / s);
                ++pairs;
                if (got != want) {
                    ++bad;
                    if (bad <= 5) {
#pragma omp critical
                        printf("mismatch amax 0x%04x x 0x%04x: got 0x%02x want 0x%02x\n", ah, xm | (sg << 15), got,
                               want);
                    }
                }
            }
        }
    }
    printf("pairs %lld\n", pairs);
    printf("mismatches %lld\n", bad);
    return bad != 0;
}
