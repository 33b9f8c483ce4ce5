/*
 * Exhaustive checks of the arithmetic by which the expert-layer kernels quantize (test
 * infrastructure; the device arithmetic of quant_f32.cuh restated in C, one IEEE rounding
 * per operation).
 *
 * 1. The scale: q = fl32(amax c), c = fl32(1/448), s = fma(fma(-q, 448, amax), c, q) must be
 *    fl32(amax / 448) for every BF16 amax in the window [2^-90, 2^100], and for every FP32
 *    mantissa at several exponents of it.
 * 2. The codes: for every such BF16 amax and every BF16 x with |x| <= amax, with a = fl32(1 / s),
 *      r = fl32(a (1 - 2^-21)), e = fma(-s, r, 1), r_lo = fl32(fma(e, e, e) r),
 *      q = fma(x, r, fl32(x r_lo))
 *    must have the E4M3 code of fl32(x / s), and r_lo must be positive.  The kernel's a is an
 *    approximation, so a one and two units to either side is tried too, for every eighth
 *    exponent of amax (the arithmetic does not change with a power of two).  The same for -x
 *    with s, r and r_lo negated, as the activation kernels have it.
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

static float step_by(float v, int units)
{
    uint32_t u;
    memcpy(&u, &v, 4);
    u += (uint32_t)units;  /* positive, far from the ends */
    memcpy(&v, &u, 4);
    return v;
}

static float scale_of(float amax)
{
    const float c = 1.0f / 448.0f, q = amax * c;
    return fmaf(fmaf(-q, 448.0f, amax), c, q);
}

int main(void)
{
    long long bad = 0, pairs = 0, scales = 0;
    for (int ex = -90; ex < 100; ex += 27) {
#pragma omp parallel for reduction(+ : bad, scales)
        for (uint32_t m = 0; m < (1u << 23); ++m) {
            const uint32_t u = ((uint32_t)(127 + ex) << 23) | m;
            float amax;
            memcpy(&amax, &u, 4);
            ++scales;
            if (scale_of(amax) != amax / 448.0f) ++bad;
        }
    }
#pragma omp parallel for schedule(dynamic, 64) reduction(+ : bad, pairs)
    for (uint32_t ah = 1; ah < 0x7F80u; ++ah) {
        const float amax = bf16(ah);
        if (!(amax >= 0x1p-90f && amax <= 0x1p100f)) continue;
        const float s = scale_of(amax);
        if (s != amax / 448.0f) ++bad;
        const int wide = ((ah >> 7) & 7u) == 0;
        for (int d = wide ? -2 : 0; d <= (wide ? 2 : 0); ++d) {
            const float r = step_by(1.0f / s, d) * (1.0f - 0x1p-21f);
            const float e = fmaf(-s, r, 1.0f), r_lo = fmaf(e, e, e) * r;
            if (!(r_lo > 0.0f)) ++bad;
            for (uint32_t xm = 0; xm <= ah; ++xm) {
                for (uint32_t sg = 0; sg < 2; ++sg) {
                    const float x = bf16(xm | (sg << 15)), n = -x;
                    const float q = fmaf(x, r, x * r_lo), q2 = fmaf(n, -r, n * -r_lo);
                    if (q != q2 || signbit(q) != signbit(x) || signbit(q2) != signbit(x)) ++bad;
                    const uint8_t got = e4m3(q), want = e4m3(x / s);
                    ++pairs;
                    if (got != want) {
                        ++bad;
                        if (bad <= 5) {
#pragma omp critical
                            printf("mismatch amax 0x%04x x 0x%04x r %+d: got 0x%02x want 0x%02x\n", ah,
                                   xm | (sg << 15), d, got, want);
                        }
                    }
                }
            }
        }
    }
    printf("scales %lld pairs %lld\n", scales, pairs);
    printf("mismatches %lld\n", bad);
    return bad != 0;
}
