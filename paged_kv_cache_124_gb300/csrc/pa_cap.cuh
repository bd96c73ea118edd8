// Scores capped by a tanh: cap tanh(x / cap), in units of log2 (x, cap and the
// result times log2(e)).  Around zero by tanh's series, up to x^9 (the next
// term is 5e-8 of it at 0.3), beyond by 1 - 2 / (e^2x + 1), which would cancel
// there: relative errors below 1e-6.  (The hardware's tanh is off by 2^-11,
// which a cap of 50 makes 0.02 of a score.)
#pragma once

#include "pa_common.cuh"

namespace pa {

__device__ __forceinline__ float capped(float x, float cap_log2, float cap_inv) {
    const float u = x * cap_inv, v = u * u;
    const float p = fmaf(fmaf(fmaf(fmaf(v, 62.f / 2835.f, -17.f / 315.f), v, 2.f / 15.f), v, -1.f / 3.f), v, 1.f);
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u * 2.8853900817779268f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
    return cap_log2 * (fabsf(u) < 0.3f ? u * p : fmaf(-2.f, r, 1.f));
}

// n scores (times c2; cap_inv is 1 / cap_log2).  Where all of a warp's are
// within 0.3 of the cap, as nearly always, by the series alone, in packed pairs.
template <int n>
__device__ __forceinline__ void cap_scores(float (&s)[n], float c2, float cap_log2, float cap_inv) {
    float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < n; ++i) top[i & 3] = fmaxf(top[i & 3], fabsf(s[i]));
    const float by = c2 * cap_inv;
    const bool far = !(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * fabsf(by) < 0.3f);
    if (!__any_sync(0xffffffffu, far)) {
        const auto both = [](float lo, float hi) {
            uint64_t r;
            asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
            return r;
        };
        const auto mul = [](uint64_t a, uint64_t b) {
            uint64_t d;
            asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
            return d;
        };
        const auto fma = [](uint64_t a, uint64_t b, float c) {
            uint64_t d;
            asm("{\n\t.reg .b64 c;\n\tmov.b64 c, {%3, %3};\n\tfma.rn.f32x2 %0, %1, %2, c;\n\t}" : "=l"(d) : "l"(a), "l"(b), "f"(c));
            return d;
        };
#pragma unroll
        for (int i = 0; i < n; i += 2) {
            const uint64_t u = mul(both(s[i], s[i + 1]), both(by, by)), v = mul(u, u);
            uint64_t p = fma(v, both(62.f / 2835.f, 62.f / 2835.f), -17.f / 315.f);
            p = fma(p, v, 2.f / 15.f);
            p = fma(p, v, -1.f / 3.f);
            p = fma(p, v, 1.f);
            p = mul(mul(u, both(cap_log2, cap_log2)), p);
            asm("mov.b64 {%0, %1}, %2;" : "=f"(s[i]), "=f"(s[i + 1]) : "l"(p));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = capped(s[i] * c2, cap_log2, cap_inv);
}

}  // namespace pa
