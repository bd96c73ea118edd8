// Scores capped by a tanh: cap tanh(x / cap), in units of log2 (x, cap and the
// result times log2(e)).  Around zero by tanh's series, up to x^9 (the next
// term is 5e-8 of it at 0.3), beyond by 1 - 2 / (e^2x + 1), which would cancel
// there: relative errors below 1e-6 (cap_scores: also 2^-22 of the cap).  (The hardware's tanh is off by 2^-11,
// which a cap of 50 makes 0.02 of a score.)
#pragma once

#include "pa_common.cuh"

namespace pa {

// A bias by distance, in units of log2, for a row that sees positions lo .. hi - 1: the distance to the nearest of them is
// the same in all its scores and leaves its softmax alone, so it is left out: slope |p - j| less slope |p - p'| is
// slope |p' - j| for the seen position p' nearest to p.  (Far from what it sees, a row's scores would lose as many bits as
// the distance has.)
__device__ __forceinline__ int bias_from(int pos, int lo, int hi) { return min(max(pos, lo), hi - 1); }
// Beyond this one position, the nearest or the farthest, has all of the weight; times 2^31 it is finite.
constexpr float kMostSlope = 1e28f;
__device__ __forceinline__ float bias_slope(float slope) { return fminf(fmaxf(1.4426950408889634f * slope, -kMostSlope), kMostSlope); }

// Caps below 1e-30 (in units of log2) are taken for it: the inverse has to be finite for scores of 0.
constexpr float kMostCapInv = 1e30f;
// Scores u = s by beyond these are not taken for near zero, as the polynomials' coefficients would not be finite.
constexpr float kMostNearBy = 1e6f;

__device__ __forceinline__ float capped(float x, float cap_log2, float cap_inv) {
    const float u = x * cap_inv, v = u * u;
    const float p = fmaf(fmaf(fmaf(fmaf(v, 62.f / 2835.f, -17.f / 315.f), v, 2.f / 15.f), v, -1.f / 3.f), v, 1.f);
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u * 2.8853900817779268f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
    return cap_log2 * (fabsf(u) < 0.3f ? u * p : fmaf(-2.f, r, 1.f));
}

// Two floats in a register pair: both of x; a b; a b + c.
__device__ __forceinline__ uint64_t pair_of(float x) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// The largest magnitude of s (of NaN none).
template <int n>
__device__ __forceinline__ float largest(const float (&s)[n]) {
    float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < n; i += 2)
        asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %1;\n\tabs.f32 y, %2;\n\tmax.f32 %0, %0, x, y;\n\t}"
            : "+f"(top[i / 2 & 3])
            : "f"(s[i]), "f"(s[i + 1]));
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}

// The cap within a quarter of it, cap tanh(c2 s / cap) = s p(s^2): tanh(u) / u
// fitted on [0, 0.25] with even ripple (relative 4e-7) by a polynomial in u^2,
// the scales of u folded into its coefficients.
struct NearCap {
    float q0, q1, q2;
    __device__ __forceinline__ NearCap(float c2, float cap_inv) {
        const float by = c2 * cap_inv, w = by * by;
        q0 = c2 * 0.999999604f;
        q1 = c2 * w * -0.333219082f;
        q2 = c2 * w * w * 0.128416134f;
    }
    __device__ __forceinline__ float operator()(float s) const {
        const float v = s * s;
        return s * fmaf(fmaf(q2, v, q1), v, q0);
    }
};

// n scores s (times c2; cap_inv is 1 / cap_log2), the largest of which is top.  Where all of this thread's are
// within half of the cap, by a polynomial in s^2 alone, in packed pairs:
// tanh(u) / u fitted on [0, 0.5] with even ripple (relative 6e-7), the scales
// of u folded into its coefficients.  (By thread, not by warp, so that a row's
// form is its own; scores that a row does not see come as zeros, for the same.)
template <int n>
__device__ __forceinline__ void cap_scores(float (&s)[n], float top, float c2, float cap_log2, float cap_inv) {
    const float by = c2 * cap_inv, w = by * by;
    const bool far = !(top * fabsf(by) < 0.5f && fabsf(by) < kMostNearBy);
    if (!far) {
        const uint64_t q0 = pair_of(c2 * 0.999999456f), q1 = pair_of(c2 * w * -0.3332632f), q2 = pair_of(c2 * w * w * 0.131903234f),
                       q3 = pair_of(c2 * w * w * w * -0.0444030606f);
#pragma unroll
        for (int i = 0; i < n; i += 2) {
            uint64_t x;
            asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(s[i]), "f"(s[i + 1]));
            const uint64_t v = pair_mul(x, x), y = pair_mul(x, pair_fma(pair_fma(pair_fma(q3, v, q2), v, q1), v, q0));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(s[i]), "=f"(s[i + 1]) : "l"(y));
        }
        return;
    }
    // else by the second form of `capped` alone, which is within 2^-22 of the cap
    const float to = by * 2.8853900817779268f;
#pragma unroll
    for (int i = 0; i < n; ++i) {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s[i] * to));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
        s[i] = fmaf(-2.f * cap_log2, r, cap_log2);
    }
}

}  // namespace pa
