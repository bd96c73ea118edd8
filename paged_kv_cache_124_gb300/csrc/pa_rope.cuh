// What the kernels of norm, rotation and cache write share: their arguments
// and a thread's part of a head, 16 elements in packed fp32 pairs.
#pragma once

#include "pa_common.cuh"

namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    uint4* q_out;
    uint8_t* k_cache;
    uint8_t* v_cache;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    long long q_stride, k_stride, v_stride;            // elements between tokens
    const float* q_weight;
    const float* k_weight;
    const float* cos_sin;                              // [max_positions][rot_dim]: cosines, then sines
    const int32_t* positions;                          // [axes][num_tokens]
    const int64_t* slots;
    int32_t* status;
    long long num_slots;
    float eps, k_scale, v_scale;
    int max_positions, rot_dim, num_tokens, n_q_heads, n_kv_heads, block_size;
    int num_axes;
    uint32_t axes[4];                                  // 2 bits a pair: the axis whose position turns it
};

// A token's positions.
template <bool kAxes>
struct Where {
    int p[kAxes ? 4 : 1];
    __device__ __forceinline__ void load(const RopeArgs& a, size_t t) {
        p[0] = a.positions[t];
        if constexpr (kAxes) {
#pragma unroll
            for (int x = 1; x < 4; ++x) p[x] = x < a.num_axes ? a.positions[(size_t)x * a.num_tokens + t] : p[0];
        }
    }
    __device__ __forceinline__ int lowest() const {
        if constexpr (kAxes) return min(min(p[0], p[1]), min(p[2], p[3]));
        else return p[0];
    }
    __device__ __forceinline__ int highest() const {
        if constexpr (kAxes) return max(max(p[0], p[1]), max(p[2], p[3]));
        else return p[0];
    }
    __device__ __forceinline__ int of(uint32_t axis) const {
        if constexpr (kAxes) return axis & 2 ? (axis & 1 ? p[3] : p[2]) : (axis & 1 ? p[1] : p[0]);
        else return p[0];
    }
};

// Two fp32 values in a register pair, for packed arithmetic.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t r) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
    return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// A thread's 16 elements of a head as 8 pairs: f[i] (i < 4) from the first
// chunk, f[i + 4] from the second.
struct Part {
    uint64_t f[8];
};

__device__ __forceinline__ void unpack8(uint4 x, uint64_t* f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const uint64_t* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpair(f[i]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 codes8(const uint64_t* f, float scale) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpair(f[i]);
        c[i] = pa::e4m3x2(__fdiv_rn(v.x, scale), __fdiv_rn(v.y, scale));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ void load8(const float* p, uint64_t* f) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = pair(a.x, a.y);
    f[1] = pair(a.z, a.w);
    f[2] = pair(b.x, b.y);
    f[3] = pair(b.z, b.w);
}

// Which of a head's 16-byte chunks thread l of it holds: pairs (c, c +
// rot_dim / 2) take one from each half of the rotated part, all else two
// neighbours.
template <bool kInterleaved>
struct Place {
    bool turns;
    int c0, c1;
    __device__ __forceinline__ Place(int l, int rot_dim) {
        turns = l < rot_dim >> 4;
        c0 = !kInterleaved && turns ? l : 2 * l;
        c1 = !kInterleaved && turns ? l + (rot_dim >> 4) : 2 * l + 1;
    }
};

// Cosines and sines of pairs 8 l .. 8 l + 7 (l < rot_dim / 16): from one row
// of the table, or, where the pairs are of several axes, from a row each.
template <bool kAxes>
__device__ __forceinline__ void load_angles(const RopeArgs& a, const Where<kAxes>& at, int l, uint64_t* cs, uint64_t* sn) {
    const int half = a.rot_dim >> 1;
    uint32_t code = 0;
    if constexpr (kAxes) code = a.axes[l >> 1] >> (16 * (l & 1)) & 0xffffu;
    if (!kAxes || code == (code & 3u) * 0x5555u) {
        const float* tab = a.cos_sin + (size_t)at.of(code & 3u) * a.rot_dim + 8 * l;
        load8(tab, cs);
        load8(tab + half, sn);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* x = a.cos_sin + (size_t)at.of(code >> (4 * i) & 3u) * a.rot_dim + 8 * l + 2 * i;
            const float* y = a.cos_sin + (size_t)at.of(code >> (4 * i + 2) & 3u) * a.rot_dim + 8 * l + 2 * i + 1;
            cs[i] = pair(__ldg(x), __ldg(y));
            sn[i] = pair(__ldg(x + half), __ldg(y + half));
        }
    }
}

// y = x * rsqrt(mean(x^2) + eps) * gain over a head's kLanes threads (mask).
template <int kLanes>
__device__ __forceinline__ void norm_part(Part& p, const uint64_t* gain, float eps, unsigned mask) {
    uint64_t sum = mul2(p.f[0], p.f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) sum = fma2(p.f[i], p.f[i], sum);
    const float2 two = unpair(sum);
    float s = two.x + two.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(mask, s, o);
    const float inv = rsqrtf(s * (1.f / (16 * kLanes)) + eps);
    const uint64_t ii = pair(inv, inv);
#pragma unroll
    for (int i = 0; i < 8; ++i) p.f[i] = mul2(mul2(p.f[i], ii), gain[i]);
}

// (a, b) -> (a cos - b sin, b cos + a sin) for the thread's 8 pairs.
template <bool kInterleaved>
__device__ __forceinline__ void turn_part(Part& p, const uint64_t* cs, const uint64_t* sn) {
    if constexpr (kInterleaved) {
        // pair i is (f[i].x, f[i].y)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = unpair(p.f[i]), cc = unpair(cs[i >> 1]), ss = unpair(sn[i >> 1]);
            const float c = i & 1 ? cc.y : cc.x, s = i & 1 ? ss.y : ss.x;
            p.f[i] = fma2(pair(f.y, f.x), pair(-s, s), mul2(p.f[i], pair(c, c)));
        }
    } else {
        // pairs are (f[i], f[i + 4]), two at a time
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t x = p.f[i], y = p.f[i + 4];
            const float2 s = unpair(sn[i]);
            p.f[i] = fma2(y, pair(-s.x, -s.y), mul2(x, cs[i]));
            p.f[i + 4] = fma2(x, sn[i], mul2(y, cs[i]));
        }
    }
}

// The map of the pairs' axes, from num_axes >= 1 and axis_of_pair (host,
// [rot_dim / 2]); false: an axis out of range.
inline bool set_axes(RopeArgs& a, int num_axes, const int8_t* axis_of_pair, int rot_dim) {
    a.num_axes = num_axes;
    for (int c = 0; c < rot_dim / 2; ++c) {
        if (axis_of_pair[c] < 0 || axis_of_pair[c] >= num_axes) return false;
        a.axes[c >> 4] |= (uint32_t)axis_of_pair[c] << (2 * (c & 15));
    }
    return true;
}

}  // namespace
