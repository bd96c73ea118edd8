// The kernel of units of up to 16 rows (pa_decode_multi.cu says what it does
// and why), for plain scores and for shaped ones, and the host's choices
// around it that its callers share.
//
// Shaped: what a row sees (its interval, its bias) lies in shared memory, as
// registers are short.  Tiles wholly outside a unit's interval are not part
// of its work, and only those at its ends, or in units with a row that sees
// nothing, take a mask.  Block-scaled: a stage's scales are a lane's own load,
// passed on by shuffles; K's multiply the scores, V's the weights, relative to
// the largest that the row has seen so far, so that a weight fits f16.  64 decodes of 512 to 4,096
// positions, 32 query heads over 8 of 128: capped over bf16 99 us, 0.90 of the
// measured copy rate, block-scaled 64 us, 0.70 (nothing is full there, issue 44
// %, ALU 42 %, DRAM 58 %: with twelve warps an SM a tile's chain of codes to
// f16, scores, softmax and products is what they wait for); 96 through windows
// of 1,024 of 100 to 8,000 positions 38 us, 0.75 (a short call: starting, the
// first tiles and the joins are a part of it).
#pragma once

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pa_multi.cuh"

namespace {

using namespace pa_multi;

constexpr int kTile = 16;                  // positions per warp and step
constexpr int kRows = 16;                  // rows of a unit
constexpr int kWarpsPerSm = 12;
constexpr int kLog2WeightScale = 7;        // FP8: weights enter f16 products times 2^7 (at most 2^15)
constexpr float kWeightScale = 1 << kLog2WeightScale;
// A block's kWarps (4 or 12) warps split a step's positions, 16 each.  What
// its shares are counted in:
__host__ __device__ constexpr int step_of(int warps) { return warps * kTile; }
// Steps that starting and joining a unit is worth.  (64 requests of 512 to
// 4096 positions, 16 rows: 2, 5, 9 steps bf16 102.5, 103.9, 105.6 us; E4M3 of
// 500 to 4096 68.5, 64.1, 66.9.)
__host__ __device__ constexpr int cost_of(int warps, bool f8) { return warps == 12 ? 1 : f8 ? 5 : 3; }
// Steps per block, at least.
__host__ __device__ constexpr int least_of(int warps) { return warps == 12 ? 1 : 4; }
// Units of at most this many steps are not split where each has a block: 4
// requests of 4 tokens, 8 KV heads, whole units against shares and their
// merge: four warps 256 positions 9.3 / 11.0 us, 768 16.8 / 16.8, 1024 20.6 /
// 16.9; twelve 1024 13.9 / 13.3 (144 units 18.0 / 20.4), 1536 16.5 / 13.7.
__host__ __device__ constexpr int direct_of(int warps) { return warps == 12 ? 6 : 12; }

template <int D, bool F8, int kWarps>
struct Geo {
    static constexpr int kSlabs = F8 ? 1 : D / 64;               // 128-byte boxes per cache row
    static constexpr int kSlabBytes = kTile * 128;
    static constexpr int kTileBytes = kSlabs * kSlabBytes;       // K or V of one warp's tile
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRingBytes = 16 * 1024 * kWarps;
    static constexpr int kStages = kRingBytes / (kWarps * kStageBytes);
    // The joining of the warps' states takes the fp32 rows of the unit: one
    // stage of all key warps (bf16), or two (E4M3).
    static constexpr int kJoinStages = F8 ? 2 : 1;
    static constexpr int kAhead = kStages - kJoinStages;         // tiles of the next unit in flight meanwhile
    static constexpr int kQStride = 2 * D + 16;                  // bytes per row of q: ldmatrix rows hit distinct banks
    static constexpr int kSmem = 1024 + kRingBytes + kRows * (kQStride + 4) + kWarps * kRows * 8 +
                                 kWarps * kStages * 8;
    static constexpr int kSteps = D / 16;
    static_assert(kAhead >= 1, "the ring has to hold a tile of the next unit beside the join");
    static_assert(kJoinStages * kStageBytes == 4 * kRows * D, "a unit's states fill the join stages");
};

// Shaped units: what a row sees, the position that its bias counts from, and
// the bias' slope times log2(e).  In shared memory: few tiles need it, and registers are short.
struct Shape {
    int lo, hi, pos;
    float slope;
};
__device__ __forceinline__ Shape shape_of(const ShapedArgs& a, const ShapedUnit& u, int r) {
    Shape s;
    const int row = u.row0 + r, i = row >> a.log2_group;
    const bool real = i < u.n;
    s.pos = u.first + i;
    s.lo = 0;
    s.hi = real ? min(s.pos + 1, u.ctx) : u.ctx;                 // a row that is not there: any finite result will do
    if (a.visible && real) {
        const int2 v = a.visible[u.q0 + i];
        s.lo = max(v.x, 0);
        s.hi = max(min(v.y, u.ctx), 0);
    }
    s.pos = pa::bias_from(s.pos, s.lo, s.hi);
    s.slope = a.slopes ? pa::bias_slope(a.slopes[(u.kvh << a.log2_group) + (row & ((1 << a.log2_group) - 1))]) : 0.f;
    return s;
}

__device__ __forceinline__ bool visible(const MultiArgs& a, const Unit& u, int row, int pos) {
    if (pos >= u.ctx) return false;
    if (pos < u.first) return true;
    const int i = (u.row0 + row) >> a.log2_group;
    return i >= u.n || sees(words_of(a, u), i, pos - u.first);      // a row that is not there: any finite result will do
}

// One warp's running state: rows g and g + 8.
template <int D>
struct State {
    float m[2], l[2];
    int top[2];                            // block-scaled values: the largest scale's byte that the row has seen, 2^(byte - 127) being acc's unit
    float acc[D / 8][4];
    __device__ __forceinline__ void reset() {
        top[0] = top[1] = 0;
        m[0] = m[1] = kNone;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
    }
};

// Fold one tile (K at shared address ks, V at vs, positions t0 .. t0 + 15)
// into the warp's state.  qr: the rows of q as A operands; c[h]: score factor
// of rows g + 8 h.  scales (shaped, E4M3): the scale bytes of K and V of the
// tile's first 8 positions, then of the others.
// kEight: no unit has more than 8 rows, so rows 8 .. 15 of the matrix instructions stay empty and
// their softmax is left out.  Only block-scaled caches have this form, whose tiles' chains are the
// longest (64 decodes over mixed lengths 68.2 -> 63.1 us, 64 x 4096 105.7 -> 97.7 when it came); of
// bf16 caches the reads bound them.
template <int D, bool F8, class Args, bool kEight>
__device__ __forceinline__ void fold_tile(State<D>& st, uint32_t ks, uint32_t vs, const float (&c)[2], int t0, const Args& a,
                                          const typename Args::Unit& u, int lane, const uint32_t (&qr)[D / 16][4],
                                          const Shape* shape, uint32_t scales, bool masked) {
    constexpr bool kShaped = Args::kShaped;
    constexpr int kH = kEight ? 1 : 2;
    constexpr int kSlabBytes = kTile * 128, kSteps = D / 16;
    const int g = lane >> 2, t4 = lane & 3;
    // ldmatrix addresses.  K as B operand: keys (lane & 7) + 8 (lane >> 4), chunk + (lane >> 3 & 1);
    // V (transposed) as B: rows (lane & 7) + 8 (lane >> 3 & 1), chunk + (lane >> 4)
    const int k_row = (lane & 7) + ((lane >> 4) << 3), k_add = (lane >> 3) & 1;
    const int v_row = (lane & 7) + (((lane >> 3) & 1) << 3), v_add = lane >> 4;
    float s[2][4];                         // [keys 0-7, 8-15]: (g, 2 t4), (g, 2 t4 + 1), rows g + 8
#pragma unroll
    for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    auto score = [&](int kk, uint32_t b00, uint32_t b01, uint32_t b10, uint32_t b11) {
        pa::mma16816<F8>(s[0], qr[kk], b00, b01);
        pa::mma16816<F8>(s[1], qr[kk], b10, b11);
    };
    if constexpr (F8) {
        // a chunk of 16 codes is one k-step; lane (g, t4) gets codes 4 t4 .. 4 t4 + 3 of key g
#pragma unroll
        for (int j = 0; j < kSteps / 2; ++j) {
            uint32_t r[4], b[4][2];
            pa::ldsm4(ks + pa::swz128(k_row, 2 * j + k_add), r);
#pragma unroll
            for (int e = 0; e < 4; ++e) pa::e4m3x4_to_f16x4(r[e], b[e][0], b[e][1]);
            score(2 * j, b[0][0], b[0][1], b[2][0], b[2][1]);
            score(2 * j + 1, b[1][0], b[1][1], b[3][0], b[3][1]);
        }
    } else {
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
            uint32_t r[4];
            pa::ldsm4(ks + (kk >> 2) * kSlabBytes + pa::swz128(k_row, 2 * (kk & 3) + k_add), r);
            score(kk, r[0], r[1], r[2], r[3]);
        }
    }
    float by[2][2];                                    // block-scaled values: factors of the weights, of 8 positions each, by row
    float f[2][2];                                     // factors of the scores: of positions 8 n on, and row g + 8 h
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < kH; ++h) f[n][h] = kShaped && F8 ? fmaxf(c[h] * scale_of(scales >> (16 * n) & 0xff), 1e-37f) : c[h];   // never 0: masked scores stay -inf
    if constexpr (kShaped) {
        if constexpr (Args::kCurved) {                 // scores in units of log2 from here on
            const float slope[2] = {shape[g].slope, shape[g + 8].slope};
            const int at[2] = {shape[g].pos, shape[g + 8].pos};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2 * kH; ++e) {
                    s[n][e] *= f[n][e >> 1];
                    if (a.cap_inv != 0.f) s[n][e] = pa::capped(s[n][e], a.cap_log2, a.cap_inv);
                    if (a.slopes) s[n][e] -= slope[e >> 1] * (float)abs(at[e >> 1] - (t0 + 8 * n + 2 * t4 + (e & 1)));
                }
#pragma unroll
            for (int h = 0; h < kH; ++h) f[0][h] = f[1][h] = 1.f;
        }
        if (masked) {
            const int lo[2] = {shape[g].lo, shape[g + 8].lo}, hi[2] = {shape[g].hi, shape[g + 8].hi};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2 * kH; ++e) {
                    const int pos = t0 + 8 * n + 2 * t4 + (e & 1);
                    if (pos < lo[e >> 1] || pos >= hi[e >> 1]) s[n][e] = -INFINITY;
                }
        }
        if constexpr (F8) {
            // (A scale of positions that a row does not see is none of its own: its weights there are zeros, and the
            // unit of the others stays.  All factors are powers of two, put together from their exponents.)
            const int v0 = scales >> 8 & 0xff, v1 = scales >> 24;
#pragma unroll
            for (int h = 0; h < kH; ++h) {
                int u0 = v0, u1 = v1;
                if (masked) {
                    const int lo = shape[g + 8 * h].lo, hi = shape[g + 8 * h].hi;
                    if (lo >= t0 + 8 || hi <= t0) u0 = 0;
                    if (lo >= t0 + kTile || hi <= t0 + 8) u1 = 0;
                }
                const int top = max(u0, u1);
                if (top > st.top[h]) {
                    const float less = scale_of(max(127 + st.top[h] - top, 0));
                    st.top[h] = top;
#pragma unroll
                    for (int d = 0; d < D / 8; ++d) {
                        st.acc[d][2 * h] *= less;
                        st.acc[d][2 * h + 1] *= less;
                    }
                }
                const int unit = 127 + kLog2WeightScale - st.top[h];
                by[0][h] = scale_of(max(unit + u0, 0));
                by[1][h] = scale_of(max(unit + u1, 0));
            }
        }
    } else if (t0 + kTile > u.first) {                 // some row may not see some position
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!visible(a, u, g + 8 * (e >> 1), t0 + 8 * n + 2 * t4 + (e & 1))) s[n][e] = -INFINITY;
    }
    // how far the tile's scores rise above the running maxima
    float over = -INFINITY;
#pragma unroll
    for (int h = 0; h < kH; ++h) {
        if constexpr (kShaped && F8) {
            over = fmaxf(over, fmaxf(fmaf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), f[0][h], -st.m[h]),
                                     fmaf(fmaxf(s[1][2 * h], s[1][2 * h + 1]), f[1][h], -st.m[h])));
        } else {
            const float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            over = fmaxf(over, fmaf(top, f[0][h], -st.m[h]));
        }
    }
    if (__any_sync(0xffffffffu, over > kRaise)) {
#pragma unroll
        for (int h = 0; h < kH; ++h) {
            float top = kShaped && F8 ? fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]) * f[0][h], fmaxf(s[1][2 * h], s[1][2 * h + 1]) * f[1][h])
                                      : fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            float m = fmaxf(st.m[h], kShaped && F8 ? top : top * f[0][h]);
            if (kShaped && !(m > st.m[h] + kRaise)) m = st.m[h];   // (a row's own scores alone raise its maximum)
            const float less = pa::exp2_approx(st.m[h] - m);
            st.m[h] = m;
            st.l[h] *= less;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                st.acc[d][2 * h] *= less;
                st.acc[d][2 * h + 1] *= less;
            }
        }
    }
    // weights as the A operand: bf16 in two terms (a relative 2^-16), f16 times 2^7 (2^-11)
    uint32_t ph[4] = {0, 0, 0, 0}, pl[4] = {0, 0, 0, 0};
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float p0 = pa::exp2_approx(fmaf(s[n][2 * h], f[n][h], -st.m[h]));
            const float p1 = pa::exp2_approx(fmaf(s[n][2 * h + 1], f[n][h], -st.m[h]));
            st.l[h] += p0 + p1;
            if constexpr (F8) {
                ph[2 * n + h] = kShaped ? pa::pack_f16x2(p0 * by[n][h], p1 * by[n][h]) : pa::pack_f16x2(p0 * kWeightScale, p1 * kWeightScale);
            } else {
                const uint32_t w = pa::pack_bf16x2(p0, p1);
                const float2 hi = pa::bf16x2_to_float2(w);
                ph[2 * n + h] = w;
                pl[2 * n + h] = pa::pack_bf16x2(p0 - hi.x, p1 - hi.y);
            }
        }
    // O += P . V; V rows past the context are zeroed (0 * NaN)
    const int nv = u.ctx - t0;
    auto values = [&](bool masked, uint32_t mlo, uint32_t mhi) {
#pragma unroll
        for (int j = 0; j < D / (F8 ? 32 : 16); ++j) {
            uint32_t r[4];
            if constexpr (F8) {
                // r[0], r[1]: keys 2 t4, 2 t4 + 1 and 2 t4 + 8, + 9, codes 2 g and 2 g + 1 of chunk
                // 2 j; r[2], r[3]: of chunk 2 j + 1.  Paired by code, they are the products of the
                // chunk's even and odd columns.
                pa::ldsm4_trans(vs + pa::swz128(v_row, 2 * j + v_add), r);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t b0[2], b1[2];
                    pa::e4m3x4_to_f16x4(pa::byte_perm(r[2 * x], 0x3120u), b0[0], b0[1]);
                    pa::e4m3x4_to_f16x4(pa::byte_perm(r[2 * x + 1], 0x3120u), b1[0], b1[1]);
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        if (masked) {
                            b0[odd] &= mlo;
                            b1[odd] &= mhi;
                        }
                        pa::mma16816<true>(st.acc[2 * (2 * j + x) + odd], ph, b0[odd], b1[odd]);
                    }
                }
            } else {
                pa::ldsm4_trans(vs + (j >> 2) * kSlabBytes + pa::swz128(v_row, 2 * (j & 3) + v_add), r);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t b0 = masked ? r[2 * x] & mlo : r[2 * x];
                    const uint32_t b1 = masked ? r[2 * x + 1] & mhi : r[2 * x + 1];
                    pa::mma16816<false>(st.acc[2 * j + x], ph, b0, b1);
                    pa::mma16816<false>(st.acc[2 * j + x], pl, b0, b1);
                }
            }
        }
    };
    if (nv < kTile) {
        const int k = 2 * t4;
        values(true, (k < nv ? 0x0000ffffu : 0u) | (k + 1 < nv ? 0xffff0000u : 0u),
               (k + 8 < nv ? 0x0000ffffu : 0u) | (k + 9 < nv ? 0xffff0000u : 0u));
    } else {
        values(false, 0u, 0u);
    }
}

template <int D, bool F8, int kWarps, class Args, bool kEight>
__global__ void __launch_bounds__(32 * kWarps, kWarpsPerSm / kWarps)
    multi_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Args a) {
    using G = Geo<D, F8, kWarps>;
    using Unit = typename Args::Unit;
    constexpr bool kShaped = Args::kShaped, kScaled = kShaped && F8;
    constexpr int kStages = G::kStages, kThreads = G::kThreads;
    constexpr int kStep = step_of(kWarps), kUnitCost = cost_of(kWarps, F8), kMinSteps = least_of(kWarps), kDirectSteps = direct_of(kWarps);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* qsm = ring + G::kRingBytes;                          // [kRows][kQStride]
    float* q_scale = reinterpret_cast<float*>(qsm + kRows * G::kQStride);   // FP8: score factor per row
    float2* stats = reinterpret_cast<float2*>(q_scale + kRows);   // [key warp][row]: maximum and sum
    uint64_t* full = reinterpret_cast<uint64_t*>(stats + kWarps * kRows);   // [key warp][stage]
    __shared__ Part parts[kWarps];
    __shared__ int unfinite[2];                                   // per unit parity: some new value is not finite
    // Thread 0 walks the share two units ahead; a unit's place is free again
    // two barriers after its join.
    __shared__ WalkOf<typename Args::Seq> walk;
    __shared__ Unit units[4];
    __shared__ Shape shape[kShaped ? kRows : 1];                  // of the unit's rows

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = 1 << a.log2_block, heads = a.n_kv_heads;
    if (threadIdx.x == 0) {
#pragma unroll 1
        for (int i = 0; i < kWarps * kStages; ++i) pa::mbar_init(&full[i], 1);
        unfinite[0] = unfinite[1] = 0;
        pa::fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (!find_share<kRows, kStep, kUnitCost, kMinSteps, kDirectSteps, kThreads>(a, walk, parts)) return;
    if (threadIdx.x == 0) {
        next_unit<kRows, kStep, kUnitCost>(walk, units[0], a);
        next_unit<kRows, kStep, kUnitCost>(walk, units[1], a);
    }
    __syncthreads();
    if (!units[0].valid) return;                                 // a share that ends in a unit's constant part

    const uint64_t policy = pa::l2_evict_first_policy();
    const uint32_t ring0 = pa::smem_addr(ring) + warp * G::kStageBytes;
    const uint32_t qs = pa::smem_addr(qsm);
    uint64_t* wfull = full + warp * kStages;
    auto base_of = [](const Unit& u) {
        if constexpr (kShaped) return u.base;
        else return 0;
    };
    auto lo_of = [](const Unit& u) {
        if constexpr (kShaped) return u.lo;
        else return 0;
    };
    auto stage_at = [&](int stage) { return ring0 + stage * (kWarps * G::kStageBytes); };

    // A warp's tile k of a unit holds positions (st0 + k) * kStep + 16 warp on (from base).  Its
    // table entries come 32 tiles at a time, one per lane, the next 32 ahead.
    // (A tile of which one block alone is seen has it in both entries: no block that the unit does not see is read.)
    auto fetch = [&](const Unit& u, int k, int& e0, int& e1) {
        e0 = e1 = -1;
        const int t0 = base_of(u) + (u.st0 + k) * kStep + warp * kTile;
        if (k < u.len && t0 < u.ctx) {
            const int32_t* table = table_of(a, u);
            const bool second = B < kTile && t0 + B < u.ctx, first = !second || t0 + B > lo_of(u);
            if (first) e0 = e1 = table[t0 >> a.log2_block];
            if (second) e1 = table[(t0 >> a.log2_block) + 1];
            if (!first) e0 = e1;
        }
    };
    // Block-scaled: the scale bytes that go with the entries, asked for when those have come and before their tiles.  Zeros
    // for a block that is not there.
    auto scales_of = [&](const Unit& u, int b0, int b1) {
        uint32_t r = 0;
        if constexpr (kScaled) {
            const size_t i0 = (size_t)b0 * heads + u.kvh, i1 = (size_t)b1 * heads + u.kvh;
            if (b0 >= 0 && b0 < a.num_blocks) r = a.k_scales[i0] | (uint32_t)a.v_scales[i0] << 8;
            if (b1 >= 0 && b1 < a.num_blocks) r |= (uint32_t)a.k_scales[i1] << 16 | (uint32_t)a.v_scales[i1] << 24;
        }
        return r;
    };
    uint32_t scales = 0, scales_next = 0;                         // of this lane's tile of the 32 in work, and of the next 32
    int e0 = -1, e1 = -1, f0 = -1, f1 = -1;
    int used = 0;                                                 // tiles of the ring before the current unit's
    auto issue = [&](const Unit& u, int k) {                      // whole warp
        if (k && (k & 31) == 0) {
            e0 = f0;
            e1 = f1;
            scales_next = scales_of(u, e0, e1);
            fetch(u, k + 32 + lane, f0, f1);
        }
        const int b0 = __shfl_sync(0xffffffffu, e0, k & 31), b1 = __shfl_sync(0xffffffffu, e1, k & 31);
        if (lane == 0) {
            const int at = used + k, stage = at % kStages;
            uint64_t* bar = &wfull[stage];
            const int t0 = base_of(u) + (u.st0 + k) * kStep + warp * kTile;
            if (t0 >= u.ctx) {
                pa::mbar_arrive(bar);                             // no such tile: the stage goes by empty
            } else {
                const int box = B < kTile ? B : kTile, boxes = (B < kTile && t0 + B < u.ctx) ? 2 : 1;
                const uint32_t dst = stage_at(stage);
                pa::mbar_arrive_expect_tx(bar, (uint32_t)(2 * G::kSlabs * boxes * box * 128));
#pragma unroll 1
                for (int r = 0; r < boxes; ++r) {
                    int blk = r ? b1 : b0;
                    if (blk < 0 || blk >= a.num_blocks) {
                        pa::set_status(a.status, PA_DEV_BAD_BLOCK_ID);
                        blk = 0;
                    }
                    const int row = (blk * heads + u.kvh) * B + (r ? 0 : t0 & (B - 1));
#pragma unroll
                    for (int h = 0; h < G::kSlabs; ++h) {
                        const uint32_t d = dst + h * G::kSlabBytes + r * box * 128;
                        pa::tma_box(d, &map_k, h * 64, row, bar, policy);
                        pa::tma_box(d + G::kTileBytes, &map_v, h * 64, row, bar, policy);
                    }
                }
            }
        }
    };
    // q of a unit's rows, 8 elements per thread and piece: loaded, then stored
    constexpr int kLanesQ = D / 8, kQPer = (kRows * kLanesQ + kThreads - 1) / kThreads;
    auto load_q = [&](const Unit& u, uint4 (&v)[kQPer]) {
#pragma unroll
        for (int x = 0; x < kQPer; ++x) {
            const int r = (x * kThreads + threadIdx.x) / kLanesQ, c = threadIdx.x % kLanesQ;
            const int row = u.row0 + r, i = row >> a.log2_group;
            v[x] = make_uint4(0, 0, 0, 0);
            if (r < kRows && i < u.n)
                v[x] = *reinterpret_cast<const uint4*>(
                    a.q + ((size_t)(u.q0 + i) * a.n_q_heads + (u.kvh << a.log2_group) +
                           (row & ((1 << a.log2_group) - 1))) * D + 8 * c);
        }
    };
    auto store_q = [&](const uint4 (&v)[kQPer]) {
#pragma unroll
        for (int x = 0; x < kQPer; ++x) {
            const int r = (x * kThreads + threadIdx.x) / kLanesQ, c = threadIdx.x % kLanesQ;
            if (r >= kRows) break;                               // (whole warps)
            uint8_t* dst = qsm + r * G::kQStride;
            const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
            if constexpr (F8) {
                // f16 after a power of two per row that brings its largest element into [2^14, 2^15)
                float f[8], top = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 p = pa::bf16x2_to_float2(w[e]);
                    f[2 * e] = p.x;
                    f[2 * e + 1] = p.y;
                    top = fmaxf(top, fmaxf(fabsf(p.x), fabsf(p.y)));
                }
#pragma unroll
                for (int o = 1; o < kLanesQ; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                int eb = (__float_as_int(top) >> 23) & 0xff;
                eb = eb < 14 ? 14 : (eb > 254 ? 254 : eb);
                const float up = __int_as_float((268 - eb) << 23);
                if (c == 0) q_scale[r] = fmaxf(a.scale_log2 / up, 1e-37f);   // never 0: masked scores stay -inf
                const float by = up * a.q_sign;
                // within 16 elements, word t4 holds d = 4 t4, 4 t4 + 1 and word t4 + 4 the next
                // two: the order in which ldmatrix hands out K's codes
                uint32_t* p = reinterpret_cast<uint32_t*>(dst + (c >> 1) * 32);
                const int j = (c & 1) * 2;
                p[j] = pa::pack_f16x2(f[0] * by, f[1] * by);
                p[j + 4] = pa::pack_f16x2(f[2] * by, f[3] * by);
                p[j + 1] = pa::pack_f16x2(f[4] * by, f[5] * by);
                p[j + 5] = pa::pack_f16x2(f[6] * by, f[7] * by);
            } else {
                const uint32_t flip = a.q_sign < 0.f ? 0x80008000u : 0u, keep = a.q_sign == 0.f ? 0u : 0xffffffffu;
                *reinterpret_cast<uint4*>(dst + 16 * c) =
                    make_uint4((w[0] ^ flip) & keep, (w[1] ^ flip) & keep, (w[2] ^ flip) & keep, (w[3] ^ flip) & keep);
            }
        }
    };

    uint4 qv[kQPer];
    fetch(units[0], lane, e0, e1);
    fetch(units[0], 32 + lane, f0, f1);
    scales = scales_of(units[0], e0, e1);
#pragma unroll 1
    for (int k = 0; k < G::kAhead; ++k)
        if (k < units[0].len) issue(units[0], k);
    load_q(units[0], qv);
#pragma unroll 1
    for (int nth = 0;; ++nth) {
        const Unit& u = units[nth & 3];
        const Unit& next = units[(nth + 1) & 3];
        store_q(qv);
        if constexpr (kShaped)
            if (threadIdx.x < kRows) shape[threadIdx.x] = shape_of(a, u, threadIdx.x);
        __syncthreads();
        const int len = u.len, ctx = u.ctx, base = base_of(u) + u.st0 * kStep + warp * kTile;
        const bool more = next.valid;
#pragma unroll 1
        for (int k = G::kAhead; k < kStages; ++k)
            if (k < len) issue(u, k);
        int n0 = -1, n1 = -1;
        if (more) fetch(next, lane, n0, n1);
        if (threadIdx.x == 0) {
            next_unit<kRows, kStep, kUnitCost>(walk, units[(nth + 2) & 3], a);
            unfinite[(nth + 1) & 1] = 0;                          // (its last readers are a barrier behind)
        }
        __syncwarp();
        uint32_t qr[G::kSteps][4];
#pragma unroll
        for (int kk = 0; kk < G::kSteps; ++kk)
            pa::ldsm4(qs + ((lane & 7) + (((lane >> 3) & 1) << 3)) * G::kQStride + (2 * kk + (lane >> 4)) * 16, qr[kk]);
        float c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) c[h] = F8 ? q_scale[(lane >> 2) + 8 * h] : a.scale_log2;

        int seen_lo = 0, seen_hi = 0, blind = 0;
        if constexpr (kShaped) {
            seen_lo = u.seen_lo;
            seen_hi = u.seen_hi;
            blind = u.blind;
        }
        State<D> st;
        st.reset();
        bool landed = true;
#pragma unroll 1
        for (int k = 0; k < len; ++k) {
            uint32_t tile_scales = 0;
            if constexpr (kScaled) {
                if (k && (k & 31) == 0) scales = scales_next;
                tile_scales = __shfl_sync(0xffffffffu, scales, k & 31);
            }
            const int at = used + k, stage = at % kStages;
            if (!__all_sync(0xffffffffu, pa::mbar_wait_bounded(&wfull[stage], (at / kStages) & 1, kMaxProbes))) {
                // give up: nothing more is issued, and the copies in flight are waited for, each within the limit
                if (lane == 0) pa::set_status(a.status, PA_DEV_WAIT_TIMEOUT);
                const int issued = min(len, k + kStages);
#pragma unroll 1
                for (int j = k; j < issued; ++j)
                    pa::mbar_wait_bounded(&wfull[(used + j) % kStages], ((used + j) / kStages) & 1, kMaxProbes);
                landed = false;
                break;
            }
            const int t0 = base + k * kStep;
            if (t0 < ctx) {
                const uint32_t ks = stage_at(stage);
                const bool some = kShaped ? t0 < seen_lo || t0 + kTile > seen_hi : t0 + kTile > u.first;
                if (some) {                                       // some row may not see some position
                    uint8_t* v = ring + stage * (kWarps * G::kStageBytes) + warp * G::kStageBytes + G::kTileBytes;
                    if (kShaped ? drop_unfinite_outside<F8, G::kSlabs>(v, G::kSlabBytes, t0, seen_lo, seen_hi, min(kTile, ctx - t0), lane, 32)
                                : drop_unfinite<F8, G::kSlabs>(v, G::kSlabBytes, max(0, u.first - t0), min(kTile, ctx - t0), lane, 32))
                        unfinite[nth & 1] = 1;
                    __syncwarp();
                }
                fold_tile<D, F8, Args, kEight>(st, ks, ks + G::kTileBytes, c, t0, a, u, lane, qr, shape, tile_scales, some || blind);
            }
            __syncwarp();
            if (k + kStages < len) issue(u, k + kStages);
        }
        used += len;
        if (!__syncthreads_and(landed)) return;                   // every tile of the unit is consumed
        if (more) {
            e0 = n0;
            e1 = n1;
            fetch(next, 32 + lane, f0, f1);
            scales = scales_of(next, e0, e1);
#pragma unroll 1
            for (int k = 0; k < G::kAhead; ++k)
                if (k < next.len) issue(next, k);
            load_q(next, qv);
        }

        // ---- join the key warps' states (the exact block merge) ----
        if constexpr (kScaled)
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.acc[d][e] *= scale_of(st.top[e >> 1]);
        const int g = lane >> 2, t4 = lane & 3;
        auto join_row = [&](int w, int r) {                       // fp32 row r of key warp w
            const int rows = kRows / G::kJoinStages, stage = (used + G::kAhead + r / rows) % kStages;
            return reinterpret_cast<float*>(ring + stage * (kWarps * G::kStageBytes)) + (w * rows + r % rows) * D;
        };
        auto spread = [](int r) { return ((r & 1) << 4) | ((r & 2) << 2); };   // rows to distinct banks
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float l = st.l[h];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int r = g + 8 * h;
            if (t4 == 0) stats[warp * kRows + r] = make_float2(st.m[h], l);
            float* row = join_row(warp, r);
            if constexpr (F8) {
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                    *reinterpret_cast<float4*>(row + ((16 * x + 4 * t4) ^ spread(r))) = make_float4(
                        st.acc[2 * x][2 * h], st.acc[2 * x + 1][2 * h], st.acc[2 * x][2 * h + 1], st.acc[2 * x + 1][2 * h + 1]);
            } else {
#pragma unroll
                for (int d = 0; d < D / 8; ++d)
                    *reinterpret_cast<float2*>(row + ((8 * d + 2 * t4) ^ spread(r))) =
                        make_float2(st.acc[d][2 * h], st.acc[d][2 * h + 1]);
            }
        }
        __syncthreads();
        const bool whole = u.whole;
        const int slot = 2 * blockIdx.x + (u.st0 == 0 ? 1 : 0);
#pragma unroll 1
        for (int x = threadIdx.x; x < kRows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), d = x % (D / 4) * 4;
            const int row = u.row0 + r, i = row >> a.log2_group;
            if (i >= u.n) continue;
            float2 ml[kWarps];
            float M = kNone;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = stats[w * kRows + r];
                M = fmaxf(M, ml[w].x);
            }
            float Z = 0.f;
            float4 U = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = pa::exp2_approx(ml[w].x - M);
                const float4 v = *reinterpret_cast<const float4*>(join_row(w, r) + (d ^ spread(r)));
                Z += f * ml[w].y;
                U.x += f * v.x;
                U.y += f * v.y;
                U.z += f * v.z;
                U.w += f * v.w;
            }
            if (whole) {
                const float f = a.v_scale / Z;
                put4(a.out, a.out_f32,
                     ((size_t)(u.q0 + i) * a.n_q_heads + (u.kvh << a.log2_group) + (row & ((1 << a.log2_group) - 1))) * D + d,
                     Z == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(U.x * f, U.y * f, U.z * f, U.w * f));
            } else {
                const size_t at = (size_t)slot * kRows + r;
                *reinterpret_cast<float4*>(a.part_u + at * D + d) = U;
                if (d == 0) {
                    a.part_m[at] = M;
                    a.part_z[at] = Z;
                }
            }
        }
        if (__builtin_expect(unfinite[nth & 1], 0))
#pragma unroll 1
            for (int x = threadIdx.x; x < kRows * (D / 4); x += kThreads) {   // (to what the thread itself has written)
                const int r = x / (D / 4), d = x % (D / 4) * 4;
                add_unfinite<D, F8>(a, u.seq, u.kvh, u.row0 + r, base_of(u) + u.st0 * kStep, base_of(u) + (u.st0 + len) * kStep, d,
                                    whole ? nullptr : a.part_u + ((size_t)slot * kRows + r) * D + d);
            }
        if (!whole && u.st0 == 0 && threadIdx.x == 0)             // this block begins the unit
            a.pieces[blockIdx.x] = begun_unit(u, a.log2_group);
        if (!more) return;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the join's stages go back to TMA (after the barrier above)
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

inline int sms() { return pa_host::sm_count(); }

// Rows of a unit: on the wide kernel 64, and 128 for bf16 where a KV head has more.
inline int unit_rows(long long rows, bool f8, bool wide) { return !wide ? kRows : f8 || rows <= 64 ? 64 : 128; }

// Resident blocks of the device.
inline int max_grid(bool wide) { return sms() * (wide ? 1 : kWarpsPerSm / 4); }

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace: the blocks' pieces, then m and z, then u; 256-byte aligned.
inline size_t workspace_size(int grid, int unit, int d) {
    const size_t rows = (size_t)2 * grid * unit;
    return up256(16 * (size_t)grid) + 2 * up256(4 * rows) + 4 * rows * d;
}

// Whether a call that the wide kernel could take goes 16 rows at a time all
// the same: contexts of one tile, and an SM for each unit of 16 (a third of
// one where the units there would be of 128).  8 KV heads of 128, 64
// positions, us here against there: 4 sequences of 32 rows 6.2 / 7.2, of 64
// 6.5 / 7.9, of 128 7.9 / 9.8, 9 of 96 7.9 / 9.2, 1 of 256 6.7 / 10.8; 18 of
// 32 at 128 positions 8.7 / 7.7; E4M3 4 of 128 at 128 9.1 / 8.3.
inline bool in_small_tiles(bool f8, long long rows, double heads, int ctx) {
    const double units = heads * (double)((rows + kRows - 1) / kRows);
    return ctx <= 128 && units <= (f8 || rows <= 64 ? 1 : 3) * sms();
}

inline void set_workspace(MultiArgs& a, void* workspace, int grid, int unit) {
    const size_t rows = (size_t)2 * grid * unit;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.pieces = reinterpret_cast<int4*>(w);
    w += up256(16 * (size_t)grid);
    a.part_m = reinterpret_cast<float*>(w);
    w += up256(4 * rows);
    a.part_z = reinterpret_cast<float*>(w);
    w += up256(4 * rows);
    a.part_u = reinterpret_cast<float*>(w);
}

// Warps of a block: four, three blocks to an SM, or twelve where every unit
// can have an SM to itself, is long enough to share (one warp alone folds its
// tile of 16 positions in 0.85 us) and the device is not filled.  Four against
// twelve, us: 32 units of 37 positions 6.6 / 7.5, 256 9.4 / 8.7, 768 17.0 /
// 11.7, 2048 18.0 / 15.8 (E4M3 19.0 / 14.3); 144 units of 1536 28.9 / 25.3;
// 68 of 411 to 8221 20.2 / 22.8; 512 of 4096 E4M3 102 / 116.
inline int block_warps(double units, int ctx) { return units <= sms() && ctx > 128 && units * ctx <= 1536.0 * sms() ? 12 : 4; }

// The grid of a call.  No more blocks than the largest possible work has
// smallest shares, or, for short contexts with an SM for each unit, one a unit.
struct Split {
    int unit, warps, grid, direct;         // rows of a unit; warps of a block (not wide); not 0: row tiles a KV head
    double units;
};
inline Split split_work(bool f8, bool wide, long long all_rows, int num_seqs, int n_kv_heads, int ctx_cap) {
    Split s;
    s.unit = unit_rows(all_rows, f8, wide);
    const long long tiles = (all_rows + s.unit - 1) / s.unit;
    s.units = (double)num_seqs * n_kv_heads * (double)tiles;
    s.warps = wide ? 0 : block_warps(s.units, ctx_cap);
    const int step = wide ? kWideStep : step_of(s.warps), cost = wide ? kWideCost : cost_of(s.warps, f8);
    const int blocks = wide || s.warps == 12 ? sms() : max_grid(wide);
    const long long seq_work = ((long long)ctx_cap + step - 1) / step + cost;
    const double shares = s.units * (double)seq_work / ((wide ? kWideMinSteps : least_of(s.warps)) + cost) + 1;
    const bool direct = ctx_cap <= step * (wide ? kWideDirectSteps : direct_of(s.warps)) && s.units <= blocks;
    s.grid = direct ? (int)s.units : shares < blocks ? (int)shares : blocks;
    s.direct = direct ? (int)tiles : 0;
    return s;
}

template <int D, bool F8, int kWarps, bool kEight, class Args>
int launch_multi(const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, int grid, cudaStream_t st) {
    static int attr[64] = {0};
    constexpr int kSmem = Geo<D, F8, kWarps>::kSmem;
    if (pa_host::ensure_smem_attr(multi_kernel<D, F8, kWarps, Args, kEight>, kSmem, attr) != cudaSuccess) return PA_ERR_CUDA;
    return pa_host::launch_dependent(multi_kernel<D, F8, kWarps, Args, kEight>, dim3(grid), dim3(32 * kWarps), kSmem, st, mk, mv, a) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

template <int D, bool F8, bool kEight = false, class Args>
int launch_multi(int warps, const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, int grid, cudaStream_t st) {
    return warps == 12 ? launch_multi<D, F8, 12, kEight>(mk, mv, a, grid, st) : launch_multi<D, F8, 4, kEight>(mk, mv, a, grid, st);
}

}  // namespace
