// Attention of a few new tokens per sequence over the paged cache: the tokens
// of a speculative draft (a chain or a tree) to verify, or a short chunk.
//
// Sequence s has C positions in the cache, of which the last n are new.  Row
// (i, g) is new token i's query head g of the KV head's group; it sees every
// position before C - n, and of the new ones those up to its own (causal) or
// those whose bit its mask word has.  out = softmax(scale q . K) V over them
// ("PagedAttention: Virtual Memory for the KV Cache", sections 7 and 13;
// "PagedAttention in vLLM: scattered memory, exact attention", sections 10
// and 11: translation, the online softmax, the exact merge).
//
// This file serves up to 16 rows a KV head (and any number with a scale that
// is not positive, or over a few contexts of one tile); pa_decode_wide.cu
// takes more.
//
// What bounds it: each K/V byte is read once for n * G rows, 4 * n * G
// operations per two bytes, so the cache's bytes bound it.  64 sequences of
// 4096 positions, 8 KV heads of 128, 16 rows: 168 us, 0.94 of the measured
// copy rate; E4M3 94 us, 0.85 (there the unpacking of codes to f16 for
// warp-level products takes 44 % of the ALU's cycles).  The smallest steps
// are a chain of latencies: 4 sequences of up to 37 positions take 4.7 us.
//  * A unit is a (sequence, KV head, tile of 16 rows); its work is counted in
//    steps of a block's positions plus a constant for starting and joining
//    it.  The grid is the resident blocks, and they take equal contiguous
//    shares of all the work, computed from the lengths by every block for
//    itself: no partition size to choose, no empty blocks on ragged batches,
//    and at most two unfinished units per block whatever the batch.
//  * The warps of a block, four or twelve, take 16 positions of a step each,
//    from rings of shared-memory stages that TMA fills through the block
//    table.  The next unit's first tiles are in flight while the warps' states
//    of a unit are joined, in the stages they leave free.
//  * Rows are the rows of the products (S[16 x 16] = Q . K^T, then
//    O[16 x D] += P . V), so the weights are the second product's operand as
//    they come out of the first.
//  * The running maximum of a row is raised only when a score exceeds it by
//    2^8 (one vote instead of a maximum's shuffles); weights stay within 2^8
//    and sums in fp32.
//  * A unit that one block covers is written at once.  Pieces of the others
//    go to the workspace as (m, z, u), and a second kernel, over the units
//    that a block began and did not finish, merges them.  Short contexts with
//    a block for every unit are not split, and then nothing is merged.

#include <math.h>

#include <algorithm>

#include "pa_multi.cuh"

using namespace pa_multi;

namespace {

constexpr int kTile = 16;                  // positions per warp and step
constexpr int kRows = 16;                  // rows of a unit
constexpr int kWarpsPerSm = 12;
constexpr float kWeightScale = 128.f;      // FP8: weights enter f16 products times 2^7 (at most 2^15)
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
    float acc[D / 8][4];
    __device__ __forceinline__ void reset() {
        m[0] = m[1] = kNone;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
    }
};

// Fold one tile (K at shared address ks, V at vs, positions t0 .. t0 + 15)
// into the warp's state.  qr: the rows of q as A operands; c[h]: score factor
// of rows g + 8 h.
template <int D, bool F8>
__device__ __forceinline__ void fold_tile(State<D>& st, uint32_t ks, uint32_t vs, const float (&c)[2], int t0, const MultiArgs& a,
                                          const Unit& u, int lane, const uint32_t (&qr)[D / 16][4]) {
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
    if (t0 + kTile > u.first) {                        // some row may not see some position
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!visible(a, u, g + 8 * (e >> 1), t0 + 8 * n + 2 * t4 + (e & 1))) s[n][e] = -INFINITY;
    }
    // how far the tile's scores rise above the running maxima
    float over = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        over = fmaxf(over, fmaf(top, c[h], -st.m[h]));
    }
    if (__any_sync(0xffffffffu, over > kRaise)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float m = fmaxf(st.m[h], top * c[h]);
            const float f = pa::exp2_approx(st.m[h] - m);
            st.m[h] = m;
            st.l[h] *= f;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                st.acc[d][2 * h] *= f;
                st.acc[d][2 * h + 1] *= f;
            }
        }
    }
    // weights as the A operand: bf16 in two terms (a relative 2^-16), f16 times 2^7 (2^-11)
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float p0 = pa::exp2_approx(fmaf(s[n][2 * h], c[h], -st.m[h]));
            const float p1 = pa::exp2_approx(fmaf(s[n][2 * h + 1], c[h], -st.m[h]));
            st.l[h] += p0 + p1;
            if constexpr (F8) {
                ph[2 * n + h] = pa::pack_f16x2(p0 * kWeightScale, p1 * kWeightScale);
            } else {
                const uint32_t w = pa::pack_bf16x2(p0, p1);
                const float2 f = pa::bf16x2_to_float2(w);
                ph[2 * n + h] = w;
                pl[2 * n + h] = pa::pack_bf16x2(p0 - f.x, p1 - f.y);
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

template <int D, bool F8, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarpsPerSm / kWarps)
    multi_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const MultiArgs a) {
    using G = Geo<D, F8, kWarps>;
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
    __shared__ Walk walk;
    __shared__ Unit units[4];

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
    auto stage_at = [&](int stage) { return ring0 + stage * (kWarps * G::kStageBytes); };

    // A warp's tile k of a unit holds positions (st0 + k) * kStep + 16 warp on.  Its
    // table entries come 32 tiles at a time, one per lane, the next 32 ahead.
    auto fetch = [&](const Unit& u, int k, int& e0, int& e1) {
        e0 = e1 = 0;
        const int t0 = (u.st0 + k) * kStep + warp * kTile;
        if (k < u.len && t0 < u.ctx) {
            const int32_t* table = table_of(a, u);
            e0 = table[t0 >> a.log2_block];
            if (B < kTile && t0 + B < u.ctx) e1 = table[(t0 >> a.log2_block) + 1];
        }
    };
    int e0 = 0, e1 = 0, f0 = 0, f1 = 0;
    int used = 0;                                                 // tiles of the ring before the current unit's
    auto issue = [&](const Unit& u, int k) {                      // whole warp
        if (k && (k & 31) == 0) {
            e0 = f0;
            e1 = f1;
            fetch(u, k + 32 + lane, f0, f1);
        }
        const int b0 = __shfl_sync(0xffffffffu, e0, k & 31), b1 = __shfl_sync(0xffffffffu, e1, k & 31);
        if (lane == 0) {
            const int at = used + k, stage = at % kStages;
            uint64_t* bar = &wfull[stage];
            const int t0 = (u.st0 + k) * kStep + warp * kTile;
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
#pragma unroll 1
    for (int k = 0; k < G::kAhead; ++k)
        if (k < units[0].len) issue(units[0], k);
    load_q(units[0], qv);
#pragma unroll 1
    for (int nth = 0;; ++nth) {
        const Unit& u = units[nth & 3];
        const Unit& next = units[(nth + 1) & 3];
        store_q(qv);
        __syncthreads();
        const int len = u.len, ctx = u.ctx, base = u.st0 * kStep + warp * kTile;
        const bool more = next.valid;
#pragma unroll 1
        for (int k = G::kAhead; k < kStages; ++k)
            if (k < len) issue(u, k);
        int n0 = 0, n1 = 0;
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

        State<D> st;
        st.reset();
        bool landed = true;
#pragma unroll 1
        for (int k = 0; k < len; ++k) {
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
                if (t0 + kTile > u.first) {
                    const int from = max(0, u.first - t0);
                    uint8_t* v = ring + stage * (kWarps * G::kStageBytes) + warp * G::kStageBytes + G::kTileBytes;
                    if (drop_unfinite<F8, G::kSlabs>(v, G::kSlabBytes, from, min(kTile, ctx - t0), lane, 32))
                        unfinite[nth & 1] = 1;
                    __syncwarp();
                }
                fold_tile<D, F8>(st, ks, ks + G::kTileBytes, c, t0, a, u, lane, qr);
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
#pragma unroll 1
            for (int k = 0; k < G::kAhead; ++k)
                if (k < next.len) issue(next, k);
            load_q(next, qv);
        }

        // ---- join the key warps' states (the exact block merge) ----
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
                const float f = Z == 0.f ? 0.f : a.v_scale / Z;
                put4(a.out, a.out_f32,
                     ((size_t)(u.q0 + i) * a.n_q_heads + (u.kvh << a.log2_group) + (row & ((1 << a.log2_group) - 1))) * D + d,
                     make_float4(U.x * f, U.y * f, U.z * f, U.w * f));
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
                add_unfinite<D, F8>(a, u.seq, u.kvh, u.row0 + r, u.st0 * kStep, (u.st0 + len) * kStep, d,
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

int sms() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && cached[dev]) return cached[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) cached[dev] = n;
    return n;
}

// Whether the units of 64 (or 128) rows of pa_decode_wide.cu serve a call:
// from more than 16 rows a KV head on, where they read the cache once and
// units of 16 twice or more.  8 KV heads of 128, us here / there (batches in
// turn, so that nothing stays in L2):
//   sequences x positions   16 rows       20 rows       32 rows       64 rows
//   bf16  64 x 4096         168 / 162     322 / 163     327 / 164     635 / 168
//         512 x 500         166 / 167     329 / 169     342 / 174     710 / 192
//         512 x 128          62 / 90      110 / 92      117 / 94      237 / 100
//         2048 x 60         184 / 316     331 / 318     373 / 327     740 / 364
//   E4M3  64 x 4096          94 / 100     174 / 100     175 / 101     338 / 108
//         512 x 500         122 / 166     233 / 166     237 / 165     470 / 167
//         512 x 128          64 / 125     117 / 133     119 / 140     237 / 157
//         2048 x 60         197 / 459     373 / 499     392 / 511     767 / 585
// (At 16 rows short contexts decide: a unit there costs some 3 to 5 us.  At 17
// to 32 rows the rule is wrong for E4M3 contexts of a tile or less in many
// sequences, which lose 14 to 30 % by it.)
// Its bf16 products take a positive scale only; others go 16 rows at a time.
bool is_wide(bool f8, float scale, long long rows) { return rows > kRows && (f8 || scale > 0.f); }

// Whether a call that the wide kernel could take goes 16 rows at a time all
// the same: contexts of one tile, and an SM for each unit of 16 (a third of
// one where the units there would be of 128).  8 KV heads of 128, 64
// positions, us here against there: 4 sequences of 32 rows 6.2 / 7.2, of 64
// 6.5 / 7.9, of 128 7.9 / 9.8, 9 of 96 7.9 / 9.2, 1 of 256 6.7 / 10.8; 18 of
// 32 at 128 positions 8.7 / 7.7; E4M3 4 of 128 at 128 9.1 / 8.3.
bool in_small_tiles(bool f8, long long rows, double heads, int ctx) {
    const double units = heads * (double)((rows + kRows - 1) / kRows);
    return ctx <= 128 && units <= (f8 || rows <= 64 ? 1 : 3) * sms();
}

// Rows of a unit: on the wide kernel 64, and 128 for bf16 where a KV head has more.
int unit_rows(long long rows, bool f8, bool wide) { return !wide ? kRows : f8 || rows <= 64 ? 64 : 128; }

// Resident blocks of the device.
int max_grid(bool wide) { return sms() * (wide ? 1 : kWarpsPerSm / 4); }

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace: the blocks' pieces, then m and z, then u; 256-byte aligned.
size_t workspace_size(int grid, int unit, int d) {
    const size_t rows = (size_t)2 * grid * unit;
    return up256(16 * (size_t)grid) + 2 * up256(4 * rows) + 4 * rows * d;
}

// Warps of a block: four, three blocks to an SM, or twelve where every unit
// can have an SM to itself, is long enough to share (one warp alone folds its
// tile of 16 positions in 0.85 us) and the device is not filled.  Four against
// twelve, us: 32 units of 37 positions 6.6 / 7.5, 256 9.4 / 8.7, 768 17.0 /
// 11.7, 2048 18.0 / 15.8 (E4M3 19.0 / 14.3); 144 units of 1536 28.9 / 25.3;
// 68 of 411 to 8221 20.2 / 22.8; 512 of 4096 E4M3 102 / 116.
int block_warps(double units, int ctx) { return units <= sms() && ctx > 128 && units * ctx <= 1536.0 * sms() ? 12 : 4; }

template <int D, bool F8, int kWarps>
int launch_multi(const CUtensorMap& mk, const CUtensorMap& mv, const MultiArgs& a, int grid, cudaStream_t st) {
    static int attr[64] = {0};
    constexpr int kSmem = Geo<D, F8, kWarps>::kSmem;
    if (pa_host::ensure_smem_attr(multi_kernel<D, F8, kWarps>, kSmem, attr) != cudaSuccess) return PA_ERR_CUDA;
    return pa_host::launch_dependent(multi_kernel<D, F8, kWarps>, dim3(grid), dim3(32 * kWarps), kSmem, st, mk, mv, a) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

template <int D, bool F8>
int launch_multi(int warps, const CUtensorMap& mk, const CUtensorMap& mv, const MultiArgs& a, int grid, cudaStream_t st) {
    return warps == 12 ? launch_multi<D, F8, 12>(mk, mv, a, grid, st) : launch_multi<D, F8, 4>(mk, mv, a, grid, st);
}

int decode_multi(void* out, int out_dtype, const void* q, const void* k_cache, const void* v_cache,
                 const int32_t* block_tables, const int32_t* query_start, const int32_t* context_lens,
                 const int64_t* tree_mask, int block_size, float scale, int n_q_heads, int n_kv_heads, int d_head,
                 int num_seqs, int num_tokens, int max_query_len, int max_blocks_per_seq, int num_blocks,
                 int max_context_len, void* workspace, size_t workspace_bytes, int32_t* status_dev, void* stream,
                 bool f8, float k_scale, float v_scale) {
    if (num_seqs < 0 || num_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || max_query_len <= 0 ||
        max_blocks_per_seq <= 0 || num_blocks <= 0 || max_context_len < 0 || !(scale == scale))
        return PA_ERR_INVALID_ARG;
    if (f8 && (!(k_scale > 0.f) || !(v_scale > 0.f) || !(k_scale < INFINITY) || !(v_scale < INFINITY)))
        return PA_ERR_INVALID_ARG;
    if (out_dtype != PA_DTYPE_BF16 && out_dtype != PA_DTYPE_F32) return PA_ERR_INVALID_ARG;
    if (!pa_host::supported_block_size(block_size) || !pa_host::supported_d_head(d_head)) return PA_ERR_UNSUPPORTED;
    if (f8 && d_head != 128) return PA_ERR_UNSUPPORTED;
    if (n_q_heads % n_kv_heads) return PA_ERR_UNSUPPORTED;
    const int group = n_q_heads / n_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8 && group != 16) return PA_ERR_UNSUPPORTED;
    if (tree_mask && max_query_len > 64) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !query_start || !context_lens || out == q)
        return PA_ERR_INVALID_ARG;
    if (!pa_host::aligned16(out) || !pa_host::aligned16(q) || !pa_host::aligned16(k_cache) ||
        !pa_host::aligned16(v_cache) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
        (reinterpret_cast<uintptr_t>(query_start) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
        return PA_ERR_MISALIGNED;
    const long long cache_rows = (long long)num_blocks * n_kv_heads * block_size;
    if (cache_rows > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    const long long all_rows = (long long)max_query_len * group;
    const long long cap = (long long)max_blocks_per_seq * block_size;
    const int ctx_cap = (int)(cap < max_context_len ? cap : max_context_len);
    const bool wide = is_wide(f8, scale, all_rows) && !in_small_tiles(f8, all_rows, (double)num_seqs * n_kv_heads, ctx_cap);
    const int unit = unit_rows(all_rows, f8, wide);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return PA_ERR_WORKSPACE;
    const int most = max_grid(wide);
    if (most <= 0) return PA_ERR_CUDA;
    if (workspace_bytes < workspace_size(most, unit, d_head)) return PA_ERR_WORKSPACE;

    MultiArgs a{};
    a.ctx_cap = ctx_cap;
    // no more blocks than the largest possible work has smallest shares
    const double units = (double)num_seqs * n_kv_heads * (double)((all_rows + unit - 1) / unit);
    const int warps = wide ? 0 : block_warps(units, a.ctx_cap);
    const int step = wide ? kWideStep : step_of(warps), cost = wide ? kWideCost : cost_of(warps, f8);
    const int blocks = wide || warps == 12 ? sms() : most;
    const long long tiles = (all_rows + unit - 1) / unit;
    const long long seq_work = ((long long)a.ctx_cap + step - 1) / step + cost;
    const double work = (double)num_seqs * n_kv_heads * (double)tiles * (double)seq_work;
    const double shares = work / ((wide ? kWideMinSteps : least_of(warps)) + cost) + 1;
    const bool direct = a.ctx_cap <= step * (wide ? kWideDirectSteps : direct_of(warps)) && units <= blocks;
    const int grid = direct ? (int)units : shares < blocks ? (int)shares : blocks;
    a.direct = direct ? (int)tiles : 0;

    a.out = out;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.query_start = query_start;
    a.context_lens = context_lens;
    a.tree_mask = reinterpret_cast<const uint64_t*>(tree_mask);
    const size_t rows = (size_t)2 * grid * unit;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.pieces = reinterpret_cast<int4*>(w);
    w += up256(16 * (size_t)grid);
    a.part_m = reinterpret_cast<float*>(w);
    w += up256(4 * rows);
    a.part_z = reinterpret_cast<float*>(w);
    w += up256(4 * rows);
    a.part_u = reinterpret_cast<float*>(w);
    a.status = status_dev;
    const float factor = fabsf(scale) * kLog2e * (f8 ? k_scale : 1.f);
    a.scale_log2 = factor == 0.f ? 1.f : factor;                // masked scores are -inf times it
    a.q_sign = factor == 0.f ? 0.f : scale > 0.f ? 1.f : -1.f;
    a.v_scale = !f8 ? 1.f : wide ? v_scale : v_scale / kWeightScale;   // (the wide kernel's sums carry its weights' factor)
    a.out_f32 = out_dtype == PA_DTYPE_F32;
    a.log2_block = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = n_kv_heads;
    a.log2_group = group == 1 ? 0 : group == 2 ? 1 : group == 4 ? 2 : group == 8 ? 3 : 4;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.num_seqs = num_seqs;
    a.num_tokens = num_tokens;
    a.max_query_len = max_query_len;
    // a box of the wide kernel is a block, of the others at most a warp's tile
    const int box = wide || block_size < kTile ? block_size : kTile;
    CUtensorMap mk, mv;
    if (!pa_host::cache_view(&mk, k_cache, cache_rows, d_head, f8 ? 1 : 2, box) ||
        !pa_host::cache_view(&mv, v_cache, cache_rows, d_head, f8 ? 1 : 2, box))
        return PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc;
    if (wide)
        rc = launch_wide(unit, d_head, f8, q, block_size, mk, mv, a, grid, st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    else
        rc = f8 ? launch_multi<128, true>(warps, mk, mv, a, grid, st)
             : d_head == 128 ? launch_multi<128, false>(warps, mk, mv, a, grid, st)
                             : launch_multi<64, false>(warps, mk, mv, a, grid, st);
    if (rc != PA_OK || direct) return rc;                        // (no unit is shared: nothing to merge)
    // Few units come in many pieces: four threads then share four columns of a row, in more blocks; else one thread
    // takes all of its pieces.  (3 units of 66 pieces 22 us against 32; 512 units over 456 blocks 105 against 101.)
    const bool few = units * 4 <= grid;
    const int columns = unit * d_head / 4, items = few ? 64 : kMergeThreads;
    const int splits = few ? std::min(columns / items, 16) : std::min((columns + items - 1) / items, 4);
    const auto merge = few ? (d_head == 128 ? merge_kernel<128, 64> : merge_kernel<64, 64>)
                           : (d_head == 128 ? merge_kernel<128, kMergeThreads> : merge_kernel<64, kMergeThreads>);
    return pa_host::launch_dependent(merge, dim3(grid, splits), dim3(kMergeThreads), 0, st, a, unit) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t pa_decode_multi_workspace_size(int max_query_len, int n_q_heads, int n_kv_heads, int d_head) {
    if (max_query_len <= 0 || n_kv_heads <= 0 || n_q_heads < n_kv_heads || d_head <= 0) return 0;
    // one size for whichever kernel a call of this shape takes
    const long long rows = (long long)max_query_len * (n_q_heads / n_kv_heads);
    size_t most = 0;
    for (int x = 0; x < 4; ++x) {
        const bool f8 = x & 1, wide = is_wide(f8, x & 2 ? 1.f : -1.f, rows);
        const int unit = unit_rows(rows, f8, wide);
        const size_t n = workspace_size(max_grid(wide), unit, d_head);
        most = n > most ? n : most;
    }
    return most;
}

int pa_decode_multi(void* out, int out_dtype, const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, const int32_t* query_start, const int32_t* context_lens,
                    const int64_t* tree_mask, int block_size, float scale, int n_q_heads, int n_kv_heads, int d_head,
                    int num_seqs, int num_tokens, int max_query_len, int max_blocks_per_seq, int num_blocks,
                    int max_context_len, void* workspace, size_t workspace_bytes, int32_t* status_dev, void* stream) {
    return decode_multi(out, out_dtype, q, k_cache, v_cache, block_tables, query_start, context_lens, tree_mask,
                        block_size, scale, n_q_heads, n_kv_heads, d_head, num_seqs, num_tokens, max_query_len,
                        max_blocks_per_seq, num_blocks, max_context_len, workspace, workspace_bytes, status_dev,
                        stream, false, 1.f, 1.f);
}

int pa_decode_multi_fp8(void* out, int out_dtype, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_tables, const int32_t* query_start, const int32_t* context_lens,
                        const int64_t* tree_mask, int block_size, float scale, float k_scale, float v_scale,
                        int n_q_heads, int n_kv_heads, int d_head, int num_seqs, int num_tokens, int max_query_len,
                        int max_blocks_per_seq, int num_blocks, int max_context_len, void* workspace,
                        size_t workspace_bytes, int32_t* status_dev, void* stream) {
    return decode_multi(out, out_dtype, q, k_cache, v_cache, block_tables, query_start, context_lens, tree_mask,
                        block_size, scale, n_q_heads, n_kv_heads, d_head, num_seqs, num_tokens, max_query_len,
                        max_blocks_per_seq, num_blocks, max_context_len, workspace, workspace_bytes, status_dev,
                        stream, true, k_scale, v_scale);
}

}  // extern "C"
