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
// What bounds it: each K/V byte is read once for n * G rows, 4 * n * G
// operations per two bytes, so up to some tens of rows the cache's bytes
// bound it and the design is the single-token kernel's, with more columns:
//  * Work is counted in steps of 64 positions of one unit (sequence, KV
//    head, tile of 8 * NT rows).  The grid's blocks take equal contiguous
//    shares of all the steps, computed from the lengths by every block for
//    itself: no partition size to choose, no empty blocks on ragged batches,
//    and at most two unfinished units per block whatever the batch.
//  * A block's 4 warps take 16 positions of a step each, from rings of
//    shared-memory stages that TMA fills through the block table.  Keys are
//    the rows of the products (S[16 x 8 NT] = K . Q^T, O^T += V^T . P^T), so
//    a K or V fragment is loaded once for all the tile's rows.
//  * The running maximum of a column is raised only when a score exceeds it
//    by 2^8 (one vote instead of the shuffles of a maximum); weights stay
//    within 2^8 and sums in fp32.
//  * A unit that one block covers is written at once.  Pieces of the others
//    go to the workspace as (m, z, u), and a second kernel, one block per
//    unit that a block began and did not finish, merges them.

#include <math.h>

#include "pa_mma.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;                  // positions per warp and step
constexpr int kStep = kWarps * kTile;
constexpr int kMaxProbes = 2000000;        // ~2 s bound on any single wait
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRaise = 8.0f;             // log2 of the largest weight before the maximum is raised
constexpr float kWeightScale = 128.f;      // FP8: weights enter f16 products times 2^7 (at most 2^15)
constexpr int kMinShare = 4;               // steps per block, at least
constexpr int kMergeThreads = 256;
constexpr int kMergeSplit = 4;             // blocks per unit to merge

struct MultiArgs {
    void* out;
    const __nv_bfloat16* q;
    const int32_t* block_tables;
    const int32_t* query_start;
    const int32_t* context_lens;
    const uint64_t* tree_mask;             // null: causal
    int4* pieces;                          // per block: {sequence or -1, KV head, row tile, last block}
    float* part_m;                         // [2 per block][rows]
    float* part_z;
    float* part_u;                         // [2 per block][rows][D]
    int32_t* status;
    float scale_log2;                      // scale * log2(e), times the K scale
    float v_scale;                         // factor on the weighted sums
    int out_f32, log2_block, n_q_heads, n_kv_heads, log2_group, max_blocks, num_blocks, ctx_cap, num_seqs, num_tokens,
        max_query_len;
};

template <int D, bool F8, int NT>
struct Geo {
    static constexpr int kRows = 8 * NT;
    static constexpr int kSlabs = F8 ? 1 : D / 64;               // 128-byte boxes per row
    static constexpr int kSlabBytes = kTile * 128;
    static constexpr int kTileBytes = kSlabs * kSlabBytes;       // K or V of one tile
    static constexpr int kStageBytes = 2 * kTileBytes;
    // bytes in flight per SM decide: 64 KB per block at three blocks, 96 at two
    static constexpr int kBlocksPerSm = NT > 2 ? 2 : 3;
    static constexpr int kStages = (NT > 2 ? 98304 : 65536) / (kWarps * kStageBytes);
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kUStride = D + 4;                       // floats per row of the merge: banks differ
    static constexpr int kMergeBytes = 4 * kWarps * kRows * (kUStride + 2);
    static constexpr int kMain = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
    static constexpr int kQStride = 2 * D + 16;                  // bytes per row of q: ldmatrix rows hit distinct banks
    static constexpr int kSmem = 1024 + kMain + kRows * (kQStride + 4) + kWarps * kStages * 8;
    static constexpr int kSteps = D / 16;
};

__device__ __forceinline__ void put(void* out, int f32, size_t i, float v) {
    if (f32)
        static_cast<float*>(out)[i] = v;
    else
        static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

// A sequence's part of the step: its work in steps is units * steps.
struct Seq {
    int q0, n, ctx, steps, tiles;
    __device__ __forceinline__ long long work(int heads) const { return (long long)heads * tiles * steps; }
};

template <int kRows>
__device__ __forceinline__ Seq read_seq(const MultiArgs& a, int s, bool flag) {
    Seq r;
    r.q0 = a.query_start[s];
    const int q1 = a.query_start[s + 1];
    int ctx = a.context_lens[s];
    bool bad = ctx < 0 || ctx > a.ctx_cap;
    ctx = ctx < 0 ? 0 : (ctx > a.ctx_cap ? a.ctx_cap : ctx);
    r.n = q1 - r.q0;
    if (r.q0 < 0 || q1 > a.num_tokens || q1 < r.q0 || r.n > ctx || r.n > a.max_query_len) {
        r.n = 0;                                        // nothing of it is computed
        bad = true;
    }
    if (bad && flag) pa::set_status(a.status, PA_DEV_BAD_CONTEXT);
    r.ctx = ctx;
    r.tiles = (int)((((long long)r.n << a.log2_group) + kRows - 1) / kRows);
    r.steps = r.n ? (ctx + kStep - 1) / kStep : 0;
    return r;
}

template <int D, bool F8, int NT>
struct Cols {                              // one warp's running state
    float m[NT][2], l[NT][2];
    float acc[NT][D / 16][4];
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) acc[t][k][0] = acc[t][k][1] = acc[t][k][2] = acc[t][k][3] = 0.f;
        }
    }
};

// What a lane needs to mask a tile: the unit's rows and the sequence's lengths.
struct Unit {
    int ctx, first, n, row0;               // first: position of new token 0; row0: the tile's first row
    const uint64_t* words;                 // mask words of the sequence's tokens, or null
};

__device__ __forceinline__ bool visible(const Unit& u, int log2_group, int row, int pos) {
    if (pos >= u.ctx) return false;
    if (pos < u.first) return true;
    const int i = (u.row0 + row) >> log2_group, j = pos - u.first;
    if (i >= u.n) return true;             // a row that is not there: any finite result will do
    return u.words ? (j < 64 && (u.words[i] >> j & 1ull)) : j <= i;
}

// Fold one tile (K at shared address ks, V at vs, positions t0 .. t0 + 15)
// into the warp's state.
template <int D, bool F8, int NT>
__device__ __forceinline__ void fold_tile(Cols<D, F8, NT>& st, uint32_t ks, uint32_t vs, uint32_t qs,
                                          const float* q_scale, int t0, const Unit& u, const MultiArgs& a, int lane,
                                          const uint32_t (&qr)[NT <= 2 ? D / 16 : 1][NT][2]) {
    using G = Geo<D, F8, NT>;
    const int g = lane >> 2, t4 = lane & 3, mi = lane >> 3;
    const int k_row = ((mi & 1) << 3) + (lane & 7), k_add = mi >> 1;
    // q fragments of k-step kk: from registers (NT <= 2) or shared memory
    auto q_frag = [&](int kk, uint32_t (&b)[NT][2]) {
        if constexpr (NT <= 2) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                b[t][0] = qr[kk][t][0];
                b[t][1] = qr[kk][t][1];
            }
        } else {
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                uint32_t r[4];
                pa::ldsm4(qs + (8 * t + ((mi >> 1) << 3) + (lane & 7)) * G::kQStride + (2 * kk + (mi & 1)) * 16, r);
                b[t][0] = r[0];
                b[t][1] = r[1];
                b[t + 1][0] = r[2];
                b[t + 1][1] = r[3];
            }
        }
    };
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
    if constexpr (F8) {
#pragma unroll
        for (int j = 0; j < G::kSteps / 2; ++j) {
            uint32_t r[4], af[4], b[NT][2];
            pa::ldsm4(ks + pa::swz128(k_row, 2 * j + k_add), r);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                pa::e4m3x4_to_f16x4(r[2 * h], af[0], af[2]);
                pa::e4m3x4_to_f16x4(r[2 * h + 1], af[1], af[3]);
                q_frag(2 * j + h, b);
#pragma unroll
                for (int t = 0; t < NT; ++t) pa::mma16816<true>(s[t], af, b[t][0], b[t][1]);
            }
        }
    } else {
#pragma unroll
        for (int kk = 0; kk < G::kSteps; ++kk) {
            uint32_t af[4], b[NT][2];
            pa::ldsm4(ks + (kk >> 2) * G::kSlabBytes + pa::swz128(k_row, 2 * (kk & 3) + k_add), af);
            q_frag(kk, b);
#pragma unroll
            for (int t = 0; t < NT; ++t) pa::mma16816<false>(s[t], af, b[t][0], b[t][1]);
        }
    }
    // s[t][0], [1]: position g, columns 2 t4 and 2 t4 + 1; [2], [3]: position g + 8
    bool raise = false;
    const bool tail = t0 + kTile > u.first;            // some row may not see some position
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float c0 = a.scale_log2, c1 = a.scale_log2;
        if constexpr (F8) {
            const float2 c = *reinterpret_cast<const float2*>(q_scale + 8 * t + 2 * t4);
            c0 = c.x;
            c1 = c.y;
        }
        s[t][0] *= c0;
        s[t][1] *= c1;
        s[t][2] *= c0;
        s[t][3] *= c1;
        if (tail) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!visible(u, a.log2_group, 8 * t + 2 * t4 + (e & 1), t0 + g + (e >> 1) * 8)) s[t][e] = -INFINITY;
        }
        raise |= fmaxf(s[t][0], s[t][2]) > st.m[t][0] + kRaise || fmaxf(s[t][1], s[t][3]) > st.m[t][1] + kRaise;
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float b0 = fmaxf(s[t][0], s[t][2]), b1 = fmaxf(s[t][1], s[t][3]);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
                b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, o));
                b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, o));
            }
            const float n0 = fmaxf(st.m[t][0], b0), n1 = fmaxf(st.m[t][1], b1);
            // a column that has seen nothing yet has sums of zero, whatever the factor
            const float f0 = n0 == -INFINITY ? 1.f : pa::exp2_approx(st.m[t][0] - n0);
            const float f1 = n1 == -INFINITY ? 1.f : pa::exp2_approx(st.m[t][1] - n1);
            st.m[t][0] = n0;
            st.m[t][1] = n1;
            st.l[t][0] *= f0;
            st.l[t][1] *= f1;
#pragma unroll
            for (int k = 0; k < G::kSteps; ++k) {
                st.acc[t][k][0] *= f0;
                st.acc[t][k][1] *= f1;
                st.acc[t][k][2] *= f0;
                st.acc[t][k][3] *= f1;
            }
        }
    }
    // weights as the B operand: bf16 in two terms (a relative 2^-16), f16 times 2^7 (2^-11)
    uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const float m0 = st.m[t][0] == -INFINITY ? 0.f : st.m[t][0], m1 = st.m[t][1] == -INFINITY ? 0.f : st.m[t][1];
        const float p0 = pa::exp2_approx(s[t][0] - m0), p1 = pa::exp2_approx(s[t][1] - m1);
        const float p2 = pa::exp2_approx(s[t][2] - m0), p3 = pa::exp2_approx(s[t][3] - m1);
        st.l[t][0] += p0 + p2;
        st.l[t][1] += p1 + p3;
        if constexpr (F8) {
            bh[t][0] = pa::transpose8(pa::pack_f16x2(p0 * kWeightScale, p1 * kWeightScale));
            bh[t][1] = pa::transpose8(pa::pack_f16x2(p2 * kWeightScale, p3 * kWeightScale));
        } else {
            const uint32_t h01 = pa::pack_bf16x2(p0, p1), h23 = pa::pack_bf16x2(p2, p3);
            const float2 f01 = pa::bf16x2_to_float2(h01), f23 = pa::bf16x2_to_float2(h23);
            bh[t][0] = pa::transpose8(h01);
            bh[t][1] = pa::transpose8(h23);
            bl[t][0] = pa::transpose8(pa::pack_bf16x2(p0 - f01.x, p1 - f01.y));
            bl[t][1] = pa::transpose8(pa::pack_bf16x2(p2 - f23.x, p3 - f23.y));
        }
    }
    // O^T += V^T . P^T; V rows past the context are zeroed (0 * NaN)
    const int nv = u.ctx - t0;
    uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
    if (nv < kTile) {
        const int t = 2 * t4;
        mlo = (t < nv ? 0x0000ffffu : 0u) | (t + 1 < nv ? 0xffff0000u : 0u);
        mhi = (t + 8 < nv ? 0x0000ffffu : 0u) | (t + 9 < nv ? 0xffff0000u : 0u);
    }
    if constexpr (F8) {
#pragma unroll
        for (int j = 0; j < G::kSteps / 2; ++j) {
            uint32_t r[4];
            pa::ldsm4_trans(vs + pa::swz128(k_row, 2 * j + k_add), r);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t af[4];
                pa::e4m3x4_to_f16x4(pa::byte_perm(r[2 * h], 0x3120u), af[0], af[1]);
                pa::e4m3x4_to_f16x4(pa::byte_perm(r[2 * h + 1], 0x3120u), af[2], af[3]);
                af[0] &= mlo;
                af[1] &= mlo;
                af[2] &= mhi;
                af[3] &= mhi;
#pragma unroll
                for (int t = 0; t < NT; ++t) pa::mma16816<true>(st.acc[t][2 * j + h], af, bh[t][0], bh[t][1]);
            }
        }
    } else {
        const int v_row = ((mi >> 1) << 3) + (lane & 7), v_add = mi & 1;
#pragma unroll
        for (int k = 0; k < G::kSteps; ++k) {
            uint32_t af[4];
            pa::ldsm4_trans(vs + (k >> 2) * G::kSlabBytes + pa::swz128(v_row, 2 * (k & 3) + v_add), af);
            af[0] &= mlo;
            af[1] &= mlo;
            af[2] &= mhi;
            af[3] &= mhi;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                pa::mma16816<false>(st.acc[t][k], af, bh[t][0], bh[t][1]);
                pa::mma16816<false>(st.acc[t][k], af, bl[t][0], bl[t][1]);
            }
        }
    }
}

template <int D, bool F8, int NT>
__global__ void __launch_bounds__(kThreads, Geo<D, F8, NT>::kBlocksPerSm)
    multi_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const MultiArgs a) {
    using G = Geo<D, F8, NT>;
    constexpr int kRows = G::kRows, kStages = G::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* qsm = ring + G::kMain;                               // [kRows][kQStride]
    float* q_scale = reinterpret_cast<float*>(qsm + kRows * G::kQStride);   // FP8: score factor per row
    uint64_t* bars = reinterpret_cast<uint64_t*>(q_scale + kRows);
    __shared__ long long sums[kWarps];
    __shared__ long long where_off;
    __shared__ int where_seq;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = 1 << a.log2_block, heads = a.n_kv_heads;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) pa::mbar_init(&bars[i], 1);
        pa::fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- this block's share: thread t counts sequences [t * per, (t + 1) * per) ----
    const int per = (a.num_seqs + kThreads - 1) / kThreads;
    const int s_lo = threadIdx.x * per, s_hi = min(a.num_seqs, s_lo + per);
    long long mine = 0;
    for (int s = s_lo; s < s_hi; ++s) mine += read_seq<kRows>(a, s, blockIdx.x == 0).work(heads);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
    }
    long long share = (total + gridDim.x - 1) / gridDim.x;
    share = share < kMinShare ? kMinShare : share;
    const long long begin = share * blockIdx.x;
    long long end = begin + share;
    end = end > total ? total : end;
    if (threadIdx.x == 0) a.pieces[blockIdx.x].x = -1;
    if (begin >= total) return;
    if (begin >= upto - mine && begin < upto) {                  // one thread's range holds the first step
        long long off = begin - (upto - mine);
        for (int s = s_lo;; ++s) {
            const long long w = read_seq<kRows>(a, s, false).work(heads);
            if (off < w) {
                where_seq = s;
                where_off = off;
                break;
            }
            off -= w;
        }
    }
    __syncthreads();
    int seq = where_seq;
    long long off = where_off;                                   // steps of the sequence before the current one
    Seq sq = read_seq<kRows>(a, seq, false);

    const uint64_t policy = pa::l2_evict_first_policy();
    uint64_t* wbars = bars + warp * kStages;
    const uint32_t wring = pa::smem_addr(ring) + warp * kStages * G::kStageBytes;
    const uint32_t qs = pa::smem_addr(qsm);
    int used = 0;                                                // stages this warp consumed in earlier segments
    Cols<D, F8, NT> st;

    for (long long cur = begin; cur < end;) {
        while (off >= sq.work(heads)) {
            off -= sq.work(heads);
            sq = read_seq<kRows>(a, ++seq, false);
        }
        const int unit = (int)(off / sq.steps), st0 = (int)(off - (long long)unit * sq.steps);
        const int len = (int)min((long long)(sq.steps - st0), end - cur);
        const int kvh = unit / sq.tiles, tile = unit - kvh * sq.tiles;
        Unit u;
        u.ctx = sq.ctx;
        u.n = sq.n;
        u.first = sq.ctx - sq.n;
        u.row0 = tile * kRows;
        u.words = a.tree_mask ? a.tree_mask + sq.q0 : nullptr;
        const int32_t* table = a.block_tables + (size_t)seq * a.max_blocks;

        // ---- this warp's tiles: positions (st0 + k) * 64 + 16 warp, k < mine_k ----
        const int base = st0 * kStep + warp * kTile;
        const int mine_k = base >= u.ctx ? 0 : min(len, (u.ctx - base + kStep - 1) / kStep);
        // table entries of 32 tiles at a time, one per lane, the next 32 fetched ahead
        auto fetch = [&](int k, int& e0, int& e1) {
            e0 = e1 = 0;
            if (k < mine_k) {
                const int t0 = base + k * kStep;
                e0 = table[t0 >> a.log2_block];
                if (B < kTile && t0 + B < u.ctx) e1 = table[(t0 >> a.log2_block) + 1];
            }
        };
        int e0, e1, f0, f1;
        fetch(lane, e0, e1);
        fetch(32 + lane, f0, f1);
        auto issue = [&](int k) {                                // whole warp
            if (k && (k & 31) == 0) {
                e0 = f0;
                e1 = f1;
                fetch(k + 32 + lane, f0, f1);
            }
            int b0 = __shfl_sync(0xffffffffu, e0, k & 31), b1 = __shfl_sync(0xffffffffu, e1, k & 31);
            if (lane == 0) {
                const int t0 = base + k * kStep;
                const int box = B < kTile ? B : kTile, boxes = (B < kTile && t0 + B < u.ctx) ? 2 : 1;
                const int stage = (used + k) % kStages;
                uint64_t* bar = &wbars[stage];
                const uint32_t dst = wring + stage * G::kStageBytes;
                pa::mbar_arrive_expect_tx(bar, (uint32_t)(2 * G::kSlabs * boxes * box * 128));
                for (int r = 0; r < boxes; ++r) {
                    int blk = r ? b1 : b0;
                    if (blk < 0 || blk >= a.num_blocks) {
                        pa::set_status(a.status, PA_DEV_BAD_BLOCK_ID);
                        blk = 0;
                    }
                    const int row = (blk * heads + kvh) * B + (r ? 0 : t0 & (B - 1));
#pragma unroll
                    for (int h = 0; h < G::kSlabs; ++h) {
                        const uint32_t d = dst + h * G::kSlabBytes + r * box * 128;
                        pa::tma_box(d, &map_k, h * 64, row, bar, policy);
                        pa::tma_box(d + G::kTileBytes, &map_v, h * 64, row, bar, policy);
                    }
                }
            }
        };
        for (int k = 0; k < kStages; ++k)
            if (k < mine_k) issue(k);

        // ---- q of the unit's rows to shared memory, 8 elements per thread ----
        constexpr int kLanesQ = D / 8;
        for (int x = threadIdx.x; x < kRows * kLanesQ; x += kThreads) {
            const int r = x / kLanesQ, c = x % kLanesQ;
            const int row = u.row0 + r, i = row >> a.log2_group;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (i < u.n)
                v = *reinterpret_cast<const uint4*>(
                    a.q + ((size_t)(sq.q0 + i) * a.n_q_heads + (kvh << a.log2_group) + (row & ((1 << a.log2_group) - 1))) * D +
                    8 * c);
            uint8_t* dst = qsm + r * G::kQStride;
            if constexpr (F8) {
                // f16 after a power of two per row that brings its largest element into [2^14, 2^15)
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
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
                if (c == 0) q_scale[r] = a.scale_log2 / up;
                // within 16 elements, place 2 j holds d = 4 j and place 2 j + 8 holds
                // d = 4 j + 2 (pairs): the order in which ldmatrix hands out K's codes
                uint32_t* p = reinterpret_cast<uint32_t*>(dst + (c >> 1) * 32);
                const int j = (c & 1) * 2;
                p[j] = pa::pack_f16x2(f[0] * up, f[1] * up);
                p[j + 4] = pa::pack_f16x2(f[2] * up, f[3] * up);
                p[j + 1] = pa::pack_f16x2(f[4] * up, f[5] * up);
                p[j + 5] = pa::pack_f16x2(f[6] * up, f[7] * up);
            } else {
                *reinterpret_cast<uint4*>(dst + 16 * c) = v;
            }
        }
        __syncthreads();
        uint32_t qr[NT <= 2 ? G::kSteps : 1][NT][2];
        if constexpr (NT <= 2) {
#pragma unroll
            for (int kk = 0; kk < G::kSteps; ++kk)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    pa::ldsm2(qs + (8 * t + (lane & 7)) * G::kQStride + (2 * kk + ((lane >> 3) & 1)) * 16, qr[kk][t][0],
                              qr[kk][t][1]);
        }

        st.reset();
        bool landed = true;
        for (int k = 0; k < mine_k; ++k) {
            const int stage = (used + k) % kStages;
            if (!__all_sync(0xffffffffu, pa::mbar_wait_bounded(&wbars[stage], ((used + k) / kStages) & 1, kMaxProbes))) {
                // give up: nothing more is issued, and the copies in flight are waited for, each within the limit
                if (lane == 0) pa::set_status(a.status, PA_DEV_WAIT_TIMEOUT);
                const int issued = min(mine_k, k + kStages);
                for (int j = k; j < issued; ++j)
                    pa::mbar_wait_bounded(&wbars[(used + j) % kStages], ((used + j) / kStages) & 1, kMaxProbes);
                landed = false;
                break;
            }
            const uint32_t ks = wring + stage * G::kStageBytes;
            fold_tile<D, F8, NT>(st, ks, ks + G::kTileBytes, qs, q_scale, base + k * kStep, u, a, lane, qr);
            __syncwarp();
            if (k + kStages < mine_k) issue(k + kStages);
        }
        used += mine_k;

        // ---- join the warps' states (the exact block merge) ----
        if (!__syncthreads_and(landed)) return;
        float* um = reinterpret_cast<float*>(ring);              // [warp][row]
        float* ul = um + kWarps * kRows;
        float* uu = ul + kWarps * kRows;                         // [warp][row][kUStride]
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
                st.l[t][0] += __shfl_xor_sync(0xffffffffu, st.l[t][0], o);
                st.l[t][1] += __shfl_xor_sync(0xffffffffu, st.l[t][1], o);
            }
            const int r0 = warp * kRows + 8 * t + 2 * t4;
            if (g == 0) {
                um[r0] = st.m[t][0];
                um[r0 + 1] = st.m[t][1];
                ul[r0] = st.l[t][0];
                ul[r0 + 1] = st.l[t][1];
            }
#pragma unroll
            for (int k = 0; k < G::kSteps; ++k) {
                float* p = uu + r0 * G::kUStride + 16 * k + (F8 ? 2 * g : g);
                constexpr int kNext = F8 ? 1 : 8;
                p[0] = st.acc[t][k][0];
                p[G::kUStride] = st.acc[t][k][1];
                p[kNext] = st.acc[t][k][2];
                p[G::kUStride + kNext] = st.acc[t][k][3];
            }
        }
        __syncthreads();
        const long long unit_begin = cur - st0;                  // in steps of the whole call
        const bool whole = len == sq.steps;
        const int slot = 2 * blockIdx.x + (unit_begin >= begin ? 1 : 0);
        for (int x = threadIdx.x; x < kRows * D; x += kThreads) {
            const int r = x / D, d = x % D;
            const int row = u.row0 + r, i = row >> a.log2_group;
            if (i >= u.n) break;                                 // rows come in order
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, um[w * kRows + r]);
            float Z = 0.f, U = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                // a warp that saw nothing adds its zeros as they are (or the NaN of a score)
                const float f = um[w * kRows + r] == -INFINITY ? 1.f : pa::exp2_approx(um[w * kRows + r] - M);
                Z += f * ul[w * kRows + r];
                U += f * uu[(w * kRows + r) * G::kUStride + d];
            }
            if (whole) {
                const size_t o = ((size_t)(sq.q0 + i) * a.n_q_heads + (kvh << a.log2_group) +
                                  (row & ((1 << a.log2_group) - 1))) * D + d;
                put(a.out, a.out_f32, o, Z == 0.f ? 0.f : U * a.v_scale / Z);
            } else {
                a.part_u[((size_t)slot * kRows + r) * D + d] = U;
                if (d == 0) {
                    a.part_m[slot * kRows + r] = M;
                    a.part_z[slot * kRows + r] = Z;
                }
            }
        }
        if (!whole && (slot & 1) && threadIdx.x == 0)            // this block began the unit
            a.pieces[blockIdx.x] = make_int4(seq, kvh, tile, (int)((unit_begin + sq.steps - 1) / share));
        cur += len;
        off += len;
        __syncthreads();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the ring goes back to TMA
    }
}

// out of the units that several blocks share: pieces of block b (its second
// slot) and of blocks b + 1 .. last (their first), in that order.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const MultiArgs a, int rows) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int4 p = a.pieces[blockIdx.x];
    if (p.x < 0) return;
    const int q0 = a.query_start[p.x], n = a.query_start[p.x + 1] - q0;
    const int G = 1 << a.log2_group;
    for (int x = blockIdx.y * kMergeThreads + threadIdx.x; x < rows * D; x += kMergeSplit * kMergeThreads) {
        const int r = x / D, d = x % D;
        const int row = p.z * rows + r, i = row >> a.log2_group;
        if (i >= n) return;
        float M = -INFINITY, Z = 0.f, U = 0.f;
        for (int b = blockIdx.x; b <= p.w; ++b) {
            const int at = (2 * b + (b == (int)blockIdx.x)) * rows + r;
            const float m = a.part_m[at];
            const float z = a.part_z[at], u = a.part_u[(size_t)at * D + d];
            const float top = fmaxf(M, m);
            const float f = M == top ? 1.f : pa::exp2_approx(M - top), h = m == top ? 1.f : pa::exp2_approx(m - top);
            Z = Z * f + z * h;
            U = U * f + u * h;
            M = top;
        }
        put(a.out, a.out_f32, ((size_t)(q0 + i) * a.n_q_heads + p.y * G + (row & (G - 1))) * D + d,
            Z == 0.f ? 0.f : U * a.v_scale / Z);
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

// n-tiles of 8 rows: the fewest that hold all rows of a KV head, at most 4.
int n_tiles(int max_query_len, int group) {
    const long long rows = (long long)max_query_len * group;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

#ifndef PA_MULTI_WAVES
#define PA_MULTI_WAVES 1
#endif
int max_grid(int nt) { return sms() * (nt > 2 ? 2 : 3) * PA_MULTI_WAVES; }

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace: the blocks' pieces, then m and z, then u; 256-byte aligned.
size_t workspace_size(int grid, int nt, int d) {
    const size_t rows = (size_t)2 * grid * 8 * nt;
    return up256(16 * (size_t)grid) + 2 * up256(4 * rows) + 4 * rows * d;
}

template <int D, bool F8, int NT>
int launch_multi(const CUtensorMap& mk, const CUtensorMap& mv, const MultiArgs& a, int grid, cudaStream_t st) {
    static int attr[64] = {0};
    using G = Geo<D, F8, NT>;
    if (pa_host::ensure_smem_attr(multi_kernel<D, F8, NT>, G::kSmem, attr) != cudaSuccess) return PA_ERR_CUDA;
    if (pa_host::launch_dependent(multi_kernel<D, F8, NT>, dim3(grid), dim3(kThreads), G::kSmem, st, mk, mv, a) !=
        cudaSuccess)
        return PA_ERR_CUDA;
    return pa_host::launch_dependent(merge_kernel<D>, dim3(grid, kMergeSplit), dim3(kMergeThreads), 0, st, a,
                                     G::kRows) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

template <int D, bool F8>
int launch_multi(int nt, const CUtensorMap& mk, const CUtensorMap& mv, const MultiArgs& a, int grid, cudaStream_t st) {
    return nt == 1   ? launch_multi<D, F8, 1>(mk, mv, a, grid, st)
           : nt == 2 ? launch_multi<D, F8, 2>(mk, mv, a, grid, st)
                     : launch_multi<D, F8, 4>(mk, mv, a, grid, st);
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
    if (!out || !q || !k_cache || !v_cache || !block_tables || !query_start || !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!pa_host::aligned16(out) || !pa_host::aligned16(q) || !pa_host::aligned16(k_cache) ||
        !pa_host::aligned16(v_cache) || (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
        return PA_ERR_MISALIGNED;
    const long long cache_rows = (long long)num_blocks * n_kv_heads * block_size;
    if (cache_rows > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    const int nt = n_tiles(max_query_len, group);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return PA_ERR_WORKSPACE;
    const int most = max_grid(nt);
    if (most <= 0) return PA_ERR_CUDA;
    if (workspace_bytes < workspace_size(most, nt, d_head)) return PA_ERR_WORKSPACE;

    MultiArgs a{};
    const long long cap = (long long)max_blocks_per_seq * block_size;
    a.ctx_cap = (int)(cap < max_context_len ? cap : max_context_len);
    // no more blocks than the largest possible work has shares of kMinShare steps
    const long long tiles = ((long long)max_query_len * group + 8 * nt - 1) / (8 * nt);
    const long long seq_steps = ((long long)a.ctx_cap + kStep - 1) / kStep;
    const double work = (double)num_seqs * n_kv_heads * (double)tiles * (double)seq_steps;
    const double shares = work / kMinShare + 1;
    const int grid = shares < most ? (int)shares : most;

    a.out = out;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.block_tables = block_tables;
    a.query_start = query_start;
    a.context_lens = context_lens;
    a.tree_mask = reinterpret_cast<const uint64_t*>(tree_mask);
    const size_t rows = (size_t)2 * grid * 8 * nt;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.pieces = reinterpret_cast<int4*>(w);
    w += up256(16 * (size_t)grid);
    a.part_m = reinterpret_cast<float*>(w);
    w += up256(4 * rows);
    a.part_z = reinterpret_cast<float*>(w);
    w += up256(4 * rows);
    a.part_u = reinterpret_cast<float*>(w);
    a.status = status_dev;
    a.scale_log2 = scale * kLog2e * (f8 ? k_scale : 1.f);
    a.v_scale = f8 ? v_scale / kWeightScale : 1.f;
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
    const int box = block_size < kTile ? block_size : kTile;
    CUtensorMap mk, mv;
    if (!pa_host::cache_view(&mk, k_cache, cache_rows, d_head, f8 ? 1 : 2, box) ||
        !pa_host::cache_view(&mv, v_cache, cache_rows, d_head, f8 ? 1 : 2, box))
        return PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return f8 ? launch_multi<128, true>(nt, mk, mv, a, grid, st)
              : d_head == 128 ? launch_multi<128, false>(nt, mk, mv, a, grid, st)
                              : launch_multi<64, false>(nt, mk, mv, a, grid, st);
}

}  // namespace

extern "C" {

size_t pa_decode_multi_workspace_size(int max_query_len, int n_q_heads, int n_kv_heads, int d_head) {
    if (max_query_len <= 0 || n_kv_heads <= 0 || n_q_heads < n_kv_heads || d_head <= 0) return 0;
    const int nt = n_tiles(max_query_len, n_q_heads / n_kv_heads);
    return workspace_size(max_grid(nt), nt, d_head);
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
