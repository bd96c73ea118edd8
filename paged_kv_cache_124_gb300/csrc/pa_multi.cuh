// Shared by the kernels that attend several new tokens per sequence: their
// arguments, the even split of the work over the grid's blocks, and the merge
// of the units that several blocks share.
//
// A unit is a (sequence, KV head, tile of rows).  Its work is the steps of
// its context plus a constant for starting and joining it; block b takes the
// work from b * share to (b + 1) * share, sequence after sequence, heads and
// row tiles within them.  A share that begins within a unit's constant part
// begins with the unit's first step.  Where few units of short contexts leave
// blocks to spare, each block takes one unit instead and nothing is merged.
#pragma once

#include "pa_cap.cuh"
#include "pa_mma.cuh"

namespace pa_multi {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.0e38f;          // a row's maximum before it has seen anything
constexpr float kRaise = 8.0f;             // log2 of the largest weight before the maximum is raised
constexpr int kMaxProbes = 2000000;        // ~2 s bound on any single wait
constexpr int kMergeThreads = 256;

// A sequence's part of the call.
struct Seq {
    int q0, n, ctx, steps, tiles;
    // tiles is 0 where nothing is to be done; cost: steps that starting and joining a unit is worth
    __device__ __forceinline__ long long work(int heads, int cost) const {
        return (long long)heads * tiles * (steps + cost);
    }
};

// The stretch of one unit that a block computes: steps st0 .. st0 + len - 1.
struct Unit {
    int q0, n, ctx, first;                 // first: position of new token 0
    int kvh, row0, st0, len, seq, last;    // last: the block that ends the unit, if this one does not
    int whole, valid;                      // valid 0: the share has ended
};

// The like where each token sees an interval of positions: ctx is the end of
// the positions that some token of the sequence sees, lo their begin, and base
// (lo down to a multiple of 16, or of 32) where step 0 starts; blocks wholly in
// front of lo are not read, nor their table entries.  All tokens that see any
// see seen_lo .. seen_hi - 1.
struct ShapedSeq : Seq {
    int lo, base, first, seen_lo, seen_hi, blind;                 // blind: some token sees nothing
};
struct ShapedUnit : Unit {
    int lo, base, seen_lo, seen_hi, blind;
};

struct MultiArgs {
    using Seq = pa_multi::Seq;
    using Unit = pa_multi::Unit;
    static constexpr bool kShaped = false, kCurved = false;
    void* out;
    const __nv_bfloat16* q;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* query_start;
    const int32_t* context_lens;
    const uint64_t* tree_mask;             // null: causal
    int4* pieces;                          // per block: the unit that it begins and others end, or x of -1 (begun_unit)
    float* part_m;                         // [2 per block][rows]
    float* part_z;
    float* part_u;                         // [2 per block][rows][D]
    int32_t* status;
    float scale_log2;                      // |scale| * log2(e), times the K scale; > 0
    float q_sign;                          // the scale's sign (0: a scale of zero, scale_log2 is 1)
    float v_scale;                         // factor on the weighted sums
    int out_f32, log2_block, n_q_heads, n_kv_heads, log2_group, max_blocks, num_blocks, ctx_cap, num_seqs, num_tokens,
        max_query_len;
    int direct;                            // not 0: a block takes one whole unit, of `direct` row tiles a KV head
};

// Scores s become cap tanh(s / cap), less slope |p - j| (pa_attend); E4M3
// caches have a scale per block and head.
struct ShapedArgs : MultiArgs {
    using Seq = ShapedSeq;
    using Unit = ShapedUnit;
    static constexpr bool kShaped = true, kCurved = false;
    const int2* visible;                   // [tokens] positions x .. y - 1 are seen; null: causal
    const float* slopes;                   // [query heads], or null
    const uint8_t* k_scales;               // [blocks][KV heads] biased exponents, or null
    const uint8_t* v_scales;
    float cap_log2, cap_inv;               // cap * log2(e) and 1 over it; 0: none
};
// With a cap or a bias: a form of the wide kernel of its own.
struct CurvedArgs : ShapedArgs {
    static constexpr bool kCurved = true;
};

// 2^(e - 127) of a scale's byte (of byte 0, 0: what 2^-127 scales is nothing beside any sum).
__device__ __forceinline__ float scale_of(uint32_t e) { return __int_as_float((int)(e << 23)); }

// Four consecutive values of a row.
__device__ __forceinline__ void put4(void* out, int f32, size_t i, float4 v) {
    if (f32)
        *reinterpret_cast<float4*>(static_cast<float*>(out) + i) = v;
    else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + i) =
            make_uint2(pa::pack_bf16x2(v.x, v.y), pa::pack_bf16x2(v.z, v.w));
}

template <int kRows, int kStep, class Args>
__device__ __forceinline__ typename Args::Seq read_seq(const Args& a, int s, bool flag) {
    typename Args::Seq r;
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
    if constexpr (Args::kShaped) {
        r.first = ctx - r.n;
        int lo = 0, hi = ctx;
        r.seen_lo = 0;
        r.seen_hi = r.first + 1;
        r.blind = 0;
        if (a.visible) {
            lo = r.seen_hi = 0x7fffffff;
            hi = 0;
#pragma unroll 8
            for (int i = 0; i < r.n; ++i) {
                const int2 v = a.visible[r.q0 + i];
                const int x = max(v.x, 0), y = min(v.y, ctx);
                if (x < y) {                            // (what a row that sees nothing comes to is not looked at)
                    lo = min(lo, x);
                    hi = max(hi, y);
                    r.seen_lo = max(r.seen_lo, x);
                    r.seen_hi = min(r.seen_hi, y);
                } else {
                    r.blind = 1;
                }
            }
            if (lo >= hi) lo = hi = 0;                  // nothing is seen: a step of no positions, and zeros
        }
        r.lo = lo;
        r.base = lo & ~(kRows == 16 ? 15 : 31);             // (a tile of the wide kernel begins with a block)
        r.ctx = hi;
        r.steps = max(1, (hi - r.base + kStep - 1) / kStep);
    } else {
        r.steps = (ctx + kStep - 1) / kStep;
    }
    return r;
}

// The mask words of a unit's tokens, or null, and its table.
__device__ __forceinline__ const uint64_t* words_of(const MultiArgs& a, const Unit& u) {
    return a.tree_mask ? a.tree_mask + u.q0 : nullptr;
}
__device__ __forceinline__ const int32_t* table_of(const MultiArgs& a, const Unit& u) {
    return a.block_tables + (size_t)u.seq * a.max_blocks;
}

// What the merge needs of a unit: its first token, its tokens (the last tile's
// may be fewer than its rows hold), KV head and last block.  (A unit's rows
// are a multiple of the group.)
__device__ __forceinline__ int4 begun_unit(const Unit& u, int log2_group) {
    const int skipped = u.row0 >> log2_group;
    return make_int4(u.q0 + skipped, u.n - skipped, u.kvh, u.last);
}

// A block's share of the work, walked unit by unit.
template <class Seq>
struct WalkOf {
    long long left, share;                 // work of this share from here on, and of a whole one
    int seq, unit, gone;                   // the sequence's unit, and how much of its work is before here
    Seq sq;
};
using Walk = WalkOf<Seq>;

// The next stretch of the share; u.valid is 0 at its end.
template <int kRows, int kStep, int kUnitCost, class Args>
__device__ __noinline__ void next_unit(WalkOf<typename Args::Seq>& w, typename Args::Unit& u, const Args& a) {
    u.valid = 0;
    while (w.left > 0) {
        if (w.unit >= a.n_kv_heads * w.sq.tiles) {
            w.unit = 0;
            w.sq = read_seq<kRows, kStep>(a, ++w.seq, false);
            continue;
        }
        const int per = w.sq.steps + kUnitCost, o = w.gone, unit = w.unit;
        const int take = (int)min((long long)(per - o), w.left);
        const int lo = max(0, o - kUnitCost), hi = max(0, o + take - kUnitCost);
        const bool ends = o + take == per;
        // a unit that goes on behind this share: the blocks from here to its end
        const unsigned rest = per - o - take, share = (unsigned)min(w.share, 1ll << 30);
        u.last = blockIdx.x + (rest ? (rest + share - 1) / share : 0);
        w.left -= take;
        w.gone = ends ? 0 : o + take;
        w.unit += ends;
        if (hi == lo) continue;            // the share ends within the unit's constant part
        u.q0 = w.sq.q0;
        u.n = w.sq.n;
        u.ctx = w.sq.ctx;
        if constexpr (Args::kShaped) {
            u.first = w.sq.first;
            u.lo = w.sq.lo;
            u.base = w.sq.base;
            u.seen_lo = w.sq.seen_lo;
            u.seen_hi = w.sq.seen_hi;
            u.blind = w.sq.blind;
        } else {
            u.first = w.sq.ctx - w.sq.n;
        }
        u.kvh = w.sq.tiles == 1 ? unit : unit / w.sq.tiles;
        u.row0 = (unit - u.kvh * w.sq.tiles) * kRows;
        u.st0 = lo;
        u.len = hi - lo;
        u.seq = w.seq;
        u.whole = u.len == w.sq.steps;
        u.valid = 1;
        return;
    }
}

// The walk of one whole unit: `unit` of sequence s.
template <int kUnitCost, class Seq>
__device__ __forceinline__ void one_unit(WalkOf<Seq>& walk, const Seq& sq, int s, int unit) {
    walk.left = walk.share = sq.steps + kUnitCost;
    walk.seq = s;
    walk.unit = unit;
    walk.gone = 0;
    walk.sq = sq;
}

// A warp's part of the batch: its work, its units and the most steps of one.
struct Part {
    long long work;
    int units, longest;
};

// This block's share, found by all its threads: thread t counts sequences
// [t * per, (t + 1) * per), and the one whose sequences hold the share's
// start sets `walk` up there.  False: the block has nothing to do.  Ends with
// a barrier; `parts` holds a value per warp until then.  The shares are whole units, one
// per block, where the grid has a block for each and none is longer than
// kDirectSteps.
template <int kRows, int kStep, int kUnitCost, int kMinSteps, int kDirectSteps, int kThreads, class Args>
__device__ __forceinline__ bool find_share(const Args& a, WalkOf<typename Args::Seq>& walk, Part* parts) {
    using Seq = typename Args::Seq;
    constexpr int kMinShare = kMinSteps + kUnitCost;
    if (a.direct) {
        int there = 0;
        if (threadIdx.x == 0) {
            const int per = a.n_kv_heads * a.direct, s = blockIdx.x / per, unit = blockIdx.x - s * per;
            const int kvh = unit / a.direct, tile = unit - kvh * a.direct;
            const Seq sq = read_seq<kRows, kStep>(a, s, unit == 0);
            one_unit<kUnitCost>(walk, sq, s, kvh * sq.tiles + tile);
            there = tile < sq.tiles;
        }
        return __syncthreads_or(there);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, heads = a.n_kv_heads;
    const int per = (a.num_seqs + kThreads - 1) / kThreads;
    const int s_lo = threadIdx.x * per, s_hi = min(a.num_seqs, s_lo + per);
    Part mine{0, 0, 0};
#pragma unroll 1
    for (int s = s_lo; s < s_hi; ++s) {
        const Seq sq = read_seq<kRows, kStep>(a, s, blockIdx.x == 0);
        mine.work += sq.work(heads, kUnitCost);
        mine.units = min(mine.units + min(heads * sq.tiles, 1 << 20), 1 << 20);   // (more than any grid is enough to know)
        if (sq.tiles) mine.longest = max(mine.longest, sq.steps);
    }
    Part upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long w = __shfl_up_sync(0xffffffffu, upto.work, o);
        const int u = __shfl_up_sync(0xffffffffu, upto.units, o);
        if (lane >= o) {
            upto.work += w;
            upto.units += u;
        }
        upto.longest = max(upto.longest, __shfl_xor_sync(0xffffffffu, upto.longest, o));
    }
    if (lane == 31) parts[warp] = upto;
    __syncthreads();
    Part all{0, 0, 0};
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
        const Part p = parts[w];
        if (w < warp) {
            upto.work += p.work;
            upto.units += p.units;
        }
        all.work += p.work;
        all.units += p.units;
        all.longest = max(all.longest, p.longest);
    }
    if (threadIdx.x == 0) a.pieces[blockIdx.x].x = -1;
    // Shaped, with four warps, also where the units are of nearly one length, as windows are, and there is one for three
    // blocks in four or more: nothing is merged then, and fewer blocks read as fast (384 units on 456 blocks, windows of
    // 1,024 positions 38.6 us whole, 43.1 in shares; 2,048 68.0 / 70.6, 4,096 131.1 / 131.7).  Block-scaled, where
    // instructions bind, only if the longest is within seven steps of a share (1,024 30.3 / 33.4, 2,048 50.4 / 51.6, but
    // 4,096 90.4 / 86.4).
    bool even = false;
    if constexpr (Args::kShaped && kRows == 16 && kThreads == 128) {
        const long long most = all.longest + kUnitCost, grid = gridDim.x;
        even = all.units * 4ll >= grid * 3 && most * all.units * 7 <= all.work * 8 &&
               (!a.k_scales || (most - 7) * grid <= all.work);
    }
    if ((all.longest <= kDirectSteps || even) && all.units <= (int)gridDim.x) {
        int unit = blockIdx.x;
        if (unit >= all.units) return false;
        if (unit < upto.units && unit >= upto.units - mine.units) {
            unit -= upto.units - mine.units;
            int s = s_lo;
            Seq sq = read_seq<kRows, kStep>(a, s, false);
#pragma unroll 1
            while (unit >= heads * sq.tiles) {
                unit -= heads * sq.tiles;
                sq = read_seq<kRows, kStep>(a, ++s, false);
            }
            one_unit<kUnitCost>(walk, sq, s, unit);
        }
        __syncthreads();
        return true;
    }
    long long share = (all.work + gridDim.x - 1) / gridDim.x;
    share = share < kMinShare ? kMinShare : share;
    const long long begin = share * blockIdx.x;
    if (begin >= all.work) return false;
    if (begin >= upto.work - mine.work && begin < upto.work) {
        long long off = begin - (upto.work - mine.work);
        int s = s_lo;
        Seq sq = read_seq<kRows, kStep>(a, s, false);
#pragma unroll 1
        while (off >= sq.work(heads, kUnitCost)) {
            off -= sq.work(heads, kUnitCost);
            sq = read_seq<kRows, kStep>(a, ++s, false);
        }
        const int per = sq.steps + kUnitCost;
        walk.left = min(all.work, begin + share) - begin;
        walk.share = share;
        walk.seq = s;
        walk.unit = (int)(off / per);
        walk.gone = (int)(off - (long long)walk.unit * per);
        walk.sq = sq;
    }
    __syncthreads();
    return true;
}

// Whether new token i of a sequence sees its new token j.
__device__ __forceinline__ bool sees(const uint64_t* words, int i, int j) {
    return words ? (j < 64 && (words[i] >> j & 1ull)) : j <= i;
}

// A value that is not finite reaches the rows that see it only.  In a product
// it would reach all (0 * inf = NaN), so at the new positions, which are all
// that a row may not see (shaped: those that some row does not see), the
// products run with zeros in its place, and the rows of such a unit add what
// they see of it when they are written.

// The elements of w (two bf16, or four E4M3 codes) that are not finite, as a mask.
template <bool F8>
__device__ __forceinline__ uint32_t unfinite_mask(uint32_t w) {
    return F8 ? ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu
              : ((((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 15) * 0xffffu;
}

// Zeros in their place in rows from .. to - 1 of a tile (slabs of 128-byte
// rows, their chunks in any order), by `threads` threads of which this is
// `thread`; whether it found any.
template <bool F8, int kSlabs>
__device__ __forceinline__ bool drop_unfinite(uint8_t* tile, int slab_bytes, int from, int to, int thread, int threads) {
    uint32_t any = 0;
#pragma unroll 1
    for (int x = from * 8 * kSlabs + thread; x < to * 8 * kSlabs; x += threads) {
        const int row = x / (8 * kSlabs), c = x % (8 * kSlabs);
        uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * slab_bytes + row * 128 + (c & 7) * 16);
        uint4 v = *p;
        const uint32_t m[4] = {unfinite_mask<F8>(v.x), unfinite_mask<F8>(v.y), unfinite_mask<F8>(v.z), unfinite_mask<F8>(v.w)};
        const uint32_t bad = m[0] | m[1] | m[2] | m[3];
        if (bad) {
            *p = make_uint4(v.x & ~m[0], v.y & ~m[1], v.z & ~m[2], v.w & ~m[3]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // for tensor cores, and copies to come
        }
        any |= bad;
    }
    return any != 0;
}

// The like outside positions seen_lo .. seen_hi - 1 of a tile that begins at
// t0, of its first `rows` rows.
template <bool F8, int kSlabs>
__device__ __forceinline__ bool drop_unfinite_outside(uint8_t* tile, int slab_bytes, int t0, int seen_lo, int seen_hi, int rows,
                                                      int thread, int threads) {
    const int lo = min(max(seen_lo - t0, 0), rows), hi = max(min(seen_hi - t0, rows), lo);
    bool any = false;
    if (lo > 0) any |= drop_unfinite<F8, kSlabs>(tile, slab_bytes, 0, lo, thread, threads);
    if (hi < rows) any |= drop_unfinite<F8, kSlabs>(tile, slab_bytes, hi, rows, thread, threads);
    return any;
}

// Add the values that are not finite, at d .. d + 3 of the positions of
// [lo, hi) that a row of sequence s sees, to the row's result: its sums at
// `part`, or `out` where that is null.
// (Shaped: positions that every row sees, within seen_lo .. seen_hi, keep theirs.)
template <int D, bool F8, class Args>
__device__ __noinline__ void add_unfinite(const Args& a, int s, int kvh, int row, int lo, int hi, int d, float* part) {
    const auto q = read_seq<1, 1>(a, s, false);
    const int i = row >> a.log2_group, B = 1 << a.log2_block;
    if (i >= q.n) return;
    int first, end = min(hi, q.ctx);
    const uint64_t* words = nullptr;
    if constexpr (Args::kShaped) {
        first = lo;
        if (a.visible) {
            const int2 v = a.visible[q.q0 + i];
            first = max(lo, v.x);
            end = min(end, v.y);
        } else {
            end = min(end, q.first + i + 1);
        }
    } else {
        first = q.ctx - q.n;
        words = a.tree_mask ? a.tree_mask + q.q0 : nullptr;
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int pos = max(lo, first); pos < end; ++pos) {
        if constexpr (Args::kShaped) {
            if (pos >= q.seen_lo && pos < q.seen_hi) {
                pos = q.seen_hi - 1;
                continue;
            }
        } else if (!sees(words, i, pos - first)) {
            continue;
        }
        const int blk = a.block_tables[(size_t)s * a.max_blocks + (pos >> a.log2_block)];
        if (blk < 0 || blk >= a.num_blocks) continue;
        const size_t at = ((size_t)(blk * a.n_kv_heads + kvh) * B + (pos & (B - 1))) * D + d;
        if constexpr (F8) {                                       // E4M3 has NaN only
            const uint32_t m = unfinite_mask<true>(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v_cache) + at));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m >> (8 * e) & 1u) sum[e] = __int_as_float(0x7fffffff);
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.v_cache) + at);
            const float2 x = pa::bf16x2_to_float2(w.x & unfinite_mask<false>(w.x));
            const float2 y = pa::bf16x2_to_float2(w.y & unfinite_mask<false>(w.y));
            sum[0] += x.x;
            sum[1] += x.y;
            sum[2] += y.x;
            sum[3] += y.y;
        }
    }
    const size_t at = ((size_t)(q.q0 + i) * a.n_q_heads + (kvh << a.log2_group) + (row & ((1 << a.log2_group) - 1))) * D + d;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (sum[e] == 0.f) continue;
        float* f = part ? part + e : static_cast<float*>(a.out) + at + e;
        __nv_bfloat16* b = static_cast<__nv_bfloat16*>(a.out) + at + e;
        if (part || a.out_f32) *f += sum[e];
        else *b = __float2bfloat16(__bfloat162float(*b) + sum[e]);
    }
}

// out of the units that several blocks share: the pieces of block b, which
// begins the unit (its second slot), and of blocks b + 1 .. last (their
// first).  kMergeThreads / kItems threads take four columns of a row and share
// its pieces.
template <int D, int kItems>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const MultiArgs a, int rows) {
    constexpr int kStep = kMergeThreads / kItems;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int4 p = a.pieces[blockIdx.x];
    if (p.x < 0) return;
    const int G = 1 << a.log2_group, mine = kStep > 1 ? threadIdx.x / kItems : 0;
    const int pieces = p.w - blockIdx.x + 1;                     // two at least
#pragma unroll 1
    for (int x = blockIdx.y * kItems + threadIdx.x % kItems; x < rows * (D / 4); x += gridDim.y * kItems) {
        const int r = x / (D / 4), d = x % (D / 4) * 4, i = r >> a.log2_group;
        const bool there = i < p.y;
        float M = kNone, Z = 0.f;
        float4 U = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float m, float z, float4 v) {
            const float top = fmaxf(M, m);
            const float f = pa::exp2_approx(M - top), h = pa::exp2_approx(m - top);
            Z = Z * f + z * h;
            U.x = U.x * f + v.x * h;
            U.y = U.y * f + v.y * h;
            U.z = U.z * f + v.z * h;
            U.w = U.w * f + v.w * h;
            M = top;
        };
        if (there) {
            // two pieces' loads together; a piece's slot is the first of its block's two but for the first piece
#pragma unroll 1
            for (int k = mine; k < pieces; k += 2 * kStep) {
                const int then = min(k + kStep, pieces - 1);
                const int at = (2 * ((int)blockIdx.x + k) + (k == 0)) * rows + r;
                const int next = (2 * ((int)blockIdx.x + then) + (then == 0)) * rows + r;
                const float m0 = a.part_m[at], m1 = a.part_m[next], z0 = a.part_z[at], z1 = a.part_z[next];
                const float4 v0 = *reinterpret_cast<const float4*>(a.part_u + (size_t)at * D + d);
                const float4 v1 = *reinterpret_cast<const float4*>(a.part_u + (size_t)next * D + d);
                add(m0, z0, v0);
                if (k + kStep < pieces) add(m1, z1, v1);
            }
        }
        if constexpr (kStep > 1) {
            __shared__ float4 sums[kMergeThreads];
            __shared__ float2 stats[kMergeThreads];
            sums[threadIdx.x] = U;
            stats[threadIdx.x] = make_float2(M, Z);
            __syncthreads();
            if (mine == 0)
#pragma unroll
                for (int k = 1; k < kStep; ++k) {
                    const float2 e = stats[k * kItems + threadIdx.x];
                    add(e.x, e.y, sums[k * kItems + threadIdx.x]);
                }
            __syncthreads();
        }
        if (mine == 0 && there) {
            const float f = a.v_scale / Z;
            put4(a.out, a.out_f32, ((size_t)(p.x + i) * a.n_q_heads + p.z * G + (r & (G - 1))) * D + d,
                 Z == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(U.x * f, U.y * f, U.z * f, U.w * f));
        }
    }
}

// The merge of the units that blocks share (pa_decode_multi.cu).
cudaError_t launch_merge(const MultiArgs& a, int unit, int d_head, double units, int grid, cudaStream_t st);

// Launches of the 64- and 128-row units on the 5th-generation tensor cores
// (pa_decode_wide.cu, pa_attend_wide.cu); cudaSuccess or the launch's error.
cudaError_t launch_shaped_wide(int rows, int d_head, bool f8, const void* q, int block_size, const CUtensorMap& map_k,
                               const CUtensorMap& map_v, const CurvedArgs& a, int grid, cudaStream_t st);
cudaError_t launch_wide(int rows, int d_head, bool f8, const void* q, int block_size, const CUtensorMap& map_k,
                        const CUtensorMap& map_v, const MultiArgs& a, int grid, cudaStream_t st);
// (Unit cost of 2, 3, 4, 6 steps: 64 requests of 8 tokens, E4M3 68.6, 67.3, 67.6, 69.5 us; 48 trees of 16, bf16
// 101.3, 102.2, 102.0, 103.7.)
constexpr int kWideCost = 3, kWideMinSteps = 2, kWideStep = 128, kWideDirectSteps = 8;

}  // namespace pa_multi
