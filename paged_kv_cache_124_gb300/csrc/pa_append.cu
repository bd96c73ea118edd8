// Norm, rotation and the append to a block-scaled cache, in one pass over a
// step's projections (pa_qk_norm_rope_cache_scaled), and the append alone
// (pa_reshape_and_cache_scaled).
//
// The arithmetic up to the codes is that of pa_rope.cu.  A block's scale for
// a head is 2^e, e the least for which no value of its positions is beyond
// 448 2^e, E4M3's largest: the whole range of the codes is used, and a
// product by 2^-e is exact, so a code is off by its own rounding alone, and
// codes that a grown scale makes smaller stay what they are (but for E4M3's
// subnormals, which lose bits).
//
// The tokens of one block follow one another (a run: consecutive slots within
// a block).  A thread block takes the runs that begin among its own tokens,
// for four or eight heads: D / 16 lanes hold a token's part of a head, as
// pa_rope.cu's do, and a token's angles are loaded once for all of its heads.
// Turned keys wait in shared memory, in 32 bits, and values in registers, as
// they came, while the largest of each run and head meet.  Queries go beside, in
// blocks of their own.
//
// Memory bounds it from prompts on: 32,048 tokens of 32 + 2 x 8 heads of 128
// take 137.9 us, 0.78 of the measured copy rate for their 725 MB (DRAM 62 %
// busy, issue 40 %: all warps of a block wait between the products and the
// codes).  A decode batch of 250 tokens takes 5.1 us, a chain of loads: slot,
// scale, then the block's codes where the scale grows.  A warp for each run
// and head with all of it in registers took 169 to 182 us, angles and gains
// folded into factors 141.  The append alone, 2 x 8 heads of 128: 6 tokens 4.0
// us, 250 of one prompt 6.5, 2,003 6.4, 32,048 58.2, 0.50 of the measured copy
// rate for 197 MB.

#include <cuda_fp16.h>
#include <math.h>

#include "pa_rope.cuh"

namespace {

struct AppendArgs : RopeArgs {
    uint8_t* k_scales;
    uint8_t* v_scales;
    int kv_blocks;                                     // thread blocks of keys and values: every (every + 1)th of the grid's
    int every;                                         // first; the others take queries
    int q_heads_per;                                   // query heads one after another in the same lanes
    int log2_block;
};

constexpr int kWarps = kRopeThreads / 32;

__device__ __forceinline__ float scale_of(int e) { return __int_as_float(e ? e << 23 : 0x00400000); }

// The least e (biased, at least 0) with top <= 448 2^(e - 127); top finite and not negative.
__device__ __forceinline__ int scale_byte(float top) {
    const int bits = __float_as_int(top);              // 448 is 1.75 2^8
    return max(0, (bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000));
}

__device__ __forceinline__ float top_of(const Part& p, float top) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = unpair(p.f[i]);
        top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));     // (a NaN is no value)
    }
    return top;
}

__device__ __forceinline__ float finite_top_of(const Part& p, float top) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = unpair(p.f[i]);
        if (fabsf(v.x) < INFINITY) top = fmaxf(top, fabsf(v.x));
        if (fabsf(v.y) < INFINITY) top = fmaxf(top, fabsf(v.y));
    }
    return top;
}

__device__ __forceinline__ uint2 codes_by(const uint64_t* f, uint64_t by) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpair(mul2(f[i], by));
        c[i] = pa::e4m3x2(v.x, v.y);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
    return d;
}

// Four codes times `by`, rounded again.
__device__ __forceinline__ uint32_t code_again(uint32_t w, float by) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return pa::e4m3x2(x.x * by, x.y * by) | (pa::e4m3x2(y.x * by, y.y * by) << 16);
}

// Rows on their way to a warp, in shared memory rather than in registers: a
// slot holds the two chunks of each lane, which alone reads them back.
__device__ __forceinline__ void copy_in(uint32_t slot, int lane, const uint4* src, int c0, int c1) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n\tcp.async.cg.shared.global [%2], [%3], 16;" ::"r"(slot + 16 * lane),
                 "l"(src + c0), "r"(slot + 512 + 16 * lane), "l"(src + c1) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }
__device__ __forceinline__ void read_slot(uint32_t slot, int lane, uint64_t* f) {
    uint4 x;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(slot + 512 * k + 16 * lane) : "memory");
        unpack8(x, f + 4 * k);
    }
}

constexpr int kFlight = 8;                             // heads of a query on their way
constexpr int kRuns = 16;                              // of a thread block at most: a run a token
constexpr int kWindow = 64;                            // tokens that a thread block looks at: its own, one before, kBlock - 1 behind

struct Shared {                                        // what a thread block of keys and values shares
    long long slot[kWindow];                           // of tokens first - 1 on; negative where nothing is written
    int4 where[kWindow];                               // their positions
    unsigned long long there, follows;                 // bit j: token first - 1 + j is written; and goes on with the run
    uint32_t top[kRuns][16];                           // largest magnitudes of each run's keys, then values; then scales
    int grown[kRuns][16];                              // log2 of what the block's other codes are to be divided by
};

// How a thread block goes over keys and values, D / 16 lanes a token and head.
//   kFew   4 heads' keys and values side by side, a part a thread, of the
//          tokens that leaves (4 of D 128): the least latency.
//   kSome  16 tokens, 4 heads, 2 of them in turn (D 128).
//   kMany  16 tokens, 8 heads, 4 in turn: a token's angles serve the most.
enum Mode { kFew, kSome, kMany };
template <int D, int kMode>
struct Share {
    static constexpr int kLanes = D / 16, kGroups = kRopeThreads / kLanes, kTile = kMode == kMany ? 8 : 4;
    static constexpr int kTokens = kMode == kFew ? kGroups / (2 * kTile) : kRuns, kSides = kGroups / kTokens;
    static constexpr int kHeads = kMode == kFew ? 1 : kTile / kSides;
    static constexpr int kTogether = kMode == kSome;           // keys and values loaded together (kMany has no registers for both)
};

// (Thread blocks an SM: 2 against 3 with many tokens, whose registers then hold the gains, 32,048 tokens 137 / 141 us; 3
// against 2 with fewer, 250 of 256 4.6 / 5.3.)
template <int D, bool kInterleaved, bool kAxes, int kMode>
__global__ void __launch_bounds__(kRopeThreads, kMode == kMany ? 2 : 3) append_kernel(const AppendArgs a) {
    using S = Share<D, kMode>;
    constexpr int kLanes = S::kLanes, kTokens = S::kTokens, kHeads = S::kHeads, kTileHeads = S::kTile;
    const int kBlock = 1 << a.log2_block;
    extern __shared__ __align__(16) uint8_t smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, l = lane % kLanes;
    const unsigned mask = ((1u << kLanes) - 1u) << (lane / kLanes * kLanes);
    const Place<kInterleaved> w(l, a.rot_dim);
    // Blocks of both kinds run side by side: queries stream, keys and values wait for their largest.
    const int turn = blockIdx.x / (a.every + 1), kv_before = min((int)(turn + (blockIdx.x % (a.every + 1) != 0)), a.kv_blocks);
    if (blockIdx.x % (a.every + 1) || turn >= a.kv_blocks) {
        // ------------------------------------------------------------ queries
        const uint32_t slots = pa::smem_addr(smem) + (threadIdx.x >> 5) * (kFlight * 1024);
        const uint32_t parts = (a.n_q_heads + a.q_heads_per - 1) / a.q_heads_per;
        const uint32_t nth = (blockIdx.x - kv_before) * (kRopeThreads / kLanes) + threadIdx.x / kLanes;
        const uint32_t t = nth / parts;
        if (t >= (uint32_t)a.num_tokens) return;               // whole heads: a head's threads leave together
        const int h0 = (nth - t * parts) * a.q_heads_per, h1 = min(h0 + a.q_heads_per, a.n_q_heads);
        Where<kAxes> at;
        at.load(a, t);
        const uint4* rows = reinterpret_cast<const uint4*>(a.q + (long long)t * a.q_stride);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (h0 + u < h1) copy_in(slots + 1024 * u, lane, rows + (h0 + u) * (D / 8), w.c0, w.c1);
            copies_end();
        }
        if (at.lowest() >= 0 && at.highest() < a.max_positions) {   // (else flagged by the keys' warps)
            uint64_t cs[4], sn[4];
            if (w.turns) load_angles<kAxes>(a, at, l, cs, sn);
            uint64_t gain[8];
            if (a.q_weight) {
                load8(a.q_weight + 8 * w.c0, gain);
                load8(a.q_weight + 8 * w.c1, gain + 4);
            }
            int u = 0;
#pragma unroll 2
            for (int h = h0; h < h1; ++h) {
                wait_copies<kFlight - 1>();
                const uint32_t slot = slots + 1024 * u;
                Part p;
                read_slot(slot, lane, p.f);
                if (a.q_weight) norm_part<kLanes>(p, gain, a.eps, mask);
                if (w.turns) turn_part<kInterleaved>(p, cs, sn);
                const uint4 y0 = pack8(p.f), y1 = pack8(p.f + 4);
                if (h + kFlight < h1) copy_in(slot, lane, rows + (h + kFlight) * (D / 8), w.c0, w.c1);
                copies_end();
                uint4* dst = a.q_out + ((size_t)t * a.n_q_heads + h) * (D / 8);
                dst[w.c0] = y0;
                dst[w.c1] = y1;
                u = (u + 1) % kFlight;
            }
        }
        wait_copies<0>();
        return;
    }
    // ---------------------------------------------------------------- keys and values
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    const int tiles = (a.n_kv_heads + kTileHeads - 1) / kTileHeads, tile = turn % tiles;
    const long long first = (long long)(turn / tiles) * kTokens;
    const int head0 = tile * kTileHeads, heads = min(kTileHeads, a.n_kv_heads - head0);
    sh.top[threadIdx.x / 16][threadIdx.x % 16] = 0;
    static_assert(kRopeThreads == 16 * kRuns, "a thread for each");
    if (threadIdx.x < 32) {                                      // a warp finds the runs
        long long slot[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j = lane + 32 * x;
            const long long t = first - 1 + j;
            slot[x] = -1;
            if (t >= 0 && t < a.num_tokens && j < kTokens + kBlock) {
                slot[x] = a.slots[t];
                if (a.positions) {
                    Where<kAxes> at;
                    at.load(a, t);
                    if (at.lowest() < 0 || at.highest() >= a.max_positions) {
                        if (tile == 0 && at.lowest() >= 0) pa::set_status(a.status, PA_DEV_BAD_POSITION);
                        slot[x] = -1;
                    }
                    sh.where[j] = make_int4(at.of(0), at.of(1), at.of(2), at.of(3));
                }
                if (slot[x] >= a.num_slots) {
                    if (tile == 0) pa::set_status(a.status, PA_DEV_BAD_SLOT);
                    slot[x] = -1;
                }
            }
            sh.slot[j] = slot[x];
        }
        const long long p0 = __shfl_up_sync(0xffffffffu, slot[0], 1), p1 = __shfl_up_sync(0xffffffffu, slot[1], 1);
        const long long last = __shfl_sync(0xffffffffu, slot[0], 31);
        const long long before[2] = {lane ? p0 : -1, lane ? p1 : last};
        unsigned b[2], f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            b[x] = __ballot_sync(0xffffffffu, slot[x] >= 0);
            f[x] = __ballot_sync(0xffffffffu, slot[x] >= 0 && before[x] >= 0 && slot[x] == before[x] + 1 && (slot[x] & (kBlock - 1)));
        }
        if (lane == 0) {
            sh.there = b[0] | (unsigned long long)b[1] << 32;
            sh.follows = f[0] | (unsigned long long)f[1] << 32;
        }
    }
    __syncthreads();
    const unsigned long long there = sh.there, follows = sh.follows;
    // The runs' first tokens, and the tokens from the first run's begin to the last one's end: theirs, but for ones that are not written.
    const unsigned long long starts = there & ~follows & (((1ull << kTokens) - 1) << 1);
    if (!starts) return;
    const int begin = __ffsll((long long)starts) - 1, last_run = 63 - __clzll((long long)starts);
    const int end = last_run + __ffsll((long long)~(follows >> (last_run + 1)));
    const int group = threadIdx.x / kLanes, side = group / kTokens, mine = begin + group % kTokens;
    const bool one_pass = end - begin <= kTokens;                // the rows stay in registers

    // This thread's parts: of heads side, side + kSides, .. both keys and values; few tokens: one of either.
    auto head_of = [&](int x) { return kMode != kFew ? x * S::kSides + side : side % kTileHeads; };
    const bool keys = kMode != kFew || side < kTileHeads, values = kMode != kFew || side >= kTileHeads;
    struct Raw {
        uint4 x0[kHeads], x1[kHeads];
    };
    Raw k, v;
    auto load = [&](const __nv_bfloat16* rows, long long stride, int j, bool in, Raw& r) {   // token j of the window
#pragma unroll
        for (int x = 0; x < kHeads; ++x) {
            r.x0[x] = r.x1[x] = make_uint4(0, 0, 0, 0);
            if (in && head_of(x) < heads) {
                const uint4* src = reinterpret_cast<const uint4*>(rows + (first - 1 + j) * stride + (head0 + head_of(x)) * D);
                r.x0[x] = src[w.c0];
                r.x1[x] = src[w.c1];
            }
        }
    };
    uint64_t cs[4], sn[4];
    auto angles = [&](int j, bool in) {
        if (!w.turns || !in) return;
        const int4 p = sh.where[j];
        Where<kAxes> at;
        at.p[0] = p.x;
        if constexpr (kAxes) {
            at.p[1] = p.y;
            at.p[2] = p.z;
            at.p[3] = p.w;
        }
        load_angles<kAxes>(a, at, l, cs, sn);
    };
    uint64_t gain[8];
    if (a.k_weight && kMode == kMany) {
        load8(a.k_weight + 8 * w.c0, gain);
        load8(a.k_weight + 8 * w.c1, gain + 4);
    }
    auto key = [&](int x) {                                      // part x of the keys ready for the cache
        Part p;
        unpack8(k.x0[x], p.f);
        unpack8(k.x1[x], p.f + 4);
        if (a.k_weight) {
            if (kMode != kMany) {                                // (from L1: registers are short)
                load8(a.k_weight + 8 * w.c0, gain);
                load8(a.k_weight + 8 * w.c1, gain + 4);
            }
            norm_part<kLanes>(p, gain, a.eps, mask);
        }
        if (w.turns) turn_part<kInterleaved>(p, cs, sn);
        return p;
    };
    // where they wait for their scale
    uint32_t kept = pa::smem_addr(smem + sizeof(Shared)) + 16 * threadIdx.x;
    auto keep = [&](int x, const Part& p) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(kept + (4 * x + q) * (16 * kRopeThreads)), "l"(p.f[2 * q]), "l"(p.f[2 * q + 1]) : "memory");
    };
    auto get = [&](int x) {
        Part p;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(p.f[2 * q]), "=l"(p.f[2 * q + 1]) : "r"(kept + (4 * x + q) * (16 * kRopeThreads)) : "memory");
        return p;
    };
    auto meet = [&](int kind, int x, bool in, int run, uint32_t top) {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
        if (in && l == 0 && head_of(x) < heads) atomicMax(&sh.top[run][kind * kTileHeads + head_of(x)], top);
    };
    auto run_of = [&](int j) { return __popcll(starts & ((2ull << j) - 1)) - 1; };
    const int stop = begin + (end - begin + kTokens - 1) / kTokens * kTokens;
#pragma unroll 1
    for (int j = mine; j < stop; j += kTokens) {
        const bool in = j < end && (there >> j & 1);
        const int run = in ? run_of(j) : 0;
        if (keys) load(a.k, a.k_stride, j, in, k);
        if (values && S::kTogether) load(a.v, a.v_stride, j, in, v);
        if (keys) {
            angles(j, in);
#pragma unroll
            for (int x = 0; x < kHeads; ++x) {
                const Part p = key(x);
                float f = top_of(p, 0.f);
                if (!(f < INFINITY)) f = finite_top_of(p, 0.f);
                if (one_pass) keep(x, p);
                meet(0, x, in, run, __float_as_uint(f));
            }
        }
        if (values) {
            if (!S::kTogether) load(a.v, a.v_stride, j, in, v);
#pragma unroll
            for (int x = 0; x < kHeads; ++x) {
                const uint4 y = v.x0[x], z = v.x1[x];
                uint32_t m = max2(max2(max2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu), max2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu)),
                                  max2(max2(z.x & 0x7fff7fffu, z.y & 0x7fff7fffu), max2(z.z & 0x7fff7fffu, z.w & 0x7fff7fffu)));
                m = max(m & 0xffffu, m >> 16);
                uint32_t top = m << 16;
                if (m >= 0x7f80u) {                              // NaN is no value, and infinities saturate
                    Part p;
                    unpack8(y, p.f);
                    unpack8(z, p.f + 4);
                    top = __float_as_uint(finite_top_of(p, 0.f));
                }
                meet(1, x, in, run, top);
            }
        }
    }
    __syncthreads();
    const int runs = __popcll(starts);
    // the block that run's tokens go to, from `off` on, and its head (an index of scales)
    auto block_of = [&](int run, int h, int& off, int& n) {
        unsigned long long rest = starts;
        for (int i = 0; i < run; ++i) rest &= rest - 1;
        const int j = __ffsll((long long)rest) - 1;
        off = (int)sh.slot[j] & (kBlock - 1);
        n = __ffsll((long long)~(follows >> (j + 1)));
        return (size_t)(sh.slot[j] >> a.log2_block) * a.n_kv_heads + head0 + h;
    };
    if (threadIdx.x < runs * 2 * kTileHeads) {                   // a thread for each run, kind and head: its scale
        const int run = threadIdx.x / (2 * kTileHeads), kh = threadIdx.x % (2 * kTileHeads), h = kh % kTileHeads;
        if (h < heads) {
            int off, n;
            uint8_t* scale = (kh < kTileHeads ? a.k_scales : a.v_scales) + block_of(run, h, off, n);
            const int old = off ? *scale : 0, now = max(old, scale_byte(__uint_as_float(sh.top[run][kh])));
            if (now != old || !off) *scale = (uint8_t)now;
            sh.top[run][kh] = now;
            sh.grown[run][kh] = off ? now - old : 0;
        } else {
            sh.grown[run][kh] = 0;
        }
    }
    __syncthreads();
    // where a scale has grown, the block's other codes again
#pragma unroll 1
    for (int x = threadIdx.x / 32; x < runs * 2 * kTileHeads; x += kWarps) {
        const int run = x / (2 * kTileHeads), kh = x % (2 * kTileHeads), by = sh.grown[run][kh];
        if (!by) continue;
        int off, n;
        const size_t place = block_of(run, kh % kTileHeads, off, n);
        const float down = by > 126 ? 0.f : scale_of(127 - by);
        uint4* codes = reinterpret_cast<uint4*>((kh < kTileHeads ? a.k_cache : a.v_cache) + place * (kBlock * D));
#pragma unroll 2
        for (int y = lane; y < kBlock * (D / 16); y += 32) {
            const int row = y / (D / 16);
            if (row >= off && row < off + n) continue;
            uint4 c = codes[y];
            c.x = code_again(c.x, down);
            c.y = code_again(c.y, down);
            c.z = code_again(c.z, down);
            c.w = code_again(c.w, down);
            codes[y] = c;
        }
    }
#pragma unroll 1
    for (int j = mine; j < stop; j += kTokens) {
        const bool in = j < end && (there >> j & 1);
        const int run = in ? run_of(j) : 0;
        const long long slot = in ? sh.slot[j] : 0;
        const size_t place = ((size_t)(slot >> a.log2_block) * a.n_kv_heads + head0) * kBlock + ((int)slot & (kBlock - 1));
        auto put = [&](int kind, int x, const Part& p) {
            const int h = head_of(x);
            if (!in || h >= heads) return;
            const float up = scale_of(254 - (int)sh.top[run][kind * kTileHeads + h]);
            uint2* dst = reinterpret_cast<uint2*>((kind ? a.v_cache : a.k_cache) + (place + (size_t)h * kBlock) * D);
            dst[w.c0] = codes_by(p.f, pair(up, up));
            dst[w.c1] = codes_by(p.f + 4, pair(up, up));
        };
        auto value = [&](int x) {
            Part p;
            unpack8(v.x0[x], p.f);
            unpack8(v.x1[x], p.f + 4);
            return p;
        };
        if (one_pass) {
            if (values)
#pragma unroll
                for (int x = 0; x < kHeads; ++x) put(1, x, value(x));
            if (keys)
#pragma unroll
                for (int x = 0; x < kHeads; ++x) put(0, x, get(x));
        } else {
            if (keys) {
                load(a.k, a.k_stride, j, in, k);
                angles(j, in);
#pragma unroll
                for (int x = 0; x < kHeads; ++x) put(0, x, key(x));
            }
            if (values) {
                load(a.v, a.v_stride, j, in, v);
#pragma unroll
                for (int x = 0; x < kHeads; ++x) put(1, x, value(x));
            }
        }
    }
}

template <int D, int kMode>
cudaError_t launch_append(const AppendArgs& a, int interleaved, cudaStream_t st) {
    using S = Share<D, kMode>;
    constexpr int kParts = kRopeThreads / S::kLanes;
    const long long kv = ((long long)a.num_tokens + S::kTokens - 1) / S::kTokens * ((a.n_kv_heads + S::kTile - 1) / S::kTile);
    const long long q = a.n_q_heads ? (long long)a.num_tokens * ((a.n_q_heads + a.q_heads_per - 1) / a.q_heads_per) : 0;
    AppendArgs b = a;
    b.kv_blocks = (int)kv;
    const int q_blocks = (int)((q + kParts - 1) / kParts);
    b.every = q_blocks / b.kv_blocks;
    const auto kernel = a.num_axes ? (interleaved ? append_kernel<D, true, true, kMode> : append_kernel<D, false, true, kMode>)
                                   : (interleaved ? append_kernel<D, true, false, kMode> : append_kernel<D, false, false, kMode>);
    // queries' rows on their way; keys that wait for their scale, in 32 bits, and what a thread block shares of its tokens
    constexpr int kKept = 64 * kRopeThreads * S::kHeads + sizeof(Shared);
    constexpr int kSmem = kWarps * kFlight * 1024 > kKept ? kWarps * kFlight * 1024 : kKept;
    static int attr[4][64] = {{0}};
    const cudaError_t e = pa_host::ensure_smem_attr(kernel, kSmem, attr[2 * (a.num_axes != 0) + (interleaved != 0)]);
    if (e != cudaSuccess) return e;
    return pa_host::launch_dependent(kernel, dim3((unsigned)(b.kv_blocks + q_blocks)), dim3(kRopeThreads), kSmem, st, b);
}

template <int D>
cudaError_t launch_append(const AppendArgs& a, int mode, int interleaved, cudaStream_t st) {
    return mode == kFew ? launch_append<D, kFew>(a, interleaved, st) : mode == kSome ? launch_append<D, kSome>(a, interleaved, st)
                                                                     : launch_append<D, kMany>(a, interleaved, st);
}

int append(void* q_out, void* k_cache, void* v_cache, uint8_t* k_scales, uint8_t* v_scales, const void* q, const void* k,
           const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_weight,
           const float* k_weight, float eps, const float* cos_sin, int max_positions, int rot_dim, int interleaved,
           const int32_t* positions, int num_axes, const int8_t* axis_of_pair, const int64_t* slot_mapping,
           int num_tokens, int n_q_heads, int n_kv_heads, int d_head, int block_size, int num_blocks,
           int32_t* status_dev, void* stream, bool turned) {
    if (num_tokens < 0 || n_q_heads < 0 || n_kv_heads <= 0 || num_blocks <= 0 || !(eps >= 0.f) ||
        !(eps < __builtin_inff()) || num_axes < 0)
        return PA_ERR_INVALID_ARG;
    if (!pa_host::supported_block_size(block_size) || !pa_host::supported_d_head(d_head)) return PA_ERR_UNSUPPORTED;
    if (turned) {
        if (n_q_heads == 0 || max_positions <= 0 || (num_axes && !axis_of_pair)) return PA_ERR_INVALID_ARG;
        if (rot_dim < 16 || rot_dim > d_head || rot_dim % 16 || num_axes > 4) return PA_ERR_UNSUPPORTED;
    }
    if (((long long)n_q_heads + 2LL * n_kv_heads) * num_tokens > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!k_cache || !v_cache || !k_scales || !v_scales || !k || !v || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (turned && (!q_out || !q || !cos_sin || !positions)) return PA_ERR_INVALID_ARG;
    if ((q_weight == nullptr) != (k_weight == nullptr)) return PA_ERR_INVALID_ARG;
    if (q_stride < (int64_t)n_q_heads * d_head || k_stride < (int64_t)n_kv_heads * d_head ||
        v_stride < (int64_t)n_kv_heads * d_head)
        return PA_ERR_INVALID_ARG;
    if (!pa_host::aligned16(q_out) || !pa_host::aligned16(k_cache) || !pa_host::aligned16(v_cache) ||
        !pa_host::aligned16(q) || !pa_host::aligned16(k) || !pa_host::aligned16(v) || !pa_host::aligned16(cos_sin) ||
        !pa_host::aligned16(q_weight) || !pa_host::aligned16(k_weight) || ((q_stride | k_stride | v_stride) & 7) ||
        (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PA_ERR_MISALIGNED;
    // in place of a strided q, rows would be written over rows still to be read
    if (turned && q_out == q && num_tokens > 1 && q_stride != (int64_t)n_q_heads * d_head) return PA_ERR_INVALID_ARG;
    AppendArgs a{};
    if (num_axes && !set_axes(a, num_axes, axis_of_pair, rot_dim)) return PA_ERR_INVALID_ARG;
    a.q_out = static_cast<uint4*>(q_out);
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.cos_sin = cos_sin;
    a.positions = positions;
    a.slots = slot_mapping;
    a.status = status_dev;
    a.num_slots = (long long)num_blocks * block_size;
    a.eps = eps;
    a.max_positions = max_positions;
    a.rot_dim = rot_dim;
    a.num_tokens = num_tokens;
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = n_kv_heads;
    a.block_size = block_size;
    a.log2_block = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    const bool many = n_q_heads >= 8 && (long long)num_tokens * (n_q_heads + 2 * n_kv_heads) * d_head >= 12000000;
    // Calls of up to 600 tokens are taken for decode batches, a token a block, larger ones for prompts (the slots are on the
    // device).  kMany where its tiles of eight heads are three quarters full or more, and 180 blocks of them, of heads of 128,
    // are there.  32 + 2 x 8 heads of 128, us of kFew / kSome / kMany: prompts of 300 tokens 10.6 / 11.5 / 13.7, 700 13.9 /
    // 12.1 / 14.4, 2003 19.4 / 17.4 / 19.5, 4006 31.5 / 26.5 / 23.0, 8012 58.6 / 47.9 / 41.5; a token each of 256 requests 5.0 /
    // 8.2 / 9.7, 1024 12.8 / 13.7 / 16.4, 4096 36.5 / 28.6 / 27.1.  Other heads (inputs in L2): 2 + 2 x 1 of 128, prompts of 300
    // 8.2 / 5.0 / 6.0, 4006 11.9 / 7.4 / 9.3, 16,000 32.4 / 19.0 / 26.7, 256 requests 3.8 / 6.0 / 7.9, 1024 4.4 / 6.0 / 8.1;
    // 16 + 2 x 2 of 64, 8012 18.9 / 17.0 / 23.2; 32 + 2 x 8 of 64, 3000 16.3 / 11.5 / 13.5, 4006 20.5 / 16.3 / 15.0, 8012 31.9 /
    // 26.4 / 23.8; 32 + 2 x 32 of 128, 700 15.6 / 10.6 / 11.1, 1024 24.1 / 16.9 / 14.5; the append alone, 8 heads of 128, 3000
    // 12.7 / 6.7 / 7.4, 4006 15.8 / 9.7 / 7.6.
    const long long tiles = (n_kv_heads + 7) / 8, blocks = ((long long)num_tokens + kRuns - 1) / kRuns * tiles;
    const bool full = n_kv_heads >= 6 * tiles;
    const int mode = num_tokens < 600 ? kFew : full && blocks * d_head >= 180 * 128 ? kMany : kSome;
    a.q_heads_per = many ? (n_q_heads + 1) / 2 : 1;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        d_head == 128 ? launch_append<128>(a, mode, interleaved, st) : launch_append<64>(a, mode, interleaved, st);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

int pa_qk_norm_rope_cache_scaled(void* q_out, void* k_cache, void* v_cache, uint8_t* k_scales, uint8_t* v_scales,
                                 const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, const float* q_weight, const float* k_weight, float eps,
                                 const float* cos_sin, int max_positions, int rot_dim, int interleaved,
                                 const int32_t* positions, int num_axes, const int8_t* axis_of_pair,
                                 const int64_t* slot_mapping, int num_tokens, int n_q_heads, int n_kv_heads, int d_head,
                                 int block_size, int num_blocks, int32_t* status_dev, void* stream) {
    return append(q_out, k_cache, v_cache, k_scales, v_scales, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight,
                  eps, cos_sin, max_positions, rot_dim, interleaved, positions, num_axes, axis_of_pair, slot_mapping,
                  num_tokens, n_q_heads, n_kv_heads, d_head, block_size, num_blocks, status_dev, stream, true);
}

int pa_reshape_and_cache_scaled(void* k_cache, void* v_cache, uint8_t* k_scales, uint8_t* v_scales, const void* k,
                                const void* v, int64_t k_stride, int64_t v_stride, const int64_t* slot_mapping,
                                int num_tokens, int n_kv_heads, int d_head, int block_size, int num_blocks,
                                int32_t* status_dev, void* stream) {
    return append(nullptr, k_cache, v_cache, k_scales, v_scales, nullptr, k, v, 0, k_stride, v_stride, nullptr, nullptr,
                  0.f, nullptr, 0, 0, 0, nullptr, 0, nullptr, slot_mapping, num_tokens, 0, n_kv_heads, d_head,
                  block_size, num_blocks, status_dev, stream, false);
}

}  // extern "C"
