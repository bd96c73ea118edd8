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
// a block).  A warp takes a run's keys or values of one head: D / 16 lanes a
// token, all of the run's tokens in registers as they came, twice through the
// arithmetic: for the largest value, then for the codes (which is cheaper
// than 32-bit values of a run in registers, and both passes are far below the
// time of its bytes).  A run belongs to the warp that has its first token
// among its own `span`; so decode batches go a token a warp, and prompts
// about a block a warp.  Queries go beside, in blocks of their own.

#include <cuda_fp16.h>
#include <math.h>

#include "pa_rope.cuh"

namespace {

struct AppendArgs : RopeArgs {
    uint8_t* k_scales;
    uint8_t* v_scales;
    int span;                                          // tokens of a warp
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

// Four codes times `by`, rounded again.
__device__ __forceinline__ uint32_t code_again(uint32_t w, float by) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return pa::e4m3x2(x.x * by, x.y * by) | (pa::e4m3x2(y.x * by, y.y * by) << 16);
}

template <int D, int kBlock, bool kInterleaved, bool kAxes>
__global__ void __launch_bounds__(kRopeThreads, 2) append_kernel(const AppendArgs a) {
    constexpr int kLanes = D / 16, kRowsAt = 32 / kLanes;      // tokens side by side in a warp
    constexpr int kRounds = (kBlock + kRowsAt - 1) / kRowsAt;  // of a run
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, l = lane % kLanes, g = lane / kLanes;
    const unsigned mask = ((1u << kLanes) - 1u) << (lane / kLanes * kLanes);
    const Place<kInterleaved> w(l, a.rot_dim);
    // Blocks of both kinds run side by side: queries stream, keys and values wait for their largest.
    const int turn = blockIdx.x / (a.every + 1), kv_before = min((int)(turn + (blockIdx.x % (a.every + 1) != 0)), a.kv_blocks);
    if (blockIdx.x % (a.every + 1) || turn >= a.kv_blocks) {
        // ------------------------------------------------------------ queries
        constexpr int kFlight = 4;
        const uint32_t parts = (a.n_q_heads + a.q_heads_per - 1) / a.q_heads_per;
        const uint32_t nth = (blockIdx.x - kv_before) * (kRopeThreads / kLanes) + threadIdx.x / kLanes;
        const uint32_t t = nth / parts;
        if (t >= (uint32_t)a.num_tokens) return;               // whole heads: a head's threads leave together
        const int h0 = (nth - t * parts) * a.q_heads_per, h1 = min(h0 + a.q_heads_per, a.n_q_heads);
        Where<kAxes> at;
        at.load(a, t);
        const __nv_bfloat16* rows = a.q + (long long)t * a.q_stride;
        uint4 x0[kFlight], x1[kFlight];
        auto load = [&](int h) {
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (h + u < h1) {
                    const uint4* src = reinterpret_cast<const uint4*>(rows + (h + u) * D);
                    x0[u] = src[w.c0];
                    x1[u] = src[w.c1];
                }
        };
        load(h0);
        uint64_t gain[8];
        if (a.q_weight) {
            load8(a.q_weight + 8 * w.c0, gain);
            load8(a.q_weight + 8 * w.c1, gain + 4);
        }
        if (at.lowest() < 0 || at.highest() >= a.max_positions) return;   // (flagged by the keys' warps)
        uint64_t cs[4], sn[4];
        if (w.turns) load_angles<kAxes>(a, at, l, cs, sn);
#pragma unroll 1
        for (int h = h0; h < h1; h += kFlight) {
            uint4 y0[kFlight], y1[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                y0[u] = x0[u];
                y1[u] = x1[u];
            }
            load(h + kFlight);
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (h + u >= h1) break;
                Part p;
                unpack8(y0[u], p.f);
                unpack8(y1[u], p.f + 4);
                if (a.q_weight) norm_part<kLanes>(p, gain, a.eps, mask);
                if (w.turns) turn_part<kInterleaved>(p, cs, sn);
                uint4* dst = a.q_out + ((size_t)t * a.n_q_heads + h + u) * (D / 8);
                dst[w.c0] = pack8(p.f);
                dst[w.c1] = pack8(p.f + 4);
            }
        }
        return;
    }
    // ---------------------------------------------------------------- keys and values
    const uint32_t per = 2 * a.n_kv_heads, item = turn * kWarps + (threadIdx.x >> 5), first = item / per * a.span;
    if (first >= (uint32_t)a.num_tokens) return;
    const int which = item % per, h = which >> 1;
    const bool is_v = which & 1;
    // Tokens first - 1 .. first + 62, two a lane: their slots, negative where nothing is written.
    long long slot[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const long long t = (long long)first - 1 + lane + 32 * x;
        slot[x] = -1;
        if (t >= 0 && t < a.num_tokens && lane + 32 * x < a.span + kBlock) {
            slot[x] = a.slots[t];
            bool there = true;
            if (a.positions) {
                Where<kAxes> at;
                at.load(a, t);
                there = at.lowest() >= 0 && at.highest() < a.max_positions;
                if (which == 0 && at.lowest() >= 0 && !there) pa::set_status(a.status, PA_DEV_BAD_POSITION);
            }
            if (!there) slot[x] = -1;
            if (slot[x] >= a.num_slots) {
                if (which == 0) pa::set_status(a.status, PA_DEV_BAD_SLOT);
                slot[x] = -1;
            }
        }
    }
    unsigned long long there, follows;                           // bit j: token first - 1 + j is written; and goes on with the run
    {
        const long long p0 = __shfl_up_sync(0xffffffffu, slot[0], 1), p1 = __shfl_up_sync(0xffffffffu, slot[1], 1);
        const long long last = __shfl_sync(0xffffffffu, slot[0], 31);
        const long long before[2] = {lane ? p0 : -1, lane ? p1 : last};
        unsigned b[2], f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            b[x] = __ballot_sync(0xffffffffu, slot[x] >= 0);
            f[x] = __ballot_sync(0xffffffffu, slot[x] >= 0 && before[x] >= 0 && slot[x] == before[x] + 1 && (slot[x] & (kBlock - 1)));
        }
        there = b[0] | (unsigned long long)b[1] << 32;
        follows = f[0] | (unsigned long long)f[1] << 32;
    }
    unsigned long long heads = there & ~follows & (((1ull << a.span) - 1) << 1);   // the runs' first tokens (span <= 32)
    const __nv_bfloat16* src = is_v ? a.v : a.k;
    const long long stride = is_v ? a.v_stride : a.k_stride;
    uint8_t* cache = is_v ? a.v_cache : a.k_cache;
    uint8_t* all_scales = is_v ? a.v_scales : a.k_scales;
    const bool norm = !is_v && a.k_weight, turns = !is_v && w.turns;
#pragma unroll 1
    for (; heads; heads &= heads - 1) {
        const int j = __ffsll((long long)heads) - 1;
        const int n = __ffsll((long long)~(follows >> (j + 1)));  // tokens of the run, kBlock at most
        const long long s0 = __shfl_sync(0xffffffffu, j < 32 ? slot[0] : slot[1], j & 31);
        const int blk = (int)(s0 >> a.log2_block), off = (int)s0 & (kBlock - 1);
        const size_t t0 = (size_t)first - 1 + j;
        uint8_t* scales = all_scales + (size_t)blk * a.n_kv_heads + h;
        uint8_t* rows = cache + ((size_t)blk * a.n_kv_heads + h) * (kBlock * D);
        uint4 x0[kRounds], x1[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int i = r * kRowsAt + g;
            x0[r] = x1[r] = make_uint4(0, 0, 0, 0);
            if (i < n) {
                const uint4* p = reinterpret_cast<const uint4*>(src + (long long)(t0 + i) * stride + h * D);
                x0[r] = p[w.c0];
                x1[r] = p[w.c1];
            }
        }
        const int old = off ? *scales : 0;
        // round r's part of the rows, ready for the cache
        auto part = [&](int r) {
            Part p;
            unpack8(x0[r], p.f);
            unpack8(x1[r], p.f + 4);
            if (norm) {
                uint64_t gain[8];                                // (from L1: registers are short)
                load8(a.k_weight + 8 * w.c0, gain);
                load8(a.k_weight + 8 * w.c1, gain + 4);
                norm_part<kLanes>(p, gain, a.eps, mask);
            }
            const int i = r * kRowsAt + g;
            if (turns && i < n) {
                Where<kAxes> at;
                at.load(a, t0 + i);
                uint64_t cs[4], sn[4];
                load_angles<kAxes>(a, at, l, cs, sn);
                turn_part<kInterleaved>(p, cs, sn);
            }
            return p;
        };
        float top = 0.f;
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (r * kRowsAt < n) top = top_of(part(r), top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (!(top < INFINITY)) {                                 // infinities saturate, at the scale of the others
            top = 0.f;
#pragma unroll
            for (int r = 0; r < kRounds; ++r)
                if (r * kRowsAt < n) top = finite_top_of(part(r), top);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        const int now = max(old, scale_byte(top));
        const float up = scale_of(254 - now);
        const uint64_t by = pair(up, up);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int i = r * kRowsAt + g;
            if (r * kRowsAt >= n) break;
            const Part p = part(r);
            if (i < n) {
                uint2* dst = reinterpret_cast<uint2*>(rows + (off + i) * D);
                dst[w.c0] = codes_by(p.f, by);
                dst[w.c1] = codes_by(p.f + 4, by);
            }
        }
        if (off && now > old) {                                  // the scale has grown: the block's other codes again
            const float down = now - old > 126 ? 0.f : scale_of(127 - (now - old));
#pragma unroll 1
            for (int x = lane; x < kBlock * (D / 16); x += 32) {
                const int row = x / (D / 16);
                if (row >= off && row < off + n) continue;
                uint4* p = reinterpret_cast<uint4*>(rows) + x;
                uint4 v = *p;
                v.x = code_again(v.x, down);
                v.y = code_again(v.y, down);
                v.z = code_again(v.z, down);
                v.w = code_again(v.w, down);
                *p = v;
            }
        }
        if (lane == 0 && (now != old || !off)) *scales = (uint8_t)now;
    }
}

template <int D, int kBlock>
cudaError_t launch_append(const AppendArgs& a, int interleaved, cudaStream_t st) {
    constexpr int kLanes = D / 16;
    const long long kv = ((long long)a.num_tokens + a.span - 1) / a.span * 2 * a.n_kv_heads;
    const long long q = a.n_q_heads ? (long long)a.num_tokens * ((a.n_q_heads + a.q_heads_per - 1) / a.q_heads_per) : 0;
    AppendArgs b = a;
    b.kv_blocks = (int)((kv + kWarps - 1) / kWarps);
    const int q_blocks = (int)((q + kRopeThreads / kLanes - 1) / (kRopeThreads / kLanes));
    b.every = q_blocks / b.kv_blocks;
    const unsigned grid = (unsigned)(b.kv_blocks + q_blocks);
    const auto kernel = a.num_axes ? (interleaved ? append_kernel<D, kBlock, true, true> : append_kernel<D, kBlock, false, true>)
                                   : (interleaved ? append_kernel<D, kBlock, true, false> : append_kernel<D, kBlock, false, false>);
    return pa_host::launch_dependent(kernel, dim3(grid), dim3(kRopeThreads), 0, st, b);
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
    a.span = num_tokens <= 2048 ? 1 : block_size;
    const bool many = n_q_heads >= 8 && (long long)num_tokens * (n_q_heads + 2 * n_kv_heads) * d_head >= 12000000;
    a.q_heads_per = many ? (n_q_heads + 1) / 2 : 1;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        d_head == 128 ? (block_size == 8    ? launch_append<128, 8>(a, interleaved, st)
                         : block_size == 16 ? launch_append<128, 16>(a, interleaved, st)
                                            : launch_append<128, 32>(a, interleaved, st))
                      : (block_size == 8    ? launch_append<64, 8>(a, interleaved, st)
                         : block_size == 16 ? launch_append<64, 16>(a, interleaved, st)
                                            : launch_append<64, 32>(a, interleaved, st));
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
