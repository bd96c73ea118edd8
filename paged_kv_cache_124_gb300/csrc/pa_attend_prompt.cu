// Prompts and long chunks of pa_attend and pa_attend_scaled: the prefill
// kernel (pa_prefill.cuh) with shaped scores, and its staging passes.
//
// What the shape changes: an item's tiles run from the first position that
// one of its rows sees to the last, rather than from 0 to its own; scores are
// capped and biased in registers before the softmax; rows mask by an interval.
// The staging leaves out blocks that no token sees, and values that are not
// finite, since the weights of rows that do not see them are zeros and 0 * inf
// is not; the rows that see them add them when they are written.  From a block-scaled cache it makes
// bf16 keys and fp16 values that hold every element exactly (a tile whose
// blocks' scales are outside fp16's range keeps bf16 values, as pa_prefill's
// do).
//
// 8 prompts of 2,003 tokens with spans: 296 us, 957 TFLOP/s of what is seen.
// With a cap: 393 us, 721 TFLOP/s, where all scores of a warp's half tile are
// within a quarter of it (scores of deviation 2 under a cap of 50: the cap is
// taken with the weights); 463 where they are within half of it (deviation 4:
// a longer polynomial before the maximum), 667 where they go beyond (deviation
// 10: two special functions a score).  Nothing is full (issue 41 %, ALU 25 %,
// tensor 34 %): both halves of a row tile wait for each other's maximum at
// every tile before they write a weight, with two warps a scheduler, and the
// code is long for the instruction cache (0.8 of a stall in each issue).  When
// it took 415, sixteen softmax warps took 466, four for each row tile by itself
// 489 and eight for each 474.  Keeping what is not seen out of the cap's form
// costs 2 % (in one loop with the mask behind it 10 %, only where scores are
// large, which is more code, 4 %).  8 chunks of 512 tokens over block-scaled
// prefixes of 2,048 to 8,192: 353 us, 925 TFLOP/s, of which the staging is some
// 30 us.  Tiles of small values (stage_shaped_v_kernel) take two-term weights:
// 8 causal prompts all of whose values are below 2^-10 401 us against 273.

#include "pa_attend.cuh"
#include "pa_prefill.cuh"

namespace {

struct ShapedStageArgs : StageArgs {
    const uint8_t* k_scales;
    const uint8_t* v_scales;
    const int32_t* query_start;
    const int2* visible;
    int num_tokens, ctx_cap, max_query_len;
    int* sched;           // zeroed for the prefill kernel's claims
};

// The positions from the first to the last that some token of the sequence
// sees (x .. y - 1), found by a whole block; what lies outside is not read.  Of
// a sequence without new tokens, or one that the prefill kernel flags and
// leaves out (by the same conditions), none.
__device__ __forceinline__ int2 seen_of(const ShapedStageArgs& a, int s, int ctx) {
    const int q0 = a.query_start[s], q1 = a.query_start[s + 1];
    if (q0 < 0 || q1 <= q0 || q1 > a.num_tokens || q1 - q0 > ctx || q1 - q0 > a.max_query_len) return make_int2(0, 0);
    if (!a.visible) return make_int2(0, ctx);
    __shared__ int2 part[8];
    int lo = INT_MAX, hi = 0;
    for (int t = q0 + threadIdx.x; t < q1; t += 256) {
        const int2 v = a.visible[t];
        const int from = max(v.x, 0), to = min(v.y, ctx);
        if (from < to) {
            lo = min(lo, from);
            hi = max(hi, to);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_int2(lo, hi);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        lo = min(lo, part[w].x);
        hi = max(hi, part[w].y);
    }
    return make_int2(lo, hi);
}

// Whether tile j has such positions; which, in `seen`.
__device__ __forceinline__ bool tile_there(const ShapedStageArgs& a, int s, int j, int2& seen) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x < 2 && blockIdx.x + blockIdx.y + blockIdx.z == 0) a.sched[threadIdx.x] = 0;
    int ctx = a.context_lens[s];
    ctx = min(max(ctx, 0), a.ctx_cap);                           // the prefill kernel flags and clamps the same
    if (j * kKv >= ctx) return false;
    seen = seen_of(a, s, ctx);
    return seen.x < (j + 1) * kKv && seen.y > j * kKv;
}

// Whether a position's block holds any of them.
__device__ __forceinline__ bool block_there(int pos, int2 seen, int block_size) {
    return pos < seen.y && (pos | (block_size - 1)) >= seen.x;
}

// Two bf16 that are not finite, as a mask.
__device__ __forceinline__ uint32_t unfinite2(uint32_t w) {
    return ((((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 15) * 0xffffu;
}

// stage_v_kernel without the values that are not finite (format bit 1: there are some), and whose tiles stay bf16 also
// where some position's values are all small: fp16 rounds them to steps of 2^-24 below 2^-14, and a row may see no others.
// So a value is off by at most 2^-25, 2^-15 of the largest of its position.  (Zeros are exact.)
constexpr uint32_t kF16Small = 0x3A80;                           // 2^-10
template <int D>
__global__ void __launch_bounds__(256) stage_shaped_v_kernel(const uint4* __restrict__ v_cache, const ShapedStageArgs a) {
    constexpr int kChunksPerRow = D / 8, kPer = kKv * kChunksPerRow / 256;
    const int j = blockIdx.x, s = blockIdx.y, h = blockIdx.z;
    int2 seen;
    if (!tile_there(a, s, j, seen)) return;
    const int32_t* table = a.block_tables + (size_t)s * a.max_blocks;
    const int log2_block = __ffs(a.block_size) - 1;
    uint4 v[kPer];
    uint32_t amax = 0, bad = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = threadIdx.x + 256 * i, pos = j * kKv + c / kChunksPerRow;
        v[i] = make_uint4(0, 0, 0, 0);
        if (block_there(pos, seen, a.block_size)) {
            const int blk = __ldg(table + (pos >> log2_block));
            if (blk >= 0 && blk < a.num_blocks)
                v[i] = __ldg(v_cache + ((((size_t)blk * a.n_kv_heads + h) << log2_block) + (pos & (a.block_size - 1))) * kChunksPerRow +
                             c % kChunksPerRow);
            // a bad entry reads zeros; the prefill kernel's K loads flag it
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint4 m = make_uint4(unfinite2(v[i].x), unfinite2(v[i].y), unfinite2(v[i].z), unfinite2(v[i].w));
        bad |= m.x | m.y | m.z | m.w;
        v[i] = make_uint4(v[i].x & ~m.x, v[i].y & ~m.y, v[i].z & ~m.z, v[i].w & ~m.w);
        amax = max_u16x2(amax, max_u16x2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu));
        amax = max_u16x2(amax, max_u16x2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
    }
    bool small = false;                                          // a position's chunks lie in neighbouring lanes
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t m = max_u16x2(max_u16x2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                     max_u16x2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
        const uint32_t mine = (kChunksPerRow == 16 ? 0xffffu : 0xffu) << (threadIdx.x & 31 & -kChunksPerRow);
        const bool large = (m & 0xffffu) >= kF16Small || (m >> 16) >= kF16Small;
        const uint32_t filled = __ballot_sync(0xffffffffu, m != 0) & mine, larges = __ballot_sync(0xffffffffu, large) & mine;
        small |= filled != 0 && larges == 0;
    }
    const bool wide = __syncthreads_or(small || (amax & 0xffffu) >= kF16Wide || (amax >> 16) >= kF16Wide) != 0;
    const bool some = __syncthreads_or(bad != 0) != 0;
    uint4* dst = reinterpret_cast<uint4*>(a.v_stage + ((size_t)(h * a.num_seqs + s) * a.l_slot + (size_t)j * kKv) * D);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        dst[threadIdx.x + 256 * i] = wide ? v[i]
                                          : make_uint4(bf16x2_to_f16x2(v[i].x), bf16x2_to_f16x2(v[i].y),
                                                       bf16x2_to_f16x2(v[i].z), bf16x2_to_f16x2(v[i].w));
    if (threadIdx.x == 0) a.v_fmt[(size_t)(h * a.num_seqs + s) * a.t_slot + j] = (wide ? 1 : 0) | (some ? 2 : 0);
}

// Two bf16, the largest for what is beyond it (infinite, it would reach rows that do not see it).
__device__ __forceinline__ uint32_t pack_bf16_finite(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A block-scaled cache's tile: K as bf16 (even blocks of z), V (odd ones) as fp16 where the blocks' scales are 2^-15 ..
// 2^7 (the values are multiples of 2^-24 below 2^16 then), else as bf16; all exact but for values beyond bf16's
// largest.
template <int D>
__global__ void __launch_bounds__(256) stage_scaled_kernel(const uint4* __restrict__ k_cache, const uint4* __restrict__ v_cache,
                                                           uint16_t* k_stage, const ShapedStageArgs a) {
    constexpr int kChunksPerRow = D / 16, kPer = kKv * kChunksPerRow / 256;
    const int j = blockIdx.x, s = blockIdx.y, h = blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    int2 seen;
    if (!tile_there(a, s, j, seen)) return;
    const int32_t* table = a.block_tables + (size_t)s * a.max_blocks;
    const uint4* cache = is_v ? v_cache : k_cache;
    const uint8_t* scales = is_v ? a.v_scales : a.k_scales;
    const int log2_block = __ffs(a.block_size) - 1;
    uint4 code[kPer];
    float scale[kPer];
    bool narrow = true;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = threadIdx.x + 256 * i, pos = j * kKv + c / kChunksPerRow;
        code[i] = make_uint4(0, 0, 0, 0);
        scale[i] = 0.f;
        if (block_there(pos, seen, a.block_size)) {
            const int blk = __ldg(table + (pos >> log2_block));
            if (blk >= 0 && blk < a.num_blocks) {
                const size_t block = (size_t)blk * a.n_kv_heads + h;
                code[i] = __ldg(cache + ((block << log2_block) + (pos & (a.block_size - 1))) * kChunksPerRow + c % kChunksPerRow);
                const int e = scales[block];
                scale[i] = __int_as_float(e ? e << 23 : 0x00400000);
                if (e && (e < 112 || e > 134)) narrow = false;   // (what 2^-127 scales is nothing to any sum)
            } else if (!is_v) {
                pa::set_status(a.status, PA_DEV_BAD_BLOCK_ID);
            }
        }
    }
    bool wide = true;
    if (is_v) {
        uint32_t bad = 0;
        auto nan4 = [](uint32_t w) { return ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu; };
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            uint4& v = code[i];                                  // NaN, E4M3's only one that is not finite
            const uint4 m = make_uint4(nan4(v.x), nan4(v.y), nan4(v.z), nan4(v.w));
            bad |= m.x | m.y | m.z | m.w;
            v = make_uint4(v.x & ~m.x, v.y & ~m.y, v.z & ~m.z, v.w & ~m.w);
        }
        wide = __syncthreads_or(!narrow) != 0;
        const bool some = __syncthreads_or(bad != 0) != 0;
        if (threadIdx.x == 0) a.v_fmt[(size_t)(h * a.num_seqs + s) * a.t_slot + j] = (wide ? 1 : 0) | (some ? 2 : 0);
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? a.v_stage : k_stage) + ((size_t)(h * a.num_seqs + s) * a.l_slot + (size_t)j * kKv) * D);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
        uint32_t f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            const float lo = x.x * scale[i], hi = x.y * scale[i];
            f[e] = wide ? pack_bf16_finite(lo, hi) : pack_f16_rn(lo, hi);
        }
        st_global_v8(dst + 2 * (threadIdx.x + 256 * i), f);      // (whole sectors; the workspace is 256-byte aligned)
    }
}

constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool kScaled, class Args>
int launch_shaped(const Args& a, const ShapedStageArgs& sa, const pa_attend_calls::Call& c, uint16_t* k_stage, int grid) {
    CUtensorMap mq, mk, mv;
    const long long cache_rows = (long long)c.num_blocks * c.n_kv_heads * c.block_size;
    if (!make_maps<D>(mq, mk, mv, a, sa, c.q, c.k_cache, kScaled ? k_stage : nullptr, c.num_tokens, cache_rows)) return PA_ERR_CUDA;
    const auto kernel = prefill_kernel<D, kScaled, Args>;
    if (pa_host::ensure_smem_attr(kernel, PGeo<D>::kSmem, g_smem_done<D, kScaled, Args>) != cudaSuccess)
        return PA_ERR_CUDA;
    const dim3 sgrid((unsigned)sa.t_slot, (unsigned)sa.num_seqs, (unsigned)(kScaled ? 2 * sa.n_kv_heads : sa.n_kv_heads));
    cudaError_t e;
    if constexpr (kScaled)
        e = pa_host::launch_dependent(stage_scaled_kernel<D>, sgrid, dim3(256), 0, c.stream, static_cast<const uint4*>(c.k_cache),
                                      static_cast<const uint4*>(c.v_cache), k_stage, sa);
    else
        e = pa_host::launch_dependent(stage_shaped_v_kernel<D>, sgrid, dim3(256), 0, c.stream, static_cast<const uint4*>(c.v_cache), sa);
    if (e != cudaSuccess) return PA_ERR_CUDA;
    return pa_host::launch_dependent(kernel, dim3(grid), dim3(kThreads), PGeo<D>::kSmem, c.stream, mq, mk, mv, a) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

namespace pa_attend_calls {

size_t prompt_workspace(int num_seqs, int max_query_len, int max_blocks, int block_size, int n_q_heads, int n_kv_heads,
                        int d_head, bool scaled) {
    const int group = n_q_heads / n_kv_heads;
    const double tiles = ((double)max_query_len * group + 2 * kRows - 1) / (2 * kRows);
    const double slots = ((double)max_blocks * block_size + kKv) * num_seqs * n_kv_heads;
    if (num_seqs > 65535 || n_kv_heads > (scaled ? 32767 : 65535) || group > kRows || slots > INT_MAX - kKv ||
        tiles * num_seqs * n_kv_heads > INT_MAX - 4096.0)
        return 0;
    return workspace_layout(num_seqs, max_blocks, block_size, n_kv_heads, d_head, scaled).total + 256;
}

int launch_prompt(const Call& c) {
    const bool scaled = c.k_scales != nullptr;
    const Workspace ws = workspace_layout(c.num_seqs, c.max_blocks, c.block_size, c.n_kv_heads, c.d_head, scaled);
    uint8_t* w8 = static_cast<uint8_t*>(c.workspace);
    int* sched = reinterpret_cast<int*>(w8 + ws.total);
    const int group = c.n_q_heads / c.n_kv_heads, tq = kRows / group;
    const long long tiles = ((long long)c.max_query_len + 2 * tq - 1) / (2 * tq), items = tiles * c.num_seqs * c.n_kv_heads;
    ShapedPrefillArgs a{};
    a.out = c.out;
    a.out_f32 = c.out_f32;
    a.out_al32 = (reinterpret_cast<uintptr_t>(c.out) & 31u) == 0;
    a.block_tables = c.block_tables;
    a.max_blocks = c.max_blocks;
    a.query_start = c.query_start;
    a.context_lens = c.context_lens;
    a.num_seqs = c.num_seqs;
    a.num_tokens = c.num_tokens;
    a.tiles_per_seq = (int)tiles;
    a.block_size = c.block_size;
    a.n_kv_heads = c.n_kv_heads;
    a.group = group;
    a.tq = tq;
    a.n_q_heads = c.n_q_heads;
    a.num_blocks = c.num_blocks;
    a.oob_row = c.num_blocks * c.n_kv_heads * c.block_size;
    a.scale_log2 = c.scale * kLog2e;
    a.v_fmt = w8 + ws.fmt_off;
    a.l_slot = ws.l_slot;
    a.t_slot = ws.t_slot;
    a.k_scale = a.v_scale = 1.f;
    a.status = c.status;
    a.sched = sched;
    a.visible = reinterpret_cast<const int2*>(c.visible);
    a.slopes = c.slopes;
    a.cap_log2 = c.softcap * kLog2e;
    a.cap_inv = c.softcap > 0.f ? fminf(1.f / a.cap_log2, pa::kMostCapInv) : 0.f;
    a.v_cache = c.v_cache;
    a.ctx_cap = c.ctx_cap;
    a.max_query_len = c.max_query_len;
    const int sms = num_sms(), grid = (int)(items < sms ? items : sms);
    const long long per_head = tiles * c.num_seqs, hpg = (2LL * grid + per_head - 1) / per_head;
    a.heads_per_group = (int)(hpg < 1 ? 1 : hpg > c.n_kv_heads ? c.n_kv_heads : hpg);
    ShapedStageArgs sa{};
    sa.block_tables = c.block_tables;
    sa.max_blocks = c.max_blocks;
    sa.context_lens = c.context_lens;
    sa.num_seqs = c.num_seqs;
    sa.block_size = c.block_size;
    sa.n_kv_heads = c.n_kv_heads;
    sa.num_blocks = c.num_blocks;
    sa.l_slot = ws.l_slot;
    sa.t_slot = ws.t_slot;
    sa.v_stage = reinterpret_cast<uint16_t*>(w8);
    sa.v_fmt = w8 + ws.fmt_off;
    sa.status = c.status;
    sa.k_scales = c.k_scales;
    sa.v_scales = c.v_scales;
    sa.query_start = c.query_start;
    sa.visible = a.visible;
    sa.num_tokens = c.num_tokens;
    sa.max_query_len = c.max_query_len;
    sa.sched = sched;
    sa.ctx_cap = c.ctx_cap;
    const auto with = [&](auto form) {
        static_cast<ShapedPrefillArgs&>(form) = a;
        return form;
    };
    const auto launch = [&](const auto& args) {
        if (scaled) return launch_shaped<128, true>(args, sa, c, reinterpret_cast<uint16_t*>(w8 + ws.k_off), grid);
        return c.d_head == 128 ? launch_shaped<128, false>(args, sa, c, nullptr, grid) : launch_shaped<64, false>(args, sa, c, nullptr, grid);
    };
    if (c.slopes) return launch(with(BiasedPrefillArgs{}));
    return c.softcap > 0.f ? launch(with(CappedPrefillArgs{})) : launch(a);
}

}  // namespace pa_attend_calls
