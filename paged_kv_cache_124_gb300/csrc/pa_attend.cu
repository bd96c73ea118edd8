// Attention of new tokens over the paged cache with shaped scores, from one
// token a sequence to whole prompts: scores capped by a tanh, less a bias by
// distance, over an interval of positions per token, and over bf16 caches or
// E4M3 codes with a power-of-two scale per block and head (pa_attend,
// pa_attend_scaled; the formulas stand in pa.h).
//
// Three kernels take them (route_of): units of 16 rows a KV head, on warp-level
// products (pa_multi_rows.cuh), units of 64 and 128 rows on the tensor cores
// (pa_wide.cuh), and whole prompts (pa_prefill.cuh).  In the first two a
// sequence's work begins at the first position that some token of it sees and
// ends behind the last; in the third that goes by items of 256 rows: so a
// window costs its own bytes.
//
// What the shape costs beside the plain kernels: with few rows, arithmetic
// that the cache's bytes hide (64 decodes of 4096 positions, capped, 170 us,
// 0.93 of the measured copy rate; block-scaled 100, 0.80, and 113 with blocks
// of 8, against 92 with one scale: a score and a weight take a factor more).
// With many, the softmax of a tile is the longer: 8 prompts of 2003 tokens 273
// us causal (272 plain), 346 with a bias, 358 with a cap beside which scores
// are small, 433 and 612 where they are not (pa_attend_prompt.cu).

#include "pa_attend.cuh"
#include "pa_cap.cuh"
#include "pa_multi_rows.cuh"

namespace {

enum Route { kUnits16, kWide, kPrompt };

// From this many rows a KV head on (new tokens times the group's heads) a call may go to the prefill kernel.
constexpr long long kPromptRows = 192;

// Which kernel takes a call.  Up to 16 rows a KV head, with a scale that is
// not positive, and over few short contexts (in_small_tiles): units of 16 rows.
// More rows: units of 64 or 128 (wide), whose contexts are split over the
// device, or the prefill kernel, whose items of 256 rows read their keys once,
// up to their own last one.  Block-scaled calls of up to 32 rows, half of what
// a wide unit holds, stay with units of 16 also where the context is one tile
// of a wide unit and there are three units of it an SM or more, so that its
// chain of a tile from beginning to end is what they wait for.
//
// The estimates (us) count wide units, at 1.55 us of an SM a tile of 128
// positions (block-scaled, 64 rows: 1.25) and 5 (4.5) to begin and end, and
// items, at 1.9 a tile of two and 5.5, most of the last wave waited for,
// behind their staging.  32 query and 8 KV heads, us of wide / prefill:
//   contexts x new tokens   bf16        block-scaled
//   8 x 8192, 64            106 / 159   143 / 185
//   8 x 8192, 128           184 / 161   264 / 187
//   8 x 4096, 192           150 / 142   218 / 158
//   8 x 1024, 128            52 / 33     63 / 35
//   64 x 2048, 64           198 / 219   312 / 259
//   64 x 512, 64             88 / 74    139 / 83
//   1 x 16384, 512          172 / 240   259 / 253
//   3 x 700, 64              16 / 23     16 / 24
//   64 x 64, 64              53 / 36     87 / 37
// and of units of 16 rows / wide, 8 tokens (32 rows), contexts of
//                           60            128           256           512
//   block-scaled, 32      17 / 17       20 / 17       23 / 21       29 / 26
//                 64      22 / 26       27 / 27       36 / 32       48 / 46
//                 256     60 / 76       73 / 84       98 / 101     145 / 136
//                 1024   227 / 305     278 / 318     370 / 388     558 / 443
//   bf16,         64      21 / 22       26 / 22       32 / 27       49 / 34
//                 1024   190 / 195     230 / 202     355 / 253     690 / 362
// (12 tokens, 48 rows, block-scaled: 64 x 60 30 / 26, 1024 x 60 337 / 331; 5 tokens, 20 rows: 110 / 141 for 512 x 60).
Route route_of(long long rows, float scale, bool f8, int num_seqs, int n_kv_heads, int group, int ctx) {
    const double heads = (double)num_seqs * n_kv_heads;
    if (rows <= kRows || !(scale > 0.f) || in_small_tiles(f8, rows, heads, ctx)) return kUnits16;
    const double sm = std::max(1, sms());
    if (f8 && rows <= 32 && ctx <= kWideStep && heads >= 3 * sm) return kUnits16;
    if (rows < kPromptRows) return kWide;
    const double units = heads * (double)((rows + (f8 ? 63 : 127)) / (f8 ? 64 : 128)), tiles = (ctx + 127) / 128;
    const double wide = 5 + units * tiles * (f8 ? 1.25 : 1.55) / sm + ceil(units / sm) * (f8 ? 4.5 : 5) + (units > sm ? 4 : 0);
    const double items = heads * (double)((rows + 255) / 256), seen = (ctx - 0.5 * (double)(rows / group)) / 128 + 0.5;
    const double waves = items <= sm ? 1 : 0.15 * items / sm + 0.85 * ceil(items / sm);
    const double prompt = 8 + waves * (1.9 * seen + 5.5) + heads * ctx * (f8 ? 0.9e-4 : 0.6e-4);
    return wide <= prompt ? kWide : kPrompt;
}

int unit_of(Route route, long long rows, bool f8) { return unit_rows(rows, f8, route == kWide); }

int attend(void* out, int out_dtype, const void* q, const void* k_cache, const void* v_cache, const uint8_t* k_scales,
           const uint8_t* v_scales, const int32_t* block_tables, const int32_t* query_start,
           const int32_t* context_lens, const int32_t* visible, const float* slopes, float softcap, int block_size,
           float scale, int n_q_heads, int n_kv_heads, int d_head, int num_seqs, int num_tokens, int max_query_len,
           int max_blocks_per_seq, int num_blocks, int max_context_len, void* workspace, size_t workspace_bytes,
           int32_t* status_dev, void* stream, bool f8) {
    if (num_seqs < 0 || num_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || max_query_len <= 0 ||
        max_blocks_per_seq <= 0 || num_blocks <= 0 || max_context_len < 0 || !(fabsf(scale) < INFINITY) ||
        !(softcap >= 0.f) || !(softcap < INFINITY))
        return PA_ERR_INVALID_ARG;
    if (out_dtype != PA_DTYPE_BF16 && out_dtype != PA_DTYPE_F32) return PA_ERR_INVALID_ARG;
    if (!pa_host::supported_block_size(block_size) || !pa_host::supported_d_head(d_head)) return PA_ERR_UNSUPPORTED;
    if (f8 && d_head != 128) return PA_ERR_UNSUPPORTED;
    if (n_q_heads % n_kv_heads) return PA_ERR_UNSUPPORTED;
    const int group = n_q_heads / n_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8 && group != 16) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !query_start || !context_lens || out == q ||
        (f8 && (!k_scales || !v_scales)))
        return PA_ERR_INVALID_ARG;
    if (!pa_host::aligned16(out) || !pa_host::aligned16(q) || !pa_host::aligned16(k_cache) ||
        !pa_host::aligned16(v_cache) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
        (reinterpret_cast<uintptr_t>(query_start) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(visible) & 7u) || (reinterpret_cast<uintptr_t>(slopes) & 3u))
        return PA_ERR_MISALIGNED;
    const long long cache_rows = (long long)num_blocks * n_kv_heads * block_size;
    if (cache_rows > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    const long long all_rows = (long long)max_query_len * group;
    const long long cap = (long long)max_blocks_per_seq * block_size;
    const int ctx_cap = (int)(cap < max_context_len ? cap : max_context_len);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return PA_ERR_WORKSPACE;
    Route route = route_of(all_rows, scale, f8, num_seqs, n_kv_heads, group, ctx_cap);
    if (route == kPrompt) {
        const size_t n = pa_attend_calls::prompt_workspace(num_seqs, max_query_len, max_blocks_per_seq, block_size, n_q_heads,
                                                           n_kv_heads, d_head, f8);
        if (n) {
            if (workspace_bytes < n) return PA_ERR_WORKSPACE;
            return pa_attend_calls::launch_prompt({out, out_dtype == PA_DTYPE_F32, q, k_cache, v_cache, k_scales, v_scales,
                                                   block_tables, query_start, context_lens, visible, slopes, softcap, scale,
                                                   block_size, n_q_heads, n_kv_heads, d_head, num_seqs, num_tokens,
                                                   max_query_len, max_blocks_per_seq, num_blocks, ctx_cap, workspace,
                                                   status_dev, static_cast<cudaStream_t>(stream)});
        }
        route = kWide;
    }
    const bool wide = route == kWide;
    const int unit = unit_of(route, all_rows, f8), most = max_grid(wide);
    if (most <= 0) return PA_ERR_CUDA;
    if (workspace_bytes < workspace_size(most, unit, d_head)) return PA_ERR_WORKSPACE;

    CurvedArgs a{};
    a.ctx_cap = ctx_cap;
    if ((double)((all_rows + unit - 1) / unit) * num_seqs * n_kv_heads > 1 << 30) return PA_ERR_UNSUPPORTED;
    const Split split = split_work(f8, wide, all_rows, num_seqs, n_kv_heads, ctx_cap);
    a.direct = split.direct;
    a.out = out;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.query_start = query_start;
    a.context_lens = context_lens;
    set_workspace(a, workspace, split.grid, unit);
    a.status = status_dev;
    const float factor = fabsf(scale) * kLog2e;
    a.scale_log2 = factor == 0.f ? 1.f : factor;
    a.q_sign = factor == 0.f ? 0.f : scale > 0.f ? 1.f : -1.f;
    a.v_scale = f8 && !wide ? 1.f / kWeightScale : 1.f;         // (the wide kernel's sums carry its weights' factor)
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
    a.visible = reinterpret_cast<const int2*>(visible);
    a.slopes = slopes;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.cap_log2 = softcap * kLog2e;
    a.cap_inv = softcap > 0.f ? fminf(1.f / a.cap_log2, pa::kMostCapInv) : 0.f;
    const int box = wide || block_size < kTile ? block_size : kTile;
    CUtensorMap mk, mv;
    if (!pa_host::cache_view(&mk, k_cache, cache_rows, d_head, f8 ? 1 : 2, box) ||
        !pa_host::cache_view(&mv, v_cache, cache_rows, d_head, f8 ? 1 : 2, box))
        return PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto launch = [&](const auto& args) {
        if (f8 && all_rows <= 8) return launch_multi<128, true, true>(split.warps, mk, mv, args, split.grid, st);
        return f8              ? launch_multi<128, true>(split.warps, mk, mv, args, split.grid, st)
               : d_head == 128 ? launch_multi<128, false>(split.warps, mk, mv, args, split.grid, st)
                               : launch_multi<64, false>(split.warps, mk, mv, args, split.grid, st);
    };
    int rc;
    if (wide)
        rc = launch_shaped_wide(unit, d_head, f8, q, block_size, mk, mv, a, split.grid, st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    else
        rc = a.cap_inv != 0.f || a.slopes ? launch(a) : launch(static_cast<const ShapedArgs&>(a));
    if (rc != PA_OK || split.direct) return rc;
    return launch_merge(a, unit, d_head, split.units, split.grid, st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t pa_attend_workspace_size(int num_seqs, int max_query_len, int max_blocks_per_seq, int block_size,
                                int n_q_heads, int n_kv_heads, int d_head, int scaled) {
    if (num_seqs <= 0 || max_query_len <= 0 || max_blocks_per_seq <= 0 || block_size <= 0 || n_kv_heads <= 0 ||
        n_q_heads < n_kv_heads || d_head <= 0)
        return 0;
    // one size for whichever kernel a call of this shape takes
    const long long rows = (long long)max_query_len * (n_q_heads / n_kv_heads);
    size_t most = 0;
    for (const Route route : {kUnits16, kWide}) {
        if (route == kWide && rows <= kRows) break;
        const size_t n = workspace_size(max_grid(route == kWide), unit_of(route, rows, scaled != 0), d_head);
        most = n > most ? n : most;
    }
    if (rows >= kPromptRows) {
        const size_t n = pa_attend_calls::prompt_workspace(num_seqs, max_query_len, max_blocks_per_seq, block_size, n_q_heads,
                                                           n_kv_heads, d_head, scaled != 0);
        most = n > most ? n : most;
    }
    return most;
}

int pa_attend(void* out, int out_dtype, const void* q, const void* k_cache, const void* v_cache,
              const int32_t* block_tables, const int32_t* query_start, const int32_t* context_lens,
              const int32_t* visible, const float* slopes, float softcap, int block_size, float scale, int n_q_heads,
              int n_kv_heads, int d_head, int num_seqs, int num_tokens, int max_query_len, int max_blocks_per_seq,
              int num_blocks, int max_context_len, void* workspace, size_t workspace_bytes, int32_t* status_dev,
              void* stream) {
    return attend(out, out_dtype, q, k_cache, v_cache, nullptr, nullptr, block_tables, query_start, context_lens, visible,
                  slopes, softcap, block_size, scale, n_q_heads, n_kv_heads, d_head, num_seqs, num_tokens, max_query_len,
                  max_blocks_per_seq, num_blocks, max_context_len, workspace, workspace_bytes, status_dev, stream, false);
}

int pa_attend_scaled(void* out, int out_dtype, const void* q, const void* k_cache, const void* v_cache,
                     const uint8_t* k_scales, const uint8_t* v_scales, const int32_t* block_tables,
                     const int32_t* query_start, const int32_t* context_lens, const int32_t* visible,
                     const float* slopes, float softcap, int block_size, float scale, int n_q_heads, int n_kv_heads,
                     int d_head, int num_seqs, int num_tokens, int max_query_len, int max_blocks_per_seq,
                     int num_blocks, int max_context_len, void* workspace, size_t workspace_bytes,
                     int32_t* status_dev, void* stream) {
    return attend(out, out_dtype, q, k_cache, v_cache, k_scales, v_scales, block_tables, query_start, context_lens, visible,
                  slopes, softcap, block_size, scale, n_q_heads, n_kv_heads, d_head, num_seqs, num_tokens, max_query_len,
                  max_blocks_per_seq, num_blocks, max_context_len, workspace, workspace_bytes, status_dev, stream, true);
}

}  // extern "C"
