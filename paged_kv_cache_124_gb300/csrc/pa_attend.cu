// Attention of new tokens over the paged cache with shaped scores, from one
// token a sequence to whole prompts: scores capped by a tanh, less a bias by
// distance, over an interval of positions per token, and over bf16 caches or
// E4M3 codes with a power-of-two scale per block and head (pa_attend,
// pa_attend_scaled; the formulas stand in pa.h).
//
// Up to 16 rows a KV head (new tokens times query heads of the group) take
// the units of pa_multi_rows.cuh.  What the shape costs them is arithmetic on
// 16 scores a tile and lane beside the cache's bytes.  A sequence's work
// begins at the first position that some token of it sees and ends behind
// the last, so a window costs its own bytes.

#include "pa_attend.cuh"
#include "pa_multi_rows.cuh"

namespace {

// Which kernel takes a call.  Up to 16 rows a KV head: units of 16.  More:
// with a scale above 0, units of 64 or 128 rows (wide), or, for long chunks and
// prompts, the prefill kernel.  (Scales of 0 or below: units of 16 rows.)
enum Route { kUnits16, kWide, kPrompt };
Route route_of(long long rows, float scale) { return rows <= kRows || !(scale > 0.f) ? kUnits16 : rows <= 256 ? kWide : kPrompt; }

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
    Route route = route_of(all_rows, scale);
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
    a.cap_inv = softcap > 0.f ? 1.f / a.cap_log2 : 0.f;
    const int box = wide || block_size < kTile ? block_size : kTile;
    CUtensorMap mk, mv;
    if (!pa_host::cache_view(&mk, k_cache, cache_rows, d_head, f8 ? 1 : 2, box) ||
        !pa_host::cache_view(&mv, v_cache, cache_rows, d_head, f8 ? 1 : 2, box))
        return PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const ShapedArgs& shaped = a;
    int rc;
    if (wide)
        rc = launch_shaped_wide(unit, d_head, f8, q, block_size, mk, mv, a, split.grid, st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    else
        rc = f8 ? launch_multi<128, true>(split.warps, mk, mv, shaped, split.grid, st)
             : d_head == 128 ? launch_multi<128, false>(split.warps, mk, mv, shaped, split.grid, st)
                             : launch_multi<64, false>(split.warps, mk, mv, shaped, split.grid, st);
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
    if (route_of(rows, 1.f) == kPrompt) {
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
