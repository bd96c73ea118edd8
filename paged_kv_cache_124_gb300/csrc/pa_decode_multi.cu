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
// The kernel of pa_multi_rows.cuh serves up to 16 rows a KV head (and any number
// with a scale that is not positive, or over a few contexts of one tile);
// pa_decode_wide.cu takes more.
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

#include "pa_multi_rows.cuh"

namespace {

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

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
    const Split split = split_work(f8, wide, all_rows, num_seqs, n_kv_heads, ctx_cap);
    a.direct = split.direct;

    a.out = out;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.query_start = query_start;
    a.context_lens = context_lens;
    a.tree_mask = reinterpret_cast<const uint64_t*>(tree_mask);
    set_workspace(a, workspace, split.grid, unit);
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
        rc = launch_wide(unit, d_head, f8, q, block_size, mk, mv, a, split.grid, st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    else
        rc = f8 ? launch_multi<128, true>(split.warps, mk, mv, a, split.grid, st)
             : d_head == 128 ? launch_multi<128, false>(split.warps, mk, mv, a, split.grid, st)
                             : launch_multi<64, false>(split.warps, mk, mv, a, split.grid, st);
    if (rc != PA_OK || split.direct) return rc;                  // (no unit is shared: nothing to merge)
    return launch_merge(a, unit, d_head, split.units, split.grid, st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

namespace pa_multi {

cudaError_t launch_merge(const MultiArgs& a, int unit, int d_head, double units, int grid, cudaStream_t st) {
    // Few units come in many pieces: four threads then share four columns of a row, in more blocks; else one thread
    // takes all of its pieces.  (3 units of 66 pieces 22 us against 32; 512 units over 456 blocks 105 against 101.)
    const bool few = units * 4 <= grid;
    const int columns = unit * d_head / 4, items = few ? 64 : kMergeThreads;
    const int splits = few ? std::min(columns / items, 16) : std::min((columns + items - 1) / items, 4);
    const auto merge = few ? (d_head == 128 ? merge_kernel<128, 64> : merge_kernel<64, 64>)
                           : (d_head == 128 ? merge_kernel<128, kMergeThreads> : merge_kernel<64, kMergeThreads>);
    return pa_host::launch_dependent(merge, dim3(grid, splits), dim3(kMergeThreads), 0, st, a, unit);
}

}  // namespace pa_multi

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
