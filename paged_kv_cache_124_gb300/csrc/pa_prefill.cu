// Paged prefill attention for sm_103a on the 5th-generation tensor cores.
//
// Operation ("PagedAttention in vLLM: scattered memory, exact attention",
// sections 4 and 8; "PagedAttention: Virtual Memory for the KV Cache",
// sections 7 and 13): a sequence with context length ctx whose last n
// positions are new (their keys and values already written to the paged
// cache) gets, for each new position p = ctx - n + i and each query head,
//     o = softmax(scale * q . K[0..p]) V[0..p]
// with K and V read through the block table (causal: a query sees only the
// positions up to its own).  The whole prompt (n = ctx), a later chunk of it
// (chunked prefill), or the suffix after a prefix-cache hit are all this
// same call.
//
// Design (a staging pass, then a persistent CTA per SM; a work item is two
// tiles of 128 query rows of one KV head):
//   * stage_v_kernel gathers V through the block table into the caller's
//     workspace, each (KV head, sequence) owning consecutive rows, so that a
//     128-position V tile is contiguous.  It stores a tile as fp16, which
//     holds every bf16 magnitude in [2^-14, 2^16) exactly and is off by at
//     most 2^-25 below that range, with the rows past the context zeroed; a
//     tile holding a magnitude of 2^16 or more (or a non-finite value)
//     stays bf16, and a format byte per tile says which.
//   * Rows are (token, grouped query head) pairs: 128 / G consecutive new
//     tokens times the G query heads that share KV head h, so every K/V tile
//     is read once for all G heads (GQA).  Each Q tile is one 3-D TMA box;
//     an item's two tiles (A, B) are consecutive token ranges and share every
//     K/V tile.
//   * Items are claimed from a counter shared by all CTAs, by group of KV
//     heads and heaviest first within a group (the group's K/V stays in L2);
//     the claiming warp decodes each item once and posts it to a ring in
//     shared memory for the other warps.  Barrier phases run on across
//     items, so the next item's loads and first products overlap the
//     current item's last products and output.
//   * K tiles of 128 positions are gathered through the block table with
//     one 2-D TMA box (64 columns x B rows, 128-byte swizzle) per block and
//     64-column half; a warp issues its boxes one lane after another, so K
//     and V have a producer warp each, and table entries are fetched four
//     tiles ahead.  Blocks past the needed range, and bad table entries, are
//     loaded from outside the tensor, which fills zeros and reads no HBM.  A
//     staged V tile is one box of 128 rows per 64 columns.
//   * S = Q K^T (M 128, N 128, K d) and O += P V (M 128, N d, K 128) are
//     tcgen05.mma kind::f16 (fp32 accumulate), one issuing thread per Q
//     tile (two issuers hide most of the pipe drain between groups of
//     products of different kinds).  Tensor memory holds S_A, S_B (128
//     columns each) and O_A, O_B (d columns each).  S takes bf16 Q and K.
//     P V takes fp16 weights (written over the first 64 columns of their
//     own S and read from there as the A operand) and the staged fp16
//     values: fp16 carries each weight to a relative 2^-11 where bf16 would
//     give 2^-8.  For a V tile that stayed bf16 each weight is split into
//     two bf16 terms, hi = bf16(p) and lo = bf16(p - hi), written over the
//     first and the second 64 columns of S (O += P_hi V + P_lo V, a relative
//     2^-16).  An item learns once whether any of its V tiles stayed bf16,
//     and the softmax and MMA warps run one of two compiled forms of their
//     tile loop (the fp16-only form checks no formats).  V is an MN-major
//     operand read straight from the TMA layout.
//   * Eight softmax warps work on tile A, then on tile B, then on tile A of
//     the next K/V tile, ...: warps w and w + 4 share the 32 rows of lane
//     quarter w (tensor-memory lane = row), each taking 64 of the 128
//     columns; the two halves of a row exchange their maxima (and, at the
//     end, their sums) through shared memory.  Per row: mask, online maximum
//     in the log2 domain, exp2, running sum, P; the scale-and-subtract and
//     the running sums use packed f32x2 arithmetic (one instruction for two
//     columns), which the softmax's instruction issue is bound by.  O is
//     rescaled in tensor memory only when a row's maximum grows by more than
//     2^8 (the weights, which carry a factor 2^7, stay below 2^15 otherwise),
//     which is rare after the first tiles.  At the end of an item each
//     thread writes its half row with 32-byte stores.
//   * Every wait is bounded; on a timeout the CTA flags PA_DEV_WAIT_TIMEOUT,
//     waits (bounded) for its own copies and products in flight, frees its
//     tensor memory and returns.

#include "pa_prefill.cuh"

namespace {

template <int D, bool kF8>
int launch(const PrefillArgs& a, const StageArgs& sa, const void* q, const void* k_cache, const void* v_cache,
           uint16_t* k_stage, int num_tokens, long long cache_rows, dim3 grid, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    if (!make_maps<D>(mq, mk, mv, a, sa, q, k_cache, kF8 ? k_stage : nullptr, num_tokens, cache_rows)) return PA_ERR_CUDA;
    if (pa_host::ensure_smem_attr(prefill_kernel<D, kF8, PrefillArgs>, PGeo<D>::kSmem, g_smem_done<D, kF8, PrefillArgs>) != cudaSuccess)
        return PA_ERR_CUDA;
    const dim3 sgrid((unsigned)sa.t_slot, (unsigned)sa.num_seqs, (unsigned)sa.n_kv_heads);
    if constexpr (kF8) {
        if (pa_host::launch_dependent(stage_kv_f8_kernel<D>, sgrid, dim3(256), 0, st,
                                      static_cast<const uint4*>(k_cache), static_cast<const uint4*>(v_cache), k_stage,
                                      sa) != cudaSuccess)
            return PA_ERR_CUDA;
    } else {
        if (pa_host::launch_dependent(stage_v_kernel<D>, sgrid, dim3(256), 0, st, static_cast<const uint4*>(v_cache),
                                      sa) != cudaSuccess)
            return PA_ERR_CUDA;
    }
    return pa_host::launch_dependent(prefill_kernel<D, kF8, PrefillArgs>, grid, dim3(kThreads), PGeo<D>::kSmem, st, mq, mk, mv,
                                     a) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

int prefill_impl(void* out, int out_dtype, const void* q, const void* k_cache, const void* v_cache,
                 const int32_t* block_tables, int max_blocks_per_seq, const int32_t* query_start,
                 const int32_t* context_lens, int num_seqs, int num_tokens, int max_query_len, int num_blocks,
                 int block_size, float scale, int n_q_heads, int n_kv_heads, int d_head, void* workspace,
                 size_t workspace_bytes, int32_t* sched_dev, int32_t* status_dev, void* stream, bool f8,
                 float k_scale, float v_scale) {
    if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || num_blocks <= 0 || max_blocks_per_seq < 0 ||
        n_q_heads <= 0 || n_kv_heads <= 0)
        return PA_ERR_INVALID_ARG;
    if (n_q_heads % n_kv_heads != 0) return PA_ERR_UNSUPPORTED;         // as pa_decode
    if (out_dtype != PA_DTYPE_BF16 && out_dtype != PA_DTYPE_F32) return PA_ERR_INVALID_ARG;
    if (f8 && (!(k_scale > 0.f) || !(v_scale > 0.f) || !(k_scale < INFINITY) || !(v_scale < INFINITY)))
        return PA_ERR_INVALID_ARG;
    if (!pa_host::supported_block_size(block_size) || !pa_host::supported_d_head(d_head)) return PA_ERR_UNSUPPORTED;
    if (f8 && d_head != 128) return PA_ERR_UNSUPPORTED;
    const int group = n_q_heads / n_kv_heads;
    if (group > kRows || kRows % group != 0) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !query_start || !context_lens)
        return PA_ERR_INVALID_ARG;
    if (max_blocks_per_seq == 0) return PA_ERR_INVALID_ARG;
    if (num_seqs > 65535) return PA_ERR_UNSUPPORTED;
    const Workspace ws = workspace_layout(num_seqs, max_blocks_per_seq, block_size, n_kv_heads, d_head, f8);
    if ((long long)n_kv_heads * num_seqs * ws.l_slot > INT_MAX - kKv) return PA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < ws.total) return PA_ERR_WORKSPACE;
    if (!pa_host::aligned16(out) || !pa_host::aligned16(q) || !pa_host::aligned16(k_cache) ||
        !pa_host::aligned16(v_cache) || !pa_host::aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
        (reinterpret_cast<uintptr_t>(query_start) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(sched_dev) & 3u))
        return PA_ERR_MISALIGNED;
    const long long cache_rows = (long long)num_blocks * n_kv_heads * block_size;
    if (cache_rows > INT_MAX - 64 || (long long)max_blocks_per_seq * block_size > INT_MAX / 2 ||
        n_kv_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    const int tq = kRows / group;
    const long long tiles = (max_query_len + 2 * tq - 1) / (2 * tq);
    if (tiles * num_seqs > INT_MAX) return PA_ERR_UNSUPPORTED;

    uint8_t* w8 = static_cast<uint8_t*>(workspace);
    PrefillArgs a;
    a.out = out;
    a.out_f32 = out_dtype == PA_DTYPE_F32;
    a.out_al32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    a.block_tables = block_tables;
    a.max_blocks = max_blocks_per_seq;
    a.query_start = query_start;
    a.context_lens = context_lens;
    a.num_seqs = num_seqs;
    a.num_tokens = num_tokens;
    a.tiles_per_seq = (int)tiles;
    a.block_size = block_size;
    a.n_kv_heads = n_kv_heads;
    a.group = group;
    a.tq = tq;
    a.n_q_heads = n_q_heads;
    a.num_blocks = num_blocks;
    a.oob_row = (int)cache_rows;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.v_fmt = w8 + ws.fmt_off;
    a.l_slot = ws.l_slot;
    a.t_slot = ws.t_slot;
    a.k_scale = f8 ? k_scale : 1.f;
    a.v_scale = f8 ? v_scale : 1.f;
    a.status = status_dev;
    a.sched = reinterpret_cast<int*>(sched_dev);
    const long long items = tiles * num_seqs * n_kv_heads;
    if (items > INT_MAX - 4096) return PA_ERR_UNSUPPORTED;    // claims run past the last item by one per CTA
    const int sms = num_sms();
    const dim3 grid((unsigned)(items < sms ? items : sms));
    const long long per_head = tiles * num_seqs;
    long long hpg = (2LL * grid.x + per_head - 1) / per_head;
    a.heads_per_group = (int)(hpg < 1 ? 1 : hpg > n_kv_heads ? n_kv_heads : hpg);
    StageArgs sa;
    sa.block_tables = block_tables;
    sa.max_blocks = max_blocks_per_seq;
    sa.context_lens = context_lens;
    sa.num_seqs = num_seqs;
    sa.block_size = block_size;
    sa.n_kv_heads = n_kv_heads;
    sa.num_blocks = num_blocks;
    sa.l_slot = ws.l_slot;
    sa.t_slot = ws.t_slot;
    sa.v_stage = reinterpret_cast<uint16_t*>(w8);
    sa.v_fmt = w8 + ws.fmt_off;
    sa.status = status_dev;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (f8)
        return launch<128, true>(a, sa, q, k_cache, v_cache, reinterpret_cast<uint16_t*>(w8 + ws.k_off), num_tokens,
                                 cache_rows, grid, st);
    return d_head == 128 ? launch<128, false>(a, sa, q, k_cache, v_cache, nullptr, num_tokens, cache_rows, grid, st)
                         : launch<64, false>(a, sa, q, k_cache, v_cache, nullptr, num_tokens, cache_rows, grid, st);
}

}  // namespace

extern "C" {

size_t pa_prefill_workspace_size(int num_seqs, int max_blocks_per_seq, int block_size, int n_kv_heads,
                                 int d_head) {
    if (num_seqs <= 0 || max_blocks_per_seq <= 0 || block_size <= 0 || n_kv_heads <= 0 || d_head <= 0) return 0;
    return workspace_layout(num_seqs, max_blocks_per_seq, block_size, n_kv_heads, d_head).total;
}

size_t pa_prefill_fp8_workspace_size(int num_seqs, int max_blocks_per_seq, int block_size, int n_kv_heads,
                                     int d_head) {
    if (num_seqs <= 0 || max_blocks_per_seq <= 0 || block_size <= 0 || n_kv_heads <= 0 || d_head <= 0) return 0;
    return workspace_layout(num_seqs, max_blocks_per_seq, block_size, n_kv_heads, d_head, true).total;
}

int pa_prefill(void* out, int out_dtype, const void* q, const void* k_cache, const void* v_cache,
               const int32_t* block_tables, int max_blocks_per_seq, const int32_t* query_start,
               const int32_t* context_lens, int num_seqs, int num_tokens, int max_query_len, int num_blocks,
               int block_size, float scale, int n_q_heads, int n_kv_heads, int d_head, void* workspace,
               size_t workspace_bytes, int32_t* sched_dev, int32_t* status_dev, void* stream) {
    return prefill_impl(out, out_dtype, q, k_cache, v_cache, block_tables, max_blocks_per_seq, query_start,
                        context_lens, num_seqs, num_tokens, max_query_len, num_blocks, block_size, scale, n_q_heads,
                        n_kv_heads, d_head, workspace, workspace_bytes, sched_dev, status_dev, stream, false, 1.f, 1.f);
}

int pa_prefill_fp8(void* out, int out_dtype, const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, int max_blocks_per_seq, const int32_t* query_start,
                   const int32_t* context_lens, int num_seqs, int num_tokens, int max_query_len, int num_blocks,
                   int block_size, float scale, float k_scale, float v_scale, int n_q_heads, int n_kv_heads,
                   int d_head, void* workspace, size_t workspace_bytes, int32_t* sched_dev, int32_t* status_dev,
                   void* stream) {
    return prefill_impl(out, out_dtype, q, k_cache, v_cache, block_tables, max_blocks_per_seq, query_start,
                        context_lens, num_seqs, num_tokens, max_query_len, num_blocks, block_size, scale, n_q_heads,
                        n_kv_heads, d_head, workspace, workspace_bytes, sched_dev, status_dev, stream, true, k_scale,
                        v_scale);
}

}  // extern "C"
