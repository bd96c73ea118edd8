// A call of pa_attend or pa_attend_scaled, checked, as its kernels' launches take it.
#pragma once

#include "pa_common.cuh"

namespace pa_attend_calls {

struct Call {
    void* out;
    int out_f32;
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const uint8_t* k_scales;               // both null: bf16 caches
    const uint8_t* v_scales;
    const int32_t* block_tables;
    const int32_t* query_start;
    const int32_t* context_lens;
    const int32_t* visible;
    const float* slopes;
    float softcap, scale;
    int block_size, n_q_heads, n_kv_heads, d_head, num_seqs, num_tokens, max_query_len, max_blocks, num_blocks, ctx_cap;
    void* workspace;
    int32_t* status;
    cudaStream_t stream;
};

// Prompts and long chunks (pa_attend_prompt.cu): bytes of workspace, 0 where
// the sizes are beyond it; and the launches, with a scale above 0.
size_t prompt_workspace(int num_seqs, int max_query_len, int max_blocks, int block_size, int n_q_heads, int n_kv_heads,
                        int d_head, bool scaled);
int launch_prompt(const Call& c);

}  // namespace pa_attend_calls
