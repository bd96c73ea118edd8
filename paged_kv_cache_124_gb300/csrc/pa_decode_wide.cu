// Attention of several new tokens per sequence for more rows (new tokens
// times query heads of the group) than warp-level products can keep up with
// the cache's bytes for: units of 64 or 128 rows on the 5th-generation tensor
// cores.  Same operation, units, shares and pieces as pa_decode_multi.cu.
//
// What bounds it: a tile of 128 positions of one KV head (64 KB of K and V at
// d_head 128) takes an SM about 1.46 us of its share of the memory's rate,
// and its products, S = Q . K^T and O += P . V at 128 rows, 0.33 us each: the
// bytes bound it as long as copies, products and softmax overlap.  64
// sequences of 4096 positions, 8 KV heads of 128: 32 rows 165 us (0.96 of the
// measured copy rate), 64 rows 170 (0.94), 128 rows 174 (0.94; 789 TFLOP/s).
// E4M3: 32 rows 101 us (0.80), 64 rows 107 (0.77); 128 rows, as two units that
// read the cache each, 196 (0.43).  No unit of the SM is full there (ALU 44 %,
// issue slots 51 %, tensor cores 39 %, DRAM 56 % on a ragged batch of 32 rows),
// and a tile costs nearly the same with 20, 32 or 64 of its rows there: what
// bounds it is a tile's chain of hand-overs, in which the softmax, with four
// terms of each weight, is longer than bf16's.  How much of that is work on
// rows that are not there, no counter tells.
//  * One block per SM walks its share.  A producer warp each fills stages of
//    K and V through the block table; one warp issues the score products of
//    whole tiles, into two buffers in turn; two groups of four warps take the
//    first and the second 64 positions of every tile, each with its own
//    running statistics and, by an issuing warp of its own, its own output
//    accumulator.  Scores and accumulators (S0, S1, O0, O1) fill the 512
//    columns of tensor memory; weights are written over their scores.  The
//    groups exchange nothing until a unit's end, where four more warps merge
//    the two accumulators exactly while the groups go on to the next unit.
//    (An issuing thread spends some 60 to 100 cycles on a product of 64 and a
//    hand-over between warps 100 to 450, so what bounds the rate of tiles is
//    the chain scores - softmax - values: two buffers and a chain of half a
//    tile keep it under the memory's 2800 cycles a tile.)
//  * Roles are many and their code together is larger than the instruction
//    cache, so what is not a tile's work is kept out of it or rolled up
//    (unroll 1): with one miss for five fetches instead of 25, 64 requests of
//    8 tokens over E4M3 took 100 us instead of 68.
//  * Every barrier is waited for in every phase, in order, by each of its
//    waiters, so no wait can take an older phase's parity for its own.  One
//    exception: the softmax groups wait for p_done only when they rescale;
//    why that wait can meet one phase alone stands there.
//  * bf16: V stays bf16, so the weights enter P . V as two bf16 terms (hi +
//    lo, a relative 2^-16).  Units of 64 rows lie in lanes 0-15 of each 32:
//    the hi terms there and the lo terms in the other 16 lanes, so a single
//    product does both and the output adds the two lanes; a row's scores are
//    read by two threads.  Units of 128 rows take two products.
//  * E4M3: the codes are operands as they lie in the cache.  q is the exact
//    sum of two E4M3 terms, in a row's two lanes, whose scores the softmax
//    adds; weights are four E5M2 terms in two products.
//  * A warp of its own zeroes V rows past the context (0 * NaN) in shared
//    memory, and new positions' values that are not finite, which the rows
//    that see them add at the unit's end.

#include "pa_wide.cuh"

namespace pa_multi {

cudaError_t launch_wide(int rows, int d_head, bool f8, const void* q, int block_size, const CUtensorMap& mk,
                        const CUtensorMap& mv, const MultiArgs& a, int grid, cudaStream_t st) {
    return launch_units(rows, d_head, f8, q, block_size, mk, mv, a, grid, st);
}

}  // namespace pa_multi
