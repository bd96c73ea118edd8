// Units of 64 and 128 rows of pa_attend and pa_attend_scaled: the kernel of
// pa_wide.cuh with shaped scores.
//
// The scores pass a softmax thread's registers 32 or 64 at a time, where they
// are capped, biased and masked before the maximum.  Block-scaled caches: a
// tile's 64 positions of a group have 2 to 8 blocks, whose scales its warps
// fetch themselves, a tile ahead (their table entries two), a lane each; K's
// multiply the scores, V's the weights, relative to the largest so far.
//
// 8 sequences of 32,000 positions and more, 8 new tokens of 32 query heads
// over 8 (32 rows), block-scaled: 121 us, 0.65 of the measured copy rate for
// 532 MB (issue 51 %, ALU 42 %: a tile's chain of scores, softmax
// and the four terms of a weight bounds it, as with one scale).

#include "pa_wide.cuh"

namespace pa_multi {

cudaError_t launch_shaped_wide(int rows, int d_head, bool f8, const void* q, int block_size, const CUtensorMap& mk,
                               const CUtensorMap& mv, const CurvedArgs& a, int grid, cudaStream_t st) {
    return a.cap_inv != 0.f || a.slopes ? launch_units(rows, d_head, f8, q, block_size, mk, mv, a, grid, st)
                                        : launch_units(rows, d_head, f8, q, block_size, mk, mv, static_cast<const ShapedArgs&>(a), grid, st);
}

}  // namespace pa_multi
