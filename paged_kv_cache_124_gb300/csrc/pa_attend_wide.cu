// Units of 64 and 128 rows of pa_attend and pa_attend_scaled: the kernel of
// pa_wide.cuh with shaped scores.
//
// The scores pass a softmax thread's registers 32 or 64 at a time, where they
// are capped, biased and masked before the maximum.  Block-scaled caches: a
// tile's 64 positions of a group have 2 to 8 blocks, whose scales its warps
// fetch themselves, a tile ahead (their table entries two), a lane each; K's
// multiply the scores, V's the weights, relative to the largest that the row
// has seen so far.
//
// 8 sequences of 32,000 positions and more, 8 new tokens of 32 query heads
// over 8 (32 rows), block-scaled: 123 us, 0.64 of the measured copy rate for
// 532 MB (issue 52 %, ALU 41 %: a tile's chain of scores, softmax
// and the four terms of a weight bounds it, as with one scale); capped 158 us,
// and 183 where scores go beyond half of the cap.  bf16, 8 of 8,192 positions,
// 64 new tokens: 104 us for 268 MB (40 us): a unit has 128 of a KV head's 256
// rows, so the cache is read twice, and the softmax of 256 rows a position is
// what there is to do (capped 118).

#include "pa_wide.cuh"

namespace pa_multi {

cudaError_t launch_shaped_wide(int rows, int d_head, bool f8, const void* q, int block_size, const CUtensorMap& mk,
                               const CUtensorMap& mv, const CurvedArgs& a, int grid, cudaStream_t st) {
    return a.cap_inv != 0.f || a.slopes ? launch_units(rows, d_head, f8, q, block_size, mk, mv, a, grid, st)
                                        : launch_units(rows, d_head, f8, q, block_size, mk, mv, static_cast<const ShapedArgs&>(a), grid, st);
}

}  // namespace pa_multi
