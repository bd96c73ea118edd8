// Per-head RMS norm of queries and keys, rotation by position, and the cache
// write, in one pass over a step's projections.
//
//   y = x * rsqrt(mean(x^2) + eps) * gain                  (q and k; optional)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t)       the first rot_dim
// elements of a head in pairs: (i, i + rot_dim / 2), or (2 i, 2 i + 1) when
// interleaved; t from a table of cosines and sines by position.  q goes to
// q_out, k and v to their slots in the paged cache ("PagedAttention: Virtual
// Memory for the KV Cache", section 7: slot = block * B + offset), as bf16 or
// as E4M3 codes of the value over the cache's scale.
//
// Everything between the bf16 inputs and the one rounding at the end is
// 32-bit.  The pass is bound by memory: each input is read once and each
// output written once.  A thread holds 16 elements of a head (two 16-byte
// chunks, chosen so that both halves of every pair are its own), so a head
// of 128 is 8 threads and the norm's sum is three shuffles; arithmetic is in
// packed pairs.  With many tokens the same threads take two heads of a token
// at a time, one pair of heads after another, so that angles and gains are
// loaded once for all of them: 32,048 tokens of 32 + 2 x 8 heads in 123 us,
// 0.95 of the measured copy rate for their 790 MB; into E4M3 caches, with an
// IEEE division for each of their elements, in 145 us, 0.74 for 724 MB.  With
// few, every head has threads of its own: 4 tokens in 2.0 us, 250 of 256 (E4M3)
// in 3.5 us.
//
// By several axes (pa_qk_norm_mrope_cache): each pair's angle is that of the
// position on its axis, so a thread's angles come from up to three rows of the
// table for a token instead of one, chosen by constants of the call.  5,003
// tokens of 32 + 2 x 4 heads of 128 take 21.6 us, 0.72 of the measured copy
// rate for 105 MB; 6 tokens 2.1 us.  32 + 2 x 8 heads, with norm, bf16 / E4M3:
// 6 tokens 2.2 / 2.6 us, 250 3.5 / 3.9, 2,003 9.2 / 11.4, 5,003 26.2 / 31.5,
// 32,048 122.7 / 144.6.

#include <algorithm>

#include "pa_rope.cuh"

namespace {

// A head's place in the caches.
template <int D>
__device__ __forceinline__ size_t cache_elem(const RopeArgs& a, long long slot, int h) {
    const long long blk = slot / a.block_size;
    return (((size_t)blk * a.n_kv_heads + h) * a.block_size + (size_t)(slot - blk * a.block_size)) * D;
}

template <bool F8>
__device__ __forceinline__ void put_part(uint8_t* cache, size_t elem, const Part& p, float scale, int c0, int c1) {
    if constexpr (F8) {
        uint2* dst = reinterpret_cast<uint2*>(cache + elem);
        dst[c0] = codes8(p.f, scale);
        dst[c1] = codes8(p.f + 4, scale);
    } else {
        uint4* dst = reinterpret_cast<uint4*>(cache + 2 * elem);
        dst[c0] = pack8(p.f);
        dst[c1] = pack8(p.f + 4);
    }
}

// Few heads in all: D / 16 threads per head and nothing shared, so that all
// loads are in flight from the start.
template <int D, bool F8, bool kInterleaved, bool kAxes>
__global__ void __launch_bounds__(kRopeThreads, 4) heads_kernel(const RopeArgs a) {
    constexpr int kLanes = D / 16;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t heads = a.n_q_heads + 2 * a.n_kv_heads;
    const uint32_t nth = blockIdx.x * (kRopeThreads / kLanes) + threadIdx.x / kLanes;
    const uint32_t t = nth / heads;
    if (t >= (uint32_t)a.num_tokens) return;           // whole heads: a head's threads leave together
    const int row = nth - t * heads, l = threadIdx.x % kLanes;
    const unsigned mask = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
    const bool is_q = row < a.n_q_heads, is_v = row >= a.n_q_heads + a.n_kv_heads;
    const int h = is_q ? row : row - a.n_q_heads - (is_v ? a.n_kv_heads : 0);
    const Place<kInterleaved> w(l, a.rot_dim);
    const uint4* src = reinterpret_cast<const uint4*>(
        (is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + h * D);
    Where<kAxes> at;
    at.load(a, t);
    const long long slot = is_q ? 0 : a.slots[t];
    const uint4 x0 = src[w.c0], x1 = src[w.c1];
    const float* gains = is_v ? nullptr : is_q ? a.q_weight : a.k_weight;
    uint64_t gain[8];
    if (gains) {
        load8(gains + 8 * w.c0, gain);
        load8(gains + 8 * w.c1, gain + 4);
    }
    if (at.lowest() < 0) return;                               // padding: nothing of the token is touched
    if (at.highest() >= a.max_positions) {
        if (l == 0 && row == 0) pa::set_status(a.status, PA_DEV_BAD_POSITION);
        return;
    }
    if (slot < 0) return;                              // a key and value that stay out of the cache
    if (slot >= a.num_slots) {
        if (l == 0) pa::set_status(a.status, PA_DEV_BAD_SLOT);
        return;
    }
    Part p;
    unpack8(x0, p.f);
    unpack8(x1, p.f + 4);
    if (!is_v) {
        uint64_t cs[4], sn[4];
        if (w.turns) load_angles<kAxes>(a, at, l, cs, sn);
        if (gains) norm_part<kLanes>(p, gain, a.eps, mask);
        if (w.turns) turn_part<kInterleaved>(p, cs, sn);
    }
    if (is_q) {
        uint4* dst = a.q_out + ((size_t)t * a.n_q_heads + h) * (D / 8);
        dst[w.c0] = pack8(p.f);
        dst[w.c1] = pack8(p.f + 4);
    } else {
        put_part<F8>(is_v ? a.v_cache : a.k_cache, cache_elem<D>(a, slot, h), p, is_v ? a.v_scale : a.k_scale, w.c0, w.c1);
    }
}

// Many: kSide heads of a token side by side (32 / (kSide D / 16) tokens per
// warp), turn after turn, kFlight turns in flight, so that the angles and
// the gains are loaded once for all of a token's heads.
constexpr int kFlight = 4;

template <int D, bool F8, bool kInterleaved, bool kAxes, int kSide>
__global__ void __launch_bounds__(kRopeThreads, 2) tokens_kernel(const RopeArgs a) {
    constexpr int kLanes = D / 16, kGroup = kLanes * kSide;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t t = blockIdx.x * (kRopeThreads / kGroup) + threadIdx.x / kGroup;
    if (t >= (uint32_t)a.num_tokens) return;           // whole tokens: a token's threads leave together
    const int lane = threadIdx.x % kGroup, l = lane % kLanes, g = lane / kLanes;
    const unsigned mask = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
    const int q_turns = (a.n_q_heads + kSide - 1) / kSide, kv_turns = (a.n_kv_heads + kSide - 1) / kSide;
    const Place<kInterleaved> w(l, a.rot_dim);
    Where<kAxes> at;
    at.load(a, t);
    const long long slot = a.slots[t];
    struct Raw {
        uint4 x0[kFlight], x1[kFlight];
    };
    // heads (turn + u) * kSide + g of a tensor's row
    auto load = [&](const __nv_bfloat16* rows, int turn, int heads, Raw& r) {
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int h = (turn + u) * kSide + g;
            if (h < heads) {
                const uint4* src = reinterpret_cast<const uint4*>(rows + h * D);
                r.x0[u] = src[w.c0];
                r.x1[u] = src[w.c1];
            }
        }
    };
    const __nv_bfloat16* q = a.q + (long long)t * a.q_stride;
    const __nv_bfloat16* k = a.k + (long long)t * a.k_stride;
    const __nv_bfloat16* v = a.v + (long long)t * a.v_stride;
    Raw raw;
    load(q, 0, a.n_q_heads, raw);                      // these do not wait for the position
    if (at.lowest() < 0) return;                               // padding: nothing of the token is touched
    if (at.highest() >= a.max_positions) {
        if (lane == 0) pa::set_status(a.status, PA_DEV_BAD_POSITION);
        return;
    }
    uint64_t cs[4], sn[4], gain[8];
    if (w.turns) load_angles<kAxes>(a, at, l, cs, sn);
    const bool norm = a.q_weight != nullptr;
    auto load_gain = [&](const float* g_) {
        if (norm) {
            load8(g_ + 8 * w.c0, gain);
            load8(g_ + 8 * w.c1, gain + 4);
        }
    };
    auto work = [&](uint4 x0, uint4 x1) {              // a head's threads
        Part p;
        unpack8(x0, p.f);
        unpack8(x1, p.f + 4);
        if (norm) norm_part<kLanes>(p, gain, a.eps, mask);
        if (w.turns) turn_part<kInterleaved>(p, cs, sn);
        return p;
    };
    load_gain(a.q_weight);
    for (int turn = 0; turn < q_turns; turn += kFlight) {
        const Raw now = raw;
        load(q, turn + kFlight, a.n_q_heads, raw);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (turn + u >= q_turns) break;
            const int h = (turn + u) * kSide + g;
            const Part p = work(now.x0[u], now.x1[u]);
            if (h < a.n_q_heads) {
                uint4* dst = a.q_out + ((size_t)t * a.n_q_heads + h) * (D / 8);
                dst[w.c0] = pack8(p.f);
                dst[w.c1] = pack8(p.f + 4);
            }
        }
    }
    if (slot < 0) return;                              // a key and value that stay out of the cache
    if (slot >= a.num_slots) {
        if (lane == 0) pa::set_status(a.status, PA_DEV_BAD_SLOT);
        return;
    }
    const size_t row0 = cache_elem<D>(a, slot, 0), head = (size_t)a.block_size * D;
    Raw vraw;
    load(k, 0, a.n_kv_heads, raw);
    load_gain(a.k_weight);
    load(v, 0, a.n_kv_heads, vraw);
    for (int turn = 0; turn < kv_turns; turn += kFlight) {
        if (turn) load(k, turn, a.n_kv_heads, raw);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (turn + u >= kv_turns) break;
            const int h = (turn + u) * kSide + g;
            const Part p = work(raw.x0[u], raw.x1[u]);
            if (h < a.n_kv_heads) put_part<F8>(a.k_cache, row0 + h * head, p, a.k_scale, w.c0, w.c1);
        }
    }
    for (int turn = 0; turn < kv_turns; turn += kFlight) {
        if (turn) load(v, turn, a.n_kv_heads, vraw);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int h = (turn + u) * kSide + g;
            if (h >= a.n_kv_heads) break;
            if constexpr (F8) {
                Part p;
                unpack8(vraw.x0[u], p.f);
                unpack8(vraw.x1[u], p.f + 4);
                put_part<true>(a.v_cache, row0 + h * head, p, a.v_scale, w.c0, w.c1);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(a.v_cache + 2 * (row0 + h * head));
                dst[w.c0] = vraw.x0[u];
                dst[w.c1] = vraw.x1[u];
            }
        }
    }
}

template <int D, bool F8, bool kInterleaved, bool kAxes, int kSide>
cudaError_t launch_tokens(const RopeArgs& a, cudaStream_t st) {
    const int per = kRopeThreads / (D / 16 * kSide);
    return pa_host::launch_dependent(tokens_kernel<D, F8, kInterleaved, kAxes, kSide>,
                                     dim3((unsigned)(((long long)a.num_tokens + per - 1) / per)), dim3(kRopeThreads), 0, st, a);
}

// Which kernel: the one per token is faster from about 12 million elements
// on (32 + 2 x 8 heads of 128: 1000 tokens 10.0 against 6.5 us, 2000 13.1 /
// 13.6, 4000 18.3 / 24.2, 32,048 122.9 / 168; E4M3 1000 13.9 / 7.0, 2000 16.8 /
// 14.6, 4000 21.8 / 25.7, 32,048 144 / 180; 16 + 2 x 2 of 64: 5000 tokens 7.6 /
// 5.7, 10,000 12.5 / 12.9, 40,000 36.2 / 42.5), if a token has heads enough to
// share its angles (2 + 2 x 1: 40,000 tokens 38.5 / 21.9).
//
// Several axes: the kernel per token with four heads side by side, in blocks
// of half the time, where its waves of resident blocks (two an SM) are at most
// 1.5 times those of two heads.  32 + 2 x 4 heads of 128, us by head / four /
// two: 500 tokens 4.0 / 4.2 / 6.0, 800 4.8 / 4.2 / 6.0, 2003 13.6 / 9.6 / 11.0,
// 4006 (one wave of two) 21.0 / 17.2 / 16.0, 5003 (three of four, two of two)
// 28.9 / 21.7 / 22.8, 8012 - / 31.5 / 29.2.
template <int D, bool F8, bool kInterleaved, bool kAxes>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
    constexpr int kLanes = D / 16;
    const int heads = a.n_q_heads + 2 * a.n_kv_heads;
    const long long rows = (long long)a.num_tokens * heads;
    if constexpr (kAxes) {
        const long long resident = 2LL * std::max(1, pa_host::sm_count()), four = kRopeThreads / (4 * kLanes), two = kRopeThreads / (2 * kLanes);
        const auto waves = [&](long long tokens) { return (a.num_tokens + tokens * resident - 1) / (tokens * resident); };
        if (heads >= 16 && rows * D >= 3000000 && 2 * waves(four) <= 3 * waves(two))
            return launch_tokens<D, F8, kInterleaved, kAxes, 4>(a, st);
    }
    if (heads >= 16 && rows * D >= 12000000) return launch_tokens<D, F8, kInterleaved, kAxes, 2>(a, st);
    const int per = kRopeThreads / kLanes;
    return pa_host::launch_dependent(heads_kernel<D, F8, kInterleaved, kAxes>, dim3((unsigned)((rows + per - 1) / per)),
                                     dim3(kRopeThreads), 0, st, a);
}

template <int D, bool F8>
cudaError_t launch_rope(const RopeArgs& a, int interleaved, cudaStream_t st) {
    if (a.num_axes)
        return interleaved ? launch_rope<D, F8, true, true>(a, st) : launch_rope<D, F8, false, true>(a, st);
    return interleaved ? launch_rope<D, F8, true, false>(a, st) : launch_rope<D, F8, false, false>(a, st);
}

int norm_rope_cache(void* q_out, void* k_cache, void* v_cache, const void* q, const void* k, const void* v,
                    int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_weight,
                    const float* k_weight, float eps, const float* cos_sin, int max_positions, int rot_dim,
                    int interleaved, const int32_t* positions, const int64_t* slot_mapping, int num_tokens,
                    int n_q_heads, int n_kv_heads, int d_head, int block_size, int num_blocks, int32_t* status_dev,
                    void* stream, bool f8, float k_scale, float v_scale, int num_axes = 0,
                    const int8_t* axis_of_pair = nullptr) {
    if (num_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || num_blocks <= 0 || max_positions <= 0 ||
        !(eps >= 0.f) || !(eps < __builtin_inff()))
        return PA_ERR_INVALID_ARG;
    if (f8 && (!(k_scale > 0.f) || !(v_scale > 0.f) || !(k_scale < __builtin_inff()) || !(v_scale < __builtin_inff())))
        return PA_ERR_INVALID_ARG;
    if (!pa_host::supported_block_size(block_size) || !pa_host::supported_d_head(d_head) || rot_dim < 16 ||
        rot_dim > d_head || rot_dim % 16)
        return PA_ERR_UNSUPPORTED;
    if (((long long)n_q_heads + 2LL * n_kv_heads) * num_tokens > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    if (num_axes < 0 || (num_axes && !axis_of_pair)) return PA_ERR_INVALID_ARG;
    if (num_axes > 4) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!q_out || !k_cache || !v_cache || !q || !k || !v || !cos_sin || !positions || !slot_mapping)
        return PA_ERR_INVALID_ARG;
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
    if (q_out == q && num_tokens > 1 && q_stride != (int64_t)n_q_heads * d_head) return PA_ERR_INVALID_ARG;
    RopeArgs a{};
    if (num_axes && !set_axes(a, num_axes, axis_of_pair, rot_dim)) return PA_ERR_INVALID_ARG;
    a.q_out = static_cast<uint4*>(q_out);
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
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
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.max_positions = max_positions;
    a.rot_dim = rot_dim;
    a.num_tokens = num_tokens;
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = n_kv_heads;
    a.block_size = block_size;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d_head == 128 ? (f8 ? launch_rope<128, true>(a, interleaved, st) : launch_rope<128, false>(a, interleaved, st))
                                        : (f8 ? launch_rope<64, true>(a, interleaved, st) : launch_rope<64, false>(a, interleaved, st));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

int pa_qk_norm_rope_cache(void* q_out, void* k_cache, void* v_cache, const void* q, const void* k, const void* v,
                          int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_weight,
                          const float* k_weight, float eps, const float* cos_sin, int max_positions, int rot_dim,
                          int interleaved, const int32_t* positions, const int64_t* slot_mapping, int num_tokens,
                          int n_q_heads, int n_kv_heads, int d_head, int block_size, int num_blocks,
                          int32_t* status_dev, void* stream) {
    return norm_rope_cache(q_out, k_cache, v_cache, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps,
                           cos_sin, max_positions, rot_dim, interleaved, positions, slot_mapping, num_tokens,
                           n_q_heads, n_kv_heads, d_head, block_size, num_blocks, status_dev, stream, false, 1.f, 1.f);
}

int pa_qk_norm_rope_cache_fp8(void* q_out, void* k_cache, void* v_cache, const void* q, const void* k, const void* v,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_weight,
                              const float* k_weight, float eps, const float* cos_sin, int max_positions, int rot_dim,
                              int interleaved, const int32_t* positions, const int64_t* slot_mapping, int num_tokens,
                              int n_q_heads, int n_kv_heads, int d_head, int block_size, int num_blocks,
                              float k_scale, float v_scale, int32_t* status_dev, void* stream) {
    return norm_rope_cache(q_out, k_cache, v_cache, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps,
                           cos_sin, max_positions, rot_dim, interleaved, positions, slot_mapping, num_tokens,
                           n_q_heads, n_kv_heads, d_head, block_size, num_blocks, status_dev, stream, true, k_scale,
                           v_scale);
}

int pa_qk_norm_mrope_cache(void* q_out, void* k_cache, void* v_cache, const void* q, const void* k, const void* v,
                           int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_weight,
                           const float* k_weight, float eps, const float* cos_sin, int max_positions, int rot_dim,
                           int interleaved, const int32_t* positions, int num_axes, const int8_t* axis_of_pair,
                           const int64_t* slot_mapping, int num_tokens, int n_q_heads, int n_kv_heads, int d_head,
                           int block_size, int num_blocks, int32_t* status_dev, void* stream) {
    if (num_axes < 1) return PA_ERR_INVALID_ARG;
    return norm_rope_cache(q_out, k_cache, v_cache, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps,
                           cos_sin, max_positions, rot_dim, interleaved, positions, slot_mapping, num_tokens,
                           n_q_heads, n_kv_heads, d_head, block_size, num_blocks, status_dev, stream, false, 1.f, 1.f,
                           num_axes, axis_of_pair);
}

int pa_qk_norm_mrope_cache_fp8(void* q_out, void* k_cache, void* v_cache, const void* q, const void* k, const void* v,
                               int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_weight,
                               const float* k_weight, float eps, const float* cos_sin, int max_positions, int rot_dim,
                               int interleaved, const int32_t* positions, int num_axes, const int8_t* axis_of_pair,
                               const int64_t* slot_mapping, int num_tokens, int n_q_heads, int n_kv_heads, int d_head,
                               int block_size, int num_blocks, float k_scale, float v_scale, int32_t* status_dev,
                               void* stream) {
    if (num_axes < 1) return PA_ERR_INVALID_ARG;
    return norm_rope_cache(q_out, k_cache, v_cache, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps,
                           cos_sin, max_positions, rot_dim, interleaved, positions, slot_mapping, num_tokens,
                           n_q_heads, n_kv_heads, d_head, block_size, num_blocks, status_dev, stream, true, k_scale,
                           v_scale, num_axes, axis_of_pair);
}

}  // extern "C"
