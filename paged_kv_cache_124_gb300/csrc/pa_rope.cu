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
// of 128 is 8 threads and the norm's sum is three shuffles.

#include "pa_common.cuh"

namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    uint4* q_out;
    uint8_t* k_cache;
    uint8_t* v_cache;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    long long q_stride, k_stride, v_stride;            // elements between tokens
    const float* q_weight;
    const float* k_weight;
    const float* cos_sin;                              // [max_positions][rot_dim]: cosines, then sines
    const int32_t* positions;
    const int64_t* slots;
    int32_t* status;
    long long num_slots;
    float eps, k_scale, v_scale;
    int max_positions, rot_dim, num_tokens, n_q_heads, n_kv_heads, block_size;
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void unpack8(uint4 x, float* f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = pa::bf16x2_to_float2(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint2 codes8(const float* f, float scale) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = pa::e4m3x2(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ void load8(const float* p, float* f) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <int D, bool F8, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_cache_kernel(const RopeArgs a) {
    constexpr int kLanes = D / 16;                     // threads per head
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int heads = a.n_q_heads + 2 * a.n_kv_heads;
    const uint32_t at = blockIdx.x * (kRopeThreads / kLanes) + threadIdx.x / kLanes;
    const int l = threadIdx.x % kLanes;
    const int t = at / heads;
    if (t >= a.num_tokens) return;                     // whole heads: a head's threads leave together
    const int row = at - t * heads;
    const unsigned mask = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
    const int pos = a.positions[t];
    if (pos < 0) return;                               // padding: nothing of the token is touched
    if (pos >= a.max_positions) {
        if (l == 0 && row == 0) pa::set_status(a.status, PA_DEV_BAD_POSITION);
        return;
    }
    const bool is_q = row < a.n_q_heads, is_v = row >= a.n_q_heads + a.n_kv_heads;
    const int h = is_q ? row : row - a.n_q_heads - (is_v ? a.n_kv_heads : 0);
    long long slot = 0;
    if (!is_q) {
        slot = a.slots[t];
        if (slot < 0) return;                          // a key and value that stay out of the cache
        if (slot >= a.num_slots) {
            if (l == 0) pa::set_status(a.status, PA_DEV_BAD_SLOT);
            return;
        }
    }
    // this thread's two chunks of 8: pairs (i, i + rot_dim / 2) take one from
    // each half of the rotated part, all else two neighbours
    const int turn_lanes = a.rot_dim >> 4;
    const bool turns = l < turn_lanes;
    const int c0 = !kInterleaved && turns ? l : 2 * l;
    const int c1 = !kInterleaved && turns ? l + turn_lanes : 2 * l + 1;
    const uint4* src = reinterpret_cast<const uint4*>(
        (is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + h * D);
    const uint4 x0 = src[c0], x1 = src[c1];
    float f[16];
    unpack8(x0, f);
    unpack8(x1, f + 8);
    if (!is_v) {
        const float* gain = is_q ? a.q_weight : a.k_weight;
        if (gain) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s += f[i] * f[i];
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(mask, s, o);
            const float inv = rsqrtf(s * (1.f / D) + a.eps);
            float g[16];
            load8(gain + 8 * c0, g);
            load8(gain + 8 * c1, g + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = f[i] * inv * g[i];
        }
        if (turns) {
            const float* cs = a.cos_sin + (size_t)pos * a.rot_dim + 8 * l;
            float c[8], s[8];
            load8(cs, c);
            load8(cs + (a.rot_dim >> 1), s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float& x = f[kInterleaved ? 2 * i : i];
                float& y = f[kInterleaved ? 2 * i + 1 : i + 8];
                const float xr = x * c[i] - y * s[i];
                y = y * c[i] + x * s[i];
                x = xr;
            }
        }
    }
    if (is_q) {
        uint4* dst = a.q_out + ((size_t)t * a.n_q_heads + h) * (D / 8);
        dst[c0] = pack8(f);
        dst[c1] = pack8(f + 8);
        return;
    }
    const long long blk = slot / a.block_size;
    const int off = (int)(slot - blk * a.block_size);
    const size_t elem = (((size_t)blk * a.n_kv_heads + h) * a.block_size + off) * D;
    uint8_t* cache = is_v ? a.v_cache : a.k_cache;
    if constexpr (F8) {
        const float scale = is_v ? a.v_scale : a.k_scale;
        uint2* dst = reinterpret_cast<uint2*>(cache + elem);
        dst[c0] = codes8(f, scale);
        dst[c1] = codes8(f + 8, scale);
    } else {
        uint4* dst = reinterpret_cast<uint4*>(cache + 2 * elem);
        dst[c0] = is_v ? x0 : pack8(f);
        dst[c1] = is_v ? x1 : pack8(f + 8);
    }
}

template <int D, bool F8>
cudaError_t launch_rope(const RopeArgs& a, int interleaved, cudaStream_t st) {
    const long long rows = (long long)a.num_tokens * (a.n_q_heads + 2 * a.n_kv_heads);
    const int per = kRopeThreads / (D / 16);
    return pa_host::launch_dependent(
        interleaved ? norm_rope_cache_kernel<D, F8, true> : norm_rope_cache_kernel<D, F8, false>,
        dim3((unsigned)((rows + per - 1) / per)), dim3(kRopeThreads), 0, st, a);
}

int norm_rope_cache(void* q_out, void* k_cache, void* v_cache, const void* q, const void* k, const void* v,
                    int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_weight,
                    const float* k_weight, float eps, const float* cos_sin, int max_positions, int rot_dim,
                    int interleaved, const int32_t* positions, const int64_t* slot_mapping, int num_tokens,
                    int n_q_heads, int n_kv_heads, int d_head, int block_size, int num_blocks, int32_t* status_dev,
                    void* stream, bool f8, float k_scale, float v_scale) {
    if (num_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || num_blocks <= 0 || max_positions <= 0 ||
        !(eps >= 0.f) || !(eps < __builtin_inff()))
        return PA_ERR_INVALID_ARG;
    if (f8 && (!(k_scale > 0.f) || !(v_scale > 0.f) || !(k_scale < __builtin_inff()) || !(v_scale < __builtin_inff())))
        return PA_ERR_INVALID_ARG;
    if (!pa_host::supported_block_size(block_size) || !pa_host::supported_d_head(d_head) || rot_dim < 16 ||
        rot_dim > d_head || rot_dim % 16)
        return PA_ERR_UNSUPPORTED;
    if (((long long)n_q_heads + 2LL * n_kv_heads) * num_tokens > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
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
    RopeArgs a{};
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

}  // extern "C"
