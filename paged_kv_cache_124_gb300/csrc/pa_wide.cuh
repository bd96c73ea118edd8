// The kernel of units of 64 or 128 rows (pa_decode_wide.cu says what it does
// and why), for plain scores and for shaped ones, and its launch.
#pragma once

#include "pa_multi.cuh"

namespace {

using namespace pa_multi;

constexpr int kKv = kWideStep;             // positions per tile
constexpr int kSoftmaxWarps = 8;
constexpr int kKWarp = 8;                  // walks the share, loads K
constexpr int kVWarp = 9;                  // loads q (free when its unit's last scores are done) and V
constexpr int kScoreWarp = 10;             // issues the score products and owns the tensor memory
constexpr int kOutWarp = 12;               // 12 .. 15 read the accumulators out at a unit's end
constexpr int kCheckWarp = 17;             // makes V's tiles fit for the products
constexpr int kThreads = 576;
// warps 11 and 16 issue the value products of groups 0 and 1
__device__ __forceinline__ int value_group(int warp) { return warp == 11 ? 0 : warp == 16 ? 1 : -1; }
constexpr float kQUp = 32.f;               // E4M3: factor on the second terms of q
constexpr int kHalfKv = kKv / 2;           // positions of a tile per group
constexpr int kUnits = 4;                  // units posted ahead
constexpr int kUnitReaders = 17;           // warps that read a posted unit
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;           // S0 at 0, S1 at 128, O0 and O1 from here

// kHalf: units of 64 rows, in lanes 0-15 of each 32 of a product, the other
// lanes taking a second term of their weights; else 128.  F8: E4M3 caches.
template <int D, bool kHalf, bool F8>
struct Wide {
    static_assert(!F8 || (kHalf && D == 128), "E4M3 caches: 64 rows, d_head 128");
    static constexpr int kRows = kHalf ? 64 : 128;
    static constexpr int kHalves = F8 ? 1 : D / 64;              // 128-byte columns of a cache row
    static constexpr int kHalfBytes = 128 * 128;                 // 128 rows of 128 bytes, 128-byte swizzle
    static constexpr int kTileBytes = kHalves * kHalfBytes;      // K or V of a tile
    static constexpr int kQBytes = kTileBytes;                   // F8: a row's two terms in its two lanes
    static constexpr int kQBuffers = F8 ? 2 : 1;
    static constexpr int kStages = F8 || D == 64 ? 6 : 3;
    static constexpr int kK0 = kQBuffers * kQBytes;
    static constexpr int kV0 = kK0 + kStages * kTileBytes;
    static constexpr int kStats = kV0 + kStages * kTileBytes;    // [group][row] maximum and sum; F8: then row factors and units
    static constexpr int kCtl = kStats + 2 * 128 * 8;
    static constexpr int kSmem = kCtl + 1024;
    static constexpr int kStepKeys = F8 ? 32 : 16;               // positions of one value product
};

constexpr int kMaxStages = 6;

template <class Args>
struct CtlOf {
    uint64_t q_full[2], q_empty[2];        // per buffer of q
    uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
    uint64_t v_ok[kMaxStages];             // V's tile may be multiplied
    uint64_t s_full[2];                    // per buffer: a tile's scores are in tensor memory
    uint64_t p_full[2][2];                 // per group and buffer: its weights are (and its O is rescaled)
    uint64_t p_done[2];                    // per buffer: the value products on both groups' weights have finished
    uint64_t o_done, o_free;               // a unit's last product has finished; its O has been read
    uint64_t stats_full, stats_free;       // the groups' statistics (and `unfinite`) are posted; the statistics are read
    uint64_t unit_full[kUnits], unit_empty[kUnits];
    union {
        typename Args::Unit units[kUnits];
        Part parts[kThreads / 32];         // before the roles begin
    };
    WalkOf<typename Args::Seq> walk;
    uint32_t tmem;
    int abort;
    int unfinite[2];                       // per unit parity: some new value is not finite
};
static_assert(sizeof(CtlOf<MultiArgs>) <= 1024 && sizeof(CtlOf<ShapedArgs>) <= 1024, "control block overflows its space");

// --- tcgen05 ------------------------------------------------------------------

// Shared-memory operand descriptors: start address and leading byte offset
// (>> 4) in the low word; stride 1024 >> 4, version 1 and 128-byte swizzle in
// the high one.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
    return ((addr & 0x3FFFF) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// fp32 accumulator, A K-major, B K-major or (b_mn) MN-major; A and B bf16 (kind::f16), or B E4M3 and A E4M3 or
// (a_e5m2) E5M2 (kind::f8f6f4, whose operands may differ).
__host__ __device__ constexpr uint32_t idesc(bool f8, int m, int n, int b_mn, bool a_e5m2 = false) {
    return (1u << 4) | (f8 ? (a_e5m2 ? 1u << 7 : 0u) : (1u << 7) | (1u << 10)) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// D = A . B (+ D if acc: a constant predicate where the compiler knows it).
#define PA_MMA(kind, a_op, setup)                                                                     \
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t" setup           \
                 "mov.b64 y, {%2, %5};\n\ttcgen05.mma.cta_group::1.kind::" kind " [%0], " a_op ", y, %3, p;\n\t}" ::"r"(d), \
                 "r"(a), "r"(b), "r"(id), "r"(acc), "n"(kDescHi))
#define PA_MMA_ADD(kind, a_op, setup)                                                                 \
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.eq.b32 p, 0, 0;\n\t" setup            \
                 "mov.b64 y, {%2, %4};\n\ttcgen05.mma.cta_group::1.kind::" kind " [%0], " a_op ", y, %3, p;\n\t}" ::"r"(d), \
                 "r"(a), "r"(b), "r"(id), "n"(kDescHi))

template <bool F8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    if constexpr (F8) PA_MMA("f8f6f4", "x", "mov.b64 x, {%1, %5};\n\t");
    else PA_MMA("f16", "x", "mov.b64 x, {%1, %5};\n\t");
}
template <bool F8>
__device__ __forceinline__ void mma_ss_add(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
    if constexpr (F8) PA_MMA_ADD("f8f6f4", "x", "mov.b64 x, {%1, %4};\n\t");
    else PA_MMA_ADD("f16", "x", "mov.b64 x, {%1, %4};\n\t");
}
// A operand from tensor memory: rows in lanes, two bf16 or four E5M2 values per column.
template <bool F8>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    if constexpr (F8) PA_MMA("f8f6f4", "[%1]", "");
    else PA_MMA("f16", "[%1]", "");
}
template <bool F8>
__device__ __forceinline__ void mma_ts_add(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
    if constexpr (F8) PA_MMA_ADD("f8f6f4", "[%1]", "");
    else PA_MMA_ADD("f16", "[%1]", "");
}
#undef PA_MMA
#undef PA_MMA_ADD

__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(pa::smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Waits for this warp's loads; `v` (their results) is not used before.
template <int N, class T>
__device__ __forceinline__ void wait_ld(T* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (T(0.5f) == T(0)) asm volatile("" : "+r"(v[i]));
        else asm volatile("" : "+f"(v[i]));
    }
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this thread's lane.
__device__ __forceinline__ void ld32(uint32_t t, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void ld16(uint32_t t, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t));
}

__device__ __forceinline__ void st16(uint32_t t, const uint32_t* w) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
        "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15]));
}

// Lanes 0-15 of the warp's 32 (or 16-31, with 16 added to the lane of t):
// thread x < 16 gets 32 columns of lane x from t on, thread x + 16 those 32
// columns further.
__device__ __forceinline__ void ld32_split32(uint32_t t, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], 32;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The like for stores: 16 columns, the second half 16 columns further, ...
__device__ __forceinline__ void st16_split16(uint32_t t, const uint32_t* w) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], 16, {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
        "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15]));
}

// ... and 8 columns, the second half 8 further.
__device__ __forceinline__ void st8_split8(uint32_t t, const uint32_t* w) {
    asm volatile("tcgen05.st.sync.aligned.16x32bx2.x8.b32 [%0], 8, {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]));
}

// E4M3 code pairs as f16 pairs, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
    return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ void tma_q(uint32_t dst, const CUtensorMap* map, int x, int head, int token, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(token),
        "r"(pa::smem_addr(bar)) : "memory");
}

// --- packed fp32 pairs --------------------------------------------------------

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(uint64_t r, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __noinline__ void flag(int32_t* status, int bit) { pa::set_status(status, bit); }

__device__ __noinline__ void give_up(int* abort, int32_t* status) {
    *reinterpret_cast<volatile int*>(abort) = 1;
    pa::set_status(status, PA_DEV_WAIT_TIMEOUT);
}

// A whole warp's bounded wait; gives up, too, once another role has.
template <class Ctl>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Ctl* ctl, int32_t* status) {
#pragma unroll 1
    for (int i = 0; i < kMaxProbes; ++i) {
        if (__all_sync(0xffffffffu, pa::mbar_try_wait(bar, parity))) return true;
        if ((i & 63) == 63 && __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&ctl->abort) != 0)) return false;
    }
    give_up(&ctl->abort, status);
    return false;
}

// One thread's.
template <class Ctl>
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, Ctl* ctl, int32_t* status) {
#pragma unroll 1
    for (int i = 0; i < kMaxProbes; ++i) {
        if (pa::mbar_try_wait(bar, parity)) return true;
        if ((i & 63) == 63 && *reinterpret_cast<volatile int*>(&ctl->abort)) return false;
    }
    give_up(&ctl->abort, status);
    return false;
}

// kRuns: how many scales 32 positions of a block-scaled cache have (blocks of 32, 16, 8: 1, 2, 4).
template <int D, bool kHalf, bool F8, class Args, int kRuns>
__global__ void __launch_bounds__(kThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const Args a, int oob_row) {
    using G = Wide<D, kHalf, F8>;
    using Unit = typename Args::Unit;
    using Ctl = CtlOf<Args>;
    constexpr bool kShaped = Args::kShaped, kScaled = kShaped && F8;
    auto base_of = [](const Unit& u) {
        if constexpr (kShaped) return u.base;
        else return 0;
    };
    constexpr int kRows = G::kRows, kStages = G::kStages;
    extern __shared__ __align__(1024) uint8_t sm[];
    Ctl* ctl = reinterpret_cast<Ctl*>(sm + G::kCtl);
    float2* stats = reinterpret_cast<float2*>(sm + G::kStats);
    const uint32_t s0 = pa::smem_addr(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = 1 << a.log2_block, group = 1 << a.log2_group;

    if (threadIdx.x == 0) {
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) {
            pa::mbar_init(&ctl->k_full[i], 1);
            pa::mbar_init(&ctl->k_empty[i], 1);
            pa::mbar_init(&ctl->v_full[i], 1);
            pa::mbar_init(&ctl->v_empty[i], 2);
            pa::mbar_init(&ctl->v_ok[i], 1);
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            pa::mbar_init(&ctl->q_full[i], F8 ? 128 : 1);
            pa::mbar_init(&ctl->q_empty[i], 1);
            pa::mbar_init(&ctl->s_full[i], 1);
            pa::mbar_init(&ctl->p_full[0][i], 128);
            pa::mbar_init(&ctl->p_full[1][i], 128);
            pa::mbar_init(&ctl->p_done[i], 2);
        }
        pa::mbar_init(&ctl->o_done, 2);
        pa::mbar_init(&ctl->o_free, 128);
        pa::mbar_init(&ctl->stats_full, 256 + 1);
        pa::mbar_init(&ctl->stats_free, 128);
#pragma unroll 1
        for (int i = 0; i < kUnits; ++i) {
            pa::mbar_init(&ctl->unit_full[i], 1);
            pa::mbar_init(&ctl->unit_empty[i], kUnitReaders);
        }
        ctl->abort = 0;
        pa::fence_mbar_init();
    }
    if (warp == kScoreWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(pa::smem_addr(&ctl->tmem)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = ctl->tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const bool busy = find_share<kRows, kKv, kWideCost, kWideMinSteps, kWideDirectSteps, kThreads>(a, ctl->walk, ctl->parts);
    // an address that is not a multiple of 1024 would break the swizzled tiles
    if (busy && (s0 & 1023)) {
        if (threadIdx.x == 0) pa::set_status(a.status, PA_DEV_WAIT_TIMEOUT);
    } else if (!busy) {
    } else if (warp == kKWarp || warp == kVWarp) {
        // ------------------------------------------------------------ producers
        // Lanes i * blocks on copy the blocks of tile i of the `per` tiles
        // that one load of table entries serves, the next load's in flight
        // meanwhile; blocks past the context or in front of what is seen, and
        // bad ids, are read from outside the tensor, which fills zeros.
        const bool is_k = warp == kKWarp;
        const int log2_blocks = 7 - a.log2_block, blocks = 1 << log2_blocks, per = 32 >> log2_blocks;
        static_assert(kKv == 128, "log2_blocks");
        uint64_t* full = is_k ? ctl->k_full : ctl->v_full;
        uint64_t* empty = is_k ? ctl->k_empty : ctl->v_empty;
        const CUtensorMap* map = is_k ? &map_k : &map_v;
        const uint64_t policy = pa::l2_evict_first_policy();
        const int sub = lane >> log2_blocks, place = (lane & (blocks - 1)) * B;
        constexpr int kNoBlock = -2147483647 - 1;
        // A unit, and the table entries of its first tiles on their way.
        struct Next {
            int valid, len, ctx, st0, kvh, token, first, base, lo;
            const int32_t* table;
        };
        auto fetch = [&](const Next& x, int j) {                 // tiles j .. j + per - 1
            const int pos = x.base + (x.st0 + j + sub) * kKv + place;
            return (j + sub < x.len && pos < x.ctx && pos + B > x.lo) ? x.table[pos >> a.log2_block] : kNoBlock;
        };
        auto take = [&](int nth, Next& x) {                      // K's warp posts it, V's waits for it
            const int slot = nth % kUnits;
            Unit* u = &ctl->units[slot];
            if (is_k) {
                if (nth >= kUnits && !wait_for(&ctl->unit_empty[slot], (nth / kUnits - 1) & 1, ctl, a.status)) return false;
                if (lane == 0) {
                    next_unit<kRows, kKv, kWideCost>(ctl->walk, *u, a);
                    if (u->valid && u->st0 == 0 && !u->whole)       // this block begins a unit that others end
                        a.pieces[blockIdx.x] = begun_unit(*u, a.log2_group);
                }
                __syncwarp();
            } else if (!wait_for(&ctl->unit_full[slot], (nth / kUnits) & 1, ctl, a.status)) {
                return false;
            }
            x.valid = u->valid;
            x.len = u->len;
            x.ctx = u->ctx;
            x.st0 = u->st0;
            x.base = u->valid ? base_of(*u) : 0;
            x.lo = 0;
            if constexpr (kShaped) x.lo = u->valid ? u->lo : 0;
            x.kvh = u->kvh;
            x.table = table_of(a, *u);
            x.token = u->q0 + (u->row0 >> a.log2_group);
            __syncwarp();
            if (lane == 0) pa::mbar_arrive(is_k ? &ctl->unit_full[slot] : &ctl->unit_empty[slot]);
            if (x.valid) x.first = fetch(x, 0);
            return true;
        };
        int loaded = 0, asked = 0;                               // tiles so far, and units' q
        Next now, next;
        bool ok = true;
#pragma unroll 1
        for (int nth = -1; ok; ++nth) {
            if (nth >= 0 && !now.valid) break;
            if (!F8 && !is_k && nth >= 0) {
                if (nth >= 1 && !wait_for(ctl->q_empty, (nth - 1) & 1, ctl, a.status)) break;
                if (lane == 0) {
                    // 16 rows a box: 16 / group tokens of the group's heads
                    pa::mbar_arrive_expect_tx(ctl->q_full, kRows * 128 * G::kHalves);
#pragma unroll 1
                    for (int r = 0; r < kRows; r += 16) {
#pragma unroll
                        for (int h = 0; h < G::kHalves; ++h)
                            tma_q(s0 + h * G::kHalfBytes + (kHalf ? 2 * r : r) * 128, &map_q, h * 64,
                                  now.kvh << a.log2_group, now.token + (r >> a.log2_group), ctl->q_full);
                    }
                }
                ++asked;
            }
            // the unit after it, so that its first table entries come beside this one's tiles
            if (!take(nth + 1, next)) break;
            if (nth < 0) {
                now = next;
                continue;
            }
            int row = 0, ahead = now.first;
#pragma unroll 1
            for (int j = 0; ok && j < now.len; ++j, ++loaded) {
                const int turn = j & (per - 1), st = loaded % kStages;
                if (turn == 0) {
                    row = oob_row;
                    if (ahead >= 0 && ahead < a.num_blocks) row = (ahead * a.n_kv_heads + now.kvh) * B;
                    else if (ahead != kNoBlock) flag(a.status, PA_DEV_BAD_BLOCK_ID);
                    ahead = fetch(now, j + per);
                }
                if (loaded >= kStages && !(ok = wait_for(&empty[st], (loaded / kStages - 1) & 1, ctl, a.status))) break;
                if (lane == 0) pa::mbar_arrive_expect_tx(&full[st], G::kTileBytes);
                __syncwarp();
                if (turn == sub) {
                    const uint32_t dst = s0 + (is_k ? G::kK0 : G::kV0) + st * G::kTileBytes + place * 128;
#pragma unroll
                    for (int h = 0; h < G::kHalves; ++h)
                        pa::tma_box(dst + h * G::kHalfBytes, map, h * 64, row, &full[st], policy);
                }
            }
            now = next;
        }
        // the copies this warp started land before the block exits
        if (lane == 0) {
            if (asked > 0) pa::mbar_wait_bounded(ctl->q_full, (asked - 1) & 1, kMaxProbes);
#pragma unroll 1
            for (int i = 0; i < kStages && i < loaded; ++i)
                pa::mbar_wait_bounded(&full[(loaded - 1 - i) % kStages], ((loaded - 1 - i) / kStages) & 1, kMaxProbes);
        }
    } else if (warp == kScoreWarp) {
        // ------------------------------------------------------------ score products, by one thread
        constexpr uint32_t id = idesc(F8, 128, kKv, 0);
        const uint32_t k_lo0 = desc_lo(s0 + G::kK0, 16);
        if (lane == 0) {
            int at = 0, st = 0, phase = 0;                       // tiles so far; K's stage and phase
            bool ok = true;
#pragma unroll 1
            for (int nth = 0; ok; ++nth) {
                const int slot = nth % kUnits;
                if (!wait_one(&ctl->unit_full[slot], (nth / kUnits) & 1, ctl, a.status)) break;
                const int valid = ctl->units[slot].valid, len = ctl->units[slot].len;
                pa::mbar_arrive(&ctl->unit_empty[slot]);
                if (!valid) break;
                const int qb = nth % G::kQBuffers;
                if (!wait_one(&ctl->q_full[qb], (nth / G::kQBuffers) & 1, ctl, a.status)) break;
                const uint32_t q_lo = desc_lo(s0 + qb * G::kQBytes, 16);
#pragma unroll 1
                for (int j = 0; j < len; ++j, ++at) {
                    const int b = at & 1;
                    // the scores go over weights of two tiles ago: their value products have to be done
                    if (!(ok = wait_one(&ctl->k_full[st], phase, ctl, a.status) &&
                               (at < 2 || wait_one(&ctl->p_done[b], ((at >> 1) - 1) & 1, ctl, a.status))))
                        break;
                    fence_after();
                    const uint32_t k_lo = k_lo0 + st * (G::kTileBytes >> 4), d = tmem + b * 128;
                    mma_ss<F8>(d, q_lo, k_lo, id, 0);
#pragma unroll
                    for (int kk = 1; kk < D / (F8 ? 32 : 16); ++kk) {
                        const uint32_t off = ((kk >> 2) * G::kHalfBytes + (kk & 3) * 32) >> 4;
                        mma_ss_add<F8>(d, q_lo + off, k_lo + off, id);
                    }
                    commit(&ctl->s_full[b]);
                    commit(&ctl->k_empty[st]);
                    if (j == len - 1) commit(&ctl->q_empty[qb]);
                    if (++st == kStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            // products in flight finish before the tensor memory is freed
            if (at > 0) pa::mbar_wait_bounded(&ctl->k_empty[(at - 1) % kStages], ((at - 1) / kStages) & 1, kMaxProbes);
        }
        __syncwarp();
    } else if (value_group(warp) >= 0) {
        // ------------------------------------------------------------ value products of group w
        constexpr uint32_t id = idesc(F8, 128, D, 1, F8);
        constexpr int kStepKeys = G::kStepKeys, kSteps = kHalfKv / kStepKeys, kSets = F8 || !kHalf ? 2 : 1;
        const int w = value_group(warp);
        const uint32_t t_o = tmem + kTmemO + w * 128;
        const uint32_t v_lo0 = desc_lo(s0 + G::kV0 + w * kHalfKv * 128, G::kHalfBytes);
        if (lane == 0) {
            int at = 0, st = 0, phase = 0;                       // tiles so far; V's stage and phase
            bool ok = true;
#pragma unroll 1
            for (int nth = 0; ok; ++nth) {
                const int slot = nth % kUnits;
                if (!wait_one(&ctl->unit_full[slot], (nth / kUnits) & 1, ctl, a.status)) break;
                const Unit* u = &ctl->units[slot];
                const int valid = u->valid, len = u->len, ctx = u->ctx - base_of(*u), st0 = u->st0;
                pa::mbar_arrive(&ctl->unit_empty[slot]);
                if (!valid) break;
                // the unit before has read its O out
                if (nth >= 1 && !wait_one(&ctl->o_free, (nth - 1) & 1, ctl, a.status)) break;
#pragma unroll 1
                for (int j = 0; j < len; ++j, ++at) {
                    const int b = at & 1;
                    // the group's positions of the tile within the context, in products
                    const int left = min(kHalfKv, ctx - (st0 + j) * kKv - w * kHalfKv);
                    const int steps = left > 0 ? (left + kStepKeys - 1) / kStepKeys : 0;
                    if (!(ok = wait_one(&ctl->v_ok[st], phase, ctl, a.status) &&
                               wait_one(&ctl->p_full[w][b], (at >> 1) & 1, ctl, a.status)))
                        break;
                    fence_after();
                    const uint32_t t_p = tmem + b * 128 + w * kHalfKv, v_lo = v_lo0 + st * (G::kTileBytes >> 4);
                    // weights of product kk: 8 columns each, a second set of them behind the first
#pragma unroll
                    for (int kk = 0; kk < kSteps; ++kk) {
                        if (kk >= steps) break;
#pragma unroll
                        for (int x = 0; x < kSets; ++x) {
                            const uint32_t t = t_p + 8 * (x * kSteps + kk), v = v_lo + kk * ((kStepKeys * 128) >> 4);
                            if (kk == 0 && x == 0)
                                mma_ts<F8>(t_o, t, v, id, j > 0 ? 1u : 0u);
                            else
                                mma_ts_add<F8>(t_o, t, v, id);
                        }
                    }
                    commit(&ctl->p_done[b]);
                    commit(&ctl->v_empty[st]);
                    if (j == len - 1) commit(&ctl->o_done);
                    if (++st == kStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            if (at > 0) pa::mbar_wait_bounded(&ctl->v_empty[(at - 1) % kStages], ((at - 1) / kStages) & 1, kMaxProbes);
        }
        __syncwarp();
    } else if (warp == kCheckWarp) {
        // ------------------------------------------------------------ V's tiles at a context's end
        // Zeros in place of values that are not finite at new positions, and in the rows from the context's end to
        // the end of the last product there; beside the softmax, so that the products need not wait.
        int st = 0, phase = 0;
        bool ok = true;
#pragma unroll 1
        for (int nth = 0; ok; ++nth) {
            const int slot = nth % kUnits;
            if (!wait_for(&ctl->unit_full[slot], (nth / kUnits) & 1, ctl, a.status)) break;
            const Unit* u = &ctl->units[slot];
            const int valid = u->valid, len = u->len, ctx = u->ctx, st0 = u->st0, first = u->first, base = base_of(*u);
            int seen_lo = 0, seen_hi = 0;
            if constexpr (kShaped) {
                seen_lo = u->seen_lo;
                seen_hi = u->seen_hi;
            }
            __syncwarp();
            if (lane == 0) pa::mbar_arrive(&ctl->unit_empty[slot]);
            if (!valid) break;
            bool unfinite = false;
#pragma unroll 1
            for (int j = 0; j < len; ++j) {
                if (!(ok = wait_for(&ctl->v_full[st], phase, ctl, a.status))) break;
                const int t0 = base + (st0 + j) * kKv, left = ctx - t0;
                uint8_t* tile = sm + G::kV0 + st * G::kTileBytes;
                if (kShaped ? t0 < seen_lo || t0 + kKv > seen_hi : t0 + kKv > first) {
                    unfinite |= kShaped ? drop_unfinite_outside<F8, G::kHalves>(tile, G::kHalfBytes, t0, seen_lo, seen_hi, min(kKv, left), lane, 32)
                                        : drop_unfinite<F8, G::kHalves>(tile, G::kHalfBytes, max(0, first - t0), min(kKv, left), lane, 32);
                    if (left < kKv && left % G::kStepKeys) {
#pragma unroll 1
                        for (int x = lane; x < (G::kStepKeys - left % G::kStepKeys) * G::kHalves * 8; x += 32) {
                            const int r = left + x / (G::kHalves * 8), c = x % (G::kHalves * 8);
                            *reinterpret_cast<uint4*>(tile + (c >> 3) * G::kHalfBytes + r * 128 + (c & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    __syncwarp();
                }
                if (lane == 0) pa::mbar_arrive(&ctl->v_ok[st]);
                if (++st == G::kStages) {
                    st = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            if (nth >= 1 && !wait_for(&ctl->stats_free, (nth - 1) & 1, ctl, a.status)) break;
            unfinite = __any_sync(0xffffffffu, unfinite);
            if (lane == 0) {
                ctl->unfinite[nth & 1] = unfinite;
                pa::mbar_arrive(&ctl->stats_full);
            }
        }
    } else if (warp < kSoftmaxWarps) {
        // ------------------------------------------------------------ softmax of group w's half of every tile
        const int w = warp >> 2, quarter = warp & 3;
        const int r = kHalf ? quarter * 16 + (lane & 15) : quarter * 32 + lane;   // row of the unit
        const int half = kHalf ? lane >> 4 : 0;                  // 64-row units: which 32 of the group's columns
        constexpr int kCols = kHalf ? 32 : 64;                   // columns per thread
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16), t_o = t_lane + kTmemO + w * 128;
        const float* factors = reinterpret_cast<const float*>(stats + 128);   // F8: [unit parity][row]
        float* tops = reinterpret_cast<float*>(stats + 192);      // block-scaled values: [group][row] the unit of the row's O
        constexpr float kSlack = F8 ? 0.5f : kRaise;             // F8: weights of at most 2^15.5 in E5M2's 57344
        constexpr float kHeadroom = F8 ? 3.f : 0.f;              // F8: a raise leaves room for the next ones (a raise
                                                                 // at every growth cost 560 cycles in half the tiles)
        constexpr float kUp = F8 ? 15.f : 0.f;                   // log2 of the weights' common factor
        constexpr uint32_t kLanes16 = 16u << 16;
        int at = 0;                                              // tiles so far
        bool ok = true;
#pragma unroll 1
        for (int nth = 0; ok; ++nth) {
            const int slot = nth % kUnits;
            if (!wait_for(&ctl->unit_full[slot], (nth / kUnits) & 1, ctl, a.status)) break;
            const Unit* u = &ctl->units[slot];
            if (!u->valid) break;                                // (the rest of it is not set then)
            const int len = u->len, first = u->first;
            const int start = base_of(*u) + u->st0 * kKv + w * kHalfKv + 32 * half;   // the thread's first position in the unit
            const int i = (u->row0 + r) >> a.log2_group;
            const bool real = i < u->n, tree = a.tree_mask != nullptr;
            // what the row sees of the new tokens: a word (tree), or positions below `lim`
            unsigned long long word = tree && real ? words_of(a, *u)[i] : ~0ull;
            if (u->n < 64) word &= (1ull << u->n) - 1;
            int lim = (tree || !real) ? u->ctx : first + i + 1, from = 0;
            int pos = first + i;                                 // which a bias counts from
            float slope = 0.f;                                   // times log2(e)
            const int32_t* table = nullptr;
            uint32_t kvh = 0;
            int end = 0, begin = 0;                              // the unit's positions
            if constexpr (kShaped) {
                if (a.visible && real) {
                    const int2 v = a.visible[u->q0 + i];
                    from = max(v.x, 0);
                    lim = max(v.y, 0);
                }
                lim = min(lim, u->ctx);
                if (Args::kCurved && a.slopes) slope = pa::bias_slope(a.slopes[(u->kvh << a.log2_group) + ((u->row0 + r) & ((1 << a.log2_group) - 1))]);
                pos = pa::bias_from(pos, from, lim);
                table = table_of(a, *u);
                kvh = u->kvh;
                end = u->ctx;
                begin = u->lo;
            }
            __syncwarp();
            if (lane == 0) pa::mbar_arrive(&ctl->unit_empty[slot]);
            // the positions from `start` on that the row sees, as 32 bits
            auto seen = [&](int start) {
                const int n = lim - start, b = start - first;
                uint32_t v = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
                if constexpr (kShaped) {
                    const int skip = from - start;
                    v &= skip <= 0 ? ~0u : skip >= 32 ? 0u : ~0u << skip;
                } else if (tree)
                    v &= b <= -32 ? ~0u
                         : b < 0  ? (uint32_t)(word << -b) | ((1u << -b) - 1u)
                         : b < 64 ? (uint32_t)(word >> b)
                                  : 0u;
                return v;
            };
            // Block-scaled: the scales of the group's 64 positions of a tile, lane i's of block i (K's byte, and V's above it),
            // asked for a tile ahead and their table entries two.
            float v_top = 0.f;                                   // the largest of V that the row has seen, 2^(this - 127) being its O's unit
            int entry = -1;
            uint32_t k_next = 0, v_next = 0;                      // (put together when their turn comes: nothing waits for them before)
            auto entry_of = [&](int j) {
                const int pos = start - 32 * half + j * kKv + lane * B;
                return kScaled && lane * B < kHalfKv && j < len && pos < end && pos + B > begin ? table[pos >> a.log2_block] : -1;
            };
            auto ask = [&](int blk) {
                k_next = v_next = 0;                             // (zeros are in place of what is not there)
                if constexpr (kScaled)
                    if (blk >= 0 && blk < a.num_blocks) {
                        const uint32_t at = (uint32_t)blk * a.n_kv_heads + kvh;   // (a cache has less than 2^31 rows)
                        k_next = a.k_scales[at];
                        v_next = a.v_scales[at];
                    }
            };
            float m = kNone, l = 0.f, c = a.scale_log2;
            if constexpr (F8) {
                if (!wait_for(&ctl->q_full[nth & 1], (nth >> 1) & 1, ctl, a.status)) break;   // the rows' factors come with q
                c = factors[(nth & 1) * 64 + r];
            }
            if constexpr (kScaled) {
                ask(entry_of(0));
                entry = entry_of(1);
            }
#pragma unroll 1
            for (int j = 0; j < len; ++j, ++at) {
                const int b = at & 1;
                const uint32_t t_s = t_lane + b * 128 + w * kHalfKv;
                uint32_t scales = 0;
                if constexpr (kScaled) {
                    scales = k_next | v_next << 8;
                    ask(entry);
                    entry = entry_of(j + 2);
                }
                if (!(ok = wait_for(&ctl->s_full[b], (at >> 1) & 1, ctl, a.status))) break;
                fence_after();
                float s[kCols];
                if constexpr (kHalf) {
                    ld32_split32(t_s, s);
                    if constexpr (F8) {                          // and the scores of q's second term, in the row's second lane
                        float s2[32];
                        ld32_split32(t_s + kLanes16, s2);
                        wait_ld<32>(s2);
                        wait_ld<32>(s);
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
                            split(fma2(pair(s2[k], s2[k + 1]), pair(1.f / kQUp, 1.f / kQUp), pair(s[k], s[k + 1])), s[k], s[k + 1]);
                    }
                } else {
                    ld32(t_s, s);
                    ld32(t_s + 32, s + 32);
                }
                wait_ld<kCols>(s);
                const int t0 = start + j * kKv;
                float cs[kRuns], by[kRuns];                      // the scores' factors; block-scaled values: log2 of the weights'
#pragma unroll
                for (int x = 0; x < kRuns; ++x) cs[x] = c;
                bool grows = false;                              // and whether V's largest scale does
                float v_new = v_top;
                // some row (shaped: this one) may not see some position
                const bool part = kShaped ? t0 < from || t0 + kCols > lim : t0 + kCols > first;
                auto where_unseen = [&](float to) {
#pragma unroll
                    for (int x = 0; x < kCols; x += 32) {
                        const uint32_t v = seen(t0 + x);
#pragma unroll
                        for (int k = 0; k < 32; ++k) s[x + k] = (v & (1u << k)) ? s[x + k] : to;
                    }
                };
                if constexpr (kShaped) {
                    if constexpr (kScaled) {
                        // (a scale of positions that the row does not see is none of its own: its weights there are zeros)
                        int most = 0, v_of[kRuns];
#pragma unroll
                        for (int x = 0; x < kRuns; ++x) {
                            const int e = __shfl_sync(0xffffffffu, scales, half * kRuns + x);
                            cs[x] = fmaxf(c * scale_of(e & 0xff), 1e-37f);   // never 0: masked scores stay -inf
                            v_of[x] = e >> 8;
                        }
                        if (part) {
                            const uint32_t some = seen(t0);
#pragma unroll
                            for (int x = 0; x < kRuns; ++x)
                                if (!(some & (~0u >> (32 - 32 / kRuns) << (x * (32 / kRuns))))) v_of[x] = 0;
                        }
#pragma unroll
                        for (int x = 0; x < kRuns; ++x) {
                            by[x] = (float)v_of[x];
                            most = max(most, v_of[x]);
                        }
                        most = max(most, __shfl_xor_sync(0xffffffffu, most, 16));
                        v_new = fmaxf((float)most, v_top);
                        grows = v_new > v_top;
                    }
                    if (Args::kCurved) {                         // scores in units of log2 from here on
                        if constexpr (kScaled) {
#pragma unroll
                            for (int k = 0; k < kCols; k += 2) split(mul2(pair(s[k], s[k + 1]), pair(cs[k * kRuns / 32], cs[k * kRuns / 32])), s[k], s[k + 1]);
                        }
                        float all = kScaled ? 1.f : c;
                        if (a.cap_inv != 0.f) {
                            if (part) where_unseen(0.f);
                            pa::cap_scores<kCols>(s, pa::largest(s), all, a.cap_log2, a.cap_inv);
                            all = 1.f;
                        }
                        if (a.slopes) {
                            const float d0 = (float)(pos - t0);
#pragma unroll
                            for (int k = 0; k < kCols; ++k) s[k] = fmaf(-slope, fabsf(d0 - (float)k), s[k] * all);
                        }
#pragma unroll
                        for (int x = 0; x < kRuns; ++x) cs[x] = 1.f;
                    }
                }
                if (part) where_unseen(-INFINITY);
                float top;
                if constexpr (kScaled) {
                    float p[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float* v = s + 8 * x;
                        p[x] = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
                    }
                    if constexpr (kRuns == 4)
                        top = fmaxf(fmaxf(cs[0] * p[0], cs[1] * p[1]), fmaxf(cs[2] * p[2], cs[3] * p[3]));
                    else
                        top = fmaxf(cs[0] * fmaxf(p[0], p[1]), cs[kRuns - 1] * fmaxf(p[2], p[3]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                } else {
                    float p[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        p[k] = fmaxf(fmaxf(s[k], s[k + 8]), fmaxf(s[k + 16], s[k + 24]));
                        if constexpr (!kHalf) p[k] = fmaxf(p[k], fmaxf(fmaxf(s[k + 32], s[k + 40]), fmaxf(s[k + 48], s[k + 56])));
                    }
                    top = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
                    if (kHalf) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                }
                const float c1 = kScaled ? 1.f : cs[0];          // (scaled: the maximum has its factors)
                const bool raise = fmaf(top, c1, -m) > kSlack;
                const float m_new = raise ? fmaf(top, c1, kHeadroom) : m;
                if (j > 0 && __any_sync(0xffffffffu, raise || (kScaled && grows))) {
                    // This group's O holds its halves of the tiles before, once their products are done.  The wait
                    // is for tile at - 1's phase of its buffer's barrier, whatever was skipped: the phase before it,
                    // tile at - 3's, is over, since the scores of tile at - 1 were issued after it and have been
                    // read; and the one after it, tile at + 1's, takes weights that this warp has yet to give.
                    // (Both hold for two score buffers; a third would need a wait in every phase.)
                    if (!(ok = wait_for(&ctl->p_done[b ^ 1], ((at - 1) >> 1) & 1, ctl, a.status))) break;
                    fence_after();
                    float f = pa::exp2_approx(m - m_new);
                    l *= f;
                    if (kScaled && grows) f *= pa::exp2_approx(v_top - v_new);
#pragma unroll 1
                    for (int x = 0; x < D; x += 16) {
                        uint32_t o[16];
                        ld16(t_o + x, o);
                        wait_ld<16>(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        st16(t_o + x, o);
                    }
                }
                m = m_new;
                if constexpr (kScaled) {
                    v_top = v_new;
#pragma unroll
                    for (int x = 0; x < kRuns; ++x) by[x] = fmaxf(by[x] - v_top, -60.f);   // (weights of less are nothing)
                }
                uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
                // two columns' weights, summed
                const uint64_t cc = pair(cs[0], cs[0]), neg = pair(kUp - m, kUp - m);
                auto weights = [&](float x0, float x1, int k) {
                    float y0, y1;
                    split(fma2(pair(x0, x1), cc, neg), y0, y1);
                    const uint64_t p = pair(pa::exp2_approx(y0), pa::exp2_approx(y1));
                    sum[k & 1] = add2(sum[k & 1], p);
                    return p;
                };
                // the like of run x, times 2^by[x]
                auto scaled_weights = [&](float x0, float x1, int x) {
                    const float n = kUp - m + by[x];
                    float y0, y1;
                    split(fma2(pair(x0, x1), pair(cs[x], cs[x]), pair(n, n)), y0, y1);
                    return pair(pa::exp2_approx(y0), pa::exp2_approx(y1));
                };
                if constexpr (F8) {
                    // Weights as f16 (a relative 2^-11), exactly the sum of four E5M2 terms: an f16's upper byte is
                    // its E5M2 value cut off, and so is what that leaves, down to 2^-16 (2^-28 of the row's
                    // largest).  (E4M3 ends at 2^-9, which would lose weights below 2^-14, and a long tail of such
                    // can be most of a row's sum.)  Two and two terms in a product's two lanes of a row.
                    uint32_t t[4][8];
                    uint64_t block = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint32_t h[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float p0, p1;
                            uint64_t p;
                            if constexpr (kScaled) {
                                p = scaled_weights(s[4 * k + 2 * e], s[4 * k + 2 * e + 1], k * kRuns / 8);
                                block = k % (8 / kRuns) + e == 0 ? p : add2(block, p);
                            } else {
                                p = weights(s[4 * k + 2 * e], s[4 * k + 2 * e + 1], e);
                            }
                            split(p, p0, p1);
                            h[e] = pa::pack_f16x2(p0, p1);
                        }
                        if constexpr (kScaled)
                            if (k % (8 / kRuns) == 8 / kRuns - 1) {   // a run's sum, without its factor
                                const float back = pa::exp2_approx(-by[k * kRuns / 8]);
                                sum[0] = fma2(block, pair(back, back), sum[0]);
                            }
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            t[x][k] = __byte_perm(h[0], h[1], 0x7531);
                            if (x < 3) {
                                h[0] = sub_f16x2(h[0], h[0] & 0xff00ff00u);
                                h[1] = sub_f16x2(h[1], h[1] & 0xff00ff00u);
                            }
                        }
                    }
                    st8_split8(t_s, t[0]);
                    st8_split8(t_s + kLanes16, t[1]);
                    st8_split8(t_s + 16, t[2]);
                    st8_split8(t_s + kLanes16 + 16, t[3]);
                } else {
                    // hi terms in the group's first 32 columns; lo terms in a row's second lane (64-row
                    // units) or in the other 32 columns
#pragma unroll
                    for (int x = 0; x < kCols; x += 32) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const uint64_t p = weights(s[x + 2 * k], s[x + 2 * k + 1], k);
                            float p0, p1, r0, r1;
                            split(p, p0, p1);
                            hi[k] = pa::pack_bf16x2(p0, p1);
                            split(sub2(p, pair(__uint_as_float(hi[k] << 16), __uint_as_float(hi[k] & 0xffff0000u))), r0, r1);
                            lo[k] = pa::pack_bf16x2(r0, r1);
                        }
                        if constexpr (kHalf) {
                            st16_split16(t_s, hi);
                            st16_split16(t_s + kLanes16, lo);
                        } else {
                            st16(t_s + x / 2, hi);
                            st16(t_s + 32 + x / 2, lo);
                        }
                    }
                }
                float a0, a1, b0, b1;
                split(sum[0], a0, a1);
                split(sum[1], b0, b1);
                l += (a0 + a1) + (b0 + b1);
                wait_st();
                fence_before();
                pa::mbar_arrive(&ctl->p_full[w][b]);
            }
            if (!ok) break;
            if (nth >= 1 && !wait_for(&ctl->stats_free, (nth - 1) & 1, ctl, a.status)) break;
            if (kHalf) l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (!half) stats[w * kRows + r] = make_float2(m, l);
            if (kScaled && !half) tops[w * kRows + r] = scale_of((int)v_top);
            pa::mbar_arrive(&ctl->stats_full);
        }
    } else {
        // ------------------------------------------------------------ a unit's end: the two accumulators, merged exactly
        const int quarter = warp & 3;
        const int r = kHalf ? quarter * 16 + (lane & 15) : quarter * 32 + lane;
        const bool second = kHalf && (lane & 16);                // a row's second lane
        // E4M3 caches: these warps make q's two terms too.  A bf16 value is the sum of two E4M3 values
        // (8 significant bits, 4 and 4), after a power of two per row that brings its largest into
        // [2^7, 2^8).  The second term is at most 2^3 then and goes 2^5 times as large, so that E4M3's
        // smallest step, 2^-9, cuts what is below 2^-14 of the largest, to within 2^-22 of it.
        // Returns false to give up.
        float* factors = reinterpret_cast<float*>(stats + 128);
        auto make_q = [&](int nth) {
            const int slot = nth % kUnits, qb = nth & 1;
            if (!wait_for(&ctl->unit_full[slot], (nth / kUnits) & 1, ctl, a.status)) return false;
            const Unit* u = &ctl->units[slot];
            if (!u->valid) return true;
            const int t = threadIdx.x - 32 * kOutWarp, row = t >> 1, part = t & 1, at = u->row0 + row, i = at >> a.log2_group;
            // read twice, for the maximum and then (from L1) for the terms: fewer instructions than keeping it
            const bool there = i < u->n;
            const uint4* src = reinterpret_cast<const uint4*>(
                a.q + ((size_t)(u->q0 + i) * a.n_q_heads + (u->kvh << a.log2_group) + (at & (group - 1))) * D + 64 * part);
            float top = 0.f;
            if (there) {
                uint32_t most = 0;                               // the largest magnitude of each half
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint4 v = src[x];
                    most = __vmaxu2(__vmaxu2(most, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu)),
                                    __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                }
                const float2 f = pa::bf16x2_to_float2(most);
                top = fmaxf(f.x, f.y);
            }
            // the buffer's last unit was two before
            if (nth >= 2 && !wait_for(&ctl->q_empty[qb], ((nth >> 1) - 1) & 1, ctl, a.status)) return false;
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            int eb = (__float_as_int(top) >> 23) & 0xff;
            eb = eb < 7 ? 7 : (eb > 254 ? 254 : eb);
            const float up = __int_as_float((261 - eb) << 23);
            const float by = top < INFINITY ? up * a.q_sign : __int_as_float(0x7fffffff);   // (E4M3 has no infinity)
            if (part == 0) factors[qb * 64 + row] = fmaxf(a.scale_log2 / up, 1e-37f);
            const int line = (row >> 4) * 32 + (row & 15);
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {                        // 16 elements: a 16-byte chunk of each term
                const uint4 none = make_uint4(0, 0, 0, 0), v0 = there ? src[2 * x] : none, v1 = there ? src[2 * x + 1] : none;
                uint32_t c0[4], c1[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint4 q = e < 2 ? v0 : v1;
                    const uint32_t w0 = e & 1 ? q.z : q.x, w1 = e & 1 ? q.w : q.y;
                    uint32_t a0[2], a1[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float2 f = pa::bf16x2_to_float2(y ? w1 : w0);
                        const float f0 = f.x * by, f1 = f.y * by;
                        a0[y] = pa::e4m3x2(f0, f1);
                        const uint32_t h = e4m3x2_to_f16x2(a0[y]);
                        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h));
                        a1[y] = pa::e4m3x2((f0 - g.x) * kQUp, (f1 - g.y) * kQUp);
                    }
                    c0[e] = a0[0] | (a0[1] << 16);
                    c1[e] = a1[0] | (a1[1] << 16);
                }
                uint8_t* dst = sm + qb * G::kQBytes + line * 128 + (((4 * part + x) ^ (line & 7)) << 4);
                *reinterpret_cast<uint4*>(dst) = make_uint4(c0[0], c0[1], c0[2], c0[3]);
                *reinterpret_cast<uint4*>(dst + 16 * 128) = make_uint4(c1[0], c1[1], c1[2], c1[3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            pa::mbar_arrive(&ctl->q_full[qb]);
            return true;
        };
        const uint32_t t_o = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemO;
#pragma unroll 1
        for (int nth = F8 ? -1 : 0;; ++nth) {
            const int slot = nth % kUnits;
            const Unit* u = &ctl->units[slot];
            if (nth >= 0 && !(wait_for(&ctl->unit_full[slot], (nth / kUnits) & 1, ctl, a.status) && u->valid)) break;
            if constexpr (F8) {                                  // the next unit's q, ahead of this unit's end
                if (!make_q(nth + 1)) break;
                if (nth < 0) continue;
            }
            const int st0 = u->st0;
            const int seq = u->seq, kvh = u->kvh, end = st0 + u->len, base = base_of(*u);
            const int row = u->row0 + r, i = row >> a.log2_group;
            const bool real = i < u->n, whole = u->whole;
            const bool both = u->len > 1 || u->ctx - base - st0 * kKv > kHalfKv;   // group 1 had positions: O1 was written
            const size_t out_row = ((size_t)(u->q0 + i) * a.n_q_heads + (kvh << a.log2_group) + (row & (group - 1))) * D;
            __syncwarp();
            if (lane == 0) pa::mbar_arrive(&ctl->unit_empty[slot]);
            if (!wait_for(&ctl->stats_full, nth & 1, ctl, a.status)) break;
            const float2 e = stats[r], o = stats[kRows + r];
            const bool unfinite = ctl->unfinite[nth & 1];
            float top0 = 1.f, top1 = 1.f;
            if constexpr (kScaled) {
                const float* tops = reinterpret_cast<const float*>(stats + 192);
                top0 = tops[r];
                top1 = tops[kRows + r];
            }
            pa::mbar_arrive(&ctl->stats_free);
            const float M = fmaxf(e.x, o.x), Z0 = pa::exp2_approx(e.x - M), Z1 = pa::exp2_approx(o.x - M);
            const float Z = Z0 * e.y + Z1 * o.y;
            const float by = whole ? (Z == 0.f ? 0.f : a.v_scale / Z) : 1.f;
            const bool none = kShaped && Z == 0.f;               // a row that sees nothing (and perhaps had no products)
            const float fe = Z0 * by, fo = Z1 * by;
            const size_t at = (size_t)(2 * blockIdx.x + (st0 == 0 ? 1 : 0)) * kRows + r;
            if (!wait_for(&ctl->o_done, nth & 1, ctl, a.status)) break;
            fence_after();
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                float v[32], v1[32];
                ld32(t_o + x, v);
                ld32(t_o + 128 + x, v1);
                wait_ld<32>(v);
                wait_ld<32>(v1);
                if (x == D - 32) {                               // O is in registers: the next unit's products may write it
                    fence_before();
                    pa::mbar_arrive(&ctl->o_free);
                }
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    v[k] = none ? 0.f
                         : kScaled ? fe * v[k] * top0 + (both ? fo * v1[k] * top1 : 0.f)   // (small scales last: their products are)
                                   : fe * v[k] + (both ? fo * v1[k] : 0.f);
                float f[kHalf ? 16 : 32];                         // of a row's two lanes, each writes half
                if constexpr (kHalf) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        // the other lane's sums of my half of the columns, for mine of its half
                        const float other = __shfl_xor_sync(0xffffffffu, second ? v[k] : v[k + 16], 16);
                        f[k] = (second ? v[k + 16] : v[k]) + other;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) f[k] = v[k];
                }
                if (real) {
                    const int col = x + (second ? 16 : 0);
#pragma unroll
                    for (int k = 0; k < (kHalf ? 16 : 32); k += 4) {
                        const float4 y = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
                        if (whole)
                            put4(a.out, a.out_f32, out_row + col + k, y);
                        else
                            *reinterpret_cast<float4*>(a.part_u + at * D + col + k) = y;
                    }
                }
            }
            if (!whole && real && !second) {
                a.part_m[at] = M;
                a.part_z[at] = Z;
            }
            if (__builtin_expect(unfinite, 0))
#pragma unroll 1
                for (int d = 0; d < D; d += 4)                   // (to what the thread itself has written)
                    if (!kHalf || (d & 16) == (lane & 16))
                        add_unfinite<D, F8>(a, seq, kvh, row, base + st0 * kKv, base + end * kKv, d, whole ? nullptr : a.part_u + at * D + d);
        }
    }
    fence_before();
    __syncthreads();
    if (warp == kScoreWarp) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

// 3-D view of q, [num_tokens][n_q_heads][d_head], in boxes of 16 rows of 64
// columns: 16 / group tokens of one KV head's group.
inline bool q_view(CUtensorMap* map, const void* q, int num_tokens, int n_q_heads, int d_head, int group) {
    const cuuint64_t dims[3] = {(cuuint64_t)d_head, (cuuint64_t)n_q_heads, (cuuint64_t)num_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d_head * 2, (cuuint64_t)d_head * n_q_heads * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)group, (cuuint32_t)(16 / group)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    auto encode = pa_host::tensor_map_encode();
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kHalf, bool F8, int kRuns = 1, class Args>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, int oob_row,
                   int grid, cudaStream_t st) {
    static int attr[64] = {0};
    constexpr int kSmem = Wide<D, kHalf, F8>::kSmem;
    const cudaError_t e = pa_host::ensure_smem_attr(wide_kernel<D, kHalf, F8, Args, kRuns>, kSmem, attr);
    if (e != cudaSuccess) return e;
    return pa_host::launch_dependent(wide_kernel<D, kHalf, F8, Args, kRuns>, dim3(grid), dim3(kThreads), kSmem, st, mq, mk, mv, a,
                                     oob_row);
}

template <class Args>
cudaError_t launch_units(int rows, int d_head, bool f8, const void* q, int block_size, const CUtensorMap& mk,
                         const CUtensorMap& mv, const Args& a, int grid, cudaStream_t st) {
    const int oob = a.num_blocks * a.n_kv_heads * block_size;    // one past the view's last row
    if (f8) {                                                    // (its q is not copied as it is)
        if constexpr (Args::kShaped) {
            if (block_size == 8) return launch<128, true, true, 4>(mk, mk, mv, a, oob, grid, st);
            if (block_size == 16) return launch<128, true, true, 2>(mk, mk, mv, a, oob, grid, st);
        }
        return launch<128, true, true>(mk, mk, mv, a, oob, grid, st);
    }
    CUtensorMap mq;
    if (!q_view(&mq, q, a.num_tokens, a.n_q_heads, d_head, 1 << a.log2_group)) return cudaErrorInvalidValue;
    return d_head == 128 ? (rows == 64 ? launch<128, true, false>(mq, mk, mv, a, oob, grid, st)
                                       : launch<128, false, false>(mq, mk, mv, a, oob, grid, st))
                         : (rows == 64 ? launch<64, true, false>(mq, mk, mv, a, oob, grid, st)
                                       : launch<64, false, false>(mq, mk, mv, a, oob, grid, st));
}


}  // namespace
