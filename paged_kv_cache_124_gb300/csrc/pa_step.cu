// A serving step's metadata on the GPU: block tables, slots and positions of
// the step's new tokens, from the requests' lengths and the pool's free
// blocks ("PagedAttention: Virtual Memory for the KV Cache", sections 7, 15
// and 20: translation, append, the free list as a stack).
//
// Request i of the batch holds L cached positions in h blocks and brings n
// new ones:
//   need_i = max(0, ceil((L + n) / B) - h)          blocks it takes
//   first_i = need_0 + ... + need_{i-1}             where its blocks start
//   entry h + k = free[count - 1 - (first_i + k)]   the stack's order
//   slot(p) = entry[p / B] * B + p % B              of each new position p
//
// Nothing may be written before the totals say whether the step fits, and no
// block may change a count that another still has to read.  Up to 2048
// requests, one cluster of eight thread blocks does it all: each scans the
// whole batch for itself, a cluster barrier stands between the reads of the
// state and its change, and then each expands its share of tables, positions
// and slots.  Larger steps take two launches: one block scans and takes the
// blocks, and a grid expands from its outputs alone.  Either way there is no
// scratch memory to share or to reset, so two captured graphs never meet in
// one.

#include "pa_common.cuh"

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = 8;                            // requests per thread, at most
constexpr int kPlanMaxSeqs = kPlanThreads * kPlanPer;
constexpr int kPlanMaxRows = 1 << 18;                  // one bit each in shared memory
constexpr int kExpandThreads = 256;

struct PlanArgs {
    const int32_t* seq_rows;
    const int32_t* new_lens;
    const int32_t* row_lens;
    int32_t* row_tables;
    int32_t* row_blocks;
    const int32_t* free_blocks;
    int32_t* free_count;
    int32_t* block_tables;
    int32_t* context_lens;
    int32_t* query_start;
    int32_t* positions;
    int64_t* slot_mapping;
    int32_t* status;
    int num_seqs, num_rows, max_blocks, free_capacity, num_blocks, log2_block, num_tokens;
};

// Exclusive scan of one pair per thread over the block; the totals go to
// every thread.
__device__ __forceinline__ void scan_pair(long long& a, long long& b, long long& total_a, long long& total_b,
                                          long long (*sh)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        sh[warp][0] = a;
        sh[warp][1] = b;
    }
    __syncthreads();
    if (warp == 0) {
        long long x = sh[lane][0], y = sh[lane][1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) {
                x += u;
                y += v;
            }
        }
        sh[lane][0] = x;
        sh[lane][1] = y;
    }
    __syncthreads();
    total_a = sh[kPlanThreads / 32 - 1][0];
    total_b = sh[kPlanThreads / 32 - 1][1];
    a = a - a0 + (warp ? sh[warp - 1][0] : 0);
    b = b - b0 + (warp ? sh[warp - 1][1] : 0);
}

// Largest i with starts[i] <= x, for starts[0] <= x (entries non-decreasing).
__device__ __forceinline__ int last_start(const int32_t* starts, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Thread t's kPer requests (entries [t * per, (t + 1) * per) of the batch) and
// what is wrong with the step; `seen`: a zeroed bit per row in shared memory.
template <int kPer>
struct Requests {
    int row[kPer], len[kPer], n[kPer], held[kPer], need[kPer];   // row -1: padding
    long long sum_n = 0, sum_need = 0;
    int bad = 0;

    __device__ __forceinline__ void read(const PlanArgs& a, int per, uint32_t* seen) {
        const long long cap = (long long)a.max_blocks << a.log2_block;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = threadIdx.x * per + k;
            row[k] = -1;
            len[k] = n[k] = held[k] = need[k] = 0;
            if (k >= per || i >= a.num_seqs) continue;
            const int r = a.seq_rows[i], m = a.new_lens[i];
            if (r < 0) continue;                       // padding of the batch
            if (r >= a.num_rows) {
                bad |= PA_DEV_BAD_ROW;
                continue;
            }
            if (atomicOr(&seen[r >> 5], 1u << (r & 31)) >> (r & 31) & 1u) bad |= PA_DEV_BAD_ROW;
            const int L = a.row_lens[r], h = a.row_blocks[r];
            if (L < 0 || L > cap) {
                bad |= PA_DEV_BAD_CONTEXT;
                continue;
            }
            // whatever else is wrong refuses the step, and a refused step shows what the row has: the same for every
            // entry that names it, whichever of them is the first to mark it
            row[k] = r;
            len[k] = L;
            if (h < 0 || h > a.max_blocks || m < 0 || (long long)L + m > cap) {
                bad |= PA_DEV_BAD_CONTEXT;
                continue;
            }
            n[k] = m;
            held[k] = h;
            const int nb = (int)(((long long)L + m + (1 << a.log2_block) - 1) >> a.log2_block);
            need[k] = nb > h ? nb - h : 0;
            sum_n += m;
            sum_need += need[k];
        }
    }
};

// What is wrong with the step's totals.
__device__ __forceinline__ int bad_totals(const PlanArgs& a, long long n, long long need, int count) {
    return (n > a.num_tokens ? PA_DEV_BAD_CONTEXT : 0) |
           (need > 0 && (count > a.free_capacity || need > count) ? PA_DEV_NO_BLOCKS : 0);
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
    extern __shared__ uint32_t dyn[];                  // first_[num_seqs], then a bit per row
    __shared__ long long sh[32][2];
    int32_t* first_ = reinterpret_cast<int32_t*>(dyn);
    uint32_t* seen = dyn + a.num_seqs;
    const int S = a.num_seqs, t = threadIdx.x;
    for (int i = t; i < (a.num_rows + 31) / 32; i += kPlanThreads) seen[i] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    const int per = (S + kPlanThreads - 1) / kPlanThreads;
    Requests<kPlanPer> q;
    q.read(a, per, seen);
    long long base_n = q.sum_n, base_need = q.sum_need, total_n, total_need;
    scan_pair(base_n, base_need, total_n, total_need, sh);
    const int count = a.free_count ? *a.free_count : 0;
    const int bad = q.bad | bad_totals(a, total_n, total_need, count);
    // all or nothing: every request of a refused step keeps what it has and brings nothing
    const bool refused = __syncthreads_or(bad);
    if (bad) pa::set_status(a.status, bad);
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
        const int i = t * per + k;
        if (k >= per || i >= S) continue;
        a.context_lens[i] = q.len[k] + (refused ? 0 : q.n[k]);
        a.query_start[i] = refused ? 0 : (int)base_n;
        first_[i] = (int)base_need;
        base_n += q.n[k];
        base_need += q.need[k];
    }
    if (refused) {
        if (t == 0) a.query_start[S] = 0;
        return;
    }
    if (t == 0) a.query_start[S] = (int)total_n;
    if (total_need == 0) return;
    __syncthreads();
    // the step's blocks, in the order they are taken, over all threads
    for (int k = t; k < total_need; k += kPlanThreads) {
        const int i = last_start(first_, S, k);
        const int r = a.seq_rows[i];
        a.row_tables[(size_t)r * a.max_blocks + a.row_blocks[r] + (k - first_[i])] = a.free_blocks[count - 1 - k];
    }
    __syncthreads();                                   // every thread has read the counts it needs
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k)
        if (q.need[k]) a.row_blocks[q.row[k]] += q.need[k];
    if (t == 0) *a.free_count = count - (int)total_need;
}

// Blocks [0, table_blocks): one warp per 1024 entries of a batch row's table;
// the rest: one thread per token.
constexpr int kSegment = 1024;

__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const PlanArgs a, int table_blocks, int segments) {
    extern __shared__ int32_t starts[];                // [num_seqs] (token blocks)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int S = a.num_seqs, B = 1 << a.log2_block;
    if ((int)blockIdx.x < table_blocks) {
        const int w = blockIdx.x * (kExpandThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
        const int i = w / segments, j0 = (w - i * segments) * kSegment;
        if (i >= S) return;
        const int r = a.seq_rows[i];
        const int nb = (r < 0 || r >= a.num_rows) ? 0 : (int)(((long long)a.context_lens[i] + B - 1) >> a.log2_block);
        const int32_t* src = a.row_tables + (size_t)(nb ? r : 0) * a.max_blocks;
        int32_t* dst = a.block_tables + (size_t)i * a.max_blocks;
        const int end = min(j0 + kSegment, a.max_blocks);
        if ((a.max_blocks & 3) == 0) {
            for (int j = j0 + 4 * lane; j < end; j += 128) {
                int4 x = make_int4(-1, -1, -1, -1);
                if (j < nb) {
                    x = *reinterpret_cast<const int4*>(src + j);
                    if (j + 1 >= nb) x.y = -1;
                    if (j + 2 >= nb) x.z = -1;
                    if (j + 3 >= nb) x.w = -1;
                }
                *reinterpret_cast<int4*>(dst + j) = x;
            }
        } else {
            for (int j = j0 + lane; j < end; j += 32) dst[j] = j < nb ? src[j] : -1;
        }
        return;
    }
    for (int i = threadIdx.x; i < S; i += kExpandThreads) starts[i] = a.query_start[i];
    const int total = a.query_start[S];
    __syncthreads();
    const int t = (blockIdx.x - table_blocks) * kExpandThreads + threadIdx.x;
    if (t >= a.num_tokens) return;
    int pos = -1;
    long long slot = -1;
    if (t < total) {
        const int i = last_start(starts, S, t);        // the last request that starts at or before t: it has t
        const int n = (i + 1 < S ? starts[i + 1] : total) - starts[i];
        pos = a.context_lens[i] - n + (t - starts[i]);
        const int blk = a.row_tables[(size_t)a.seq_rows[i] * a.max_blocks + (pos >> a.log2_block)];
        if (blk < 0 || blk >= a.num_blocks)
            pa::set_status(a.status, PA_DEV_BAD_BLOCK_ID);
        else
            slot = ((long long)blk << a.log2_block) + (pos & (B - 1));
    }
    a.positions[t] = pos;
    a.slot_mapping[t] = slot;
}

// The whole step in one cluster, for up to kFusedSeqs requests.
constexpr int kFusedSeqs = 2048;
constexpr int kFusedPer = kFusedSeqs / kPlanThreads;
constexpr int kCluster = 8;

struct Planned {
    int row, ctx, held, first;             // row -1: padding; entries from `held` on are the step's
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads, 1) fused_plan_kernel(const PlanArgs a) {
    extern __shared__ uint32_t dyn[];      // Planned[S], start[S + 1], a bit per row
    __shared__ long long sh[32][2];
    const int S = a.num_seqs, t = threadIdx.x, me = blockIdx.x * kPlanThreads + t;
    Planned* plan = reinterpret_cast<Planned*>(dyn);
    int32_t* start = reinterpret_cast<int32_t*>(plan + S);
    uint32_t* seen = reinterpret_cast<uint32_t*>(start + S + 1);
    for (int i = t; i < (a.num_rows + 31) / 32; i += kPlanThreads) seen[i] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    const int per = (S + kPlanThreads - 1) / kPlanThreads, B = 1 << a.log2_block;
    const int count = a.free_count ? *a.free_count : 0;
    Requests<kFusedPer> q;
    q.read(a, per, seen);
    long long base_n = q.sum_n, base_need = q.sum_need, total_n, total_need;
    scan_pair(base_n, base_need, total_n, total_need, sh);
    const int bad = q.bad | bad_totals(a, total_n, total_need, count);
    // all or nothing: every request of a refused step keeps what it has and brings nothing
    const bool refused = __syncthreads_or(bad);
    if (bad && blockIdx.x == 0) pa::set_status(a.status, bad);
#pragma unroll
    for (int k = 0; k < kFusedPer; ++k) {
        const int i = t * per + k;
        if (k >= per || i >= S) continue;
        // (a refused step's tables are what the rows have, even where that is too little for their lengths)
        plan[i] = Planned{q.row[k], q.len[k] + (refused ? 0 : q.n[k]), refused ? a.max_blocks : q.held[k], (int)base_need};
        start[i] = refused ? 0 : (int)base_n;
        base_n += q.n[k];
        base_need += q.need[k];
    }
    const int total = refused ? 0 : (int)total_n;
    if (t == 0) start[S] = total;
    __syncthreads();
    // every block of the cluster has read the counts
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    // block b of a request: one that it holds, or the step's
    auto entry = [&](const Planned& p, int b) {
        return b < p.held ? a.row_tables[(size_t)p.row * a.max_blocks + b]
                          : a.free_blocks[count - 1 - (p.first + b - p.held)];
    };
    constexpr int kAll = kCluster * kPlanThreads;
    for (int i = me; i < S; i += kAll) {
        const Planned p = plan[i];
        a.context_lens[i] = p.ctx;
        a.query_start[i] = start[i];
        const int nb = (p.ctx + B - 1) >> a.log2_block;
        if (!refused && p.row >= 0 && nb > p.held) a.row_blocks[p.row] = nb;
    }
    if (me == 0) {
        a.query_start[S] = total;
        if (!refused && total_need > 0) *a.free_count = count - (int)total_need;
    }
    // tables: a warp per 1024 entries of a batch row; the step's blocks go into the request's own table too
    const int lane = t & 31, segments = (a.max_blocks + kSegment - 1) / kSegment;
    for (int w = me >> 5; w < S * segments; w += kAll / 32) {
        const int i = w / segments, j0 = (w - i * segments) * kSegment, end = min(j0 + kSegment, a.max_blocks);
        const Planned p = plan[i];
        const int nb = p.row < 0 ? 0 : (p.ctx + B - 1) >> a.log2_block, old = min(nb, p.held);
        int32_t* dst = a.block_tables + (size_t)i * a.max_blocks;
        int32_t* own = a.row_tables + (size_t)(p.row < 0 ? 0 : p.row) * a.max_blocks;
        const bool wide = (a.max_blocks & 3) == 0;
        if (wide) {
            for (int j = j0 + 4 * lane; j < end; j += 128) {
                int4 x = make_int4(-1, -1, -1, -1);
                if (j < old) {
                    x = *reinterpret_cast<const int4*>(own + j);
                    if (j + 1 >= old) x.y = -1;
                    if (j + 2 >= old) x.z = -1;
                    if (j + 3 >= old) x.w = -1;
                }
                if (j + 3 < p.held || j >= nb) {
                    *reinterpret_cast<int4*>(dst + j) = x;
                } else {                   // some of the four are the step's
                    const int v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        int id = v[e];
                        if (j + e >= p.held && j + e < nb) own[j + e] = id = entry(p, j + e);
                        dst[j + e] = id;
                    }
                }
            }
        } else {
            for (int j = j0 + lane; j < end; j += 32) {
                int id = j < old ? own[j] : -1;
                if (j >= p.held && j < nb) own[j] = id = entry(p, j);
                dst[j] = id;
            }
        }
    }
    for (int x = me; x < a.num_tokens; x += kAll) {
        int pos = -1;
        long long slot = -1;
        if (x < total) {
            const int i = last_start(start, S, x);     // the last request that starts at or before x: it has x
            const Planned p = plan[i];
            pos = p.ctx - (start[i + 1] - x);
            const int blk = entry(p, pos >> a.log2_block);
            if (blk < 0 || blk >= a.num_blocks)
                pa::set_status(a.status, PA_DEV_BAD_BLOCK_ID);
            else
                slot = ((long long)blk << a.log2_block) + (pos & (B - 1));
        }
        a.positions[x] = pos;
        a.slot_mapping[x] = slot;
    }
}

// Rows given back: their blocks go onto the stack in table order, row after
// row, as the host manager's release does.  One block whatever the size: 4 rows
// of 50 blocks 3.3 us, 32 3.8, 256 10.9, 1000 38, 8000 of 5 blocks 47; a search
// of the row and two dependent accesses a block, so 1000 rows of 5 take 7.3.
__global__ void __launch_bounds__(kPlanThreads) release_kernel(const int32_t* rows, int num, const int32_t* row_tables,
                                                               int32_t* row_blocks, int num_rows, int max_blocks,
                                                               int32_t* free_blocks, int32_t* free_count,
                                                               int free_capacity, int32_t* status) {
    extern __shared__ uint32_t dyn[];                  // first_[num], then a bit per row
    __shared__ long long sh[32][2];
    int32_t* first_ = reinterpret_cast<int32_t*>(dyn);
    uint32_t* seen = dyn + num;
    const int t = threadIdx.x;
    for (int i = t; i < (num_rows + 31) / 32; i += kPlanThreads) seen[i] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    const int per = (num + kPlanThreads - 1) / kPlanThreads;
    int held[kPlanPer];
    int bad = 0;
    long long mine = 0;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
        const int i = t * per + k;
        held[k] = 0;
        if (k >= per || i >= num) continue;
        const int r = rows[i];
        if (r < 0) continue;
        if (r >= num_rows || (atomicOr(&seen[r >> 5], 1u << (r & 31)) >> (r & 31) & 1u)) {
            bad |= PA_DEV_BAD_ROW;
            continue;
        }
        held[k] = row_blocks[r];
        if (held[k] < 0 || held[k] > max_blocks) bad |= PA_DEV_BAD_CONTEXT;
        mine += held[k];
    }
    long long base = mine, other = 0, total, unused;
    scan_pair(base, other, total, unused, sh);
    const int count = *free_count;
    if (count < 0 || count + total > free_capacity) bad |= PA_DEV_BAD_CONTEXT;
    if (__syncthreads_or(bad)) {
        if (bad) pa::set_status(status, bad);
        return;
    }
    long long at = base;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
        const int i = t * per + k;
        if (k >= per || i >= num) continue;
        first_[i] = (int)at;
        at += held[k];
    }
    __syncthreads();
    for (int k = t; k < total; k += kPlanThreads) {
        const int i = last_start(first_, num, k);
        free_blocks[count + k] = row_tables[(size_t)rows[i] * max_blocks + (k - first_[i])];
    }
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k)
        if (held[k]) row_blocks[rows[t * per + k]] = 0;
    if (t == 0) *free_count = count + (int)total;
}

// Shared memory of the kernels for a call's sizes.  Past 40 KiB a kernel is
// given what its largest call needs, whatever this one does: threads that call
// with different sizes then never set a limit below one that another relies on.
constexpr int fused_smem(int seqs, int rows) { return (int)sizeof(Planned) * seqs + 4 * (seqs + 1) + 4 * ((rows + 31) / 32); }
constexpr int list_smem(int seqs, int rows) { return 4 * seqs + 4 * ((rows + 31) / 32); }

template <typename K>
bool has_smem(K kernel, int bytes, int most, int* granted) {
    return bytes <= 40 * 1024 || pa_host::ensure_smem_attr(kernel, most, granted) == cudaSuccess;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

int pa_plan_step(int32_t* block_tables, int32_t* context_lens, int32_t* query_start, int32_t* positions,
                 int64_t* slot_mapping, const int32_t* seq_rows, const int32_t* new_lens, const int32_t* row_lens,
                 int32_t* row_tables, int32_t* row_blocks, const int32_t* free_blocks, int32_t* free_count,
                 int free_capacity, int num_seqs, int num_rows, int max_blocks_per_seq, int num_tokens,
                 int block_size, int num_blocks, int32_t* status_dev, void* stream) {
    if (num_seqs < 0 || num_rows <= 0 || max_blocks_per_seq <= 0 || num_tokens < 0 || num_blocks <= 0 ||
        free_capacity < 0)
        return PA_ERR_INVALID_ARG;
    if (!pa_host::supported_block_size(block_size)) return PA_ERR_UNSUPPORTED;
    if (num_seqs > kPlanMaxSeqs || num_rows > kPlanMaxRows ||
        (long long)max_blocks_per_seq * block_size > 0x7fffffffLL)
        return PA_ERR_UNSUPPORTED;
    if (!query_start || (num_seqs > 0 && (!block_tables || !context_lens || !seq_rows || !new_lens || !row_lens ||
                                          !row_tables || !row_blocks)) ||
        (num_tokens > 0 && (!positions || !slot_mapping)) || ((free_blocks == nullptr) != (free_count == nullptr)))
        return PA_ERR_INVALID_ARG;
    if (!pa_host::aligned16(block_tables) || !pa_host::aligned16(row_tables) || !aligned4(context_lens) ||
        !aligned4(query_start) || !aligned4(positions) || !aligned4(seq_rows) || !aligned4(new_lens) ||
        !aligned4(row_lens) || !aligned4(row_blocks) || !aligned4(free_blocks) || !aligned4(free_count) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PA_ERR_MISALIGNED;
    PlanArgs a{};
    a.seq_rows = seq_rows;
    a.new_lens = new_lens;
    a.row_lens = row_lens;
    a.row_tables = row_tables;
    a.row_blocks = row_blocks;
    a.free_blocks = free_blocks;
    a.free_count = free_count;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.positions = positions;
    a.slot_mapping = slot_mapping;
    a.status = status_dev;
    a.num_seqs = num_seqs;
    a.num_rows = num_rows;
    a.max_blocks = max_blocks_per_seq;
    a.free_capacity = free_capacity;
    a.num_blocks = num_blocks;
    a.log2_block = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    a.num_tokens = num_tokens;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // One cluster is faster while its eight SMs keep up with the tables and
    // the tokens: 4 requests 4.7 us against 5.8, 256 of up to 256 blocks 6.0 /
    // 7.4, of 1024 7.6 / 8.3, 512 of 256 7.2 / 7.9, 1024 of 256 9.9 / 8.4,
    // 1000 of 2048 24 / 8.7 (one new token each, and behind a copy of some 1.3
    // to 1.6 us; 1000 of 2048 that bring 32,048 tokens take 11.6 without it).
    if (num_seqs <= kFusedSeqs && (long long)num_seqs * max_blocks_per_seq + 8LL * num_tokens <= 270000) {
        static int attr_fused[64] = {0};
        const int smem = fused_smem(num_seqs, num_rows);
        if (!has_smem(fused_plan_kernel, smem, fused_smem(kFusedSeqs, kPlanMaxRows), attr_fused)) return PA_ERR_CUDA;
        return pa_host::launch_dependent(fused_plan_kernel, dim3(kCluster), dim3(kPlanThreads), smem, st, a) == cudaSuccess
                   ? PA_OK
                   : PA_ERR_CUDA;
    }
    static int attr_plan[64] = {0};
    const int smem = list_smem(num_seqs, num_rows);
    if (!has_smem(plan_kernel, smem, list_smem(kPlanMaxSeqs, kPlanMaxRows), attr_plan)) return PA_ERR_CUDA;
    if (pa_host::launch_dependent(plan_kernel, dim3(1), dim3(kPlanThreads), smem, st, a) != cudaSuccess)
        return PA_ERR_CUDA;
    const int segments = (max_blocks_per_seq + kSegment - 1) / kSegment;
    const long long warps = (long long)num_seqs * segments;
    const int table_blocks = (int)((warps + kExpandThreads / 32 - 1) / (kExpandThreads / 32));
    const int token_blocks = (int)(((long long)num_tokens + kExpandThreads - 1) / kExpandThreads);
    if (table_blocks + token_blocks == 0) return PA_OK;
    return pa_host::launch_dependent(expand_kernel, dim3(table_blocks + token_blocks), dim3(kExpandThreads),
                                     4 * num_seqs, st, a, table_blocks, segments) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

int pa_release_rows(const int32_t* rows, int num_released, const int32_t* row_tables, int32_t* row_blocks,
                    int num_rows, int max_blocks_per_seq, int32_t* free_blocks, int32_t* free_count,
                    int free_capacity, int32_t* status_dev, void* stream) {
    if (num_released < 0 || num_rows <= 0 || max_blocks_per_seq <= 0 || free_capacity < 0) return PA_ERR_INVALID_ARG;
    if (num_released > kPlanMaxSeqs || num_rows > kPlanMaxRows) return PA_ERR_UNSUPPORTED;
    if (num_released == 0) return PA_OK;
    if (!rows || !row_tables || !row_blocks || !free_blocks || !free_count) return PA_ERR_INVALID_ARG;
    if (!aligned4(rows) || !aligned4(row_tables) || !aligned4(row_blocks) || !aligned4(free_blocks) ||
        !aligned4(free_count))
        return PA_ERR_MISALIGNED;
    static int attr_release[64] = {0};
    const int smem = list_smem(num_released, num_rows);
    if (!has_smem(release_kernel, smem, list_smem(kPlanMaxSeqs, kPlanMaxRows), attr_release)) return PA_ERR_CUDA;
    return pa_host::launch_dependent(release_kernel, dim3(1), dim3(kPlanThreads), smem,
                                     static_cast<cudaStream_t>(stream), rows, num_released, row_tables, row_blocks,
                                     num_rows, max_blocks_per_seq, free_blocks, free_count, free_capacity,
                                     status_dev) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // extern "C"
