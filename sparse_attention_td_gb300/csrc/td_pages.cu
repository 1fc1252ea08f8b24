// td_pages.cu -- the cache side of a speculative-decoding step: block tables
// and slot maps from request lengths, the append of a packed batch of new K/V
// rows through a slot map, and the commit of the accepted drafted rows.
// All of them move whole values; what bounds them is launch latency for a
// decode step's few rows and the HBM copy rate for prompts.
#include <cuda_runtime.h>
#include <stdint.h>

#include "td_spec.h"

namespace td {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// Every kernel here is launched while the one before it in the stream may still
// end (programmatic serialization) and waits for it before it touches memory.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename Args, typename... More>
cudaError_t launch_behind(void (*kernel)(Args, More...), dim3 grid, int threads, cudaStream_t stream,
                          const Args &a, More... more)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = host_pdl();
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, more...);
}

constexpr int kRowChunks = kHeadDim / 8;      // 16-byte chunks of one row

// ------------------------------------------------------------ block tables
constexpr int kTableThreads = 1024;
// Up to this many slots the block-table CTA writes the slot map itself; more are
// a second kernel's.  Measured on GB300 (256 requests, own / second kernel): 1280
// slots 6.3 / 9.2 us, 4096 8.3 / 8.2, 8192 11.4 / 8.1.
constexpr int kOwnSlots = 4096;

template <typename T> __device__ __forceinline__ T scan_warp(T x, int lane)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(kAll, x, d);
        if (lane >= d)
            x += y;
    }
    return x;
}

// Exclusive prefix sum over the CTA's threads, and its total.
template <typename T> __device__ __forceinline__ T scan_block(T x, T *sm_warp, T &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T inc = scan_warp(x, lane);
    if (lane == 31)
        sm_warp[warp] = inc;
    __syncthreads();
    const T w = sm_warp[lane], winc = scan_warp(w, lane);
    total = __shfl_sync(kAll, winc, 31);
    const T before = __shfl_sync(kAll, winc - w, warp);
    __syncthreads();
    return before + inc - x;
}

// The last of n ascending values that is <= e (the first one is).
template <typename T> __device__ __forceinline__ int owner_of(const T *prefix, int n, T e)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= e)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

struct Want {
    int n, fresh, held, target;
};

__device__ __forceinline__ Want want_of(const TablesArgs &a, int b, uint32_t &bad)
{
    const int cap = a.max_blocks * a.page_size;
    const int n = a.seq_lens[b], fresh = a.new_lens[b], held = a.held[b];
    Want w;
    w.n = min(max(n, 0), cap);
    w.fresh = min(max(fresh, 0), w.n);
    w.held = min(max(held, 0), a.max_blocks);
    if (w.n != n || w.fresh != fresh)
        bad |= kFlagSeqLenOutOfRange;
    if (w.held != held)
        bad |= kFlagPageOutOfRange;
    w.target = (int)((w.n + a.page_size - 1u) / (unsigned)a.page_size);
    return w;
}

// Slot of position p of request b, which holds `held` pages.
__device__ __forceinline__ int slot_of(const TablesArgs &a, int b, int p, int held, uint32_t &bad)
{
    const int j = p / a.page_size;
    if (j >= held)
        return -1;
    const int page = a.table[(size_t)b * a.max_blocks + j];
    if (page < 0 || page >= a.num_pages) {
        bad |= kFlagPageOutOfRange;
        return -1;
    }
    return page * a.page_size + (p - j * a.page_size);
}

// Pages: one CTA, requests in chunks of its threads.  Pass 1 pushes what
// requests give back, pass 2 pops what they need, so a page given back in a
// call can be taken in the same call.  Each changed table entry is one
// thread's work (its request found by a search of the chunk's prefix sums), so
// one long prompt does not make one thread walk all of its pages.  What bounds
// it is the chain of dependent loads and barriers, not its bytes: 256 requests that
// grow by up to 9 tokens each 6.1 us, slot map included; 61 prompts of 1K to 8K
// tokens 10.0 us with the slot map's kernel.
__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(const TablesArgs a)
{
    __shared__ long long sm_warp64[32];
    __shared__ int sm_warp[32];
    __shared__ int sm_prefix[kTableThreads], sm_first[kTableThreads], sm_cu[kTableThreads];
    __shared__ int sm_fit;
    const int tid = threadIdx.x;
    wait_before();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the slot map's blocks may come
    uint32_t bad = 0;
    int count = *a.count;
    if (count < 0 || count > a.num_pages) {
        count = count < 0 ? 0 : a.num_pages;
        bad |= kFlagPageOutOfRange;
    }
    const bool single = a.B <= kTableThreads;
    Want w{};
    long long top = count;
    for (int b0 = 0; b0 < a.B; b0 += kTableThreads) {
        const int b = b0 + tid;
        w = Want{};
        if (b < a.B)
            w = want_of(a, b, bad);
        const int back = w.held > w.target ? w.held - w.target : 0;
        if (!__syncthreads_or(back))
            continue;
        int total;
        const int at = scan_block(back, sm_warp, total);
        sm_prefix[tid] = at;
        sm_first[tid] = w.target;
        __syncthreads();
        const int n = min(kTableThreads, a.B - b0);
        for (int e = tid; e < total; e += kTableThreads) {
            const int i = owner_of(sm_prefix, n, e);
            const int j = sm_first[i] + e - sm_prefix[i];
            if (top + e < a.num_pages)
                a.free_pages[top + e] = a.table[(size_t)(b0 + i) * a.max_blocks + j];
            else
                bad |= kFlagPageOutOfRange;   // more pages given back than there are
        }
        top = min(top + total, (long long)a.num_pages);
        __syncthreads();      // the pushes are visible to the pops
    }
    long long taken = 0, used = 0, fresh = 0;
    for (int b0 = 0; b0 < a.B; b0 += kTableThreads) {
        const int b = b0 + tid;
        if (!single) {
            w = Want{};
            if (b < a.B)
                w = want_of(a, b, bad);
        }
        const int need = w.target > w.held ? w.target - w.held : 0;
        int total;
        long long total_new;
        const int rel = scan_block(need, sm_warp, total);
        const long long cu = fresh + scan_block((long long)w.fresh, sm_warp64, total_new);
        const bool fits = taken + rel + need <= top;
        sm_prefix[tid] = rel;
        sm_first[tid] = w.held;
        sm_cu[tid] = (int)min(cu, 0x7fffffffLL);
        // pages popped in this chunk: up to the first request that does not fit
        int fit_end = total;
        if (taken + total > top) {            // (the same for all threads)
            if (tid == 0)
                sm_fit = total;
            __syncthreads();
            if (need && !fits) {
                bad |= kFlagPagesExhausted;
                atomicMin(&sm_fit, rel);
            }
            __syncthreads();
            fit_end = sm_fit;
        }
        if (need && fits)
            w.held = w.target;
        else if (!need)
            w.held = w.target;
        if (b < a.B) {
            a.held_out[b] = w.held;
            a.cu_new[b] = sm_cu[tid];
        }
        __syncthreads();
        const int n = min(kTableThreads, a.B - b0);
        constexpr int kAhead = 4;      // pops in flight per thread
        for (int e0 = tid; e0 < fit_end; e0 += kAhead * kTableThreads) {
            int page[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int e = e0 + u * kTableThreads;
                page[u] = e < fit_end ? a.free_pages[top - 1 - (taken + e)] : 0;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int e = e0 + u * kTableThreads;
                if (e >= fit_end)
                    break;
                const int i = owner_of(sm_prefix, n, e);
                const int j = sm_first[i] + e - sm_prefix[i];
                if (page[u] < 0 || page[u] >= a.num_pages)
                    bad |= kFlagPageOutOfRange;
                a.table[(size_t)(b0 + i) * a.max_blocks + j] = page[u];
            }
        }
        taken += total;
        used += fit_end;
        fresh += total_new;
        __syncthreads();
    }
    if (tid == 0) {
        a.cu_new[a.B] = (int)min(fresh, 0x7fffffffLL);
        *a.count_out = (int)(top - used);
        if (fresh > a.max_new)
            bad |= kFlagPagesExhausted;
    }
    if (single && a.max_new <= kOwnSlots) {
        // the slots of a decode step: the chunk's sums are still in shared memory
        sm_prefix[tid] = w.held;
        sm_first[tid] = w.n - w.fresh;
        __syncthreads();
        for (int i = tid; i < a.max_new; i += kTableThreads) {
            int slot = -1;
            if (i < fresh) {
                const int b = owner_of(sm_cu, a.B, i);
                slot = slot_of(a, b, sm_first[b] + i - sm_cu[b], sm_prefix[b], bad);
            }
            a.slots[i] = slot;
        }
    }
    if (bad)
        atomicOr(a.status, bad);
}

constexpr int kSlotThreads = 256;
constexpr int kSlotsPerThread = 4;

// The slots of prompts: what a block's tokens need of the batch's prefix sums is
// searched in shared memory where it fits.
__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const TablesArgs a)
{
    __shared__ int sm_cu[1024];
    wait_before();
    const int *cu = a.cu_new;
    const int total = a.cu_new[a.B];
    const int base = blockIdx.x * kSlotThreads * kSlotsPerThread;
    if (a.B <= 1024 && base < total) {
        for (int b = threadIdx.x; b < a.B; b += kSlotThreads)
            sm_cu[b] = a.cu_new[b];
        __syncthreads();
        cu = sm_cu;
    }
    const int cap = a.max_blocks * a.page_size;
    uint32_t bad = 0;
#pragma unroll
    for (int u = 0; u < kSlotsPerThread; ++u) {
        const int i = base + u * kSlotThreads + threadIdx.x;
        if (i >= a.max_new)
            break;
        int slot = -1;
        if (i < total) {
            const int b = owner_of(cu, a.B, i);
            const int n = min(max(a.seq_lens[b], 0), cap), fresh = min(max(a.new_lens[b], 0), n);
            slot = slot_of(a, b, n - fresh + i - cu[b], a.held_out[b], bad);
        }
        a.slots[i] = slot;
    }
    if (bad)
        atomicOr(a.status, bad);
}

// -------------------------------------------------------------- slot append
// One thread per 16 bytes: consecutive threads take consecutive chunks of a
// token's K row (all heads), then of its V row.  32749 tokens of 8 KV heads (268 MB
// read and written) take 44 us, 6.0 TB/s, bound by HBM; 257 tokens 1.6 us, a launch.
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) append_slots_kernel(const AppendSlotsArgs a)
{
    wait_before();
    const int per = a.Hkv * kRowChunks;                 // chunks of one token's K (or V)
    const long long total = (long long)a.tokens * 2 * per;
    const long long limit = (long long)a.num_pages * a.page_size;
    for (long long e = (long long)blockIdx.x * kAppendThreads + threadIdx.x; e < total;
         e += (long long)gridDim.x * kAppendThreads) {
        const int i = (int)(e / (2 * per));
        int c = (int)(e - (long long)i * 2 * per);
        const bool isv = c >= per;
        c -= isv ? per : 0;
        const int slot = a.slots[i];
        if (slot < 0 || slot >= limit)
            continue;
        const uint16_t *src = (isv ? a.v_new : a.k_new) + (size_t)i * a.new_stride + c * 8;
        const int page = slot / a.page_size, r = slot % a.page_size;
        uint16_t *dst = (isv ? a.v : a.k) +
                        (((size_t)page * a.Hkv + c / kRowChunks) * a.page_size + r) * kHeadDim +
                        (c % kRowChunks) * 8;
        *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(src);
    }
}

// ------------------------------------------------------------------- commit
// A CTA takes the accepted rows of one request for up to kCommitTasks (layer, KV
// head, K or V) tasks per warp, fewer where the launch has few CTAs: the rows are
// found once, then each warp moves its tasks' rows, half a warp per 256-byte row.  A row may be both a source and a
// destination.  Where no accepted token comes before its place (a path of a tree
// whose parents have lower numbers), sixteen rows at a time can be read and then
// written in order: a later source lies behind every earlier destination.  In any
// other order the whole CTA holds all rows of a task before it writes any.
// Bound by latency: one dependent read behind the row search, then the write.
// 32 requests x 32 layers x 8 KV heads, trees of 32 (71 MB): 14.9 us, 4.8 TB/s;
// 3 requests x 4 layers 2.3 us.  The first at 4 / 3 / 2 tasks per warp: 15.4 /
// 16.9 / 15.7 us (launched in plain stream order).
constexpr int kCommitWarps = 8;
constexpr int kCommitTasks = 4;
constexpr int kCommitRows = 16;       // rows a warp holds at a time

__global__ void __launch_bounds__(32 * kCommitWarps) tree_commit_kernel(const CommitArgs a, int tasks, int per_warp)
{
    __shared__ long long sm_src[TD_MAX_TREE], sm_dst[TD_MAX_TREE];   // cache rows of KV head 0, -1: stays
    __shared__ int sm_behind, sm_moves;
    const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t bad = 0;
    wait_before();
    const TreeLens len = tree_lens_of(a.seq_lens, a.tree_lens, b, a.T, a.Nmax, bad);
    const int ctx = len.n - len.nt;
    const int raw = a.accepted_lens[b];
    const int acc = min(max(raw, 0), len.nt);
    if (acc != raw)
        bad |= kFlagTreeOutOfRange;
    if (tid == 0) {
        sm_behind = sm_moves = 0;
        if (blockIdx.x == 0 && a.seq_lens_out)
            a.seq_lens_out[b] = ctx + acc;
    }
    __syncthreads();
    auto row_of = [&](int p) -> long long {   // of KV head 0; -1: no such page
        long long page = b;
        int r = p;
        if (a.table) {
            page = a.table[(size_t)b * a.max_blocks + p / a.page_size];
            r = p % a.page_size;
        }
        return page < 0 || page >= a.num_pages ? -1 : page * a.Hkv * a.page_size + r;
    };
    for (int i = tid; i < acc; i += 32 * kCommitWarps) {
        const int j = a.accepted[(size_t)b * a.T + i];
        long long src = -1, dst = -1;
        if (j < 0 || j >= len.nt) {
            bad |= kFlagTreeOutOfRange;
        } else {
            src = row_of(ctx + j);
            dst = row_of(ctx + i);
            if (src < 0 || dst < 0)
                bad |= kFlagPageOutOfRange;
            if (j == i || src < 0 || dst < 0)
                dst = -1;
            else if (j < i)
                sm_behind = 1;
        }
        sm_src[i] = src;
        sm_dst[i] = dst;
        if (dst >= 0)
            sm_moves = 1;
    }
    __syncthreads();
    if (bad && blockIdx.x == 0)
        atomicOr(a.status, bad);
    if (!sm_moves)
        return;
    const int hi = lane >> 4, c = lane & 15;
    const int task0 = (blockIdx.x * kCommitWarps + warp) * per_warp;
    const bool in_order = !sm_behind;
    // task: layer, then K or V, then head (neighbouring warps read neighbouring rows)
    auto rows_of = [&](int task, int c) {
        const int g = task % a.Hkv, kv = task / a.Hkv & 1, l = task / a.Hkv >> 1;
        return (kv ? a.v[l] : a.k[l]) + (size_t)g * a.page_size * kHeadDim + c * 8;
    };
    if (in_order) {
        for (int task = task0; task < min(task0 + per_warp, tasks); ++task) {
            uint16_t *rows = rows_of(task, c);
#pragma unroll 1
            for (int i0 = 0; i0 < acc; i0 += kCommitRows) {
                uint4 x[kCommitRows / 2];
#pragma unroll
                for (int u = 0; u < kCommitRows / 2; ++u) {
                    const int i = i0 + 2 * u + hi;
                    if (i < acc && sm_dst[i] >= 0)
                        x[u] = *reinterpret_cast<const uint4 *>(rows + sm_src[i] * kHeadDim);
                }
                __syncwarp();
#pragma unroll
                for (int u = 0; u < kCommitRows / 2; ++u) {
                    const int i = i0 + 2 * u + hi;
                    if (i < acc && sm_dst[i] >= 0)
                        *reinterpret_cast<uint4 *>(rows + sm_dst[i] * kHeadDim) = x[u];
                }
                __syncwarp();
            }
        }
        return;
    }
    const int first = blockIdx.x * kCommitWarps * per_warp;
    constexpr int kHold = TD_MAX_TREE / (2 * kCommitWarps);
    for (int task = first; task < min(first + kCommitWarps * per_warp, tasks); ++task) {
        uint16_t *rows = rows_of(task, c);
        uint4 x[kHold];
#pragma unroll
        for (int u = 0; u < kHold; ++u) {
            const int i = 2 * (u * kCommitWarps + warp) + hi;
            if (i < acc && sm_dst[i] >= 0)
                x[u] = *reinterpret_cast<const uint4 *>(rows + sm_src[i] * kHeadDim);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kHold; ++u) {
            const int i = 2 * (u * kCommitWarps + warp) + hi;
            if (i < acc && sm_dst[i] >= 0)
                *reinterpret_cast<uint4 *>(rows + sm_dst[i] * kHeadDim) = x[u];
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_block_tables(const TablesArgs &a, cudaStream_t stream)
{
    const cudaError_t err = launch_behind(block_tables_kernel, dim3(1), kTableThreads, stream, a);
    if (err != cudaSuccess || a.max_new == 0 || (a.B <= kTableThreads && a.max_new <= kOwnSlots))
        return err;
    constexpr int kPer = kSlotThreads * kSlotsPerThread;
    const dim3 grid((unsigned)(((long long)a.max_new + kPer - 1) / kPer));
    return launch_behind(slot_map_kernel, grid, kSlotThreads, stream, a);
}

cudaError_t launch_append_slots(const AppendSlotsArgs &a, cudaStream_t stream)
{
    const long long total = (long long)a.tokens * 2 * a.Hkv * kRowChunks;
    const long long most = (long long)host_sm_count() * 8;
    long long grid = (total + kAppendThreads - 1) / kAppendThreads;
    if (grid > most)
        grid = most;
    return launch_behind(append_slots_kernel, dim3((unsigned)grid), kAppendThreads, stream, a);
}

cudaError_t launch_tree_commit(const CommitArgs &a, int num_layers, cudaStream_t stream)
{
    const int tasks = num_layers * 2 * a.Hkv;
    const long long fill = (long long)host_sm_count() * 2 * kCommitWarps;   // two CTAs per SM
    int per_warp = (int)((long long)tasks * a.B / fill);
    per_warp = per_warp < 1 ? 1 : per_warp > kCommitTasks ? kCommitTasks : per_warp;
    const int per = kCommitWarps * per_warp;
    return launch_behind(tree_commit_kernel, dim3((tasks + per - 1) / per, a.B), 32 * kCommitWarps, stream, a,
                         tasks, per_warp);
}

}  // namespace td
