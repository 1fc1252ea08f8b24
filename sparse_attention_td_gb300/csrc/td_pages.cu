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
constexpr int kRowChunks = kHeadDim / 8;      // 16-byte chunks of one row

// ------------------------------------------------------------ block tables
constexpr int kTableThreads = 1024;

// Exclusive prefix sum over the CTA's threads, and its total.
__device__ __forceinline__ long long block_scan(long long x, long long *sm_warp, long long &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(kAll, inc, d);
        if (lane >= d)
            inc += y;
    }
    if (lane == 31)
        sm_warp[warp] = inc;
    __syncthreads();
    long long w = sm_warp[lane];
    long long winc = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(kAll, winc, d);
        if (lane >= d)
            winc += y;
    }
    total = __shfl_sync(kAll, winc, 31);
    const long long before = __shfl_sync(kAll, winc - w, warp);
    __syncthreads();
    return before + inc - x;
}

// The last request of the chunk whose prefix is <= e (prefix[0] = 0, ascending).
__device__ __forceinline__ int owner_of(const long long *prefix, int n, long long e)
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
    Want w;
    int raw = a.seq_lens[b];
    w.n = raw < 0 ? 0 : (raw > cap ? cap : raw);
    if (w.n != raw)
        bad |= kFlagSeqLenOutOfRange;
    raw = a.new_lens[b];
    w.fresh = raw < 0 ? 0 : (raw > w.n ? w.n : raw);
    if (w.fresh != raw)
        bad |= kFlagSeqLenOutOfRange;
    raw = a.held[b];
    w.held = raw < 0 ? 0 : (raw > a.max_blocks ? a.max_blocks : raw);
    if (w.held != raw)
        bad |= kFlagPageOutOfRange;
    w.target = (int)(((long long)w.n + a.page_size - 1) / a.page_size);
    return w;
}

// Pages: one CTA, requests in chunks of its threads.  Pass 1 pushes what
// requests give back, pass 2 pops what they need, so a page given back in a
// call can be taken in the same call.  Each changed table entry is one
// thread's work (its request found by a search of the chunk's prefix sums), so
// one long prompt does not make one thread walk all of its pages.
__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(const TablesArgs a)
{
    __shared__ long long sm_warp[32];
    __shared__ long long sm_prefix[kTableThreads];
    __shared__ int sm_first[kTableThreads];
    const int tid = threadIdx.x;
    uint32_t bad = 0;
    int count = *a.count;
    if (count < 0 || count > a.num_pages) {
        count = count < 0 ? 0 : a.num_pages;
        bad |= kFlagPageOutOfRange;
    }
    long long top = count;
    for (int b0 = 0; b0 < a.B; b0 += kTableThreads) {
        const int b = b0 + tid;
        Want w{};
        if (b < a.B)
            w = want_of(a, b, bad);
        long long total;
        const long long at = block_scan(w.held > w.target ? w.held - w.target : 0, sm_warp, total);
        if (total == 0)
            continue;
        sm_prefix[tid] = at;
        sm_first[tid] = w.target;
        __syncthreads();
        const int n = min(kTableThreads, a.B - b0);
        for (long long e = tid; e < total; e += kTableThreads) {
            const int i = owner_of(sm_prefix, n, e);
            const int j = sm_first[i] + (int)(e - sm_prefix[i]);
            if (top + e < a.num_pages)
                a.free_pages[top + e] = a.table[(size_t)(b0 + i) * a.max_blocks + j];
            else
                bad |= kFlagPageOutOfRange;   // more pages given back than there are
        }
        top += total;
        if (top > a.num_pages)
            top = a.num_pages;
        __syncthreads();
    }
    __syncthreads();      // the pushes are visible to the pops
    long long taken = 0, used = 0, fresh = 0;
    for (int b0 = 0; b0 < a.B; b0 += kTableThreads) {
        const int b = b0 + tid;
        Want w{};
        if (b < a.B)
            w = want_of(a, b, bad);
        const int need = w.target > w.held ? w.target - w.held : 0;
        long long total, total_new;
        const long long at = taken + block_scan(need, sm_warp, total);
        const long long cu = fresh + block_scan(w.fresh, sm_warp, total_new);
        const bool fits = at + need <= top;
        if (need && !fits)
            bad |= kFlagPagesExhausted;
        sm_prefix[tid] = at - taken;
        sm_first[tid] = w.held;
        long long fit_end = 0, dummy;
        // pages popped in this chunk: the prefix up to its last request that fits
        {
            long long mine = need && fits ? need : 0;
            block_scan(mine, sm_warp, dummy);
            fit_end = dummy;
        }
        if (b < a.B) {
            a.held_out[b] = need && !fits ? w.held : w.target;
            a.cu_new[b] = (int)min(cu, 0x7fffffffLL);
        }
        __syncthreads();
        const int n = min(kTableThreads, a.B - b0);
        for (long long e = tid; e < fit_end; e += kTableThreads) {
            const int i = owner_of(sm_prefix, n, e);
            const int j = sm_first[i] + (int)(e - sm_prefix[i]);
            const int page = a.free_pages[top - 1 - (taken + e)];
            if (page < 0 || page >= a.num_pages)
                bad |= kFlagPageOutOfRange;
            a.table[(size_t)(b0 + i) * a.max_blocks + j] = page;
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
    if (bad)
        atomicOr(a.status, bad);
}

constexpr int kSlotThreads = 256;

__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const TablesArgs a)
{
    const int i = blockIdx.x * kSlotThreads + threadIdx.x;
    if (i >= a.max_new)
        return;
    int slot = -1;
    if (i < a.cu_new[a.B]) {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu_new[mid] <= i)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int cap = a.max_blocks * a.page_size;
        const int raw = a.seq_lens[lo];
        const int n = raw < 0 ? 0 : (raw > cap ? cap : raw);
        const int p = n - (a.cu_new[lo + 1] - a.cu_new[lo]) + (i - a.cu_new[lo]);
        const int j = p / a.page_size;
        if (j < a.held_out[lo]) {
            const int page = a.table[(size_t)lo * a.max_blocks + j];
            if (page >= 0 && page < a.num_pages)
                slot = page * a.page_size + p % a.page_size;
            else
                atomicOr(a.status, kFlagPageOutOfRange);
        }
    }
    a.slots[i] = slot;
}

// -------------------------------------------------------------- slot append
// One thread per 16 bytes: consecutive threads take consecutive chunks of a
// token's K row (all heads), then of its V row.
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) append_slots_kernel(const AppendSlotsArgs a)
{
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
// One CTA per (request, KV head, layer): it alone reads and writes that head's
// drafted rows, and holds all of them in registers before it writes any, so a
// row may be both a source and a destination.
constexpr int kCommitThreads = 256;

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const CommitArgs a)
{
    const int g = blockIdx.x, b = blockIdx.y, l = blockIdx.z, tid = threadIdx.x;
    uint32_t bad = 0;
    const TreeLens len = tree_lens_of(a.seq_lens, a.tree_lens, b, a.T, a.Nmax, bad);
    const int ctx = len.n - len.nt;
    const int raw = a.accepted_lens[b];
    const int acc = raw < 0 ? 0 : (raw > len.nt ? len.nt : raw);
    if (acc != raw)
        bad |= kFlagTreeOutOfRange;
    if (g == 0 && l == 0 && tid == 0 && a.seq_lens_out)
        a.seq_lens_out[b] = ctx + acc;
    auto row_of = [&](int p) -> long long {   // -1: no such page
        long long page = b;
        int r = p;
        if (a.table) {
            page = a.table[(size_t)b * a.max_blocks + p / a.page_size];
            r = p % a.page_size;
        }
        if (page < 0 || page >= a.num_pages)
            return -1;
        return ((page * a.Hkv + g) * a.page_size + r) * kHeadDim;
    };
    constexpr int kPer = TD_MAX_TREE * kRowChunks / kCommitThreads;
    uint4 kr[kPer], vr[kPer];
    long long to[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int e = tid + u * kCommitThreads;
        const int i = e / kRowChunks, c = e % kRowChunks;
        to[u] = -1;
        if (i < acc) {
            const int j = a.accepted[(size_t)b * a.T + i];
            if (j < 0 || j >= len.nt) {
                bad |= kFlagTreeOutOfRange;
                continue;
            }
            const long long src = row_of(ctx + j), dst = row_of(ctx + i);
            if (src < 0 || dst < 0) {
                bad |= kFlagPageOutOfRange;
                continue;
            }
            if (j == i)
                continue;
            kr[u] = *reinterpret_cast<const uint4 *>(a.k[l] + src + c * 8);
            vr[u] = *reinterpret_cast<const uint4 *>(a.v[l] + src + c * 8);
            to[u] = dst + c * 8;
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPer; ++u)
        if (to[u] >= 0) {
            *reinterpret_cast<uint4 *>(a.k[l] + to[u]) = kr[u];
            *reinterpret_cast<uint4 *>(a.v[l] + to[u]) = vr[u];
        }
    if (bad)
        atomicOr(a.status, bad);
}

}  // namespace

cudaError_t launch_block_tables(const TablesArgs &a, cudaStream_t stream)
{
    block_tables_kernel<<<1, kTableThreads, 0, stream>>>(a);
    if (a.max_new > 0)
        slot_map_kernel<<<(a.max_new + kSlotThreads - 1) / kSlotThreads, kSlotThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_append_slots(const AppendSlotsArgs &a, cudaStream_t stream)
{
    const long long total = (long long)a.tokens * 2 * a.Hkv * kRowChunks;
    const long long most = (long long)host_sm_count() * 8;
    long long grid = (total + kAppendThreads - 1) / kAppendThreads;
    if (grid > most)
        grid = most;
    append_slots_kernel<<<(unsigned)grid, kAppendThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_tree_commit(const CommitArgs &a, int num_layers, cudaStream_t stream)
{
    tree_commit_kernel<<<dim3(a.Hkv, a.B, num_layers), kCommitThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace td
