// td_cache_rows.cu -- rows of small caches: quantising new rows into a 4-bit cache, and
// the eviction of the positions with the least attention weight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "td_attn_common.cuh"
#include "td_cache.h"

namespace td {
namespace {

template <typename Args, typename... More>
cudaError_t launch_behind(void (*kernel)(Args, More...), long long grid, int threads, cudaStream_t stream,
                          const Args &a, More... more)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = host_pdl();
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, more...);
}

// ------------------------------------------------------------------- append
// A thread per 16 values: their scale s = e4m3(largest magnitude / 6), their codes the e2m1
// values nearest to x / s (ties to the even code).  Exact decisions in fp32: x has 8
// significant bits, s 4, a border between codes at most 3, so x / s either is the border
// or differs from it by 2^-11 relative; the quotient below is within 2^-23 and exact
// where the result is that short (one step from a rounded reciprocal: the remainder
// x - q s is exact in an fma).  The same holds for the largest value / 6 and the borders of e4m3.
constexpr int kQuantThreads = 256;

__global__ void __launch_bounds__(kQuantThreads) q4_append_kernel(const Q4AppendArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kBlocks = kHeadDim / 16;
    const int per = a.Hkv * kBlocks;              // blocks of one token's K (or V)
    const long long total = (long long)a.tokens * 2 * per;
    const long long limit = (long long)a.num_pages * a.page_size;
    for (long long e = (long long)blockIdx.x * kQuantThreads + threadIdx.x; e < total;
         e += (long long)gridDim.x * kQuantThreads) {
        const int i = (int)(e / (2 * per));
        int j = (int)(e - (long long)i * 2 * per);
        const bool isv = j >= per;
        j -= isv ? per : 0;
        const int slot = a.slots[i];
        if (slot < 0 || slot >= limit)
            continue;
        const uint4 *src = reinterpret_cast<const uint4 *>((isv ? a.v_new : a.k_new) + (size_t)i * a.new_stride + j * 16);
        const uint4 y0 = src[0], y1 = src[1];
        const uint32_t x[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            top = __vmaxu2(top, x[k] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
        const float amax = __uint_as_float(top << 16);
        uint32_t scale;                            // e4m3, saturated at 448
        asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
            : "=r"(scale)
            : "f"(0.0f), "f"(__fdiv_rn(amax, 6.0f)));
        uint32_t half;                             // its value, exact in fp16
        asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(half) : "r"(scale));
        float s;
        asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.f32.f16 %0, t;\n\t}" : "=f"(s) : "r"(half));
        uint32_t codes[2] = {0, 0};
        if (top > 0x7f80u) {
            scale = 0x7f;                          // a value that is not a number: none of the 16 is
        } else if (s > 0.0f) {
            const float inv = __frcp_rn(s), most = 8.0f * s;       // (beyond 6 s the code saturates)
            auto quotient = [&](uint32_t bits) {
                const float v = fmaxf(fminf(__uint_as_float(bits), most), -most);
                const float q = v * inv;
                return copysignf(fmaf(fmaf(-q, s, v), inv, q), v);       // (-0 keeps its sign)
            };
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float lo = quotient(x[k] << 16), hi = quotient(x[k] & 0xffff0000u);
                uint32_t two;
                asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b32 %0, {t, 0, 0, 0};\n\t}"
                    : "=r"(two)
                    : "f"(hi), "f"(lo));
                codes[k >> 2] |= two << 8 * (k & 3);
            }
        }
        const int page = slot / a.page_size, r = slot % a.page_size;
        const size_t row = ((size_t)page * a.Hkv + j / kBlocks) * a.page_size + r;
        const int block = j % kBlocks;
        *reinterpret_cast<uint2 *>((isv ? a.v : a.k) + row * kCodeBytes + block * 8) = make_uint2(codes[0], codes[1]);
        a.scales[row * kScaleBytes + (isv ? kBlocks : 0) + block] = (uint8_t)scale;
    }
}

// ------------------------------------------------------------------- eviction
// Of request b's n > budget positions and KV head g: the first `sinks`, the last `recent`, and
// of the others the `heavy` = budget - sinks - recent with the most weight (ties: the lower
// position).  A CTA per (request, KV head) finds the weight of the last one kept by three
// radix passes over order-preserving keys (11, 11 and 10 bits, counts in shared
// memory), then walks the row once, writing the kept positions in order and their
// weights.  In place a weight moves to a lower or its own place, and every place that a
// chunk writes lies below the next chunk's, so the block's barrier per chunk orders
// reads before writes.
constexpr int kSelectThreads = 512;
constexpr int kSelectPer = 4;

// A weight that is not a number counts as the largest.
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0xffffffffu : order_key(w); }

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a)
{
    __shared__ unsigned hist[2048];
    __shared__ unsigned sums[kSelectThreads / 32];
    __shared__ unsigned sm_digit, sm_rest;
    pdl_wait();
    pdl_launch_dependents();
    const int unit = blockIdx.x, b = unit / a.Hkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t bad = 0;
    const int n = seq_len_of(a.seq_lens, b, a.Nmax, bad);
    const float *w = a.weights + (size_t)unit * a.Nmax;
    float *out = a.weights_out + (size_t)unit * a.out_row;
    int32_t *kept = a.kept + (size_t)unit * a.budget;
    if (unit % a.Hkv == 0 && tid == 0) {
        a.seq_lens_out[b] = min(n, a.budget);
        if (bad)
            atomicOr(a.status, bad);
    }
    if (n <= a.budget) {
        for (int i = tid; i < a.budget; i += kSelectThreads) {
            kept[i] = i < n ? i : -1;
            if (i < n && out != w)
                out[i] = w[i];
        }
        return;
    }
    const int c0 = a.sinks, c1 = n - a.recent;       // the candidates
    const int heavy = a.budget - a.sinks - a.recent;
    // The key of the heavy-th candidate, digit by digit, and how many of that key are kept.
    uint32_t key = 0, mask = 0;
    unsigned rest = heavy;
    if (heavy > 0) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
            for (int i = tid; i < bins; i += kSelectThreads)
                hist[i] = 0;
            __syncthreads();
            for (int i = c0 + tid; i < c1; i += kSelectThreads) {
                const uint32_t k = weight_key(w[i]);
                if ((k & mask) == key)
                    atomicAdd(&hist[k >> shift & (bins - 1)], 1u);
            }
            __syncthreads();
            // Counts from the highest digit down: a thread has a run of bins.
            const int run = bins / kSelectThreads, top = bins - 1 - tid * run;
            unsigned mine = 0;
            for (int k = 0; k < run; ++k)
                mine += hist[top - k];
            unsigned inc = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned y = __shfl_up_sync(kFull, inc, d);
                if (lane >= d)
                    inc += y;
            }
            if (lane == 31)
                sums[warp] = inc;
            __syncthreads();
            unsigned before = inc - mine;
            for (int i = 0; i < warp; ++i)
                before += sums[i];
            if (before < rest && rest <= before + mine) {
                int d = top;
                for (; before + hist[d] < rest; --d)
                    before += hist[d];
                sm_digit = d;
                sm_rest = rest - before;
            }
            __syncthreads();
            key |= sm_digit << shift;
            mask |= (uint32_t)(bins - 1) << shift;
            rest = sm_rest;
        }
    }
    // ---- the kept positions in order.  Both counts pass through one scan: those kept in
    // any case in the low half, those of the last key in the high one.
    unsigned sure0 = 0, same0 = 0;                 // before this chunk
    for (int base = 0; base < n; base += kSelectThreads * kSelectPer) {
        const int at = base + tid * kSelectPer;
        float x[kSelectPer];
        unsigned sure = 0, same = 0;               // bits of this thread's positions
#pragma unroll
        for (int k = 0; k < kSelectPer; ++k) {
            const int i = at + k;
            x[k] = i < n ? w[i] : 0.0f;
            const uint32_t y = weight_key(x[k]);
            const bool always = i < c0 || i >= c1;
            if (i < n && (always || (heavy > 0 && y > key)))
                sure |= 1u << k;
            else if (i < n && heavy > 0 && y == key)
                same |= 1u << k;
        }
        const unsigned mine = __popc(sure) | __popc(same) << 16;       // (at most 2048 of either)
        unsigned inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned y = __shfl_up_sync(kFull, inc, d);
            if (lane >= d)
                inc += y;
        }
        __syncthreads();                           // (the sums of the chunk before have been read)
        if (lane == 31)
            sums[warp] = inc;
        __syncthreads();                           // every weight of this chunk has been read, too
        unsigned before = inc - mine, all = 0;
        for (int i = 0; i < kSelectThreads / 32; ++i) {
            if (i < warp)
                before += sums[i];
            all += sums[i];
        }
        unsigned nsure = sure0 + (before & 0xffff), nsame = same0 + (before >> 16);
#pragma unroll
        for (int k = 0; k < kSelectPer; ++k) {
            const bool eq = same >> k & 1u;
            const bool keep = (sure >> k & 1u) || (eq && nsame < rest);
            if (keep) {
                const unsigned to = nsure + min(nsame, rest);
                kept[to] = at + k;
                out[to] = x[k];
            }
            nsure += sure >> k & 1u;
            nsame += eq;
        }
        sure0 += all & 0xffff;
        same0 += all >> 16;
    }
}

// The kept rows, in order, to rows 0 .. of the cache they go to.  kept[i] >= i, so a row that is
// read lies at or behind the row that it goes to: a CTA that takes its rows in order, in
// chunks that are read before they are written, overwrites no row that is still to be read.
// A CTA has K or V of one (request, KV head), whole rows or a slice of each, where there are
// few; between two caches the rows are also cut into runs.  The next chunk is read before
// this one is written.
constexpr int kMoveThreads = 256;
constexpr int kMovePer = 4;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int log_slices, int runs)
{
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    const int slices = 1 << log_slices;
    int id = blockIdx.x;
    const int run = id % runs;
    id /= runs;
    const int slice = id & (slices - 1);
    id >>= log_slices;
    const bool isv = id & 1;
    const int unit = id >> 1, b = unit / a.Hkv, h = unit % a.Hkv;
    uint32_t bad = 0;
    const int n = seq_len_of(a.seq_lens, b, a.Nmax, bad);
    const int count = min(n, a.budget);
    if (a.place && n <= a.budget)
        return;
    const int lanes = 16 >> log_slices;            // of a row (or its slice), 16 bytes each
    const int rows = kMoveThreads / lanes * kMovePer;           // of a chunk
    const int chunks = (count + rows - 1) / rows;
    const int first = (int)((long long)chunks * run / runs) * rows, end = min(count, (int)((long long)chunks * (run + 1) / runs) * rows);
    const int32_t *kept = a.kept + (size_t)unit * a.budget;
    const uint8_t *from = isv ? a.from.v : a.from.k;
    uint8_t *to = (uint8_t *)(isv ? a.to_v : a.to_k);
    const int off = (slice * lanes + tid % lanes) * 16;
    uint32_t flags = 0;
    uint4 x[kMovePer], y[kMovePer];
    int to_row[kMovePer], to_next[kMovePer];       // -1: nothing to write
    auto read = [&](int base, uint4 (&v)[kMovePer], int (&dst)[kMovePer]) {
        int p[kMovePer];
#pragma unroll
        for (int k = 0; k < kMovePer; ++k) {
            const int i = base + tid / lanes + k * (kMoveThreads / lanes);
            p[k] = i < end ? kept[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < kMovePer; ++k) {
            const int i = base + tid / lanes + k * (kMoveThreads / lanes);
            dst[k] = -1;
            if (p[k] < 0 || p[k] >= n || (a.place && p[k] == i))
                continue;
            const int src = row_of(a.from, a.Hkv, h, p[k], page_of(a.from, b, p[k]));
            dst[k] = row_of(a.to, a.Hkv, h, i, page_of(a.to, b, i));
            if (src < 0 || dst[k] < 0) {
                flags |= kFlagPageOutOfRange;
                dst[k] = -1;
                continue;
            }
            v[k] = __ldcg(reinterpret_cast<const uint4 *>(from + (size_t)src * (kHeadDim * 2) + off));
        }
    };
    if (first < end)
        read(first, x, to_row);
    for (int base = first; base < end; base += rows) {
        if (base + rows < end)
            read(base + rows, y, to_next);
        if (a.place)
            __syncthreads();                       // every row of this chunk has been read
#pragma unroll
        for (int k = 0; k < kMovePer; ++k) {
            if (to_row[k] >= 0)
                *reinterpret_cast<uint4 *>(to + (size_t)to_row[k] * (kHeadDim * 2) + off) = x[k];
            x[k] = y[k];
            to_row[k] = to_next[k];
        }
    }
    if (flags)
        atomicOr(a.status, flags);
}

}  // namespace

cudaError_t launch_q4_append(const Q4AppendArgs &a, cudaStream_t stream)
{
    const long long total = (long long)a.tokens * 2 * a.Hkv * (kHeadDim / 16);
    const long long most = (long long)host_sm_count() * 8;
    long long grid = (total + kQuantThreads - 1) / kQuantThreads;
    if (grid > most)
        grid = most;
    return launch_behind(q4_append_kernel, grid, kQuantThreads, stream, a);
}

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream)
{
    const long long units = (long long)a.B * a.Hkv;
    const cudaError_t err = launch_behind(evict_select_kernel, units, kSelectThreads, stream, a);
    if (err != cudaSuccess)
        return err;
    // Slices of rows (in place) or runs of them (else) until there are about four CTAs per SM.
    int log_slices = 0, runs = 1;
    if (a.place) {
        while (log_slices < 2 && (units * 2 << log_slices) < 2ll * sms)
            ++log_slices;
    } else {
        const int chunks = (a.budget + kMoveThreads / 16 * kMovePer - 1) / (kMoveThreads / 16 * kMovePer);
        while (runs < chunks && units * 2 * runs < 8ll * sms)
            ++runs;
    }
    return launch_behind(evict_move_kernel, (units * 2 << log_slices) * runs, kMoveThreads, stream, a, log_slices, runs);
}

}  // namespace td
