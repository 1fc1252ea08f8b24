// td_cache_rows.cu -- rows of small caches: quantising new rows into a 4-bit cache, and
// the eviction of the positions with the least attention weight.
#include <cooperative_groups.h>
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
// where the result is that short (Markstein's correction, IBM J. Res. Dev. 34 (1990) 111: one step
// from a rounded reciprocal, as the remainder x - q s is exact in an fma).  The same holds for the largest value / 6 and the borders of e4m3.
//
// Bound by memory: 32749 tokens of 8 KV heads take 28.1 us (6.1 TB/s).  A block of 16 values a thread,
// 16 CTAs per SM that walk (32: 28.6 us; as many as there are blocks: 31.3).
constexpr int kQuantThreads = 256;
constexpr int kQuantCtas = 16;                // per SM, at most
constexpr int kQuantBlocks = kHeadDim / 16;   // of a row

__global__ void __launch_bounds__(kQuantThreads) q4_append_kernel(const Q4AppendArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t per = a.Hkv * kQuantBlocks;    // blocks of one token's K (or V)
    const uint32_t total = (uint32_t)a.tokens * 2 * per;        // (below 2^31)
    const uint32_t limit = (uint32_t)a.num_pages * a.page_size;
    for (uint32_t e = blockIdx.x * kQuantThreads + threadIdx.x; e < total; e += gridDim.x * kQuantThreads) {
        const uint32_t i = (uint32_t)((uint64_t)e * a.token_magic >> a.token_shift);      // e / (2 per)
        uint32_t j = e - i * 2 * per;
        const bool isv = j >= per;
        j -= isv ? per : 0;
        const uint32_t slot = a.slots[i];                       // (negative ones lie beyond the limit)
        if (slot >= limit)
            continue;
        const uint4 *src = reinterpret_cast<const uint4 *>((isv ? a.v_new : a.k_new) + (size_t)i * a.new_stride + j * 16);
        const uint4 y0 = src[0], y1 = src[1];
        const uint32_t x[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            top = __vmaxu2(top, x[k] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
        // largest / 6, by the step that the quotients below take
        const float amax = __uint_as_float(top << 16), sixth = amax * (1.0f / 6.0f);
        const float want = top >= 0x7f80u ? amax : fmaf(-fmaf(sixth, 6.0f, -amax), 1.0f / 6.0f, sixth);
        uint32_t scale;                        // e4m3, saturated at 448
        float s;                               // its value (exact in fp16 on the way)
        asm("{\n\t.reg .b16 t, u, v;\n\t.reg .b32 w;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 t, %2, %3;\n\tcvt.u32.u16 %0, t;\n\t"
            "cvt.rn.f16x2.e4m3x2 w, t;\n\tmov.b32 {u, v}, w;\n\tcvt.f32.f16 %1, u;\n\t}"
            : "=r"(scale), "=f"(s)
            : "f"(0.0f), "f"(want));
        uint2 codes = make_uint2(0, 0);
        if (top > 0x7f80u) {
            scale = 0x7f;                      // a value that is not a number: none of the 16 is
        } else if (s > 0.0f) {
            float inv;                         // (within a step: the quotient's last step corrects it)
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
            // Beyond 6 s the code saturates; 8 s stands for what is larger (only 16 values of
            // which the largest is beyond 448 * 8 have any, as a smaller scale is at
            // least half of the largest / 6).
            float2 q[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                q[k] = make_float2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xffff0000u));
            if (__builtin_expect(amax > 8.0f * 448.0f, 0)) {
                const float most = 8.0f * s;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    q[k] = make_float2(fmaxf(fminf(q[k].x, most), -most), fmaxf(fminf(q[k].y, most), -most));
            }
            // Minus the quotient, so that the zeros' signs come out right too.
            const float2 ninv = make_float2(-inv, -inv), s2 = make_float2(s, s);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 y = __fmul2_rn(q[k], ninv);
                q[k] = __ffma2_rn(__ffma2_rn(y, s2, q[k]), ninv, y);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 *z = q + 4 * h;
                uint32_t &out = h ? codes.y : codes.x;
                asm("{\n\t.reg .b8 a, b, c, d;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
                    "mov.b32 %0, {a, b, c, d};\n\t}"
                    : "=r"(out)
                    : "f"(z[0].x), "f"(z[0].y), "f"(z[1].x), "f"(z[1].y), "f"(z[2].x), "f"(z[2].y), "f"(z[3].x), "f"(z[3].y));
                out ^= 0x88888888u;
            }
        }
        const uint32_t page = (uint32_t)((uint64_t)slot * a.page_magic >> a.page_shift);
        const uint32_t r = slot - page * a.page_size, block = j % kQuantBlocks;
        const size_t row = ((size_t)page * a.Hkv + j / kQuantBlocks) * a.page_size + r;
        *reinterpret_cast<uint2 *>((isv ? a.v : a.k) + row * kCodeBytes + block * 8) = codes;
        a.scales[row * kScaleBytes + (isv ? kQuantBlocks : 0) + block] = (uint8_t)scale;
    }
}

// ------------------------------------------------------------------- eviction
// Of request b's n > budget positions and KV head g: the first `sinks`, the last `recent`, and
// of the others the `heavy` = budget - sinks - recent with the most weight (ties: the lower
// position).  A CTA, or a cluster of them, per (request, KV head) finds the weight of the last one
// kept, then writes the kept positions in order and their weights.
//
// The weight is found by at most three radix passes over order-preserving keys (11 bits each,
// counts in shared memory, a cluster's added up by each rank in order: with every thread's own
// bins read from the other ranks four CTAs take 35 us, not 17).  Rows of up to 131072 positions
// stay in registers.  In place, 32 requests x 8 heads from up to 4224 to 4096 positions: 174 us with
// the rows' moves, 6.2 TB/s; 7 prompts of 9K .. 16K to 2048: 34.8 us, of which the selection
// is 13 (integer instructions and its barriers).  (Found bit by bit with block-wide counts, without
// atomics, it takes two to three times as long.)
constexpr int kBins = 2048;

// A weight that is not a number counts as the largest, -0 as 0.  No key is 0 or kAnyCase.
constexpr uint32_t kAnyCase = 0xffffffffu;
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0xff800001u : order_key(w); }

// A row's CTAs, a cluster of C of them or one.
template <int C> __device__ __forceinline__ void row_sync()
{
    if constexpr (C > 1)
        cooperative_groups::this_cluster().sync();
    else
        __syncthreads();
}
template <int C, typename X> __device__ __forceinline__ X *of_rank(X *p, int rank)
{
    if constexpr (C > 1)
        return cooperative_groups::this_cluster().map_shared_rank(p, rank);
    else
        return p;
}

template <int T, int C> struct SelectShared {
    unsigned hist[C > 1 ? 3 : 1][kBins];             // a cluster: this rank's in two of them in turn, the row's
    unsigned ends[2][T / 32], sums[T / 32], found[4];
    unsigned totals[2][C];           // of each rank's positions: kept in any case, of the last weight
};

// The key of the heavy-th largest candidate (heavy > 0), and in `rest` how many of that key are among
// the heavy ones.  each(f) calls f(key) for every candidate of the thread; it may do so with 0, which
// counts for nothing, and with kAnyCase, which it does `others` times in the row.  The digits begin
// behind the bits that all candidates share: weights of a few magnitudes else meet in a few bins,
// whose counts are then added to one after the other.
template <int T, int C, typename Each>
__device__ __forceinline__ uint32_t last_key(SelectShared<T, C> &x, int heavy, int others, unsigned &rest, Each each)
{
    constexpr int W = T / 32, kDigit = 11, kRun = kBins / T;
    static_assert(kBins == 1 << kDigit && kBins % T == 0 && W <= 32, "bins per thread");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t least = 0xffffffffu, most = 0;
    each([&](uint32_t k) {
        least = min(least, k - 1);
        most = max(most, k + 1);
    });
    least = __reduce_min_sync(kFull, least);
    most = __reduce_max_sync(kFull, most);
    if (lane == 0) {
        x.ends[0][warp] = least;
        x.ends[1][warp] = most;
    }
    row_sync<C>();
#pragma unroll
    for (int q = 0; q < C; ++q) {
        least = min(least, of_rank<C>(x.ends[0], q)[lane % W]);
        most = max(most, of_rank<C>(x.ends[1], q)[lane % W]);
    }
    least = __reduce_min_sync(kFull, least) + 1;
    most = __reduce_max_sync(kFull, most) - 1;
    int left = 32 - __clz(least ^ most);             // bits of the key that are open
    uint32_t mask = left == 32 ? 0u : 0xffffffffu << left, key = most & mask;
    rest = heavy + (key == (kAnyCase & mask) ? others : 0);
#pragma unroll 1
    for (int pass = 0; left > 0; ++pass) {
        const int shift = max(left - kDigit, 0);
        const unsigned digits = (1u << (left - shift)) - 1;
        // (In a cluster two arrays in turn: one is cleared when every rank has read it, two passes ago.)
        unsigned *const hist = x.hist[C > 1 ? pass & 1 : 0];
        for (int i = tid; i < kBins; i += T)
            hist[i] = 0;
        __syncthreads();
        each([&](uint32_t k) {
            if ((k & mask) == key)
                atomicAdd(&hist[k >> shift & digits], 1u);
        });
        row_sync<C>();
        if constexpr (C > 1) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                unsigned sum = 0;
#pragma unroll
                for (int q = 0; q < C; ++q)
                    sum += of_rank<C>(hist, q)[i * T + tid];
                x.hist[2][i * T + tid] = sum;
            }
            __syncthreads();
        }
        const unsigned *const all = x.hist[C > 1 ? 2 : 0];
        // Counts from the highest digit down: a thread has a run of bins.
        const int top = kBins - 1 - tid * kRun;
        unsigned bins[kRun], mine = 0;
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            bins[k] = all[top - k];
            mine += bins[k];
        }
        unsigned inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned y = __shfl_up_sync(kFull, inc, d);
            if (lane >= d)
                inc += y;
        }
        if (lane == 31)
            x.sums[warp] = inc;
        __syncthreads();
        unsigned before = inc - mine + __reduce_add_sync(kFull, lane < warp ? x.sums[lane] : 0u);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            if (before < rest && rest <= before + bins[k]) {
                x.found[0] = top - k;
                x.found[1] = rest - before;
                x.found[2] = bins[k];
            }
            before += bins[k];
        }
        __syncthreads();
        key |= x.found[0] << shift;
        mask |= digits << shift;
        rest = x.found[1];
        left = shift;
        if (C == 1 && left > 0 && x.found[2] == 1) {         // one candidate is left
            each([&](uint32_t k) {
                if ((k & mask) == key)
                    x.found[3] = k;
            });
            __syncthreads();
            return x.found[3];
        }
    }
    return key;
}

// Rows of up to C T NR positions, which stay in registers; a rank has the rank-th part of its row.
template <int T, int NR, int C> __global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(T) evict_select_short_kernel(const EvictArgs a)
{
    constexpr int W = T / 32;
    __shared__ SelectShared<T, C> x;
    __shared__ uint32_t counts[NR * W];            // kept in any case, and (high half) of the last weight
    pdl_wait();
    pdl_launch_dependents();
    const int unit = blockIdx.x / C, rank = blockIdx.x % C, b = unit / a.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t bad = 0;
    const int n = seq_len_of(a.seq_lens, b, a.Nmax, bad);
    const float *w = a.weights + (size_t)unit * a.Nmax;
    float *out = a.weights_out + (size_t)unit * a.out_row;
    int32_t *kept = a.kept + (size_t)unit * a.budget;
    if (unit % a.Hkv == 0 && rank == 0 && tid == 0) {
        a.seq_lens_out[b] = min(n, a.budget);
        if (bad)
            atomicOr(a.status, bad);
    }
    if (n <= a.budget) {
        for (int i = rank * T + tid; i < a.budget; i += C * T) {
            kept[i] = i < n ? i : -1;
            if (i < n && out != w)
                out[i] = w[i];
        }
        return;
    }
    const int c0 = a.sinks, c1 = n - a.recent;       // the candidates
    const int heavy = a.budget - a.sinks - a.recent;
    const int part = (n + C - 1) / C, base = rank * part, count = min(part, n - base);
    const int rounds = (part + T - 1) / T;           // position base + j T + tid
    float v[NR];
    uint32_t k[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        const int i = j * T + tid;
        v[j] = j < rounds && i < count ? w[base + i] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        const int i = j * T + tid, at = base + i;
        k[j] = i >= count ? 0u : at < c0 || at >= c1 ? kAnyCase : weight_key(v[j]);
    }
    uint32_t key = kAnyCase - 1;
    unsigned rest = 0;                               // how many of that key are kept, the lowest positions
    if (heavy > 0)
        key = last_key(x, heavy, a.sinks + a.recent, rest, [&](auto f) {
#pragma unroll
            for (int j = 0; j < NR; ++j)
                if (j < rounds)
                    f(k[j]);
        });
    else
        row_sync<C>();       // (last_key's: every rank has begun before its shared memory is written below)
    // Counts of every warp and round, their prefix sums in the positions' order, the places.
    auto flags = [&](int j, uint32_t &sure, uint32_t &equal) {
        sure = __ballot_sync(kFull, k[j] > key);
        equal = __ballot_sync(kFull, k[j] == key);
    };
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        uint32_t sure, equal;
        flags(j, sure, equal);
        if (lane == 0)
            counts[j * W + warp] = __popc(sure) | __popc(equal) << 16;
    }
    __syncthreads();
    if (warp == 0) {
        constexpr int kPer = NR * W / 32;
        uint32_t mine[kPer], all = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            mine[i] = all;
            all += counts[lane * kPer + i];          // (at most 16384 of either)
        }
        uint32_t inc = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, inc, d);
            if (lane >= d)
                inc += y;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            counts[lane * kPer + i] = mine[i] + inc - all;
        const uint32_t total = __shfl_sync(kFull, inc, 31);
        if (lane < C) {
            of_rank<C>(x.totals[0], lane)[rank] = total & 0xffff;
            of_rank<C>(x.totals[1], lane)[rank] = total >> 16;
        }
    }
    row_sync<C>();                                   // (every weight of the row has been read, too)
    unsigned sure0 = 0, same0 = 0;                   // of the ranks before
    for (int q = 0; q < rank; ++q) {
        sure0 += x.totals[0][q];
        same0 += x.totals[1][q];
    }
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        if (j >= rounds)
            break;
        uint32_t sure, equal;
        flags(j, sure, equal);
        const uint32_t before = counts[j * W + warp];
        const uint32_t nsure = sure0 + (before & 0xffff) + __popc(sure & below);
        const uint32_t nsame = same0 + (before >> 16) + __popc(equal & below);
        if ((sure >> lane & 1u) || ((equal >> lane & 1u) && nsame < rest)) {
            const uint32_t to = nsure + min(nsame, rest);
            kept[to] = base + j * T + tid;
            out[to] = v[j];
        }
    }
}

// Longer rows are read again for each pass, then walked over.  In place a weight moves to a lower or its own
// place, and every place that a chunk writes lies below the next chunk's, so the block's
// barrier per chunk orders reads before writes.
constexpr int kSelectThreads = 512;
constexpr int kSelectPer = 4;

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a)
{
    __shared__ SelectShared<kSelectThreads, 1> x;
    unsigned *const sums = x.sums;
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
    uint32_t key = 0xffffffffu;
    unsigned rest = 0;                               // how many of that key are kept
    if (heavy > 0)
        key = last_key(x, heavy, 0, rest, [&](auto f) {
            constexpr int kAhead = 8;
            for (int i0 = c0 + tid; i0 < c1; i0 += kAhead * kSelectThreads) {
                float v[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (i0 + k * kSelectThreads < c1)
                        v[k] = w[i0 + k * kSelectThreads];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (i0 + k * kSelectThreads < c1)
                        f(weight_key(v[k]));
            }
        });
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
// few; between two caches, or to other pages, the rows are also cut into runs.  Cache rows are looked up
// kMoveList at a time; a chunk is read while the one before is written.
constexpr int kMoveThreads = 256;
constexpr int kMovePer = 8;       // (4 with 3 or 4 CTAs per SM: 219 and 191 us where this takes 176)
constexpr int kMoveList = 1024;

// POOL: two tables of one pool (the other calls have no register for that: 174 us in place became 179).
template <bool POOL> __global__ void __launch_bounds__(kMoveThreads, 2) evict_move_kernel(const EvictArgs a, int log_slices, int runs)
{
    __shared__ int sm_from[kMoveList], sm_to[kMoveList];        // cache rows; to -1: nothing to move
    // The first entry of a list that moves.  Two words in turn: no barrier lies between a warp's read of one
    // and the reset for the next list, but one lies between that read and the reset after it.
    __shared__ int sm_first[2];
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
    uint32_t bad = 0, flags = 0;
    const int n = seq_len_of(a.seq_lens, b, a.Nmax, bad);
    const int count = min(n, a.budget);
    if (a.place && n <= a.budget)
        return;
    const int lanes = 16 >> log_slices;            // of a row (or its slice), 16 bytes each
    const int step = kMoveThreads / lanes, rows = step * kMovePer;      // rows of a chunk
    const int chunks = (count + rows - 1) / rows;
    int first = (int)((long long)chunks * run / runs) * rows;
    int end = min(count, (int)((long long)chunks * (run + 1) / runs) * rows);
    bool ordered = a.place;
    if (POOL && count > 0) {
        // A request with a block of the same page in both moves as in place, by its first CTA.
        bool same = false;
        for (int j = tid; j <= block_of(a.to, count - 1); j += kMoveThreads)
            same = same || a.from.table[(size_t)b * a.from.max_blocks + j] == a.to.table[(size_t)b * a.to.max_blocks + j];
        ordered = __syncthreads_or(same);
        if (ordered) {
            if (run > 0)
                return;
            first = 0;
            end = count;
        }
    }
    const int32_t *kept = a.kept + (size_t)unit * a.budget;
    const int off = (slice * lanes + tid % lanes) * 16;
    const uint8_t *from = (isv ? a.from.v : a.from.k) + off;
    uint8_t *to = (uint8_t *)(isv ? a.to_v : a.to_k) + off;
    for (int base = first, pass = 0; base < end; base += kMoveList, pass ^= 1) {
        const int list = min(kMoveList, end - base);
        if (tid == 0)
            sm_first[pass] = list;
        __syncthreads();                           // (the list before has been read)
        constexpr int kFind = kMoveList / kMoveThreads;
        int p[kFind], pages[kFind], to_pages[kFind];
#pragma unroll
        for (int k = 0; k < kFind; ++k) {
            const int i = tid + k * kMoveThreads;
            p[k] = i < list ? kept[base + i] : -1;
        }
#pragma unroll
        for (int k = 0; k < kFind; ++k) {
            const int i = base + tid + k * kMoveThreads;
            if (p[k] >= n || (a.place && p[k] == i))
                p[k] = -1;
            pages[k] = p[k] >= 0 ? page_of(a.from, b, p[k]) : 0;
            to_pages[k] = p[k] >= 0 ? page_of(a.to, b, i) : 0;
        }
#pragma unroll
        for (int k = 0; k < kFind; ++k) {
            const int i = tid + k * kMoveThreads;
            int f = 0, t = -1;
            if (p[k] >= 0) {
                f = row_of(a.from, a.Hkv, h, p[k], pages[k]);
                t = row_of(a.to, a.Hkv, h, base + i, to_pages[k]);
                if (f < 0 || t < 0) {
                    flags |= kFlagPageOutOfRange;
                    t = -1;
                } else if (POOL && f == t) {
                    t = -1;                        // (stays where it is)
                } else {
                    atomicMin(&sm_first[pass], i);
                }
            }
            sm_from[i] = f;
            sm_to[i] = t;
        }
        __syncthreads();
        uint4 x[2][kMovePer];
        int row[2][kMovePer];                      // -1: nothing to write
        auto read = [&](int i0, uint4 (&v)[kMovePer], int (&dst)[kMovePer]) {
#pragma unroll
            for (int k = 0; k < kMovePer; ++k) {
                const int i = i0 + tid / lanes + k * step;
                dst[k] = i < list ? sm_to[i] : -1;
                if (dst[k] >= 0)
                    v[k] = __ldcg(reinterpret_cast<const uint4 *>(from + (size_t)sm_from[i] * (kHeadDim * 2)));
            }
        };
        auto write = [&](const uint4 (&v)[kMovePer], const int (&dst)[kMovePer]) {
            if (ordered)
                __syncthreads();                   // every row of this chunk has been read
#pragma unroll
            for (int k = 0; k < kMovePer; ++k)
                if (dst[k] >= 0)
                    *reinterpret_cast<uint4 *>(to + (size_t)dst[k] * (kHeadDim * 2)) = v[k];
        };
        int i0 = sm_first[pass] / rows * rows;
        if (i0 < list)
            read(i0, x[0], row[0]);
        for (; i0 < list; i0 += 2 * rows) {
            if (i0 + rows < list)
                read(i0 + rows, x[1], row[1]);
            write(x[0], row[0]);
            if (i0 + rows >= list)
                break;
            if (i0 + 2 * rows < list)
                read(i0 + 2 * rows, x[0], row[0]);
            write(x[1], row[1]);
        }
    }
    if (flags)
        atomicOr(a.status, flags);
}

}  // namespace

// x / d = x * m >> shift for 0 <= x < 2^31.
static void magic(uint32_t d, uint32_t &m, int &shift)
{
    int s = 0;
    while ((uint64_t(1) << s) < d)
        ++s;
    shift = 31 + s;
    m = (uint32_t)(((uint64_t(1) << shift) + d - 1) / d);
}

cudaError_t launch_q4_append(const Q4AppendArgs &args, cudaStream_t stream)
{
    const long long per = 2ll * args.Hkv * kQuantBlocks;        // blocks of a token
    const long long most = (long long)host_sm_count() * kQuantCtas;
    // (blocks are counted in 31 bits)
    const int piece = (int)((1ll << 30) / per) > 0 ? (int)((1ll << 30) / per) : 1;
    for (int t = 0; t < args.tokens; t += piece) {
        Q4AppendArgs a = args;
        a.k_new += (size_t)t * a.new_stride;
        a.v_new += (size_t)t * a.new_stride;
        a.slots += t;
        a.tokens = args.tokens - t < piece ? args.tokens - t : piece;
        magic((uint32_t)per, a.token_magic, a.token_shift);
        magic((uint32_t)a.page_size, a.page_magic, a.page_shift);
        long long grid = (a.tokens * per + kQuantThreads - 1) / kQuantThreads;
        if (grid > most)
            grid = most;
        const cudaError_t err = launch_behind(q4_append_kernel, grid, kQuantThreads, stream, a);
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream)
{
    const long long units = (long long)a.B * a.Hkv;
    // Rows are cut over a cluster where one CTA's registers do not hold them (100K positions: 24 us, walked
    // over 121), and in two where they are long and there are SMs enough (8 rows of 16384: 13.4 us, of
    // one CTA each 15.0; of 3000 positions 12.8 and 12.1; four CTAs a row: 13.2, but 43 for 35 with 56 rows).
    cudaError_t err;
    if (a.Nmax > 131072)
        err = launch_behind(evict_select_kernel, units, kSelectThreads, stream, a);
    else if (a.Nmax > 16384)
        err = launch_behind(evict_select_short_kernel<1024, 16, 8>, units * 8, 1024, stream, a);
    else if (a.Nmax > 4096 && units * 2 <= sms)
        err = launch_behind(evict_select_short_kernel<1024, 8, 2>, units * 2, 1024, stream, a);
    else if (a.Nmax <= 8192)
        err = launch_behind(evict_select_short_kernel<512, 16, 1>, units, 512, stream, a);
    else
        err = launch_behind(evict_select_short_kernel<1024, 16, 1>, units, 1024, stream, a);
    if (err != cudaSuccess)
        return err;
    // In place: slices of rows, up to four, until there are two CTAs per SM, as many as are resident.  Else
    // runs of rows, up to eight CTAs per SM: rows of different lengths end together.
    int log_slices = 0, runs = 1;
    if (a.place) {
        while (log_slices < 2 && (units * 2 << log_slices) < 2ll * sms)
            ++log_slices;
    } else {
        const int chunks = (a.budget + kMoveThreads / 16 * kMovePer - 1) / (kMoveThreads / 16 * kMovePer);
        while (runs < chunks && units * 2 * runs < 8ll * sms)
            ++runs;
    }
    return launch_behind(a.pool && !a.place ? evict_move_kernel<true> : evict_move_kernel<false>,
                         (units * 2 << log_slices) * runs, kMoveThreads, stream, a, log_slices, runs);
}

}  // namespace td
